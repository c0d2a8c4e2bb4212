"""The router's choice against the 64-bit form: ids equal, weights within bounds."""
import math

import pytest
import torch

import layer_reference as L

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def mx():
    import mxfp4_block_quantization_gb300 as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def check(mx, logits, k, **kw):
    ids, w = mx.moe_topk(logits, k, **kw)
    want_ids, want, bound = L.topk(logits, k, **kw)
    assert torch.equal(ids, want_ids)
    assert ids.dtype is torch.int32 and w.dtype is torch.float32
    assert ((w.double() - want).abs() <= bound).all()
    return ids, w


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 2), (7, 31, 4), (5, 32, 32), (70, 33, 8), (33, 128, 8),
                                   (9, 129, 5), (64, 256, 6), (17, 257, 1), (40, 384, 8), (8, 385, 10),
                                   (6, 512, 16), (5, 1024, 8), (3, 1025, 8), (2, 8192, 32)])
def test_sizes(mx, dtype, T, E, k):
    logits = (torch.randn(T, E, device="cuda", generator=gen(E + k)) * 2).to(dtype)
    bias = torch.randn(E, device="cuda", generator=gen(1)) * 0.1
    check(mx, logits, k)
    check(mx, logits, k, renormalize=False, scale=2.5)
    check(mx, logits, k, score="sigmoid", bias=bias, scale=2.5)
    check(mx, logits, k, score="sigmoid", renormalize=False)
    check(mx, logits, k, bias=bias, renormalize=False)


@pytest.mark.parametrize("E,groups,top", [(8, 8, 3), (24, 4, 2), (33, 3, 1), (64, 32, 5), (62, 31, 31), (384, 8, 4),
                                          (256, 2, 1), (35, 7, 2), (8192, 16, 4)])
@pytest.mark.parametrize("group_score", ["max", "sum2"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_groups(mx, E, groups, top, group_score, score, with_bias):
    logits = torch.randn(19, E, device="cuda", generator=gen(E))
    bias = torch.randn(E, device="cuda", generator=gen(2)) * 0.2 if with_bias else None
    check(mx, logits, min(E // groups + 1, 9), score=score, bias=bias, groups=groups, top_groups=top,
          group_score=group_score)


def test_equal_picks_go_to_the_lowest_index(mx):
    logits = torch.zeros(4, 100, device="cuda")
    logits[1] = torch.arange(100, device="cuda") // 10 * -1.0
    logits[2, ::2] = -0.0
    logits[3] = torch.randint(0, 3, (100,), device="cuda", generator=gen(3)).float()
    for kw in ({}, {"score": "sigmoid"}, {"score": "sigmoid", "bias": torch.full((100,), 0.25, device="cuda")},
               {"groups": 10, "top_groups": 3}, {"groups": 10, "top_groups": 3, "group_score": "sum2"},
               {"bias": torch.zeros(100, device="cuda"), "groups": 4, "top_groups": 2}):
        ids, _ = check(mx, logits, 8, **kw)
        assert ids[0].tolist() == list(range(8))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups", [1, 4])
def test_picks_that_float32_cannot_tell_apart(mx, score, groups):
    """Biases that undo the scores to half a float32 step: every pick is near
    every other, and their order is that of the roundings."""
    E = 128
    one = torch.randn(E, device="cuda", generator=gen(4))
    s = torch.sigmoid(one.double()) if score == "sigmoid" else torch.softmax(one.double(), 0)
    bias = (0.75 - s).float()
    logits = one.repeat(6, 1)
    logits[3:] += torch.randn(3, E, device="cuda", generator=gen(5)) * 1e-6
    for group_score in ("max", "sum2"):
        check(mx, logits, 8, score=score, bias=bias, groups=groups, top_groups=max(1, groups // 2),
              group_score=group_score)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups", [(64, 1), (384, 8), (129, 1), (2000, 4)])
@pytest.mark.parametrize("alike", [2, 3, 9])
def test_a_few_picks_near_each_other(mx, score, E, groups, alike):
    """Runs of picks that differ by float32 roundings, others well apart, anywhere
    in the order and over the border of the chosen; and groups that are near."""
    g = gen(E + alike)
    one = torch.randn(E, device="cuda", generator=g)
    s = torch.sigmoid(one.double()) if score == "sigmoid" else torch.softmax(one.double(), 0)
    level = torch.rand(-(-E // alike), device="cuda", generator=g).repeat_interleave(alike)[:E]
    order = torch.randperm(E, device="cuda", generator=g)
    bias = (level[order].double() - s).float()
    logits = one.repeat(9, 1)
    for k in (1, 5, 8, 16):
        for group_score in ("max", "sum2"):
            check(mx, logits, k, score=score, bias=bias, groups=groups, top_groups=max(1, groups // 2),
                  group_score=group_score)
    if groups > 1:      # the groups all alike, in another order each
        size = E // groups
        first, fs = one[:size], s[:size]
        bias = torch.cat([(torch.rand(size, device="cuda", generator=gen(5)).double() - fs).float()] * groups)
        shuffled = torch.cat([torch.arange(size, device="cuda").roll(3 * i) + i * size for i in range(groups)])
        logits = first.repeat(groups)[shuffled].repeat(3, 1) if score == "sigmoid" else logits[:3]
        check(mx, logits, 8, score=score, bias=bias[shuffled], groups=groups, top_groups=groups // 2, group_score="sum2")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_logits_that_are_not_finite_are_out(mx, dtype, score):
    logits = torch.randn(8, 40, device="cuda", generator=gen(6)).to(dtype)
    logits[0] = -math.inf
    logits[1, 1:] = -math.inf
    logits[2, ::2] = math.nan
    logits[3, 5] = math.inf
    logits[4, :37] = -math.inf
    logits[5] = math.nan
    logits[6, 10:] = -math.inf
    bias = torch.randn(40, device="cuda", generator=gen(7))
    for kw in ({}, {"bias": bias}, {"groups": 4, "top_groups": 2},
               {"bias": bias, "groups": 4, "top_groups": 3, "group_score": "sum2"}, {"renormalize": False}):
        ids, w = check(mx, logits, 6, score=score, **kw)
        assert (ids[0] == -1).all() and (w[0] == 0).all() and (ids[5] == -1).all()
        assert ids[1, 0] == 0 and (ids[1, 1:] == -1).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_values_far_apart(mx, score):
    """Logits and biases of any size; weights of small sigmoids do not vanish."""
    big = torch.tensor([[3e38, -3e38, 1e30, 0.0, -80.0, 88.0], [-100.0, -101.0, -102.0, -300.0, -90.5, -91.0],
                        [1e-40, -1e-40, 0.0, 2e-40, 1.0, -1.0]], device="cuda")
    _, w = check(mx, big, 3, score=score)
    assert (w.sum(1) - 1).abs().max() < 1e-6
    check(mx, big, 6, score=score, renormalize=False)
    bias = torch.tensor([1e30, -1e30, 5.0, -5.0, 1e-30, math.inf], device="cuda")
    ids, _ = check(mx, big, 6, score=score, bias=bias)
    assert not (ids == 5).any()


def test_rows_with_a_stride_and_outputs_at_odd_places(mx):
    whole = torch.randn(50, 100, device="cuda", generator=gen(8)).to(torch.bfloat16)
    logits = whole[:, 7:66]
    ids, w = torch.full((302,), 77, dtype=torch.int32, device="cuda"), torch.full((303,), 5.0, device="cuda")
    mx.mxfp4_moe_topk(logits, 6, ids[1:301].view(50, 6), w[2:302].view(50, 6), score="sigmoid")
    want, ww, bound = L.topk(logits, 6, score="sigmoid")
    assert torch.equal(ids[1:301].view(50, 6), want)
    assert ((w[2:302].view(50, 6).double() - ww).abs() <= bound).all()
    assert ids[0] == 77 and ids[301] == 77 and (w[:2] == 5).all() and w[302] == 5


def test_no_tokens(mx):
    ids, w = mx.moe_topk(torch.zeros(0, 16, device="cuda"), 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)


def test_refusals(mx):
    x = torch.zeros(4, 16, device="cuda")
    for kw in ({"top_k": 17}, {"top_k": 0}, {"top_k": 4, "groups": 3}, {"top_k": 4, "groups": 4, "top_groups": 5},
               {"top_k": 4, "scale": math.nan}):
        with pytest.raises(mx.MXFP4Error):
            mx.moe_topk(x, **kw)
    with pytest.raises(ValueError, match="score"):
        mx.moe_topk(x, 4, score="tanh")
    with pytest.raises(ValueError, match="group_score"):
        mx.moe_topk(x, 4, group_score=2)
    with pytest.raises(ValueError, match="bias"):
        mx.moe_topk(x, 4, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(ValueError, match="ids"):
        mx.moe_topk(x, 4, ids=torch.zeros(4, 4, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="logits"):
        mx.moe_topk(x.double(), 4)
