"""The decode-step calls through the bounds-checking build of the library: the
same bytes as the normal build, and no access outside a buffer; and the
example that runs them together."""
import contextlib
import os
import sys

import pytest
import torch

import workloads as W
from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def libs():
    assert torch.cuda.is_available()
    import mxfp4_block_quantization_gb300 as mx
    dbg = mx._load(mx.DEBUG_LIB_PATH)
    assert dbg.mxfp4_debug_bounds_violations() == 0
    return mx, mx._lib, dbg


@contextlib.contextmanager
def using(mx, lib):
    saved = mx._lib
    mx._lib = lib
    try:
        yield
    finally:
        mx._lib = saved


def check(libs, fn):
    mx, rel, dbg = libs
    got = []
    for lib in (rel, dbg):
        with using(mx, lib):
            got.append([t.cpu().clone() for t in fn()])
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert dbg.mxfp4_debug_bounds_violations() == 0


def rand(shape, seed, dtype=torch.bfloat16):
    return W.normal_bf16(shape, seed, device="cuda").to(dtype)


@pytest.mark.parametrize("T,N,K", [(1, 1, 32), (9, 200, 2880), (16, 300, 7168), (40, 33, 96),
                                   (3, 4097, 512), (4, 64, 16), (7, 130, 272)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_matvec_in_bounds(libs, T, N, K, dtype):
    mx = libs[0]
    x = rand((T, K), 1, dtype)
    w = rand((N, K), 2)
    g = torch.tensor([300.0], device="cuda")
    if K % 32 == 0:
        c, s = mx.quantize(w)
        check(libs, lambda: (mx.matvec(x, c, s),))
        wide = rand((T, K + 64), 3, dtype)
        check(libs, lambda: (mx.matvec(wide[:, 32:K + 32], c, s, out_dtype=torch.float32),))
    nc, ns = mx.quantize_nvfp4(w, g)
    check(libs, lambda: (mx.matvec_nvfp4(x, nc, ns, g),))


def test_matvec_by_block_in_bounds(libs):
    """x whose rows need a factor for every block."""
    mx = libs[0]
    e = torch.randint(-100, 100, (9, 2880), device="cuda")
    x = (rand((9, 2880), 1).float() * torch.exp2(e.float())).bfloat16()
    c, s = mx.quantize(rand((300, 2880), 2))
    check(libs, lambda: (mx.matvec(x, c, s, out_dtype=torch.float32),))


@pytest.mark.parametrize("offsets", [[0, 0, 5, 5, 30, 33], [0, 33, 33, 33, 33, 33], [0, 0, 0, 0, 0, 0],
                                     [0, 1, 2, 3, 4, 4], [0, 40, 2, 3, 4, 4]])
def test_moe_matvec_in_bounds(libs, offsets):
    mx = libs[0]
    E, N, K = 5, 200, 288
    q = [mx.quantize(rand((N, K), e)) for e in range(E)]
    codes, scales = torch.stack([c for c, _ in q]), torch.cat([s for _, s in q])
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    rows = torch.randint(-1, 13, (33,), device="cuda").to(torch.int32)     # some out of range
    x = rand((12, K), 9)

    def call(index, src):
        y = torch.zeros((33, N), dtype=torch.bfloat16, device="cuda")
        return mx.moe_matvec(src, index, off, codes, scales, out=y)

    check(libs, lambda: call(rows, x))
    check(libs, lambda: call(None, rand((33, K), 4)))


@pytest.mark.parametrize("H,D,S", [(1, 32, 1), (5, 96, 7), (2, 256, 16), (3, 160, 33)])
@pytest.mark.parametrize("nvfp4", [False, True])
def test_cache_and_attention_in_bounds(libs, H, D, S, nvfp4):
    mx = libs[0]
    g = (torch.tensor([300.0], device="cuda"),) * 2 if nvfp4 else ()
    pages, T = 12, 60
    slots = torch.randperm(pages * S, device="cuda")[:T].to(torch.int32)
    slots[::7] = -1
    slots[3] = pages * S + 5
    n = slots.numel()
    kv = rand((n, 2, H, D), 1)
    table = torch.stack([torch.randperm(pages, device="cuda") for _ in range(4)]).to(torch.int32)
    table[2, 1] = 99
    lens = torch.tensor([pages * S, 1, min(3 * S, pages * S), 0], dtype=torch.int32, device="cuda")
    q = rand((4, 3 * H, D), 2)

    def run(window):
        c = mx.cache_alloc(pages, S, H, D, *g)
        st = mx.cache_write(kv[:, 0], kv[:, 1], slots, c)
        k, v, st2 = mx.cache_read(c, slots)
        o, lse, st3 = mx.cache_attention(q, c, table, lens, 0.1, window=window)
        return (*c[:4], st, k, v, st2, o, lse, st3)

    check(libs, lambda: run(0))
    check(libs, lambda: run(5))


def test_decode_step_example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import decode_step
    finally:
        sys.path.pop(0)
    # BF16 activations between the calls: each of about ten roundings adds up to
    # 2^-8 of its value, some of them by chance of one sign
    assert decode_step.main(sequences=4, steps=20) < 10 * 2.0 ** -8
