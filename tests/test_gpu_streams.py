"""Calls on a stream that is not the current one: what they allocate is not shared
with the work of other streams."""
import pytest
import torch

from test_gpu_attention_split import with_room
from test_gpu_cache import filled, mx, rand, tables  # noqa: F401
from test_gpu_matvec import make_experts, make_weights, route

pytestmark = pytest.mark.gpu

SEQS, HEADS, D = 4, 8, 64


def attention_calls(mx):  # noqa: F811
    """(call(i, stream) -> out, lse; bytes of its workspace): three queries over one
    cache, their parts joined through the workspace."""
    c = filled(mx, 300, 16, 2, D, False, 4)
    table = with_room(tables(SEQS, 256, 300, 1), 16)
    n = torch.tensor([4096, 3001, 1, 2500], dtype=torch.int32, device="cuda")
    q = [rand((SEQS, HEADS, D), 5 + i) for i in range(3)]

    def call(i, stream=None):
        return mx.cache_attention(q[i], c, table, n, 0.1, stream=stream)[:2]

    nbytes = mx.mxfp4_cache_attention_workspace_bytes(SEQS, HEADS, 2, D, 16, table.shape[1])
    assert nbytes > 0
    return call, nbytes


def side_streams(count):
    torch.cuda.synchronize()
    return [torch.cuda.Stream() for _ in range(count)]


def test_attention_beside_work_on_the_current_stream(mx):  # noqa: F811
    call, nbytes = attention_calls(mx)
    want = [call(i) for i in range(3)]
    s, = side_streams(1)
    got, other = [], []
    for i in range(30):
        got.append(call(i % 3, s))
        other.append(torch.full((nbytes,), i + 1, dtype=torch.uint8, device="cuda"))
        if i % 4 == 3:
            del other[-3:]                       # freed while the calls run
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 3][0]) and torch.equal(lse, want[i % 3][1])
    for t in other:
        assert (t == t[0]).all()


def test_attention_on_two_streams_at_once(mx):  # noqa: F811
    call, _ = attention_calls(mx)
    want = [call(i) for i in range(3)]
    streams = side_streams(2)
    got = [call(i % 3, streams[i % 2]) for i in range(30)]
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 3][0]) and torch.equal(lse, want[i % 3][1])


def decode_calls(mx):  # noqa: F811
    """name -> call(i, stream) that returns its outputs, for two inputs i."""
    codes, scales, _ = make_weights(mx, 1000, 512, False, 8)
    x = [rand((4, 512), 9 + i) for i in range(2)]
    e_codes, e_scales, _ = make_experts(mx, 6, 200, 512, False, 3)
    off, rows = route(mx, 4, 2, 6, 1)
    c = filled(mx, 30, 16, 2, D, False, 4)
    slots = [torch.randperm(480, device="cuda").to(torch.int32) for _ in range(2)]
    attention, _ = attention_calls(mx)
    return {"matvec": lambda i, s=None: (mx.matvec(x[i], codes, scales, stream=s),),
            "moe_matvec": lambda i, s=None: mx.moe_matvec(x[i], rows, off, e_codes, e_scales, stream=s),
            "cache_read": lambda i, s=None: mx.cache_read(c, slots[i], stream=s),
            "cache_attention": attention}


@pytest.mark.parametrize("name", ["matvec", "moe_matvec", "cache_read", "cache_attention"])
def test_outputs_used_and_freed_on_the_current_stream(mx, name):  # noqa: F811
    """An output of a call on another stream that the current stream still reads
    when it is freed is not the next call's."""
    call = decode_calls(mx)[name]
    want = [t.clone() for t in call(0)]
    s, = side_streams(1)
    here = torch.cuda.current_stream()
    busy = torch.randn(4096, 4096, device="cuda")
    for _ in range(5):
        s.wait_stream(here)
        got = call(0, s)
        here.wait_stream(s)
        for _ in range(4):
            busy = busy @ busy * 1e-4                       # the reads below wait for this
        kept = [t.clone() for t in got]
        del got
        for _ in range(3):
            call(1, s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want))


def quantize_calls(mx):  # noqa: F811
    """name -> call(i, stream) of the calls with a workspace or zeroed outputs."""
    T, k, E, K = 600, 4, 12, 512
    x = [rand((T, K), 20 + i) for i in range(2)]
    ids = [torch.rand((T, E), device="cuda").topk(k, 1).indices.to(torch.int32) for _ in range(2)]
    routes = [mx.moe_route(t, E) for t in ids]
    g = torch.linspace(100.0, 400.0, E, device="cuda")

    def cut(outputs, i):
        """Without the bytes past the last expert's scales, which no call writes."""
        codes, scales, sro, status = outputs
        return codes, scales[:int(routes[i][0][-1])], sro, status

    return {
        "route": lambda i, s=None: mx.moe_route(ids[i], E, stream=s),
        "gather": lambda i, s=None: cut(mx.quantize_grouped_gather(x[i], routes[i][2], routes[i][0], stream=s), i),
        "scatter": lambda i, s=None: mx.quantize_grouped_scatter(x[i], routes[i][1], routes[i][0], stream=s),
        "nvfp4_scatter": lambda i, s=None: mx.quantize_nvfp4_grouped_scatter(x[i], routes[i][1], routes[i][0], g,
                                                                             stream=s),
        "quantize": lambda i, s=None: mx.quantize(x[i], stream=s)}


@pytest.mark.parametrize("name", ["route", "gather", "scatter", "nvfp4_scatter", "quantize"])
def test_quantize_calls_beside_work_on_the_current_stream(mx, name):  # noqa: F811
    call = quantize_calls(mx)[name]
    want = [[t.clone() for t in call(i)] for i in range(2)]
    s, = side_streams(1)
    sizes = [t.numel() * t.element_size() for t in want[0]] + [1 << 16, 1 << 20]
    got, other = [], []
    for i in range(20):
        got.append(call(i % 2, s))
        other += [torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") for n in sizes]
        if i % 4 == 3:
            del other[-2 * len(sizes):]
    torch.cuda.synchronize()
    for i, outputs in enumerate(got):
        for a, b in zip(outputs, want[i % 2]):
            assert torch.equal(a, b)
    for t in other:
        assert (t == 0xA5).all()
