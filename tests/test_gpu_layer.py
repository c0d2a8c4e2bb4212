"""A mixture-of-experts layer over many tokens with every step in the library
(router, dispatch, quantize, products, way back), step by step against the 64-bit
forms; the same calls on other streams, captured and replayed, and through the
bounds-checking build."""
import pytest
import torch

import decode_reference as R
import layer_reference as L
import workloads as W
from test_gpu_decode_bounds import check, libs, rand  # noqa: F401

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def mx():
    import mxfp4_block_quantization_gb300 as m
    return m


class Layer:
    """Weights of E experts, quantized once, w13 swapped to [w3; w1]."""

    def __init__(self, mx, E=12, hidden=256, width=192, top_k=3, nv=False):
        self.mx, self.E, self.hidden, self.width, self.top_k, self.nv = mx, E, hidden, width, top_k, nv
        self.router = rand((E, hidden), 1).float() * hidden ** -0.5
        self.bias = rand((E,), 2).float() * 0.05
        w13, w2 = rand((E, 2 * width, hidden), 3) * hidden ** -0.5, rand((E, hidden, width), 4) * width ** -0.5
        self.b13, self.b2 = rand((E, 2 * width), 5) * 0.1, rand((E, hidden), 6) * 0.1
        self.g13, self.g2, self.gx, self.gh = (
            (torch.linspace(lo, 2 * lo, E, device="cuda") for lo in (2000.0, 2000.0, 400.0, 150.0)) if nv else [None] * 4)
        self.w13, self.w2 = (self.weights(w, g) for w, g in ((w13, self.g13), (w2, self.g2)))
        if not nv:
            codes, scales, b, _ = mx.swap_w13(*self.w13, self.b13.float())
            self.w13, self.b13 = (codes, scales), b

    def weights(self, w, g):
        q = [self.mx.quantize(e) if g is None else self.mx.quantize_nvfp4(e, g[i:i + 1]) for i, e in enumerate(w)]
        return torch.stack([c for c, _ in q]), torch.cat([s for _, s in q])

    def run(self, x, stream=None):
        """Every step's outputs, the layer's last."""
        mx, s = self.mx, stream
        ids, w = mx.moe_topk(self.logits(x), self.top_k, score="sigmoid", bias=self.bias, scale=2.5, stream=s)
        off, dest, _, _ = mx.moe_route(ids, self.E, stream=s)
        gate = "first" if self.nv else "second"
        if self.nv:
            xc, xs, _, _ = mx.quantize_nvfp4_grouped_scatter(x, dest, off, self.gx, stream=s)
            h, st1 = mx.moe_gemm_nvfp4(xc, xs, self.gx, off, *self.w13, self.g13, bias=self.b13, activation="silu", gate=gate, stream=s)
            hc, hs, _, _ = mx.quantize_nvfp4_grouped(h, off, self.gh, stream=s)
            rows, st2 = mx.moe_gemm_nvfp4(hc, hs, self.gh, off, *self.w2, self.g2, bias=self.b2, stream=s)
        else:
            xc, xs, _, _ = mx.quantize_grouped_scatter(x, dest, off, stream=s)
            h, st1 = mx.moe_gemm(xc, xs, off, *self.w13, bias=self.b13, activation="silu", gate=gate, stream=s)
            hc, hs, _, _ = mx.quantize_grouped(h, off, stream=s)
            rows, st2 = mx.moe_gemm(hc, hs, off, *self.w2, bias=self.b2, stream=s)
        y, st3 = mx.moe_combine(rows, dest, w, residual=x, stream=s)
        return dict(ids=ids, w=w, off=off, dest=dest, xc=xc, xs=xs, h=h, hc=hc, hs=hs, rows=rows, st=(st1, st2, st3), y=y)

    def logits(self, x):
        return x.float() @ self.router.T

    def segment(self, o, codes, scales, g, e):
        """The values of expert e's rows from the grouped calls' codes and scales."""
        off = o["off"].tolist()
        first = sum(-(-(off[i + 1] - off[i]) // 128) for i in range(e))
        per = 512 * -(-(2 * codes.shape[1]) // (64 if self.nv else 128))
        return R.weights(codes[off[e]:off[e + 1]], scales[first * per:], self.nv, 1.0 if g is None else g[e])

    def check(self, x, o):
        assert all(int(st) == 0 for st in o["st"])
        ids, w, bound = L.topk(self.logits(x), self.top_k, score="sigmoid", bias=self.bias, scale=2.5)
        assert torch.equal(o["ids"], ids) and ((o["w"].double() - w).abs() <= bound).all()
        off = o["off"].tolist()
        for e in range(self.E):
            at = slice(off[e], off[e + 1])
            if off[e] == off[e + 1]:
                continue
            per13, per2 = (t[1].numel() // self.E for t in (self.w13, self.w2))
            w13 = R.weights(self.w13[0][e], self.w13[1][e * per13:], self.nv, 1.0 if not self.nv else self.g13[e])
            w2 = R.weights(self.w2[0][e], self.w2[1][e * per2:], self.nv, 1.0 if not self.nv else self.g2[e])
            L.close(o["h"][at], *L.gemm(self.segment(o, o["xc"], o["xs"], self.gx, e), w13, BF, self.b13[e], "silu",
                                        "first" if self.nv else "second"))
            L.close(o["rows"][at], *L.gemm(self.segment(o, o["hc"], o["hs"], self.gh, e), w2, BF, self.b2[e]))
        L.close(o["y"], *L.combine(o["rows"], o["dest"], o["w"], BF, x))


@pytest.mark.parametrize("nv", [False, True])
@pytest.mark.parametrize("T", [1, 7, 300])
def test_layer(mx, nv, T):
    layer = Layer(mx, nv=nv)
    x = rand((T, layer.hidden), 10 + T)
    layer.check(x, layer.run(x))


def test_routes_that_are_not_dispatched(mx):
    """Experts closed to a token leave routes of -1, which nothing after takes."""
    layer = Layer(mx)
    x = rand((50, layer.hidden), 20)
    closed = torch.full((50, layer.E), float("-inf"), device="cuda")
    closed[:, 3:5] = 0.0
    closed[7] = float("-inf")
    plain = layer.logits
    layer.logits = lambda t: plain(t) + closed
    o = layer.run(x)
    assert (o["ids"][:, 2] == -1).all() and int(o["off"][-1]) == 98
    assert torch.equal(o["y"][7], x[7])
    layer.check(x, o)


@pytest.mark.parametrize("nv", [False, True])
def test_captured_and_replayed(mx, nv):
    layer = Layer(mx, nv=nv)
    x = rand((40, layer.hidden), 30)
    want = [layer.run(rand((40, layer.hidden), 31 + i))["y"].clone() for i in range(3)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer.run(x)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = layer.run(x)
    for i in range(3):
        x.copy_(rand((40, layer.hidden), 31 + i))
        g.replay()
        assert torch.equal(o["y"], want[i])


@pytest.mark.parametrize("name", ["topk", "gemm", "split", "moe_gemm", "combine"])
def test_calls_on_two_streams_at_once(mx, name):
    """Equal calls on two streams, beside work on the current one."""
    layer = Layer(mx, E=6, hidden=512, width=128)
    T = 400
    xs = [rand((T, layer.hidden), 40 + i) for i in range(2)]
    o = [layer.run(x) for x in xs]
    logits = [layer.logits(x) for x in xs]
    dense = mx.quantize(rand((1500, 2048), 42))
    few = [mx.quantize(rand((T if name == "gemm" else 3, 2048), 43 + i)) for i in range(2)]
    call = {
        "topk": lambda i, s: mx.moe_topk(logits[i], 3, bias=layer.bias, stream=s),
        "gemm": lambda i, s: (mx.gemm(*few[i], *dense, activation="gelu", stream=s),),
        "split": lambda i, s: (mx.gemm(*few[i], *dense, stream=s),),
        "moe_gemm": lambda i, s: mx.moe_gemm(o[i]["xc"], o[i]["xs"], o[i]["off"], *layer.w13, gate="second", activation="silu", stream=s),
        "combine": lambda i, s: mx.moe_combine(o[i]["rows"], o[i]["dest"], o[i]["w"], stream=s),
    }[name]
    want = [[t.clone() for t in call(i, None)] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got, other = [], []
    for i in range(24):
        got.append(call(i % 2, streams[i // 2 % 2]))
        other.append(torch.full((want[0][0].numel() * want[0][0].element_size(),), i, dtype=torch.uint8, device="cuda"))
        if i % 5 == 4:
            del other[-3:]
    torch.cuda.synchronize()
    for i, outputs in enumerate(got):
        for a, b in zip(outputs, want[i % 2]):
            assert torch.equal(a, b)
    for t in other:
        assert (t == t[0]).all()


# ------------------------------------------------- the bounds-checking build
@pytest.mark.parametrize("nv", [False, True])
@pytest.mark.parametrize("T", [3, 150])
def test_layer_in_bounds(libs, nv, T):  # noqa: F811
    layer = Layer(libs[0], nv=nv)
    x = rand((T, layer.hidden), 50 + T)

    def steps():
        o = layer.run(x)
        return [o["ids"], o["w"], o["h"][:int(o["off"][-1])], o["rows"][:int(o["off"][-1])], o["y"]]

    check(libs, steps)


@pytest.mark.parametrize("T,N,K", [(1, 1, 32), (3, 130, 7168), (129, 257, 96), (300, 514, 288), (64, 1024, 1024)])
@pytest.mark.parametrize("nv", [False, True])
@pytest.mark.parametrize("dtype", [BF, torch.float16])
def test_gemm_in_bounds(libs, T, N, K, nv, dtype):  # noqa: F811
    mx = libs[0]
    g = [torch.tensor([v], device="cuda") for v in (400.0, 900.0)]
    quantize = (lambda t, i: mx.quantize_nvfp4(t, g[i])) if nv else (lambda t, i: mx.quantize(t))
    xq, wq = quantize(rand((T, K), 1), 0), quantize(rand((N, K), 2), 1)
    bias, residual = rand((N,), 3, dtype), rand((T, N + 3), 4, dtype)

    def call(**kw):
        kw["out_dtype"] = dtype
        return mx.gemm_nvfp4(*xq, g[0], *wq, g[1], **kw) if nv else mx.gemm(*xq, *wq, **kw)

    check(libs, lambda: [call(bias=bias, residual=residual[:, 1:N + 1]), call(activation="gelu")])
    if N % 2 == 0:
        check(libs, lambda: [call(bias=bias, gate="second", activation="silu", residual=residual[:, :N // 2]), call(gate="first")])


@pytest.mark.parametrize("T,E,k,groups", [(1, 1, 1, 1), (9, 129, 5, 3), (5, 384, 8, 8), (3, 1030, 4, 2), (2, 8192, 32, 32)])
@pytest.mark.parametrize("dtype", [BF, torch.float16, torch.float32])
def test_topk_in_bounds(libs, T, E, k, groups, dtype):  # noqa: F811
    mx = libs[0]
    logits, bias = rand((T, E + 1), 5).to(dtype)[:, :E], rand((E,), 6).float()
    aligned = rand((T, E), 7).to(dtype)
    for x in (logits, aligned):
        check(libs, lambda: mx.moe_topk(x, k))
        check(libs, lambda: mx.moe_topk(x, k, score="sigmoid", bias=bias, groups=groups, top_groups=max(1, groups // 2),
                                        group_score="sum2"))
        check(libs, lambda: mx.moe_topk(torch.zeros_like(x), k, bias=torch.zeros_like(bias), groups=groups,
                                        top_groups=max(1, groups // 2)))


@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (5, 3, 40), (9, 4, 2047), (3, 9, 4096)])
@pytest.mark.parametrize("f32", [False, True])
def test_combine_in_bounds(libs, T, k, N, f32):  # noqa: F811
    mx = libs[0]
    rows = rand((T * k, N), 8).to(torch.float32 if f32 else BF)
    dest = torch.randperm(T * k, generator=torch.Generator().manual_seed(1)).view(T, k).to(torch.int32).cuda()
    dest[0, 0] = -1
    dest[-1, -1] = T * k if T > 1 else -1
    w = W.normal_bf16((T, k), 9, device="cuda").float()
    check(libs, lambda: mx.moe_combine(rows, dest, w, residual=rand((T, N), 10), out_dtype=BF))
