"""Products of 4-bit operands at values where a float32 step could leave the
formula: global scales far apart, scales at the ends of their range,
activations where they are small."""
import math

import pytest
import torch

import decode_reference as R
import layer_reference as L
from test_gpu_gemm import BF, FP, gen, operand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import mxfp4_block_quantization_gb300 as m
    return m


# the tokens' and the weights' global scale: one's inverse overflows the sums that
# the other's brings back, one of them is subnormal or its inverse is, both at one end
PAIRS = [(2.0 ** -120, 2.0 ** 120), (2.0 ** 120, 2.0 ** -120), (1e-30, 3e30), (2.0 ** -127, 2.0 ** 126),
         (2.0 ** -140, 2.0 ** 127), (2.0 ** 127, 2.0 ** -149), (-2.0 ** -115, 1.7 * 2.0 ** 112),
         (2.0 ** -149, 2.0 ** -149), (2.0 ** 127, 2.0 ** 127), (2.0 ** 70, 2.0 ** 55), (2.0 ** -80, 2.0 ** -30)]


@pytest.mark.parametrize("a,b", PAIRS)
@pytest.mark.parametrize("T,K", [(5, 128), (140, 128), (5, 1024)])
@pytest.mark.parametrize("gate", [None, "first"])
def test_global_scales_at_any_distance(mx, a, b, T, K, gate):
    """sum / a / b wherever that is a number of y's type: the product of the
    scales (2^-24), its fast inverse (2^-23) and two products (2^-24 each) are within the
    sum's own bound of (K + 8) 2^-23, and the last may be a subnormal's half step, 2^-150."""
    g = gen(21)
    N = 96
    (xc, xs), (wc, ws) = operand(T, K, True, g), operand(N, K, True, g)
    xc[1], wc[3], wc[51] = 0, 0, 0
    ga, gb = torch.tensor([a], device="cuda"), torch.tensor([b], device="cuda")
    y = mx.gemm_nvfp4(xc, xs, ga, wc, ws, gb, gate=gate)
    x, w = (R.weights(c, s, True) for c, s in ((xc, xs), (wc, ws)))
    z, off = x @ w.T / a / b, (K + 8) * 2.0 ** -23 * (x.abs() @ w.abs().T) / abs(a) / abs(b) + 2.0 ** -150
    if gate:
        h = N // 2
        off = off[:, :h] * z[:, h:].abs() + z[:, :h].abs() * off[:, h:] + off[:, :h] * off[:, h:]
        z = z[:, :h] * z[:, h:]
        off = off + 2.0 ** -24 * z.abs() + 2.0 ** -150
        # (a factor may overflow, or vanish, where the product is a number: not asked)
        there = torch.isfinite(y) & (off > 2.0 ** -149)
    else:
        assert (y[1] == 0).all() and (y[:, 3] == 0).all()
        there = torch.ones_like(y, dtype=torch.bool)
    L.close(y[there], z[there], (off + R.unit(BF) * (z.abs() + off) + R.smallest(BF))[there])


@pytest.mark.parametrize("T", [5, 140])
@pytest.mark.parametrize("far", [60, 100, 120, 127])
def test_scales_at_the_ends_of_their_range(mx, T, far):
    """Scales of 2^far beside scales of 2^-far, whose products are ordinary."""
    g = gen(22)
    K, N = 256, 140
    (xc, xs), (wc, ws) = operand(T, K, False, g, pad=127), operand(N, K, False, g, pad=127)
    xs[:], ws[:] = 127 + far, 127 - far
    y = mx.gemm(xc, xs, wc, ws)
    want, bound = L.gemm(R.elements(xc), R.elements(wc), BF)
    L.close(y, want, bound)
    y = mx.gemm(wc, ws, xc, xs)
    L.close(y, want.T, bound.T)


def values(act):
    lo = {"silu": -87.0, "gelu": -13.0, "gelu_tanh": -10.0}[act]
    return torch.cat((torch.linspace(lo, 0, 1500), torch.linspace(0, 12, 500), -torch.logspace(-4, 0, 48)))


def exactly(z, act):
    """act(z) in 64 bits without cancellation: of the tails, not of 1 minus them."""
    z = z.double()
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z * math.sqrt(0.5))
    return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gate", [None, "first", "second"])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_activations_relative_to_their_own_size(mx, act, gate, dtype):
    """act(z) alone (no terms, z from the bias), relative to itself: a half step of
    y's type and 2^-14.  The exponential's argument, up to 88, is off by 5.5 float32
    roundings at most (2^-24 of it each: two of z^3, its factor, the sum, log2 e and its
    product), 2^-15, and the rest by 2^-19.  An intermediate below 2^-126 may count as 0:
    2^-119 of a result."""
    z = values(act).to(dtype).cuda()
    one = torch.ones_like(z)
    bias = {None: z, "first": torch.cat((z, one)), "second": torch.cat((one, z))}[gate].contiguous()
    T, N = 3, bias.numel()
    none = torch.zeros(0, dtype=torch.uint8, device="cuda")
    y = mx.gemm(none.new_zeros(T, 0), none, none.new_zeros(N, 0), none, bias=bias, activation=act, gate=gate,
                out_dtype=dtype)
    want = exactly(z, act).expand(T, -1)
    bound = (R.unit(dtype) + 2.0 ** -14) * want.abs() + R.smallest(dtype) + 2.0 ** -119
    R.close(y, want, bound)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_gelu_at_the_ends(mx, dtype):
    """Infinities keep their limits, infinity and 0, and NaN stays NaN."""
    bias = torch.tensor([math.inf, -math.inf, math.nan, 0.0, -0.0, 60000.0, -60000.0], dtype=dtype, device="cuda")
    none = torch.zeros(0, dtype=torch.uint8, device="cuda")
    y = mx.gemm(none.new_zeros(2, 0), none, none.new_zeros(7, 0), none, bias=bias, activation="gelu", out_dtype=dtype)
    want = torch.tensor([math.inf, 0.0, math.nan, 0.0, 0.0, float(bias[5]), 0.0], device="cuda").expand(2, -1)
    R.close(y, want, torch.zeros_like(want))
