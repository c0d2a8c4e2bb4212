"""Products of 4-bit operands at values where a float32 step could leave the
formula: global scales far apart."""
import pytest
import torch

import decode_reference as R
import layer_reference as L
from test_gpu_gemm import BF, gen, operand

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
