"""Host-side checks of the calls of a layer over many tokens: argument
validation returns the documented status before anything reaches the GPU (no
compute call here)."""
import math

import pytest

A = 1 << 32   # fake, 16-byte aligned addresses: validation fails before any use


@pytest.fixture(scope="module")
def lib():
    import mxfp4_block_quantization_gb300 as m
    return m


def caller(fn, names, args):
    def call(**kw):
        a = dict(zip(names.split(), args))
        assert set(kw) <= set(a)
        a.update(kw)
        return fn(*a.values())
    return call


@pytest.mark.parametrize("tail,size", [("", 2), ("_f16", 2), ("_f32", 4)])
def test_topk_validation(lib, tail, size):
    call = caller(getattr(lib._lib, "mxfp4_moe_topk" + tail),
                  "l T E ld bias score G tg sum2 k renorm scale ids w st",
                  [A, 5, 64, 64, 2 * A, 1, 8, 4, 1, 6, 1, 1.0, 3 * A, 4 * A, None])
    assert call(T=-1) == call(E=0) == call(k=0) == call(G=0) == call(tg=0) == lib.MXFP4_EINVAL
    assert call(score=2) == call(score=-1) == call(sum2=2) == call(renorm=3) == lib.MXFP4_EINVAL
    assert call(scale=math.nan) == call(scale=math.inf) == lib.MXFP4_EINVAL
    assert call(l=None) == call(ids=None) == call(w=None) == lib.MXFP4_EINVAL
    assert call(E=8200, ld=8200) == call(k=65) == call(k=33) == call(ld=63) == lib.MXFP4_ESHAPE
    assert call(G=7) == call(tg=9) == call(G=64) == call(T=1 << 31) == lib.MXFP4_ESHAPE
    assert call(ld=1 << 62) == lib.MXFP4_ESHAPE
    assert call(l=A + size // 2) == call(bias=2 * A + 2) == lib.MXFP4_EALIGN
    assert call(ids=3 * A + 2) == call(w=4 * A + 1) == lib.MXFP4_EALIGN
    last = A + (4 * 64 + 64) * size - 4
    assert call(ids=last) == call(w=last) == call(ids=2 * A) == call(w=3 * A + 4) == lib.MXFP4_EALIAS
    assert call(T=0, l=None, ids=None, w=None) == lib.MXFP4_OK


GEMM = "x xs T K c s N bias act gate r ldr y ldy st"
GEMM_ARGS = [A, 2 * A, 5, 64, 3 * A, 4 * A, 40, 5 * A, 1, 0, 6 * A, 40, 7 * A, 40, None]


@pytest.mark.parametrize("tail", ["", "_f16"])
def test_gemm_validation(lib, tail):
    call = caller(getattr(lib._lib, "mxfp4_gemm" + tail), GEMM, GEMM_ARGS)
    assert call(T=-1) == call(K=-32) == call(N=-1) == call(act=4) == call(act=-1) == lib.MXFP4_EINVAL
    assert call(gate=3) == call(gate=-1) == lib.MXFP4_EINVAL
    for name in ("x", "xs", "c", "s", "y"):
        assert call(**{name: None}) == lib.MXFP4_EINVAL
    assert call(K=48) == call(ldy=39) == call(ldr=39) == call(gate=1, N=41) == lib.MXFP4_ESHAPE
    assert call(N=2 ** 31, ldy=2 ** 31, ldr=2 ** 31) == call(T=2 ** 31) == lib.MXFP4_ESHAPE
    assert call(ldy=2 ** 62) == call(ldr=2 ** 62) == call(K=2 ** 31) == lib.MXFP4_ESHAPE
    for name in ("x", "xs", "c", "s"):
        assert call(**{name: dict(zip(GEMM.split(), GEMM_ARGS))[name] + 8}) == lib.MXFP4_EALIGN
    assert call(bias=5 * A + 1) == call(r=6 * A + 1) == call(y=7 * A + 1) == lib.MXFP4_EALIGN
    for base in (A, 2 * A, 3 * A, 4 * A, 5 * A):
        assert call(y=base) == lib.MXFP4_EALIAS
    # the residual may be y, but only element for element
    assert call(y=6 * A + 2) == call(y=6 * A, ldy=42) == lib.MXFP4_EALIAS
    assert call(T=0, x=None, xs=None, y=None, r=None) == lib.MXFP4_OK
    assert call(N=0, c=None, s=None, y=None, r=None) == lib.MXFP4_OK


def test_gemm_nvfp4_validation(lib):
    call = caller(lib._lib.mxfp4_gemm_nvfp4, "x xs xg T K c s g N bias act gate r ldr y ldy st",
                  [A, 2 * A, 8 * A, 5, 64, 3 * A, 4 * A, 9 * A, 40, None, 0, 0, None, 0, 7 * A, 40,
                   None])
    assert call(xg=None) == call(g=None) == lib.MXFP4_EINVAL
    assert call(K=48) == lib.MXFP4_ESHAPE                  # rows of codes in whole 16-byte pieces
    assert call(xg=8 * A + 2) == call(g=9 * A + 1) == lib.MXFP4_EALIGN
    assert call(y=8 * A) == call(y=9 * A) == lib.MXFP4_EALIAS


def test_moe_gemm_validation(lib):
    call = caller(lib._lib.mxfp4_moe_gemm, "x xs rows K off E c s N bias act gate y ldy status st",
                  [A, 2 * A, 50, 64, 10 * A, 4, 3 * A, 4 * A, 40, 5 * A, 0, 2, 7 * A, 20, 11 * A,
                   None])
    assert call(off=None) == call(E=-1) == call(E=0) == call(rows=-1) == lib.MXFP4_EINVAL
    assert call(E=lib.MXFP4_ROUTE_MAX_EXPERTS + 1) == call(N=2 ** 30) == lib.MXFP4_ESHAPE
    assert call(ldy=19) == lib.MXFP4_ESHAPE
    assert call(off=10 * A + 2) == call(status=11 * A + 1) == lib.MXFP4_EALIGN
    assert call(y=10 * A) == call(status=10 * A + 8) == call(status=7 * A + 4) == lib.MXFP4_EALIAS
    assert call(status=2 * A) == call(y=5 * A + 300) == lib.MXFP4_EALIAS


@pytest.mark.parametrize("f32", [0, 1])
def test_combine_validation(lib, f32):
    call = caller(lib._lib.mxfp4_moe_combine, "rows f32 R N ldr d w T k r ldres y ldy status st",
                  [A, f32, 20, 24, 24, 2 * A, 3 * A, 5, 4, 4 * A, 24, 5 * A, 24, 6 * A, None])
    assert call(R=-1) == call(N=-1) == call(T=-1) == call(k=0) == call(f32=2) == lib.MXFP4_EINVAL
    assert call(rows=None) == call(d=None) == call(w=None) == call(y=None) == lib.MXFP4_EINVAL
    assert call(ldr=23) == call(ldy=23) == call(ldres=23) == lib.MXFP4_ESHAPE
    assert call(T=2 ** 30) == call(R=2 ** 32) == call(ldy=2 ** 62) == lib.MXFP4_ESHAPE
    assert call(rows=A + 1 + f32) == call(d=2 * A + 2) == call(w=3 * A + 2) == lib.MXFP4_EALIGN
    assert call(r=4 * A + 1) == call(y=5 * A + 1) == call(status=6 * A + 2) == lib.MXFP4_EALIGN
    assert call(y=A) == call(y=2 * A) == call(y=3 * A) == call(y=4 * A + 2) == lib.MXFP4_EALIAS
    assert call(status=5 * A) == call(status=2 * A) == call(status=4 * A) == lib.MXFP4_EALIAS


def test_python_refusals(lib):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        lib.gemm(x, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        lib.moe_topk(torch.zeros(4, 8), 2)
    with pytest.raises(ValueError, match="CUDA"):
        lib.moe_combine(torch.zeros(4, 8), x[:, :2].int(), torch.zeros(4, 2))
