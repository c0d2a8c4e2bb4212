"""Host-side checks of the decode-step entry points: argument validation
returns the documented status before anything reaches the GPU, and the
workspace query (no compute call here)."""
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


@pytest.mark.parametrize("tail", ["", "_f16"])
def test_matvec_validation(lib, tail):
    call = caller(getattr(lib._lib, "mxfp4_matvec" + tail), "x T K ldx c s N y ldy f32 st",
                  [A, 3, 64, 64, 2 * A, 3 * A, 40, 4 * A, 40, 0, None])
    assert call(T=-1) == call(N=-1) == call(K=-32) == call(f32=2) == lib.MXFP4_EINVAL
    assert call(x=None) == call(c=None) == call(s=None) == call(y=None) == lib.MXFP4_EINVAL
    assert call(K=48, ldx=48) == call(ldx=32) == call(ldy=39) == lib.MXFP4_ESHAPE
    assert call(x=A + 8) == call(c=2 * A + 8) == call(s=3 * A + 4) == lib.MXFP4_EALIGN
    assert call(y=4 * A + 1) == call(y=4 * A + 2, f32=1) == call(ldx=68) == lib.MXFP4_EALIGN
    assert call(y=A + 64) == call(y=2 * A + 64) == call(y=3 * A + 64) == lib.MXFP4_EALIAS
    assert call(T=0, x=None, y=None) == call(N=0, c=None, s=None, y=None) == lib.MXFP4_OK
    assert call(N=2 ** 40, ldy=2 ** 40) == lib.MXFP4_ESHAPE


def test_matvec_nvfp4_validation(lib):
    call = caller(lib._lib.mxfp4_matvec_nvfp4, "x T K ldx c s g N y ldy f32 st",
                  [A, 3, 48, 48, 2 * A, 3 * A, 5 * A, 40, 4 * A, 40, 0, None])
    assert call(g=None) == lib.MXFP4_EINVAL
    assert call(K=40, ldx=40) == lib.MXFP4_ESHAPE
    assert call(g=5 * A + 2) == lib.MXFP4_EALIGN
    assert call(y=5 * A) == lib.MXFP4_EALIAS


def test_moe_matvec_validation(lib):
    call = caller(lib._lib.mxfp4_moe_matvec, "x n K ldx idx rows off E c s N y ldy f32 status st",
                  [A, 3, 64, 64, 6 * A, 12, 7 * A, 4, 2 * A, 3 * A, 40, 4 * A, 40, 0, 8 * A, None])
    assert call(off=None) == call(E=-1) == call(E=0) == call(rows=-1) == lib.MXFP4_EINVAL
    assert call(idx=None) == lib.MXFP4_ESHAPE                    # 3 rows of x for 12 of y
    assert call(E=lib.MXFP4_ROUTE_MAX_EXPERTS + 1) == lib.MXFP4_ESHAPE
    assert call(idx=6 * A + 2) == call(off=7 * A + 1) == call(status=8 * A + 2) == lib.MXFP4_EALIGN
    assert call(y=6 * A) == call(y=7 * A) == call(status=7 * A + 4) == lib.MXFP4_EALIAS
    assert call(status=4 * A + 8) == lib.MXFP4_EALIAS


def test_cache_validation(lib):
    names = "k v T H D kt kh vt vh slots P S kc ks vc vs status st"
    ok = [A, 2 * A, 5, 2, 64, 128, 64, 128, 64, 3 * A, 4, 16, 4 * A, 5 * A, 6 * A, 7 * A, 8 * A,
          None]
    call = caller(lib._lib.mxfp4_cache_write, names, ok)
    assert call(T=-1) == call(H=-1) == call(S=0) == call(P=-1) == lib.MXFP4_EINVAL
    assert call(k=None) == call(slots=None) == call(kc=None) == call(vs=None) == lib.MXFP4_EINVAL
    assert call(kt=-8) == lib.MXFP4_EINVAL
    assert call(D=48) == call(P=2 ** 31, S=1) == call(P=2 ** 28, S=16) == lib.MXFP4_ESHAPE
    assert call(k=A + 8) == call(kt=132) == call(vh=4) == call(kc=4 * A + 8) == lib.MXFP4_EALIGN
    assert call(vc=4 * A + 16) == call(ks=A) == call(status=5 * A) == call(slots=7 * A) == \
        lib.MXFP4_EALIAS
    call = caller(lib._lib.mxfp4_cache_read, "kc ks vc vs P S H D slots T ko vo status st",
                  [4 * A, 5 * A, 6 * A, 7 * A, 4, 16, 2, 64, 3 * A, 5, A, 2 * A, 8 * A, None])
    assert call(ko=None) == call(T=-1) == call(vc=None) == lib.MXFP4_EINVAL
    assert call(D=40) == lib.MXFP4_ESHAPE
    assert call(ko=A + 2) == call(slots=3 * A + 1) == lib.MXFP4_EALIGN
    assert call(ko=2 * A + 64) == call(vo=6 * A) == call(status=3 * A) == lib.MXFP4_EALIAS
    nv = caller(lib._lib.mxfp4_cache_write_nvfp4, names.replace("kc", "kg vg kc", 1),
                ok[:12] + [9 * A, 10 * A] + ok[12:])
    assert nv(kg=None) == nv(vg=None) == lib.MXFP4_EINVAL
    assert nv(kg=4 * A) == lib.MXFP4_EALIAS


def test_attention_validation(lib):
    names = "q B Hq D qs qh kc ks vc vs P S H tab ts mp len scale win ws wsb out lse status st"
    ok = [A, 3, 8, 64, 512, 64, 2 * A, 3 * A, 4 * A, 5 * A, 9, 16, 2, 6 * A, 4, 4, 7 * A, 0.1, 0,
          8 * A, 1 << 31, 9 * A, 10 * A, 11 * A, None]
    call = caller(lib._lib.mxfp4_cache_attention, names, ok)
    assert call(B=-1) == call(win=-1) == call(scale=float("nan")) == call(mp=-1) == lib.MXFP4_EINVAL
    assert call(scale=float("inf")) == call(q=None) == call(out=None) == lib.MXFP4_EINVAL
    assert call(tab=None) == call(len=None) == call(kc=None) == call(qs=-8) == lib.MXFP4_EINVAL
    assert call(Hq=7) == call(D=288) == call(ts=3) == call(mp=2 ** 28, ts=2 ** 28) == \
        lib.MXFP4_ESHAPE
    assert call(q=A + 8) == call(qh=68) == call(out=9 * A + 8) == call(lse=10 * A + 2) == \
        lib.MXFP4_EALIGN
    assert call(out=A) == call(lse=9 * A) == call(status=6 * A) == call(lse=7 * A) == \
        lib.MXFP4_EALIAS
    big = dict(B=1, Hq=8, H=1, mp=8192, ts=8192)
    need = lib.mxfp4_cache_attention_workspace_bytes(1, 8, 1, 64, 16, 8192)
    if need:
        assert call(**big, ws=None) == call(**big, wsb=need - 1) == lib.MXFP4_EINVAL
        assert call(**big, ws=8 * A + 8) == lib.MXFP4_EALIGN
        assert call(**big, ws=4 * A) == lib.MXFP4_EALIAS


def test_attention_workspace_query(lib):
    q = lib.mxfp4_cache_attention_workspace_bytes
    assert q(-1, 8, 1, 64, 16, 10) == q(1, 8, 3, 64, 16, 10) == q(1, 8, 1, 288, 16, 10) == 0
    assert q(1, 8, 1, 48, 16, 10) == q(1, 8, 1, 64, 0, 10) == q(1, 8, 0, 64, 16, 10) == 0
    assert q(1, 8, 1, 64, 16, 2 ** 28) == 0 and q(0, 8, 1, 64, 16, 10) == 0


def test_attention_workspace_of_short_and_long_contexts(lib):
    """Short contexts are joined inside the kernel; long ones need room for the
    parts of 8 heads (16 where a kv head has more and the call is large)."""
    q = lib.mxfp4_cache_attention_workspace_bytes
    assert q(1, 64, 8, 128, 16, 2) == q(1, 64, 8, 128, 16, 44) == q(1, 128, 8, 128, 16, 44) == 0
    for D in (32, 64, 96, 128, 256):
        for heads in (8, 64, 128, 256):
            need = q(1, heads, 8, D, 16, 8192)
            assert need > 0 and need % 4 == 0
            assert q(2, heads, 8, D, 16, 8192) >= need
