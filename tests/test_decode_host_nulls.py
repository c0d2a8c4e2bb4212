"""Tensors that the decode calls read without any work, for the status word alone:
NULL is refused before anything is launched."""
import pytest

from test_decode_host import A, caller, lib  # noqa: F401


@pytest.mark.parametrize("without", [dict(Hq=0), dict(Hq=0, D=0), dict(D=0)])
@pytest.mark.parametrize("tail", ["", "_f16"])
def test_the_status_word_needs_lengths_and_pages(lib, without, tail):  # noqa: F811
    names = "q B Hq D qs qh kc ks vc vs P S H tab ts mp len scale win ws wsb out lse status st"
    call = caller(getattr(lib._lib, "mxfp4_cache_attention" + tail), names,
                  [A, 3, 8, 64, 512, 64, 2 * A, 3 * A, 4 * A, 5 * A, 9, 16, 2, 6 * A, 4, 4, 7 * A, 0.1, 0, 8 * A,
                   1 << 31, 9 * A, 10 * A, 11 * A, None])
    assert call(**without, len=None) == lib.MXFP4_EINVAL
    assert call(**without, tab=None) == lib.MXFP4_EINVAL
    assert call(**without, len=None, tab=None, status=None) == lib.MXFP4_OK      # nothing is read
    assert call(**without, B=2 ** 31, tab=None, len=None) == lib.MXFP4_ESHAPE
