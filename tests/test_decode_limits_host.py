"""The decode-step calls at the largest sizes that they accept.  No GPU: an
accepted call stops at the missing workspace."""
import pytest

from tests.test_decode_host import L, append, attention   # noqa: F401  (L: the fixture)

UNSUPPORTED, NO_WORKSPACE = -3, -4


@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_longest_text(L, block):   # noqa: F811
    """Positions a little past the end have to fit 32 bits."""
    most = ((1 << 31) - (1 << 14)) // block
    kw = dict(block=block, ws=None, ws_bytes=0)
    assert attention(L, max_pages=most, ld_table=most, **kw) == NO_WORKSPACE
    for pages in (most + 1, ((1 << 31) - 1) // block, (1 << 31) // block):
        assert attention(L, max_pages=pages, ld_table=pages, **kw) == UNSUPPORTED
        assert append(L, max_pages=pages, ld_table=pages, block=block) == UNSUPPORTED


@pytest.mark.parametrize("rows", [1 << 31, 1 << 47, (1 << 62) + 4])
def test_most_queries(L, rows):   # noqa: F811
    assert attention(L, T=rows, cu=0x10000, Hq=1 << 16, H=1 << 10, ldq_t=1 << 23, ldo_t=1 << 23) == UNSUPPORTED
    assert attention(L, T=rows, cu=0x10000) == UNSUPPORTED
