"""Limits of the operators between a layer's linears that follow from their number
ranges and workspaces.  No GPU: the pointers are never dereferenced."""
import pytest

from tests.test_layer_host import L, linear  # noqa: F401  (L: a fixture)


@pytest.mark.parametrize("scale,status", [(2.0 ** 65, -1), (-2.0 ** 65, -1), (1e30, -1)])
def test_scale(L, scale, status):  # noqa: F811
    """Outputs' factors are the scale times 2^40."""
    assert linear(L, scale=scale) == status


@pytest.mark.parametrize("seqs,rows,max_len,heads,most", [
    (1, 131071, 131071, 40, 8), (1, 1 << 20, 1 << 20, 40, 8), (3, 1 << 20, 1 << 20, 40, 24), (1, 131071, 131071, 8, 19),
    (1, 1 << 20, 1 << 20, 2, 76), (64, 64 * 2048, 2048, 40, 256), (5, 1 << 20, 1536, 40, 15)])
def test_workspace_by_segments(L, seqs, rows, max_len, heads, most):  # noqa: F811
    """A sequence has no more segments than its heads fill SMs with, however long it is."""
    f = L.prism_linear_attention_workspace_bytes
    need = f(seqs, rows, max_len, heads, 128, 128)
    assert 0 < need <= most * heads * (128 * 128 + 4) * 4
    assert linear(L, S=seqs, T=rows, max_len=max_len, hv=heads, hk=heads, ldq_t=heads * 128, ldk_t=heads * 128, ldv_t=heads * 128,
                  ldo_t=heads * 128, ldd=heads, bytes=need - 1) == -4


@pytest.mark.parametrize("kw", [dict(seqs=1 << 62), dict(seqs=(1 << 24) + 1), dict(rows=1 << 31), dict(rows=1 << 62), dict(heads=65536),
                                dict(heads=1 << 40), dict(seqs=1 << 23, heads=64)])
def test_workspace_of_what_is_refused(L, kw):  # noqa: F811
    """No workspace for sizes that the call refuses, rather than one that has wrapped around."""
    d = dict(seqs=4, rows=1 << 20, max_len=1 << 20, heads=40)
    d.update(kw)
    assert L.prism_linear_attention_workspace_bytes(d["seqs"], d["rows"], d["max_len"], d["heads"], 128, 128) == 0
    h = d["heads"]
    assert linear(L, S=d["seqs"], T=d["rows"], max_len=d["max_len"], hv=h, hk=h, ldd=h) == -3
