"""The attention's workspace: bounded by the call's queries, not by the number of
sequences times the longest one.  No GPU."""
import pytest


@pytest.fixture(scope="module")
def need():
    from deterministic_w8a8_int8_gb300 import build
    build.build()
    import deterministic_w8a8_int8_gb300 as p
    return p.lib().prism_kv_attention_workspace_bytes


@pytest.mark.parametrize("seqs,rows,max_q,max_pages,heads,kv,d,most", [
    (64, 64, 1, 64, 40, 8, 128, 6e6),            # a decode step
    (64, 64, 64, 64, 40, 8, 128, 12e6),          # the same without a bound on a sequence's queries
    (64, 64 + 511, 512, 64, 40, 8, 128, 100e6),  # and one piece of a prompt among them
    (256, 256 + 511, 512, 64, 40, 8, 128, 140e6),
    (256, 256 + 511, 512, 64, 32, 8, 256, 400e6),
    (1, 8192, 8192, 1024, 40, 8, 128, 24e6),     # a prompt by itself
])
def test_sizes(need, seqs, rows, max_q, max_pages, heads, kv, d, most):
    assert 0 < need(seqs, rows, max_q, max_pages, heads, kv, d, 64) <= most


def test_more_of_anything_takes_no_less(need):
    base = dict(seqs=5, rows=40, max_q=20, max_pages=40, heads=16, kv=4, d=128, block=64)
    at = need(*base.values())
    for name, values in (("seqs", (6, 50)), ("rows", (41, 400)), ("max_q", (21, 40)), ("max_pages", (41, 4000))):
        for v in values:
            assert need(*{**base, name: v}.values()) >= at
