"""The workspace of long texts: a place for each segment that a sequence may have,
or by tokens where that makes fewer, and nothing written behind it."""
import numpy as np
import pytest
import torch

import deterministic_w8a8_int8_gb300 as prism
from tests.test_gpu_linear_attention import check, dev, index, make, offsets, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,hk,hv,dim", [([6000, 5200], 2, 8, 64), ([5100, 3, 17, 5000, 4900], 1, 8, 128), ([20100], 1, 2, 64)],
                         ids=lambda x: str(x))
def test_places_by_sequence(lens, hk, hv, dim):
    """More tokens than the segments that they may be cut into hold: against the recurrence,
    in a workspace of just the size asked for."""
    data = make(31, lens, hk, hv, dim, dim)
    n = len(lens)
    size = prism.prism_linear_attention_workspace_bytes(n, sum(lens), max(lens), hv, dim, dim)
    buf = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
    state = np.random.default_rng(13).standard_normal((n, hv, dim, dim)).astype(np.float32)
    dstate = dev(state, torch.float32)
    own = index(list(range(n)))
    got = run(data, lens, dstate, own, own, workspace=buf[:size])
    assert bool((buf[size:] == 255).all())
    check(data, lens, state, got, dstate)


def test_bits_do_not_depend_on_where_places_lie():
    """The same texts beside many short ones (places by tokens), by themselves (by sequence) and alone."""
    long, short = [9000, 8800], [1] * 12
    lens = long + short
    data = [dev(x) for x in make(32, lens, 8, 40, 64, 64)[:3]]
    g = -torch.rand((sum(lens), 40), device="cuda") * 0.1
    n = len(lens)
    state = torch.randn((n, 40, 64, 64), device="cuda")
    own = index(list(range(n)))
    size = prism.prism_linear_attention_workspace_bytes
    assert size(2, 17800, 9000, 40, 64, 64) < size(14, 17812, 9000, 40, 64, 64)

    def call(first, last):
        at, end = sum(lens[:first]), sum(lens[:last])
        mine = state.clone()
        out = prism.prism_linear_attention(*(x[at:end] for x in data), g[at:end], mine, own[first:last], own[first:last],
                                           cu=offsets(lens[first:last]), max_len=9000)
        return out, mine

    out, after = call(0, n)
    for first, last in ((0, 2), (0, 1), (1, 2), (1, n)):
        at, end = sum(lens[:first]), sum(lens[:last])
        got, mine = call(first, last)
        assert torch.equal(got, out[at:end]) and torch.equal(mine[first:last], after[first:last])
