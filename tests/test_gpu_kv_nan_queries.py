"""Attention with a query that is not a number, in either kernel."""
import pytest
import torch

from tests.test_gpu_kv_attention import _case, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,counts", [([40], [2]), ([5000], [2]), ([40], [20]), ([5000], [20])],
                         ids=["few", "few, pieces", "many", "many, pieces"])
def test_a_query_that_is_not_a_number(cuda_device, lens, counts):
    """Its row and log-sum are NaN; the other rows are as without it."""
    cache, table, q, _ = _case(3, 4, 2, 64, 16, lens, counts)
    want, want_lse = _run(cache, table, lens, q, counts)
    spoilt = q.clone()
    spoilt[1, 2, 5] = float("nan")
    got, lse = _run(cache, table, lens, spoilt, counts)
    assert got[1, 2].isnan().all() and bool(lse[1, 2].isnan())
    rest = torch.ones(lse.shape, dtype=torch.bool, device="cuda")
    rest[1, 2] = False
    assert torch.equal(got[rest], want[rest]) and torch.equal(lse[rest], want_lse[rest])
