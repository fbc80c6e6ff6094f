"""Attention with queries that are not numbers, and with queries and scales at
the ends of their ranges, in either kernel."""
import numpy as np
import pytest
import torch

from tests import decode_util as du
from tests.test_gpu_kv_attention import _case, _check, _run

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


@pytest.mark.parametrize("power", [-100, 100, 117, 123])
@pytest.mark.parametrize("counts", [[1, 1], [5, 2], [20, 9]], ids=["one", "few", "many"])
def test_large_queries_on_small_keys(cuda_device, counts, power):
    """Queries of 2^p on keys of 2^-p: the scores are ordinary ones."""
    lens = [50, 300]
    cache, table, q, _ = _case(21, 4, 2, 64, 16, lens, counts)
    q = (q.float() * 2.0 ** power).to(torch.bfloat16)
    cache[2] = (cache[2].astype(np.float64) * 2.0 ** -power).astype(np.float32)
    got, lse = _run(cache, table, lens, q, counts)
    _check(got, lse, du.attention(q.double().numpy(), cache, table, lens, counts, 16, 0.125))
