"""Attention with queries and key scales at the ends of their ranges, in either kernel."""
import numpy as np
import pytest
import torch

from tests import decode_util as du
from tests.test_gpu_kv_attention import _case, _check, _run

pytestmark = pytest.mark.gpu


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
