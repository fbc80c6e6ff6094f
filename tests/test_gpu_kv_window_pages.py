"""Attention with a window over a cache whose pages before the window are gone:
their table entries and scales do not matter."""
import numpy as np
import pytest
import torch

from tests import decode_util as du
from tests.test_gpu_kv_attention import _case, _check, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fill", [-1, 1 << 30, "other"], ids=str)
@pytest.mark.parametrize("d,block", [(64, 16), (128, 16), (128, 32), (256, 16), (64, 128)])
@pytest.mark.parametrize("counts", [[1, 1, 1], [5, 1, 7], [70, 45, 33]], ids=["decode", "few", "many"])
def test_pages_before_the_window(cuda_device, counts, d, block, fill):
    lens, window, hq = [1203, 391, 77], 40, 4
    cache, table, q, qf = _case(d + block, hq, 1, d, block, lens, counts)
    want = du.attention(qf.astype(np.float64), cache, table, lens, counts, block, d ** -0.5, window=window)
    gone = table.copy()
    if fill == "other":   # a page in another's use, with values far from these
        cache = [np.concatenate((c, c[:1])) for c in cache]
        spare = cache[0].shape[0] - 1
        cache[2][spare], cache[3][spare] = 1e30, 1e30
    for s, (n, m) in enumerate(zip(lens, counts)):
        first = max(0, n - m + 1 - window)            # of the first query
        gone[s, :first // block] = spare if fill == "other" else fill
    got, lse = _run(cache, gone, lens, q, counts, window=window)
    _check(got, lse, want)
