"""Attention of many rows whose lines of blocks are cut inside of tiles, at
their ends and past them: against the 64-bit statement, and whatever the batch
and the order of its sequences."""
import numpy as np
import pytest
import torch

from tests import decode_util as du
from tests.test_gpu_kv_attention import _case, _check, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d,block", [(3, 1, 64, 16), (2, 1, 128, 64), (4, 2, 256, 32), (8, 8, 128, 128)])
@pytest.mark.parametrize("lens,counts,kw", [
    ([3000], [100], {}),                          # several tiles, cuts inside of them
    ([2500], [17], dict(causal=False)),           # one tile in many pieces (few rows for hq / hkv = 1)
    ([400], [400], {}),                           # a prompt by itself: tiles of growing length
    ([2600], [150], dict(window=600)),            # tiles that begin at different keys
    ([130, 1900, 129], [129, 43, 1], {}),         # whole tiles, pieces and few rows in one call
], ids=["pieces", "one tile", "prompt", "window", "mixed"])
def test_matches_64_bits(cuda_device, hq, hkv, d, block, lens, counts, kw):
    cache, table, q, qf = _case(d + len(lens), hq, hkv, d, block, lens, counts)
    got, lse = _run(cache, table, lens, q, counts, **kw)
    _check(got, lse, du.attention(qf.astype(np.float64), cache, table, lens, counts, block, d ** -0.5, **kw))


@pytest.mark.parametrize("hkv,d", [(1, 128), (2, 64)])
def test_a_sequence_does_not_see_the_others(cuda_device, hkv, d):
    lens, counts, block, hq = [2600, 40, 3100, 700], [90, 40, 130, 5], 64, 4
    cache, table, q, _ = _case(11, hq, hkv, d, block, lens, counts)
    whole, whole_lse = _run(cache, table, lens, q, counts)
    at = np.concatenate(([0], np.cumsum(counts)))
    for order in ([2], [0], [3, 2, 1, 0]):
        rows = np.concatenate([np.arange(at[s], at[s + 1]) for s in order])
        got, lse = _run(cache, table[order], [lens[s] for s in order], q[rows], [counts[s] for s in order])
        assert torch.equal(got, whole[torch.from_numpy(rows).cuda()])
        assert torch.equal(lse, whole_lse[torch.from_numpy(rows).cuda()])
