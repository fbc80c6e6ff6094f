"""Attention of batches that mix long and short texts, one query and many: the
pieces' places in the workspace follow the sequences or their queries, and the
results are those of each sequence by itself."""
import numpy as np
import pytest
import torch

from tests import decode_util as du
from tests.test_gpu_kv_attention import _case, _check, _dev

import deterministic_w8a8_int8_gb300 as prism

pytestmark = pytest.mark.gpu


def _call(cache, table, lens, q, counts, max_q=None, **kw):
    """With a workspace of the stated size between two guards."""
    cu = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    hkv, block, d = cache[0].shape[1:]
    most = len(q) if max_q is None else max_q
    size = prism.prism_kv_attention_workspace_bytes(len(lens), len(q), most, table.shape[1], q.shape[1], hkv, d, block)
    guard = 1 << 20
    buf = torch.full((size + 2 * guard,), 0xff, dtype=torch.uint8, device="cuda")   # NaN as binary32
    err, lse = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full(q.shape[:2], 7.0, device="cuda")
    out = prism.prism_kv_attention(q.cuda(), _dev(cache), torch.from_numpy(table).cuda(),
                                   torch.tensor(lens, dtype=torch.int32, device="cuda"), cu_q=torch.from_numpy(cu).cuda(),
                                   lse=lse, err=err, max_q=max_q, workspace=buf[guard:guard + size], **kw)
    assert int(err) == 0
    assert bool((buf[:guard] == 0xff).all()) and bool((buf[guard + size:] == 0xff).all())
    return out, lse


BATCHES = {
    "decode and a piece": ([900] * 3 + [2500, 60, 1700, 2048, 1, 0, 1300], [1, 1, 1, 70, 1, 1, 1, 1, 1, 1]),
    "drafts": ([2100, 1500, 700, 1900, 2400], [9, 12, 3, 30, 9]),
    "two pieces among empty ones": ([1500, 0, 10, 2300, 0, 77, 5], [100, 0, 0, 140, 0, 1, 0]),
    "few and long": ([3000, 2900], [60, 1]),
}


@pytest.mark.parametrize("hq,hkv,d,block", [(5, 1, 128, 64), (8, 2, 64, 16), (4, 2, 256, 128)])
@pytest.mark.parametrize("lens,counts", BATCHES.values(), ids=BATCHES)
def test_against_64_bits_and_alone(cuda_device, lens, counts, hq, hkv, d, block):
    cache, table, q, qf = _case(len(lens) + d, hq, hkv, d, block, lens, counts)
    got, lse = _call(cache, table, lens, q, counts)
    _check(got, lse, du.attention(qf.astype(np.float64), cache, table, lens, counts, block, d ** -0.5))
    same, same_lse = _call(cache, table, lens, q, counts, max_q=max(counts))
    assert torch.equal(got, same) and torch.equal(lse, same_lse)
    at = np.concatenate(([0], np.cumsum(counts)))
    for s in np.flatnonzero(counts):
        rows = slice(at[s], at[s + 1])
        alone, alone_lse = _call(cache, table[s:s + 1], lens[s:s + 1], q[rows], counts[s:s + 1], max_q=counts[s])
        assert torch.equal(alone, got[rows]) and torch.equal(alone_lse, lse[rows])


def test_a_call_repeats_itself(cuda_device):
    lens, counts = BATCHES["drafts"]
    cache, table, q, _ = _case(4, 8, 2, 128, 64, lens, counts)
    first, first_lse = _call(cache, table, lens, q, counts)
    for _ in range(20):
        got, lse = _call(cache, table, lens, q, counts)
        assert torch.equal(got, first) and torch.equal(lse, first_lse)
