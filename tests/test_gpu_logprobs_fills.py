"""Token log probabilities of rows whose masked logits hold a finite fill, and of
rows that lie far from zero, against 64 bits."""
import numpy as np
import pytest
import torch

import deterministic_w8a8_int8_gb300 as prism

pytestmark = pytest.mark.gpu

HALF_F32 = 2.0 ** -24


def _check(x, ids, k=7):
    """Every finite value has to be met by a finite one: a binary32 sum in pieces
    of exponentials good to 2^-21, so ln of it to 2^-16, and half a step each for
    x - max, the last difference and the two roundings of ln's multiple."""
    x64 = x.double().numpy()
    y = x64 - x64.max(axis=1, keepdims=True)
    e = np.exp(y)
    total = e.sum(axis=1, keepdims=True)
    z = np.log(total)
    lp = np.take_along_axis(y, ids, axis=1) - z
    mean = (e * np.where(e > 0, y, 0.0)).sum(axis=1) / total[:, 0]
    top = np.argsort(-x64, axis=1, kind="stable")[:, :k]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = prism.prism_token_logprobs(x.cuda(), torch.from_numpy(ids.astype(np.int32)).cuda(), top_k=k, err=err)
    assert int(err) == 0
    g_lp, g_ent, g_top, g_top_lp = (t.cpu().numpy() for t in got)
    assert np.array_equal(g_top, top)
    for g, want, extra in ((g_lp, lp, 0.0), (g_ent, z[:, 0] - mean, 2.0 ** -16 * np.abs(mean)),
                           (g_top_lp, np.take_along_axis(y, top, axis=1) - z, 0.0)):
        assert np.isfinite(g).all()
        off = np.abs(g.astype(np.float64) - want)
        assert (off <= 2.0 ** -16 + extra + 4 * HALF_F32 * np.abs(want)).all()


FILLS = [-1e4, -1e5, -3e5, -6e5, -1e6, -1.1e6, -1e9, -1e10, -1e18, -1e30, -5e36, -9e36, -1e38]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("v", [1003, 20000, 70001])
@pytest.mark.parametrize("fill", FILLS, ids=str)
def test_finite_fills(cuda_device, fill, v, dtype):
    """A masked tail, a masked head, whole pieces of 8, all but a few logits, and
    every piece of some threads (they come again every 4096 logits)."""
    rng = np.random.default_rng(v)
    x = rng.standard_normal((6, v)) * 3.0
    at = np.arange(v)
    hidden = np.zeros((6, v), bool)
    hidden[0] = at >= v * 2 // 3
    hidden[1] = at < v * 3 // 4
    hidden[2] = (at // 8) % 3 != 1
    hidden[3] = ~np.isin(at, rng.permutation(v)[:5])
    hidden[4] = at % 4096 < 2560
    hidden[5] = at != v - 1
    hidden[:, v - 9] = hidden[:, 4] = False   # a few stay, in the head and in the tail
    x[hidden] = fill
    ids = np.stack([rng.integers(0, v, 6), np.full(6, 4), at[rng.integers(0, v, 6)]], axis=1)
    _check(torch.from_numpy(x).to(dtype), ids)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("centre", [3e5, 5.2e5, 5.3e5, 1.04e6, 1.05e6, 1e10, 1e20, 1e35], ids=str)
def test_rows_far_from_zero(cuda_device, centre, dtype):
    """Both signs; differences of a few units and of a few of the type's steps."""
    v, rng = 9001, np.random.default_rng(5)
    noise = rng.standard_normal((4, v))
    step = centre * torch.finfo(dtype).eps
    x = np.stack([centre + noise[0], -centre + noise[1], centre + 4 * step * noise[2], -centre + 4 * step * noise[3]])
    ids = rng.integers(0, v, (4, 2))
    _check(torch.from_numpy(x).to(dtype), ids)


def test_a_fill_next_to_infinities(cuda_device):
    rng = np.random.default_rng(8)
    x = torch.from_numpy(rng.standard_normal((3, 5000)).astype(np.float32))
    x[0, 64:4000] = -1e10
    x[0, 4100:] = -torch.inf
    x[1] = -1e30                      # all filled: a row of ties
    x[2, 8:] = -torch.inf
    x[2, :8] = -1e30
    ids = torch.tensor([[5], [5], [5]], dtype=torch.int32, device="cuda")
    lp, ent, top, top_lp = (t.cpu().double() for t in prism.prism_token_logprobs(x.cuda(), ids, top_k=3))
    want = x.double().log_softmax(-1)
    assert (lp[:, 0] - want[:, 5]).abs().max() <= 2.0 ** -15
    assert abs(ent[1] - np.log(5000.0)) <= 2.0 ** -15 and abs(ent[2] - np.log(8.0)) <= 2.0 ** -15
    assert top[1:].tolist() == [[0, 1, 2]] * 2 and (top_lp[1] + np.log(5000.0)).abs().max() <= 2.0 ** -15
