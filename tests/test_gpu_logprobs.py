"""Token log probabilities, entropy and top alternatives against 64 bits."""
import numpy as np
import pytest
import torch

import deterministic_w8a8_int8_gb300 as prism

pytestmark = pytest.mark.gpu

HALF_F32 = 2.0 ** -24


def _want(x, ids, k):
    """x float64 [R, V].  Bounds: a binary32 sum of V terms in pieces (at most
    2^7 additions deep) of exponentials good to 2^-21, so ln of it to 2^-16;
    x - max and the last difference half a step each; the entropy adds the same
    error times the mean of |x - max|."""
    m = x.max(axis=1, keepdims=True)
    y = x - m
    e = np.exp(y)
    z = np.log(e.sum(axis=1, keepdims=True))
    p = e / e.sum(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        mean = np.where(p > 0, p * np.where(p > 0, y, 0.0), 0.0).sum(axis=1)
    lp = np.take_along_axis(y, ids, axis=1) - z
    order = np.argsort(-x, axis=1, kind="stable")[:, :k]
    return lp, z[:, 0] - mean, order, np.take_along_axis(y, order, axis=1) - z, np.abs(mean)


def _check(x, ids, k):
    """x: torch CPU logits."""
    x64 = x.double().numpy()
    lp, ent, top, toplp, mean = _want(x64, ids, k)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    g_lp, g_ent, g_top, g_toplp = prism.prism_token_logprobs(
        x.cuda(), torch.from_numpy(ids.astype(np.int32)).cuda(), top_k=k, err=err)
    assert int(err) == 0

    def near(got, want, extra=0.0):
        got = got.cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isneginf(got), np.isneginf(want.astype(np.float32)))
        fine = np.isfinite(want) & np.isfinite(got)
        bound = 2.0 ** -16 + extra + 4 * HALF_F32 * np.abs(np.where(fine, want, 0.0))
        assert (np.abs(np.where(fine, got - want, 0.0)) <= bound).all()

    near(g_lp, lp)
    near(g_ent, ent, 2.0 ** -16 * mean)
    if k:
        assert np.array_equal(g_top.cpu().numpy(), top)
        near(g_toplp, toplp)
    else:
        assert g_top is None and g_toplp is None


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,V", [(1, 1), (2, 7), (3, 33), (1, 1000), (5, 4097), (2, 32003), (1, 248000), (3, 300001)])
def test_matches_64_bits(cuda_device, dtype, R, V):
    rng = np.random.default_rng(R + V)
    x = torch.from_numpy((rng.standard_normal((R, V)) * 3).astype(np.float32)).to(dtype)
    ids = rng.integers(0, V, (R, 3))
    for k in sorted({0, 1, min(V, 5), min(V, 20), min(V, 32)}):
        _check(x, ids, k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "two_values", "masked", "lowest", "one_left", "far",
                                  "signed_zeros", "top_in_one_place"])
@pytest.mark.parametrize("V", [50, 6000, 70001])
def test_orders_ties_and_masks(cuda_device, dtype, kind, V):
    rng = np.random.default_rng(V)
    x = np.zeros((2, V), np.float32)
    if kind == "rising":
        x[:] = np.arange(V) * (8.0 / V)
    elif kind == "falling":
        x[:] = -np.arange(V) * (8.0 / V)
    elif kind == "two_values":
        x[:] = rng.integers(0, 2, (2, V))
    elif kind == "masked":
        x[:] = rng.standard_normal((2, V))
        x[rng.random((2, V)) < 0.95] = -np.inf
        x[:, 3] = 0.5
    elif kind == "lowest":
        x[:] = torch.finfo(dtype).min
        x[:, V // 2] = 1.0
    elif kind == "one_left":
        x[:] = -np.inf
        x[:, V - 1] = -4.0
    elif kind == "far":
        x[:] = rng.standard_normal((2, V)) * 1e4
    elif kind == "signed_zeros":
        x[:, ::2] = -0.0
    elif kind == "top_in_one_place":
        x[:] = rng.standard_normal((2, V))
        x[:, V // 3:V // 3 + 40] += 20.0
    _check(torch.from_numpy(x).to(dtype), rng.integers(0, V, (2, 2)), min(V, 32))
    _check(torch.from_numpy(x).to(dtype), rng.integers(0, V, (2, 1)), 3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_without_a_finite_maximum(cuda_device, dtype):
    x = torch.randn(5, 5000).to(dtype)
    x[0] = -float("inf")
    x[1, 77] = float("nan")
    x[2, 4999] = float("inf")
    lp, ent, top, toplp = prism.prism_token_logprobs(x.cuda(), torch.zeros((5, 1), dtype=torch.int32, device="cuda"),
                                                     top_k=4)
    assert lp[:3].isnan().all() and ent[:3].isnan().all() and toplp[:3].isnan().all() and (top[:3] == -1).all()
    assert not lp[3:].isnan().any() and not ent[3:].isnan().any() and (top[3:] >= 0).all()


def test_ids_out_of_range(cuda_device):
    x = torch.randn(3, 100)
    ids = torch.tensor([[0, 100], [-1, 5], [99, 7]], dtype=torch.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lp = prism.prism_token_logprobs(x.cuda(), ids.cuda(), err=err)[0]
    assert int(err) == prism.PRISM_DEV_ERR_ID_RANGE
    assert lp.isnan().cpu().tolist() == [[False, True], [True, False], [False, False]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unaligned_strided_rows_and_batch(cuda_device, dtype):
    """Rows of odd stride at odd addresses; the same bits as each row alone."""
    rng = np.random.default_rng(4)
    buf = torch.from_numpy(rng.standard_normal((6, 9013)).astype(np.float32)).to(dtype).cuda()
    x = buf[:, 3:9008]
    ids = torch.from_numpy(rng.integers(0, 9005, (6, 2)).astype(np.int32)).cuda()
    whole = prism.prism_token_logprobs(x, ids, top_k=7)
    for r in range(6):
        alone = prism.prism_token_logprobs(x[r:r + 1].clone(), ids[r:r + 1], top_k=7)
        assert torch.equal(alone[2], whole[2][r:r + 1])
        for a, b in zip(alone, whole):
            assert torch.equal(a, b[r:r + 1])
    _check(x.cpu(), ids.cpu().numpy().astype(np.int64), 7)


def test_graph_and_no_entropy(cuda_device):
    x = torch.randn(4, 20000, device="cuda")
    ids = torch.arange(4, dtype=torch.int32, device="cuda")[:, None]
    want = prism.prism_token_logprobs(x, ids, top_k=5)
    none = prism.prism_token_logprobs(x, ids, top_k=5, entropy=False)
    assert none[1] is None and torch.equal(none[0], want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = prism.prism_token_logprobs(x, ids, top_k=5)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
