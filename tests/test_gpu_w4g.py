"""The 4-bit linear with group scales against a 64-bit statement."""
import numpy as np
import pytest
import torch

import workloads as wl
from tests import decode_util as du

import deterministic_w8a8_int8_gb300 as prism

pytestmark = pytest.mark.gpu


def _problem(seed, M, N, K, g, offset, extremes=False):
    rng = np.random.default_rng(seed)
    q = rng.integers(-127, 128, (M, K)).astype(np.int8)
    codes = rng.integers(-8, 8, (N, K)).astype(np.int8)
    if extremes:   # the largest group sums
        q[:] = np.where(rng.random((M, 1)) < 0.5, 127, -127)
        codes[: N // 2] = -8
        codes[N // 2:] = 7
    a = rng.uniform(0.001, 0.02, M).astype(np.float32)
    s = rng.uniform(0.001, 0.02, (N, K // g)).astype(np.float16)
    b = (rng.standard_normal((N, K // g)) * 0.02).astype(np.float16) if offset else None
    r, rf = du.bf16(rng, (M, N), 3.0)
    return q, a, codes, s, b, r, rf


def _want(q, a, codes, s, b, rf, g):
    """(values, bound): half a bf16 step, and binary32 sums of two terms a group
    (each product and sum one step) with up to 16 pieces joined."""
    M, K = q.shape
    groups = K // g
    x = q.reshape(M, groups, g).astype(np.float64)
    dot = np.einsum("mgk,ngk->mng", x, codes.reshape(-1, groups, g).astype(np.float64))
    terms = dot * s.astype(np.float64)[None]
    size = np.abs(terms).sum(axis=2)
    y = terms.sum(axis=2)
    if b is not None:
        more = x.sum(axis=2)[:, None, :] * b.astype(np.float64)[None]
        y, size = y + more.sum(axis=2), size + np.abs(more).sum(axis=2)
    y = y * a[:, None].astype(np.float64)
    bound = (2 * groups + 18) * du.HALF_F32 * size * a[:, None]
    if rf is not None:
        y = y + rf
    return y, bound + (du.HALF_BF16 + 2 * du.HALF_F32) * (np.abs(y) + bound)


def _run(q, a, codes, s, b, r, **kw):
    dev = lambda x: None if x is None else torch.from_numpy(x).cuda()  # noqa: E731
    return prism.prism_w4g_linear(dev(q), dev(a), dev(wl.pack_w4(codes)), dev(s), group_offset=dev(b),
                                  residual=None if r is None else r.cuda(), **kw)


@pytest.mark.parametrize("g", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 5, 128), (1, 64, 5120), (2, 1027, 256), (8, 200, 17408), (9, 130, 640),
                                   (17, 48, 1152), (37, 96, 2048), (64, 33, 384), (150, 70, 384)])
def test_matches_64_bits(cuda_device, g, M, N, K):
    for offset in (False, True):
        q, a, codes, s, b, r, rf = _problem(M + N + g, M, N, K, g, offset)
        for res, resf in ((None, None), (r, rf)):
            got = _run(q, a, codes, s, b, res).float().cpu().numpy()
            want, bound = _want(q, a, codes, s, b, resf, g)
            assert (np.abs(got - want) <= bound).all(), (offset, res is not None)


@pytest.mark.parametrize("g", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 8, 20])
def test_largest_group_sums(cuda_device, g, M):
    q, a, codes, s, b, r, rf = _problem(5, M, 40, 1024, g, True, extremes=True)
    want, bound = _want(q, a, codes, s, b, rf, g)
    assert (np.abs(_run(q, a, codes, s, b, r).float().cpu().numpy() - want) <= bound).all()


def test_group_sums_are_exact(cuda_device):
    """One group, scale 1: integers come out as integers."""
    rng = np.random.default_rng(1)
    for g in (32, 64, 128):
        q = rng.integers(-127, 128, (8, g)).astype(np.int8)
        codes = rng.integers(-8, 8, (64, g)).astype(np.int8)
        got = _run(q, np.ones(8, np.float32), codes, np.ones((64, 1), np.float16), None, None)
        exact = torch.from_numpy(q.astype(np.float64) @ codes.T.astype(np.float64)).to(torch.bfloat16)
        assert torch.equal(got.cpu(), exact)


@pytest.mark.parametrize("K,g", [(640, 32), (5120, 128), (17408, 64)])
def test_rows_do_not_depend_on_the_batch(cuda_device, K, g):
    q, a, codes, s, b, r, _ = _problem(3, 70, 300, K, g, True)
    whole = _run(q, a, codes, s, b, r)
    for rows in ([0], [69], [5, 6], list(range(3, 20)), list(range(60, 9, -1))):
        part = _run(np.ascontiguousarray(q[rows]), np.ascontiguousarray(a[rows]), codes, s, b, r[rows])
        assert torch.equal(part, whole[rows])


def test_strides_in_place_residual_and_graph(cuda_device):
    q, a, codes, s, b, r, rf = _problem(8, 6, 50, 512, 64, True)
    plain = _run(q, a, codes, s, b, r)
    wide = lambda x, extra: torch.nn.functional.pad(torch.from_numpy(x).cuda(), (0, extra))  # noqa: E731
    buf = torch.full((6, 61), 4.0, dtype=torch.bfloat16, device="cuda")
    buf[:, 3:53] = r.cuda()
    out = buf[:, 3:53]
    args = (wide(q, 16)[:, :512], torch.from_numpy(a).cuda(), wide(wl.pack_w4(codes), 32)[:, :256], wide(s, 3)[:, :8])
    offset = wide(b, 1)[:, :8]
    prism.prism_w4g_linear(*args, group_offset=offset, residual=out, out=out)
    assert torch.equal(out, plain) and (buf[:, :3] == 4.0).all() and (buf[:, 53:] == 4.0).all()
    graph = torch.cuda.CUDAGraph()
    res = r.cuda()
    with torch.cuda.graph(graph):
        captured = prism.prism_w4g_linear(*args, group_offset=offset, residual=res)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured, plain)
