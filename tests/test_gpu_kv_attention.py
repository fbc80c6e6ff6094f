"""Attention over the paged int8 cache against a 64-bit statement."""
import numpy as np
import pytest
import torch

from tests import decode_util as du

import deterministic_w8a8_int8_gb300 as prism

pytestmark = pytest.mark.gpu


def _case(seed, hq, hkv, d, block, lens, counts, q_scale=1.0, shared=0):
    rng = np.random.default_rng(seed)
    table, pages = du.page_table(lens, block, rng, shared=shared)
    cache = du.random_cache(rng, pages, hkv, block, d)
    q, qf = du.bf16(rng, (sum(counts), hq, d), q_scale)
    return cache, table, q, qf


def _dev(cache):
    return [torch.from_numpy(c).cuda() for c in cache]


def _run(cache, table, lens, q, counts, **kw):
    cu = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = prism.prism_kv_attention(q.cuda(), _dev(cache), torch.from_numpy(table).cuda(),
                                   torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                   cu_q=torch.from_numpy(cu).cuda(), lse=lse, err=err,
                                   max_q=max(1, max(counts)), **kw)
    torch.cuda.synchronize()
    assert int(err) == 0
    return out, lse


def _check(got, lse, want):
    out, bound, w_lse, lse_bound = want
    off = np.abs(got.float().cpu().numpy().astype(np.float64) - out)
    assert (off <= bound).all(), (off - bound).max()
    l = lse.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isneginf(l), np.isneginf(w_lse))
    fine = np.isfinite(w_lse)
    assert (np.abs(l[fine] - w_lse[fine]) <= lse_bound[fine]).all()


@pytest.mark.parametrize("hq,hkv,d,block", [(4, 4, 64, 16), (5, 1, 128, 64), (6, 2, 256, 32), (16, 2, 128, 128),
                                            (40, 1, 64, 64)])
@pytest.mark.parametrize("lens,counts", [
    ([1], [1]), ([0, 1, 17, 300], [1, 1, 1, 1]), ([63, 64, 65, 0], [1, 1, 1, 0]), ([1500, 700], [1, 1]),
    ([20, 130, 3], [20, 7, 5]), ([700, 33], [70, 33])],
    ids=["one", "decode", "edges", "long", "queries", "piece"])
def test_matches_64_bits(cuda_device, hq, hkv, d, block, lens, counts):
    cache, table, q, qf = _case(hq + d + len(lens), hq, hkv, d, block, lens, counts)
    got, lse = _run(cache, table, lens, q, counts)
    _check(got, lse, du.attention(qf.astype(np.float64), cache, table, lens, counts, block, d ** -0.5))


@pytest.mark.parametrize("kw", [dict(causal=False), dict(window=1), dict(window=40), dict(window=5000),
                                dict(scale=0.5)], ids=str)
@pytest.mark.parametrize("counts", [[1, 1, 1], [9, 50, 1]], ids=["decode", "queries"])
def test_masks_and_scale(cuda_device, kw, counts):
    lens = [77, 900, 2]
    cache, table, q, qf = _case(5, 8, 2, 64, 32, lens, counts)
    got, lse = _run(cache, table, lens, q, counts, **kw)
    args = dict(kw)
    scale = args.pop("scale", 64 ** -0.5)
    _check(got, lse, du.attention(qf.astype(np.float64), cache, table, lens, counts, 32, scale, **args))


def test_queries_that_see_nothing(cuda_device):
    """More queries than tokens: the first ones stand before the text."""
    lens, counts = [3, 0], [8, 4]
    cache, table, q, qf = _case(9, 4, 2, 64, 16, lens, counts)
    got, lse = _run(cache, table, lens, q, counts)
    assert (got[:5] == 0).all() and (got[8:] == 0).all() and torch.isneginf(lse[8:]).all()
    _check(got, lse, du.attention(qf.astype(np.float64), cache, table, lens, counts, 16, 0.125))


@pytest.mark.parametrize("counts", [[1, 1], [40, 1]], ids=["decode", "queries"])
def test_peaked_scores_and_uneven_scales(cuda_device, counts):
    """Scores far apart (one key takes all), and pages whose value scales differ by 10^6."""
    lens = [600, 333]
    cache, table, q, qf = _case(13, 4, 1, 128, 16, lens, counts, q_scale=30.0)
    cache[3] *= np.float32(10.0) ** np.random.default_rng(1).integers(-3, 4, cache[3].shape).astype(np.float32)
    cache[3][table[0, 5]] = 0.0
    got, lse = _run(cache, table, lens, q, counts)
    _check(got, lse, du.attention(qf.astype(np.float64), cache, table, lens, counts, 16, 128 ** -0.5))


def test_tiny_and_huge_queries(cuda_device):
    lens, counts = [50, 50], [1, 1]
    cache, table, q, qf = _case(21, 2, 2, 64, 16, lens, counts)
    q = q.clone()
    q[0] *= 2.0 ** -100
    q[1] *= 2.0 ** 20
    got, lse = _run(cache, table, lens, q, counts)
    _check(got, lse, du.attention(q.float().numpy().astype(np.float64), cache, table, lens, counts, 16, 0.125))


@pytest.mark.parametrize("counts", [[1, 1, 1, 1], [16, 16, 16, 3], [100, 16, 1, 70]], ids=["decode", "few", "many"])
def test_a_sequence_does_not_see_the_others(cuda_device, counts):
    """Bit-identical alone, in a batch and in another order; shared pages too."""
    lens = [900, 640, 2000, 700]
    cache, table, q, _ = _case(17, 8, 2, 128, 64, lens, counts, shared=9)
    whole, _ = _run(cache, table, lens, q, counts)
    first = np.concatenate(([0], np.cumsum(counts)))
    for s in range(4):
        rows = slice(first[s], first[s + 1])
        alone, _ = _run(cache, table[s:s + 1], lens[s:s + 1], q[rows], counts[s:s + 1])
        assert torch.equal(alone, whole[rows])
    order = [2, 0, 3, 1]
    turned, _ = _run(cache, table[order], [lens[s] for s in order],
                     torch.cat([q[first[s]:first[s + 1]] for s in order]), [counts[s] for s in order])
    assert torch.equal(turned, torch.cat([whole[first[s]:first[s + 1]] for s in order]))


def test_strides_out_and_no_offsets(cuda_device):
    lens = [90, 5, 140]
    cache, table, q, qf = _case(23, 6, 2, 64, 16, lens, [1, 1, 1])
    buf = torch.zeros((3, 6, 80), dtype=torch.bfloat16, device="cuda")
    buf[..., :64] = q.cuda()
    out = torch.full((3, 7, 72), 3.0, dtype=torch.bfloat16, device="cuda")
    prism.prism_kv_attention(buf[..., :64], _dev(cache), torch.from_numpy(table).cuda(),
                             torch.tensor(lens, dtype=torch.int32, device="cuda"), out=out[:, :6, :64])
    assert (out[:, 6] == 3.0).all() and (out[:, :, 64:] == 3.0).all()
    want = du.attention(qf.astype(np.float64), cache, table, lens, [1, 1, 1], 16, 0.125)
    off = np.abs(out[:, :6, :64].float().cpu().numpy() - want[0])
    assert (off <= want[1]).all()


@pytest.mark.parametrize("counts", [[1, 1, 1], [40, 2, 33]], ids=["decode", "queries"])
def test_bad_pages_and_lengths_set_the_error_word(cuda_device, counts):
    lens, block = [600, 40, 700], 16
    cache, table, q, qf = _case(29, 4, 2, 64, block, lens, counts)
    want = du.attention(qf.astype(np.float64), cache, table, lens, counts, block, 0.125)
    first = np.concatenate(([0], np.cumsum(counts)))

    def call(table, lens, cu=None, max_q=None):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        cu = np.concatenate(([0], np.cumsum(counts))) if cu is None else cu
        out = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
        prism.prism_kv_attention(q.cuda(), _dev(cache), torch.from_numpy(table).cuda(),
                                 torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                 cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                 max_q=max_q or max(counts), out=out, err=err)
        torch.cuda.synchronize()
        return out, int(err)

    def good(out, s):
        rows = slice(first[s], first[s + 1])
        return (np.abs(out[rows].float().cpu().numpy() - want[0][rows]) <= want[1][rows]).all()

    for page in (-1, cache[0].shape[0], 1 << 30):
        bad = table.copy()
        bad[0, 20] = page
        out, err = call(bad, lens)
        assert err == prism.PRISM_DEV_ERR_PAGE_RANGE
        assert out[:first[1]].isnan().any() and good(out, 1) and good(out, 2)
    for wrong in (-5, 16 * table.shape[1] + 1):
        out, err = call(table, [600, wrong, 700])
        assert err == prism.PRISM_DEV_ERR_SEQ_RANGE
        assert out[first[1]:first[2]].isnan().all() and good(out, 0) and good(out, 2)
    if max(counts) > 1:
        out, err = call(table, lens, max_q=39)
        assert err == prism.PRISM_DEV_ERR_SEQ_RANGE and good(out, 1) and good(out, 2)
    out, err = call(table, lens, cu=[0, first[1], first[3] + 1, first[3]])   # past T, then decreasing
    assert err == prism.PRISM_DEV_ERR_SEQ_RANGE and good(out, 0)


def test_far_pages_pass_32_bits(cuda_device):
    """Pages beyond 2^31 code bytes."""
    block, d, heads = 128, 256, 8
    pages = (1 << 31) // (block * d * heads) + 3
    kc = torch.zeros((pages, heads, block, d), dtype=torch.int8, device="cuda")
    vc = torch.zeros_like(kc)
    scales = torch.full((pages, heads), 0.01, device="cuda")
    rng = np.random.default_rng(2)
    table = np.array([[pages - 1, 0, pages - 2]], np.int32)
    small = du.random_cache(rng, 3, heads, block, d)
    for i, p in enumerate(table[0]):
        kc[p], vc[p] = torch.from_numpy(small[0][i]).cuda(), torch.from_numpy(small[1][i]).cuda()
    small[2][:] = 0.01
    small[3][:] = 0.01
    q, qf = du.bf16(rng, (1, 16, d))
    out = prism.prism_kv_attention(q.cuda(), (kc, vc, scales, scales), torch.from_numpy(table).cuda(),
                                   torch.tensor([300], dtype=torch.int32, device="cuda"))
    want = du.attention(qf.astype(np.float64), small, np.array([[0, 1, 2]]), [300], [1], block, d ** -0.5)
    assert (np.abs(out.float().cpu().numpy() - want[0]) <= want[1]).all()


def test_streams_and_graph(cuda_device):
    """A call on a side stream, and one captured and replayed on new inputs."""
    lens, counts = [1500, 900], [1, 1]
    cache, table, q, qf = _case(31, 8, 2, 128, 64, lens, counts)
    want = du.attention(qf.astype(np.float64), cache, table, lens, counts, 64, 128 ** -0.5)
    c, t, n = _dev(cache), torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    q_dev = q.cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out = prism.prism_kv_attention(q_dev, c, t, n)
    side.synchronize()
    assert (np.abs(out.float().cpu().numpy() - want[0]) <= want[1]).all()
    static = torch.zeros_like(q_dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = prism.prism_kv_attention(static, c, t, n)
    static.copy_(q_dev)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured, out)
