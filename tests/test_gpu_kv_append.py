"""The paged int8 cache's append against a plain restatement: codes and scales
equal, whatever calls brought the tokens; bad pages and offsets answered by the
error word."""
import numpy as np
import pytest
import torch

from tests import decode_util as du

import deterministic_w8a8_int8_gb300 as prism

pytestmark = pytest.mark.gpu


def _filled(pages, heads, d, block, seqs):
    """A cache whose every byte is known, so that stray writes show."""
    c = prism.new_kv_cache(pages, heads, d, block, seqs)
    c.k_codes.fill_(77), c.v_codes.fill_(-77), c.k_scale.fill_(5.0), c.v_scale.fill_(6.0)
    c.k_open.fill_(9.0), c.v_open.fill_(-9.0)
    return c


def _expected(c, tokens, table, lens, block):
    """The buffers of ``c`` (copies) with every sequence's tokens in them; tokens[s] = (k, v) float32 [len, H, D]."""
    out = [t.cpu().float().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy() for t in c]
    out = [t.copy() for t in out]
    for s, n in enumerate(lens):
        for side in range(2):
            x = tokens[s][side]
            for b0 in range(0, n, block):
                rows = x[b0:min(n, b0 + block)]
                codes, scale = du.quantise_block(rows)
                page = table[s, b0 // block]
                out[side][page][:, :len(rows)] = codes.transpose(1, 0, 2)
                out[2 + side][page] = scale
    return out


def _compare(c, want, lens, block):
    for i, name in enumerate(("k_codes", "v_codes", "k_scale", "v_scale")):
        assert np.array_equal(c[i].cpu().numpy(), want[i]), name


def _run(rng, heads, d, block, steps, shape_seed=None, strided=False):
    """Appends steps[j][s] tokens in call j to sequence s; the final buffers and what they have to be."""
    seqs = len(steps[0])
    lens = [sum(st[s] for st in steps) for s in range(seqs)]
    table, pages = du.page_table(lens, block, rng)
    tokens = []
    for n in lens:
        x = rng.standard_normal((2, n, heads, d)).astype(np.float32) * rng.uniform(0.1, 4.0, (2, n, 1, 1))
        tokens.append(torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16))
    c = _filled(pages, heads, d, block, seqs)
    want = _expected(c, [t.float().numpy() for t in tokens], table, lens, block)
    t_table = torch.from_numpy(table).cuda()
    before = np.zeros(seqs, np.int32)
    for st in steps:
        cu = np.concatenate(([0], np.cumsum(st))).astype(np.int32)
        rows = [torch.cat([tokens[s][side, before[s]:before[s] + st[s]] for s in range(seqs)]) for side in range(2)]
        if strided:   # [T, H, D] views of a fused [T, H, 2D + 8] projection
            buf = torch.zeros((rows[0].shape[0], heads, 2 * d + 8), dtype=torch.bfloat16)
            buf[..., :d], buf[..., d + 8:] = rows[0], rows[1]
            buf = buf.cuda()
            k, v = buf[..., :d], buf[..., d + 8:]
        else:
            k, v = rows[0].cuda(), rows[1].cuda()
        one = all(n == 1 for n in st)
        prism.prism_kv_append(k, v, c, t_table, torch.from_numpy(before).cuda(),
                              cu_new=None if one else torch.from_numpy(cu).cuda())
        before = before + np.array(st, np.int32)
    torch.cuda.synchronize()
    return c, want, tokens, lens


@pytest.mark.parametrize("heads,d,block", [(1, 64, 16), (3, 128, 64), (2, 256, 32), (8, 128, 128)])
@pytest.mark.parametrize("steps", [
    [[1]], [[200, 0, 1, 63]], [[64, 128]], [[1, 1, 1]] * 5, [[70, 3, 0], [1, 1, 1], [1, 1, 1], [0, 130, 64], [1, 1, 1]]],
    ids=["one", "ragged", "whole", "steps", "mixed"])
def test_append_matches_restatement(cuda_device, heads, d, block, steps):
    rng = np.random.default_rng(heads * 1000 + d + block)
    c, want, tokens, lens = _run(rng, heads, d, block, steps)
    _compare(c, want, lens, block)
    for s, n in enumerate(lens):   # the open page's rows are held in bf16
        for side in range(2):
            tail = n % block
            got = c[4 + side][s, :, :tail].transpose(0, 1).cpu()
            assert torch.equal(got, tokens[s][side, n - tail:n])


def test_codes_do_not_depend_on_the_calls(cuda_device):
    """One token at a time, in uneven pieces, or at once: the same cache."""
    got = []
    for steps in ([[90, 41]], [[1, 1]] * 41 + [[1, 0]] * 49, [[17, 40], [60, 0], [13, 1]]):
        rng = np.random.default_rng(7)
        c, want, _, lens = _run(rng, 2, 64, 32, steps)
        _compare(c, want, lens, 32)
        got.append([t.cpu() for t in c[:4]])
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


def test_strided_rows(cuda_device):
    rng = np.random.default_rng(11)
    c, want, _, lens = _run(rng, 4, 64, 16, [[33, 5], [1, 1]], strided=True)
    _compare(c, want, lens, 16)


@pytest.mark.parametrize("value", [0.0, 2.0 ** -121, 2.0 ** -120, 3e38])
def test_extreme_blocks(cuda_device, value):
    x = torch.full((3, 1, 64), value, dtype=torch.float32).to(torch.bfloat16)
    x[1] = -x[1]
    c = prism.new_kv_cache(2, 1, 64, 16, 1)
    prism.prism_kv_append(x.cuda(), x.cuda(), c, torch.tensor([[1]], dtype=torch.int32, device="cuda"),
                          torch.zeros(1, dtype=torch.int32, device="cuda"),
                          cu_new=torch.tensor([0, 3], dtype=torch.int32, device="cuda"))
    codes, scale = du.quantise_block(x.float().numpy())
    assert np.array_equal(c.k_codes[1, 0, :3].cpu().numpy(), codes[:, 0])
    assert np.array_equal(c.v_scale[1].cpu().numpy(), scale)


def test_bad_pages_and_offsets_set_the_error_word(cuda_device):
    rng = np.random.default_rng(3)
    block, d = 16, 64
    k, _ = du.bf16(rng, (40, 1, d))
    k = k.cuda()
    table = torch.tensor([[0, 1], [-1, 2], [3, 99], [4, 5]], dtype=torch.int32, device="cuda")

    def call(lens, cu):
        c = _filled(6, 1, d, block, 4)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        prism.prism_kv_append(k, k, c, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                              cu_new=torch.tensor(cu, dtype=torch.int32, device="cuda"), err=err)
        torch.cuda.synchronize()
        return c, int(err)

    # pages -1 and 99: those pages stay out, every other one is written
    c, err = call([0, 0, 0, 0], [0, 1, 18, 36, 40])
    assert err == prism.PRISM_DEV_ERR_PAGE_RANGE
    assert float(c.k_scale[0]) != 5.0 and float(c.k_scale[2]) != 5.0 and float(c.k_scale[3]) != 5.0
    assert float(c.k_scale[4]) != 5.0 and float(c.k_scale[1]) == 5.0 and float(c.k_scale[5]) == 5.0
    # malformed sequences are not appended, the others are
    for lens, cu in (([0, -1, 0, 0], [0, 1, 2, 3, 4]), ([0, 31, 0, 0], [0, 1, 3, 4, 5]),
                     ([0, 0, 0, 0], [0, 1, 0, 1, 2]), ([0, 0, 0, 0], [0, 1, 1, 1, 41])):
        c, err = call(lens, cu)
        assert err & prism.PRISM_DEV_ERR_SEQ_RANGE
        assert float(c.k_scale[0]) != 5.0
