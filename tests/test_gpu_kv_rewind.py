"""A sequence set back within its open page (a rejected draft, a step tried
again): what is appended next is coded as if the dropped rows had never been."""
import numpy as np
import pytest
import torch

from tests import decode_util as du

import deterministic_w8a8_int8_gb300 as prism

pytestmark = pytest.mark.gpu


def _append(cache, table, rows, before):
    """rows: a (k, v) pair [n, H, D] for each sequence."""
    cu = torch.tensor([0] + [len(r[0]) for r in rows]).cumsum(0).to(torch.int32).cuda()
    k, v = (torch.cat([r[side] for r in rows]).cuda() for side in range(2))
    prism.prism_kv_append(k, v, cache, table, torch.tensor(before, dtype=torch.int32, device="cuda"), cu_new=cu)


def _rows(rng, n, heads, d, scale):
    return [du.bf16(rng, (n, heads, d), scale)[0] for _ in range(2)]


@pytest.mark.parametrize("heads,d,block", [(1, 64, 16), (3, 128, 64), (2, 256, 32), (8, 128, 128)])
@pytest.mark.parametrize("draft_scale,next_scale", [(50.0, 0.1), (1e-3, 1.0), (50.0, 0.0), (1.0, 50.0)],
                         ids=["larger draft", "smaller draft", "then zeros", "then larger"])
def test_rows_after_a_rejected_draft(cuda_device, heads, d, block, draft_scale, next_scale):
    rng = np.random.default_rng(block + d)
    kept = [block + 5, 3, block * 2]                 # two open pages, and one that the draft begins
    drafts = [4, block - 4, 2]
    table_np, pages = du.page_table([n + block for n in kept], block, rng)
    table = torch.from_numpy(table_np).cuda()
    cache = prism.new_kv_cache(pages, heads, d, block, 3)
    first = [_rows(rng, n, heads, d, 1.0) for n in kept]
    _append(cache, table, first, [0, 0, 0])
    _append(cache, table, [_rows(rng, n, heads, d, draft_scale) for n in drafts], kept)
    back = [kept[0], kept[1] - 1, kept[2]]           # the second loses a kept row too
    then = [_rows(rng, n, heads, d, next_scale) for n in (1, 2, 1)]
    _append(cache, table, then, back)
    for s in range(3):
        for side in range(2):
            x = torch.cat((first[s][side][:back[s]], then[s][side])).float().numpy()
            for b0 in range(0, len(x), block):
                codes, scale = du.quantise_block(x[b0:b0 + block])
                page = table_np[s, b0 // block]
                n = len(codes)
                assert np.array_equal(cache[2 + side][page].cpu().numpy(), scale), (s, side, b0)
                assert np.array_equal(cache[side][page, :, :n].cpu().numpy(), codes.transpose(1, 0, 2)), (s, side, b0)


def test_a_step_tried_again(cuda_device):
    """The same position appended three times; the last row counts."""
    rng = np.random.default_rng(3)
    heads, d, block = 2, 64, 16
    cache = prism.new_kv_cache(1, heads, d, block, 1)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    head = _rows(rng, 6, heads, d, 1.0)
    _append(cache, table, [head], [0])
    for scale in (30.0, 300.0, 0.5):
        row = _rows(rng, 1, heads, d, scale)
        _append(cache, table, [row], [6])
        for side in range(2):
            codes, scales = du.quantise_block(torch.cat((head[side], row[side])).float().numpy())
            assert np.array_equal(cache[side][0, :, :7].cpu().numpy(), codes.transpose(1, 0, 2))
            assert np.array_equal(cache[2 + side][0].cpu().numpy(), scales)


@pytest.mark.parametrize("rows", [1, 3])
def test_a_step_that_completed_a_page_tried_again(cuda_device, rows):
    """The rows before it are still held while the next page has none."""
    rng = np.random.default_rng(rows)
    heads, d, block = 2, 64, 16
    cache = prism.new_kv_cache(1, heads, d, block, 1)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    head = _rows(rng, block - rows, heads, d, 1.0)
    _append(cache, table, [head], [0])
    for n, scale in ((rows, 30.0), (rows, 0.5), (1, 0.25)):
        new = _rows(rng, n, heads, d, scale)
        _append(cache, table, [new], [block - rows])
        for side in range(2):
            codes, scales = du.quantise_block(torch.cat((head[side], new[side])).float().numpy())
            assert np.array_equal(cache[side][0, :, :len(codes)].cpu().numpy(), codes.transpose(1, 0, 2))
            assert np.array_equal(cache[2 + side][0].cpu().numpy(), scales)
