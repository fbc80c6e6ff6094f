"""Calls whose kernels start ahead of their predecessors' end, captured in a
graph: what reads their results next sees all of them."""
import pytest
import torch

import deterministic_w8a8_int8_gb300 as prism

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,queries,max_pages", [
    ([300, 4000], [1, 200], 64),          # few rows and many, in pieces
    ([130, 90], [130, 60], 512),          # many rows, whole, in a call that could have pieces
    ([700], [64], 64),
])
def test_attention_and_its_reader(cuda_device, lens, queries, max_pages):
    g = torch.Generator().manual_seed(3)
    heads, kv, d, block = 8, 2, 128, 64
    used = [-(-n // block) for n in lens]
    cache = prism.new_kv_cache(sum(used), kv, d, block, len(lens))
    table = torch.zeros((len(lens), max_pages), dtype=torch.int32)
    at = 0
    for s, n in enumerate(used):
        table[s, :n] = torch.arange(at, at + n)
        at += n
    table = table.cuda()
    rows = torch.randn((sum(lens), 2, kv, d), generator=g).to(torch.bfloat16).cuda()
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    start = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
    lens_dev = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn((sum(queries), heads, d), generator=g).to(torch.bfloat16).cuda()
    cu_q = torch.tensor([0] + queries).cumsum(0).to(torch.int32).cuda()
    out = torch.empty_like(q)

    def step():
        prism.prism_kv_append(rows[:, 0], rows[:, 1], cache, table, start, cu_new=cu, max_new=max(lens))
        prism.prism_kv_attention(q, cache, table, lens_dev, cu_q=cu_q, max_q=max(queries), out=out)
        return out.clone()

    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        copies = []
        for _ in range(4):
            out.zero_()
            copies.append(step())
    for _ in range(5):
        graph.replay()
        for c in copies:
            assert torch.equal(c, want)
    assert not want.isnan().any() and want.abs().sum() > 0
