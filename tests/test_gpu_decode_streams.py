"""The decode-step calls on a stream that is not the current one: what they take
from the allocator is theirs for as long as that stream works on it."""
import pytest
import torch

import deterministic_w8a8_int8_gb300 as prism

pytestmark = pytest.mark.gpu

WAIT = 20_000_000   # cycles, some 10 ms: longer than all that the host does meanwhile


def _attention(queries):
    """Long texts, so that rows are in pieces and a workspace is needed."""
    g = torch.Generator().manual_seed(2)
    heads, kv, d, block, seqs, length = 8, 2, 128, 64, 3, 6000
    pages = -(-length // block)
    cache = prism.new_kv_cache(pages * seqs, kv, d, block, seqs)
    rows = torch.randn((seqs * length, 2, kv, d), generator=g).to(torch.bfloat16).cuda()
    table = torch.arange(pages * seqs, dtype=torch.int32, device="cuda").view(seqs, pages)
    cu = torch.arange(seqs + 1, dtype=torch.int32, device="cuda") * length
    prism.prism_kv_append(rows[:, 0], rows[:, 1], cache, table, torch.zeros(seqs, dtype=torch.int32, device="cuda"), cu_new=cu)
    q = torch.randn((seqs * queries, heads, d), generator=g).to(torch.bfloat16).cuda()
    args = dict(q=q, cache=cache, page_table=table, seq_lens=torch.full((seqs,), length, dtype=torch.int32, device="cuda"),
                cu_q=torch.arange(seqs + 1, dtype=torch.int32, device="cuda") * queries, max_q=queries)
    size = prism.prism_kv_attention_workspace_bytes(seqs, seqs * queries, queries, pages, heads, kv, d, block)
    assert size > 0
    return (lambda **kw: (prism.prism_kv_attention(**args, **kw),)), size


def _w4g(m):
    g = torch.Generator().manual_seed(4)
    n, k = 1024, 512
    args = dict(q=torch.randint(-127, 128, (m, k), generator=g, dtype=torch.int8).cuda(), a_scale=torch.ones(m, device="cuda"),
                w4=torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8).cuda(),
                group_scale=torch.rand((n, k // 64), generator=g).half().cuda())
    return (lambda **kw: (prism.prism_w4g_linear(**args, **kw),)), 0


def _logprobs(rows):
    g = torch.Generator().manual_seed(5)
    args = dict(logits=torch.randn((rows, 30000), generator=g).cuda(), top_k=5,
                token_ids=torch.randint(0, 30000, (rows, 2), generator=g, dtype=torch.int32).cuda())
    return (lambda **kw: prism.prism_token_logprobs(**args, **kw)), 0


CALLS = [(_attention, 1), (_attention, 40), (_w4g, 4), (_w4g, 30), (_logprobs, 600)]
IDS = ["attention", "attention of many rows", "linear", "linear of many rows", "log probabilities"]


def _blocks(outs, workspace):
    return [t.numel() * t.element_size() for t in outs] + ([workspace] if workspace else [])


@pytest.mark.parametrize("make,rows", CALLS, ids=IDS)
def test_memory_given_out_during_the_call(cuda_device, make, rows):
    """The current stream fills every block that it can get while the call waits for its turn."""
    call, workspace = make(rows)
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(WAIT)
    got = call(stream=side)
    noise = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in _blocks(want, workspace) for _ in range(2)]
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(bool((t == 255).all()) for t in noise)


@pytest.mark.parametrize("make,rows", CALLS, ids=IDS)
def test_memory_given_back_before_the_call(cuda_device, make, rows):
    """The current stream still has work on blocks that were given back to it."""
    call, workspace = make(rows)
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.empty((n,), dtype=torch.uint8, device="cuda") for n in _blocks(want, workspace)]
    side = torch.cuda.Stream()
    torch.cuda._sleep(WAIT)
    for t in old:
        t.fill_(255)
    del old, t
    got = call(stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_the_current_stream_stays(cuda_device):
    call, _ = _w4g(3)
    side = torch.cuda.Stream()
    before = torch.cuda.current_stream()
    side.wait_stream(before)
    call(stream=side)
    assert torch.cuda.current_stream() == before
    with pytest.raises(prism.PrismError):
        prism.prism_token_logprobs(torch.zeros((1, 8), device="cuda"), torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                                   top_k=-1, stream=side)
    assert torch.cuda.current_stream() == before
    side.synchronize()
