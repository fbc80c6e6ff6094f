"""The linears, the quantiser and the read-out on a stream that is not the current
one: outputs, and workspaces that have to start zeroed, belong to that stream."""
import pytest
import torch

import deterministic_w8a8_int8_gb300 as prism

pytestmark = pytest.mark.gpu

WAIT = 20_000_000   # cycles, some 10 ms: longer than all that the host does meanwhile


def _codes(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, dtype=torch.int8).cuda()


def _linear(g):
    m, n, k = 304, 1536, 5120
    args = (_codes(g, m, k), torch.rand(m, generator=g).cuda(), _codes(g, n, k), torch.rand(n, generator=g).cuda())
    return lambda **kw: [prism.prism_w8a8_linear(*args, split_k=4, **kw)]


def _linear_f16(g):
    m, n, k = 304, 1536, 5120
    x, w = (prism.prism_codes_to_f16(_codes(g, rows, k)) for rows in (m, n))
    args = (x, torch.rand(m, generator=g).cuda(), w, torch.rand(n, generator=g).cuda())
    return lambda **kw: [prism.prism_w8a8_linear_f16(*args, split_k=4, **kw)]


def _quant(g):
    x = torch.randn((300, 4096), generator=g).to(torch.bfloat16).cuda()
    return lambda **kw: list(prism.prism_quant_act(x, **kw))


@pytest.mark.parametrize("make", [_linear, _linear_f16, _quant])
def test_blocks_with_work_of_the_current_stream(cuda_device, make):
    """Blocks given back with work on them, and every block of those sizes taken again."""
    call = make(torch.Generator().manual_seed(6))
    want = [t.clone() for t in call()]
    sizes = [t.numel() * t.element_size() for t in want] + [prism.prism_w8a8_workspace_bytes(304, 1536, 5120, 4),
                                                            prism.prism_w8a8_f16_workspace_bytes(304, 1536, 5120, 4)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.empty((n,), dtype=torch.uint8, device="cuda") for n in sizes if n]
    side = torch.cuda.Stream()
    torch.cuda._sleep(WAIT)
    for t in old:
        t.fill_(255)
    del old, t
    early = call(stream=side)                  # runs while the current stream sleeps
    side.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(WAIT)
    late = call(stream=side)                   # waits, while the current stream takes what it can get
    noise = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes if n]
    torch.cuda.synchronize()
    for got in (early, late):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(bool((t == 255).all()) for t in noise)


def test_streams_by_place_and_by_handle(cuda_device):
    x = torch.randn((3, 64)).to(torch.bfloat16).cuda()
    want = prism.prism_quant_act(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for got in (prism.prism_quant_act(x, None, None, None, side),
                prism.prism_quant_act(x, stream=torch.cuda.ExternalStream(side.cuda_stream))):
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.cuda.current_stream() != side
