"""The device of a decode-step call is its operands': a stream of another one is
refused, and the caller's current device stays."""
from types import SimpleNamespace

import pytest
import torch

import deterministic_w8a8_int8_gb300 as prism

pytestmark = pytest.mark.gpu


def _calls():
    device = "cuda"
    cache = prism.new_kv_cache(4, 2, 64, 16, 1, device=device)
    row = torch.ones((1, 2, 64), dtype=torch.bfloat16, device=device)
    table = torch.arange(4, dtype=torch.int32, device=device)[None]
    lens = torch.ones(1, dtype=torch.int32, device=device)
    return [lambda **kw: prism.prism_kv_append(row, row, cache, table, lens - 1, **kw),
            lambda **kw: prism.prism_kv_attention(row, cache, table, lens, **kw),
            lambda **kw: prism.prism_w4g_linear(torch.ones((1, 32), dtype=torch.int8, device=device), torch.ones(1, device=device),
                                                torch.zeros((4, 16), dtype=torch.uint8, device=device),
                                                torch.ones((4, 1), dtype=torch.float16, device=device), **kw),
            lambda **kw: prism.prism_token_logprobs(torch.ones((1, 8), device=device),
                                                    torch.zeros((1, 1), dtype=torch.int32, device=device), **kw)]


@pytest.mark.parametrize("i", range(4), ids=["append", "attention", "linear", "log probabilities"])
def test_a_stream_of_another_device_is_refused(cuda_device, i):
    call = _calls()[i]
    with pytest.raises(ValueError, match="stream must be of cuda:0, got one of cuda:1"):
        call(stream=SimpleNamespace(cuda_stream=0, device_index=1))   # no such stream is ever used
    call(stream=torch.cuda.current_stream())
    call(stream=torch.cuda.ExternalStream(torch.cuda.current_stream().cuda_stream))
    call(stream=SimpleNamespace(cuda_stream=torch.cuda.current_stream().cuda_stream))
    assert torch.cuda.current_device() == 0
    torch.cuda.synchronize()
