"""The bounded on-chip waits of linear attention on tcgen05, made to expire on
purpose: prism_debug_wait_expiry has every CTA withhold one signal, so that a wait
cannot complete and runs out.  The kernel returns, the status bit is raised, and
the next ordinary call is right."""
import numpy as np
import pytest
import torch

import deterministic_w8a8_int8_gb300 as prism
from tests.test_gpu_linear_attention import check, dev, index, make, run

pytestmark = pytest.mark.gpu

LIMIT_NS = 20_000_000   # 20 ms


@pytest.mark.parametrize("lens", [[90], [17, 3, 200, 64], [1100, 40]], ids=["two chunks", "several", "segments"])
def test_linear_attention(cuda_device, lens):
    data = make(21, lens, 2, 4, 128, 128)
    state = np.random.default_rng(11).standard_normal((len(lens), 4, 128, 128)).astype(np.float32)
    own = index(list(range(len(lens))))
    torch.cuda.synchronize()
    assert prism.prism_device_status() == 0
    prism.prism_debug_wait_expiry(LIMIT_NS)
    try:
        run(data, lens, dev(state, torch.float32), own, own)
        torch.cuda.synchronize()   # returns: the kernel ran out without waiting
    finally:
        prism.prism_debug_wait_expiry(0)
    assert prism.prism_device_status() == prism.PRISM_DEVSTATUS_WAIT_TIMEOUT
    assert prism.prism_device_status() == 0
    dstate = dev(state, torch.float32)
    got = run(data, lens, dstate, own, own)
    check(data, lens, state, got, dstate)
