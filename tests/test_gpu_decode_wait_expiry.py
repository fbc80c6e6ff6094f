"""The bounded on-chip waits of the attention of many rows and of the 4-bit linear
of more than 8 rows, made to expire on purpose: prism_debug_wait_expiry has every
CTA withhold one signal, so that a wait cannot complete and runs out.  The kernel
returns, the status bit is raised, and the next ordinary call is right."""
import numpy as np
import pytest
import torch

from tests import decode_util as du
from tests.test_gpu_kv_attention import _case, _check, _run
from tests.test_gpu_w4g import _problem
from tests.test_gpu_w4g import _run as _w4g
from tests.test_gpu_w4g import _want as _w4g_want

import deterministic_w8a8_int8_gb300 as prism

pytestmark = pytest.mark.gpu

LIMIT_NS = 20_000_000   # 20 ms


def _expires(call):
    torch.cuda.synchronize()
    assert prism.prism_device_status() == 0
    prism.prism_debug_wait_expiry(LIMIT_NS)
    try:
        call()
        torch.cuda.synchronize()   # returns: the kernel ran out without waiting
    finally:
        prism.prism_debug_wait_expiry(0)
    assert prism.prism_device_status() == prism.PRISM_DEVSTATUS_WAIT_TIMEOUT
    assert prism.prism_device_status() == 0


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,counts", [([90], [40]), ([1500, 130, 33], [90, 70, 1])], ids=["one block", "pieces"])
def test_attention(cuda_device, lens, counts, d):
    cache, table, q, qf = _case(d, 4, 2, d, 64, lens, counts)
    _expires(lambda: _run(cache, table, lens, q, counts))
    got, lse = _run(cache, table, lens, q, counts)
    _check(got, lse, du.attention(qf.astype(np.float64), cache, table, lens, counts, 64, d ** -0.5))


@pytest.mark.parametrize("g,offset", [(32, True), (128, False)])
@pytest.mark.parametrize("M,N,K", [(9, 40, 256), (12, 200, 2048), (37, 130, 8192), (64, 6000, 5120)])
def test_linear(cuda_device, M, N, K, g, offset):
    """One chunk of weights, several, and more than the ring holds."""
    q, a, codes, s, b, r, rf = _problem(M, M, N, K, g, offset)
    _expires(lambda: _w4g(q, a, codes, s, b, r))
    got = _w4g(q, a, codes, s, b, r).double().cpu().numpy()
    want, bound = _w4g_want(q, a, codes, s, b, rf, g)
    assert (np.abs(got - want) <= bound).all()
