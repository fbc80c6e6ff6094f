"""The 4-bit group-scaled linear at every number of rows up to two turns of its
largest tile, and with fewer input channels than a stage of weights holds."""
import numpy as np
import pytest
import torch

from tests.test_gpu_w4g import _problem, _run, _want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("g,offset", [(32, True), (64, False), (128, True)])
def test_a_row_does_not_see_the_others(cuda_device, g, offset):
    """Bit-identical in batches of 1 to 130 rows."""
    q, a, codes, s, b, r, rf = _problem(g, 130, 200, 1152, g, offset)
    whole = _run(q, a, codes, s, b, r)
    want, bound = _want(q, a, codes, s, b, rf, g)
    assert (np.abs(whole.double().cpu().numpy() - want) <= bound).all()
    for m in range(1, 130):
        assert torch.equal(_run(q[:m], a[:m], codes, s, b, r[:m]), whole[:m]), m


@pytest.mark.parametrize("M", [1, 8, 9, 31, 33, 47, 49, 64, 70])
@pytest.mark.parametrize("K,g", [(32, 32), (64, 32), (64, 64), (96, 32), (128, 64), (128, 128), (192, 64), (224, 32)])
def test_short_rows(cuda_device, M, K, g):
    """Fewer than 256 input channels; the group sums at their largest are exact."""
    for offset, extremes in ((False, False), (True, True)):
        q, a, codes, s, b, r, rf = _problem(M + K, M, 37, K, g, offset, extremes)
        want, bound = _want(q, a, codes, s, b, rf, g)
        got = _run(q, a, codes, s, b, r).double().cpu().numpy()
        assert (np.abs(got - want) <= bound).all()
