"""Linear attention on values far from 1: what a chunk's decays are divided by must
not take products out of binary32's range where the result is well inside it."""
import numpy as np
import pytest
import torch

from tests.test_gpu_linear_attention import check, dev, index, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [2.0 ** -20, 2.0 ** 14, 2.0 ** 25], ids=["2^-20", "2^14", "2^25"])
@pytest.mark.parametrize("rate", [0.01, 0.3, 0.6, 0.9, 3.0, "late"], ids=str)
@pytest.mark.parametrize("n,dim", [(9, 128), (64, 64), (200, 128), (1200, 64), (1200, 128)])
def test_large_values(n, dim, rate, size):
    """The decays of a chunk of 64 tokens come to 1, 27, 55 and 83 powers of two and more, or
    to 300 in its middle.  With values of 2^25 a chunk's sum of |q.k| |v| is 2^(25 + 25 + 3.5 + 25)
    times 64 tokens at most, below the 2^87 that include/prism.h allows; with 2^-20 scores and
    states lie above 2^-60, from where on they have all their bits."""
    q, k, v, g = make(int(n + dim), [n], 1, 2, dim, dim)
    q, k, v = (x * np.float32(size) for x in (q, k, v))     # powers of two: still bf16
    if rate == "late":
        g[:] = -0.01
        g[min(n, 64) // 2::64] = -200.0
    else:
        g[:] = -rate
    state = (np.random.default_rng(n).standard_normal((1, 2, dim, dim)) * size ** 2).astype(np.float32)
    dstate = dev(state, torch.float32)
    got = run((q, k, v, g), [n], dstate, index([0]), index([0]))
    check((q, k, v, g), [n], state, got, dstate)
