"""What linear attention's chunks keep of values that are not bf16: three bf16 parts of
what is added to a state, two of a score and of a state that is read out.  The cases
show a part that is missing: by an exact result, or by one that is good to 2^-20."""
import numpy as np
import pytest
import torch

from tests import layer_util as u
from tests.test_gpu_linear_attention import dev, index, run

pytestmark = pytest.mark.gpu

F = np.float32
DIMS = [(128, 128), (64, 128), (128, 64), (64, 64)]
LENS = [9, 64, 100, 200, 1200]      # one chunk, several, in segments
HV = 2


def empty(n, dk, dv):
    return (np.zeros((n, 1, dk), F), np.zeros((n, 1, dk), F), np.zeros((n, HV, dv), F), np.zeros((n, HV), F))


def parts(y, count):
    """The sum of ``count`` bf16 parts of binary32 values."""
    kept = np.zeros_like(y)
    for _ in range(count):
        kept = kept + u.bf16(y - kept)
    return kept


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("n,at", [(9, 2), (64, 10), (100, 70), (200, 130), (1200, 300), (1200, 1190)])
def test_what_is_added_to_a_state(n, at, dk, dv):
    """One token with a key (of ones), and decays after it in its chunk alone: the state is its
    decayed v.  The exponential is good to 2^-22, its argument (1 at most) to 2^-25, the product to
    2^-24, three parts to 2^-25 and their two additions in the tensor cores to 2^-23 each: in all
    (1 + 1/8 + 1/4 + 1/8 + 1) 2^-22 < 2^-20.  Two parts are off by up to 2^-17."""
    rng = np.random.default_rng(n + at)
    q, k, v, g = empty(n, dk, dv)
    v[:] = u.bf16(rng.standard_normal(v.shape))
    k[at] = 1
    end = min(n, (at // 64 + 1) * 64)
    g[at + 1:end] = -rng.uniform(0.2, 0.6, (end - at - 1, HV)) / (end - at - 1)
    state = torch.full((1, HV, dk, dv), 7.0, device="cuda")
    run((q, k, v, g), [n], state, None, index([0]))
    left = np.exp(g[at + 1:].astype(np.float64).sum(0))
    want = left[:, None] * v[at].astype(np.float64)
    off = np.abs(state[0].double().cpu().numpy() - want[:, None, :])
    assert np.all(off <= 2.0 ** -20 * np.abs(want)[:, None, :]), f"{np.max(off / np.abs(want)[:, None, :]) * 2 ** 20} of the bound"
    y = want.astype(F)
    assert np.max(np.abs(parts(y, 2) - y) / np.abs(y)) > 2.0 ** -18.5     # a third part missing would show


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("n", [5] + LENS)
def test_scores(n, dk, dv):
    """Two tokens whose keys differ in the last place and whose values are opposite, no decay: what
    is left of their scores is exact in two parts, and in bf16."""
    rng = np.random.default_rng(n)
    q, k, v, g = empty(n, dk, dv)
    c = int(rng.integers(dk))
    q[:, 0, c] = u.bf16(rng.uniform(1, 2, n))
    k[0, 0, c] = 1 + F(77) / 128
    k[1, 0, c] = 1 + F(76) / 128
    v[0] = np.exp2(rng.integers(-3, 4, (HV, dv))) * rng.choice([-1, 1], (HV, dv))
    v[1] = -v[0]
    got = run((q, k, v, g), [n], None, None, None, scale=1.0).double().cpu().numpy()
    score = q[:, 0, c].astype(np.float64)[:, None, None]
    want = score * v[0] * F(1) / 128
    want[0] = u.bf16(score[0] * k[0, 0, c] * v[0])
    assert np.array_equal(got, want)
    one = [parts((q[:, 0, c] * k[j, 0, c]).astype(F), 1) for j in (0, 1)]
    assert np.any(one[0] - one[1] != q[:, 0, c] / 128)                    # a second part missing would show


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("n", [5] + LENS)
def test_a_state_that_is_read_out(n, dk, dv):
    """Two rows of a state, of 16 bits each, whose difference is exact in bf16."""
    rng = np.random.default_rng(n + 1)
    q, k, v, g = empty(n, dk, dv)
    a, b = rng.choice(dk, 2, replace=False)
    size = np.exp2(rng.integers(-4, 5, n))
    q[:, 0, a], q[:, 0, b] = size, -size
    x = rng.integers(1 << 15, (1 << 16) - 256, (HV, dv))
    m = rng.integers(1, 256, (HV, dv))
    state = rng.standard_normal((1, HV, dk, dv)).astype(F)
    state[0, :, a], state[0, :, b] = x / F(1 << 15), (x + m) / F(1 << 15)
    dstate = dev(state, torch.float32)
    got = run((q, k, v, g), [n], dstate, index([0]), index([0]), scale=1.0).double().cpu().numpy()
    assert np.array_equal(got, size[:, None, None] * (-m / float(1 << 15)))
    assert torch.equal(dstate.cpu(), torch.from_numpy(state))
    one = [parts(s[0, :, c].astype(F), 1) for s, c in ((state, a), (state, b))]
    assert np.any(one[1] - one[0] != m / F(1 << 15))                      # a second part missing would show
