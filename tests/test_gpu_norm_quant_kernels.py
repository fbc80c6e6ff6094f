"""The norms and the gated activation in each of their kernels: 1, 2 and 4 to 8 vectors of
8 channels a thread, with sigmoids formed and looked up, and CTAs that go on to a second
and third row."""
import numpy as np
import pytest
import torch

import deterministic_w8a8_int8_gb300 as prism
from tests import layer_util as u
from tests.test_gpu_norm_quant import check, dev, normal

pytestmark = pytest.mark.gpu

FEW, MANY = 7, 1400            # 1400 rows: more than two turns of two CTAs an SM, and enough for the look-up
LONG = [16384, 17408, 20496, 24576, 24592, 28672, 28688, 32768]


def again(call, few, times, form):
    """``call(times)``: the rows of ``few`` that often, the same codes each time."""
    many = call(times)
    assert torch.equal(many[0], few[0].repeat(times, 1))
    assert form == "bf16" or torch.equal(many[1], few[1].repeat(times))
    return many


@pytest.mark.parametrize("form", ["int8", "f16", "bf16"])
@pytest.mark.parametrize("k", [256, 512] + LONG)
def test_norm(k, form):
    rng = np.random.default_rng(k)
    x, d, w = normal(rng, (FEW, k), 2.0), normal(rng, (FEW, k), 0.6), rng.uniform(0.3, 2.0, k).astype(np.float32)
    post = rng.uniform(0.3, 2.0, k).astype(np.float32)
    dx, dd, dw, dp = dev(x), dev(d), dev(w, torch.float32), dev(post, torch.float32)
    for delta, p in ((None, None), (d, None), (d, post)):

        def call(n):
            return prism.prism_norm_quant(dx.repeat(n, 1), dw, delta=None if delta is None else dd.repeat(n, 1),
                                          post_weight=None if p is None else dp, form=form)

        y, h = u.norm(x, w, delta=delta, post=p)
        few = call(1)
        check(few[:2], y, form)
        assert np.array_equal(few[2].float().cpu().numpy(), h)
        many = again(call, few, MANY // FEW, form)
        assert torch.equal(many[2], few[2].repeat(MANY // FEW, 1))


@pytest.mark.parametrize("form", ["int8", "f16", "bf16"])
@pytest.mark.parametrize("f", [256, 512, 4096] + LONG)
def test_glu(f, form):
    rng = np.random.default_rng(f + 1)
    x, inv = normal(rng, (FEW, 2 * f), 1.5), rng.uniform(0.3, 2.0, f).astype(np.float32)
    dx, di = dev(x), dev(inv, torch.float32)
    times = max(MANY, 152 * 32768 // f + FEW) // FEW + 1
    for smooth in (None, inv):

        def call(n):
            return prism.prism_glu_quant(dx.repeat(n, 1), None if smooth is None else di, form=form)

        few = call(1)
        check(few, u.glu(x, inv=smooth), form)
        again(call, few, times, form)


@pytest.mark.parametrize("form", ["int8", "f16", "bf16"])
@pytest.mark.parametrize("h,d", [(2, 128), (8, 64), (16, 128), (64, 128), (65, 128), (96, 128), (128, 128), (129, 128), (160, 128), (128, 256), (512, 64)])
def test_heads(h, d, form):
    rng = np.random.default_rng(h * 7 + d)
    x, z, w = normal(rng, (FEW, h, d), 0.5), normal(rng, (FEW, h, d), 1.5), rng.uniform(0.3, 2.0, d).astype(np.float32)
    inv = rng.uniform(0.3, 2.0, h * d).astype(np.float32)
    dx, dz, dw, di = dev(x), dev(z), dev(w, torch.float32), dev(inv, torch.float32)
    times = max(MANY, 152 * 32768 // (h * d) + FEW) // FEW + 1
    for gate, smooth in ((None, inv), (z, None), (z, inv)):

        def call(n):
            return prism.prism_head_norm_quant(dx.repeat(n, 1, 1), dw, gate=None if gate is None else dz.repeat(n, 1, 1),
                                               inv_s=None if smooth is None else di, form=form)

        few = call(1)
        check(few, u.head_norm(x, w, gate=gate, inv=smooth), form)
        again(call, few, times, form)


def test_codes_are_the_quantisers():
    """Gates of 100, whose silu is 100, and values of three bits: their products are bf16 values,
    whose codes are prism_quant_act's."""
    g = torch.Generator(device="cuda").manual_seed(4)
    m = torch.randint(-7, 8, (33, 512), generator=g, device="cuda")
    up = m * torch.exp2(torch.randint(-9, 3, (33, 512), generator=g, device="cuda").float())
    x = (up * 100).to(torch.bfloat16)
    assert torch.equal(x.float(), up * 100) and torch.equal(up.to(torch.bfloat16).float(), up)
    inv = torch.rand((512,), generator=g, device="cuda") + 0.5
    both = torch.cat((torch.full_like(x, 100.0), up.to(torch.bfloat16)), dim=1)
    for smooth in (None, inv):
        got, scale = prism.prism_glu_quant(both, smooth)
        want, want_scale = prism.prism_quant_act(x, smooth)
        assert torch.equal(got, want) and torch.equal(scale, want_scale)
