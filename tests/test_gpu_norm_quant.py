"""Norms and the gated activation down to codes: bit for bit their restatement in
binary32, whatever the batch, the strides and the form."""
import numpy as np
import pytest
import torch

import deterministic_w8a8_int8_gb300 as prism
from tests import layer_util as u

pytestmark = pytest.mark.gpu

ROWS = [(1, 16), (3, 64), (37, 256), (305, 1040), (1700, 80), (5, 4096), (7, 5120), (2, 8208), (3, 17408), (2, 20480), (2, 24592),
        (2, 28672), (2, 32768)]


def normal(rng, shape, std=1.0):
    x = rng.standard_normal(shape) * std
    x[..., rng.integers(0, shape[-1], max(1, shape[-1] // 50))] *= 30.0
    return u.bf16(x)


def dev(x, dtype=torch.bfloat16):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(dtype).cuda()


def check(got, want_y, form):
    q, scale = u.codes(want_y, form)
    if form == "bf16":
        assert got[1] is None and np.array_equal(got[0].float().cpu().numpy(), q)
    else:
        assert np.array_equal(got[1].cpu().numpy(), scale)
        assert got[0].dtype == (torch.int8 if form == "int8" else torch.float16)
        assert np.array_equal(got[0].cpu().numpy(), q)


@pytest.mark.parametrize("form", ["int8", "f16", "bf16"])
@pytest.mark.parametrize("m,k", ROWS)
def test_norm(m, k, form):
    rng = np.random.default_rng(m * 100003 + k)
    x, w = normal(rng, (m, k), 2.0), rng.uniform(0.3, 2.0, k).astype(np.float32)
    delta, post = normal(rng, (m, k), 0.6), rng.uniform(0.3, 2.0, k).astype(np.float32)
    for kw in (dict(), dict(delta=delta), dict(delta=delta, alpha=0.37), dict(delta=delta, alpha=-1.5, post=post)):
        y, h = u.norm(x, w, **kw)
        q, scale, got_h = prism.prism_norm_quant(dev(x), dev(w, torch.float32), delta=dev(kw.get("delta")),
                                                 alpha=kw.get("alpha", 1.0), post_weight=dev(kw.get("post"), torch.float32),
                                                 form=form)
        assert np.array_equal(got_h.float().cpu().numpy(), h)
        check((q, scale), y, form)


@pytest.mark.parametrize("form", ["int8", "f16", "bf16"])
@pytest.mark.parametrize("m,h,d", [(1, 1, 64), (3, 5, 64), (305, 3, 128), (41, 40, 128), (9, 7, 256), (2, 64, 256), (2, 128, 256), (3, 100, 128)])
def test_head_norm(m, h, d, form):
    rng = np.random.default_rng(m * 1009 + h * 31 + d)
    x, gate = normal(rng, (m, h, d), 0.5), normal(rng, (m, h, d), 1.5)
    w, inv = rng.uniform(0.3, 2.0, d).astype(np.float32), rng.uniform(0.3, 2.0, h * d).astype(np.float32)
    for kw in (dict(), dict(gate=gate), dict(inv=inv), dict(gate=gate, inv=inv)):
        got = prism.prism_head_norm_quant(dev(x), dev(w, torch.float32), gate=dev(kw.get("gate")),
                                          inv_s=dev(kw.get("inv"), torch.float32), form=form)
        check(got, u.head_norm(x, w, **kw), form)


@pytest.mark.parametrize("form", ["int8", "f16", "bf16"])
@pytest.mark.parametrize("m,f", ROWS)
def test_glu(m, f, form):
    rng = np.random.default_rng(m * 7919 + f)
    x, inv = normal(rng, (m, 2 * f), 1.5), rng.uniform(0.3, 2.0, f).astype(np.float32)
    for kw in (dict(), dict(inv=inv)):
        check(prism.prism_glu_quant(dev(x), dev(kw.get("inv"), torch.float32), form=form), u.glu(x, **kw), form)


def test_rows_at_48_kb_of_shared_memory():
    """Two operands' rows of 12288 channels ahead, and a kernel's own arrays."""
    rng = np.random.default_rng(48)
    x, d, w = normal(rng, (3, 12288), 2.0), normal(rng, (3, 12288)), rng.uniform(0.3, 2.0, 12288).astype(np.float32)
    y, h = u.norm(x, w, delta=d)
    q, scale, got_h = prism.prism_norm_quant(dev(x), dev(w, torch.float32), delta=dev(d))
    check((q, scale), y, "int8")
    assert np.array_equal(got_h.float().cpu().numpy(), h)
    check(prism.prism_glu_quant(dev(np.concatenate((x, d), axis=1))), u.glu(np.concatenate((x, d), axis=1)), "int8")
    x, d, w = x.reshape(3, 96, 128), d.reshape(3, 96, 128), w[:128]
    check(prism.prism_head_norm_quant(dev(x), dev(w, torch.float32), gate=dev(d)), u.head_norm(x, w, gate=d), "int8")


def test_every_gate():
    """silu of every finite bf16 gate of magnitude below 2^40."""
    bits = np.arange(1 << 16, dtype=np.uint32)
    z = (bits << 16).view(np.float32)
    z = np.where(np.abs(z) < 2.0 ** 40, z, 0).astype(np.float32)
    x = np.concatenate((z.reshape(16, 4096), np.ones((16, 4096), np.float32)), axis=1)
    for form in ("bf16", "int8"):
        check(prism.prism_glu_quant(dev(x), form=form), u.glu(x), form)
    for up in (1.0, 1.203125, 1.6640625):       # to the last bits: a row's scale is its one value's, over 127
        rows = np.stack([z] * 16 + [np.full_like(z, up)] * 16, axis=1)
        check(prism.prism_glu_quant(dev(rows)), u.glu(rows), "int8")
    exact = z.astype(np.float64) / (1.0 + np.exp(-np.clip(z.astype(np.float64), -700, 700)))
    # the exponential and three more steps: 2^-21 of the value; results below 2^-126 become 0
    assert np.all(np.abs(u.silu(z) - exact) <= 2.0 ** -21 * np.abs(exact) + 2.0 ** -86)


@pytest.mark.parametrize("k", [2048, 4096])
def test_every_gate_of_many_rows(k):
    """The same codes where CTAs look the sigmoids up."""
    z = (np.arange(1 << 16, dtype=np.uint32) << 16).view(np.float32)
    z = np.where(np.abs(z) < 2.0 ** 40, z, 0).astype(np.float32).reshape(-1, k)
    m, rng = z.shape[0], np.random.default_rng(9)
    times = -(-5200000 // (m * k)) + 1
    up, x, w = normal(rng, (m, k)), normal(rng, (m, k // 128, 128)), rng.uniform(0.3, 2.0, 128).astype(np.float32)
    for form in ("bf16", "int8"):
        few = prism.prism_glu_quant(dev(np.concatenate((z, up), axis=1)), form=form)
        many = prism.prism_glu_quant(dev(np.tile(np.concatenate((z, up), axis=1), (times, 1))), form=form)
        check(few, u.glu(np.concatenate((z, up), axis=1)), form)
        assert torch.equal(many[0], few[0].repeat(times, 1)) and (form == "bf16" or torch.equal(many[1], few[1].repeat(times)))
        gate = z.reshape(x.shape)
        few = prism.prism_head_norm_quant(dev(x), dev(w, torch.float32), gate=dev(gate), form=form)
        many = prism.prism_head_norm_quant(dev(np.tile(x, (times, 1, 1))), dev(w, torch.float32), gate=dev(np.tile(gate, (times, 1, 1))),
                                           form=form)
        check(few, u.head_norm(x, w, gate=gate), form)
        assert torch.equal(many[0], few[0].repeat(times, 1)) and (form == "bf16" or torch.equal(many[1], few[1].repeat(times)))


def test_strides_and_in_place():
    rng = np.random.default_rng(5)
    m, k = 19, 272
    x, delta, w = normal(rng, (m, k), 2.0), normal(rng, (m, k)), rng.uniform(0.3, 2.0, k).astype(np.float32)
    y, h = u.norm(x, w, delta=delta, alpha=0.5)

    def wide(v, ld):
        buf = torch.full((m, ld), 7.0, dtype=torch.bfloat16, device="cuda")
        buf[:, :k] = dev(v)
        return buf

    for place in ("x", "delta", "other"):
        bx, bd = wide(x, k + 24), wide(delta, k + 8)
        bh = dict(x=bx, delta=bd, other=wide(x, k + 40))[place]
        q, s, got = prism.prism_norm_quant(bx[:, :k], dev(w, torch.float32), delta=bd[:, :k], alpha=0.5, h=bh[:, :k])
        assert got.data_ptr() == bh.data_ptr() and np.array_equal(got.float().cpu().numpy(), h)
        check((q, s), y, "int8")
        assert bool((bh[:, k:] == 7).all())
    buf = torch.full((m, 3 * k + 8), 9.0, dtype=torch.bfloat16, device="cuda")      # gate/up inside wider rows
    buf[:, k:3 * k] = dev(np.concatenate((x, delta), axis=1))
    check(prism.prism_glu_quant(buf[:, k:3 * k]), u.glu(np.concatenate((x, delta), axis=1)), "int8")
    heads = torch.full((m, 6, 64), 9.0, dtype=torch.bfloat16, device="cuda")       # heads 1 .. 4 of six
    heads[:, 1:5] = dev(x[:, :256].reshape(m, 4, 64))
    check(prism.prism_head_norm_quant(heads[:, 1:5], dev(w[:64], torch.float32)), u.head_norm(x[:, :256].reshape(m, 4, 64), w[:64]), "int8")


def test_zero_tiny_and_large_rows():
    rng = np.random.default_rng(6)
    k = 1024
    x = normal(rng, (6, k), 1.0)
    x[0] = 0
    x[1] *= 2.0 ** -70
    x[2] *= 2.0 ** 34
    x[3] = 0
    x[3, 17] = 2.0 ** 39
    x[4] = u.bf16(x[4] * np.exp2(rng.integers(-60, 30, k)))
    w = np.ones(k, np.float32)
    for form in ("int8", "bf16"):
        q, s, _ = prism.prism_norm_quant(dev(x), dev(w, torch.float32), form=form)
        check((q, s), u.norm(x, w)[0], form)
    q, s, _ = prism.prism_norm_quant(dev(x), dev(w, torch.float32), eps=1e-20)
    check((q, s), u.norm(x, w, eps=1e-20)[0], "int8")
    assert float(s[0]) == 0 and not q[0].any()
    wz = np.concatenate((x, np.ones_like(x)), axis=1)
    check(prism.prism_glu_quant(dev(wz)), u.glu(wz), "int8")


def test_a_row_does_not_depend_on_the_batch():
    g = torch.Generator(device="cuda").manual_seed(3)
    x, d = (torch.randn((4000, 5120), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = torch.rand((5120,), generator=g, device="cuda") + 0.5
    q, s, h = prism.prism_norm_quant(x, w, delta=d, post_weight=w)
    for i in (0, 1, 1234, 3999):
        qi, si, hi = prism.prism_norm_quant(x[i:i + 1], w, delta=d[i:i + 1], post_weight=w)
        assert torch.equal(qi[0], q[i]) and torch.equal(si[0], s[i]) and torch.equal(hi[0], h[i])


def test_codes_are_the_quantisers():
    """The codes of bf16 values that need no norm: prism_quant_act's."""
    g = torch.Generator(device="cuda").manual_seed(4)
    up = torch.randn((33, 512), generator=g, device="cuda").to(torch.bfloat16)
    inv = torch.rand((512,), generator=g, device="cuda") + 0.5
    gate = torch.full_like(up, 100.0)                 # silu(100) = 100
    got, scale = prism.prism_glu_quant(torch.cat((gate, up / 128), dim=1), inv)
    want, want_scale = prism.prism_quant_act((up / 128 * 100).to(torch.bfloat16), inv)
    exact = (up / 128).float() * 100.0
    if torch.equal(exact.to(torch.bfloat16).float(), exact):
        assert torch.equal(got, want) and torch.equal(scale, want_scale)
    gate = torch.full_like(up, 64.0)                  # silu(64) = 64, exactly in bf16 afterwards
    got, scale = prism.prism_glu_quant(torch.cat((gate, up / 64), dim=1), inv)
    want, want_scale = prism.prism_quant_act(up, inv)
    assert torch.equal(got, want) and torch.equal(scale, want_scale)


def test_streams_and_graphs():
    g = torch.Generator(device="cuda").manual_seed(5)
    x, d = (torch.randn((65, 640), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = torch.rand((640,), generator=g, device="cuda") + 0.5
    want = prism.prism_norm_quant(x, w, delta=d)
    glu = prism.prism_glu_quant(torch.cat((x, d), 1))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = prism.prism_norm_quant(x, w, delta=d, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    buf = torch.zeros_like(x)
    both = torch.cat((x, d), 1)
    with torch.cuda.graph(graph):
        q, s, h = prism.prism_norm_quant(buf, w, delta=d)
        q2, s2 = prism.prism_glu_quant(both)
    for _ in range(2):
        buf.copy_(x)
        graph.replay()
        assert torch.equal(q, want[0]) and torch.equal(s, want[1]) and torch.equal(h, want[2])
        assert torch.equal(q2, glu[0]) and torch.equal(s2, glu[1])


def test_one_row_of_any_stride():
    x = torch.randn((4096, 1), device="cuda").to(torch.bfloat16).t()
    w = torch.rand((4096,), device="cuda") + 0.5
    assert x.stride() == (1, 1)
    got, want = prism.prism_norm_quant(x, w, delta=x), prism.prism_norm_quant(x.contiguous(), w, delta=x.contiguous())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got, want = prism.prism_glu_quant(x), prism.prism_glu_quant(x.clone(memory_format=torch.contiguous_format))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    heads = x.reshape(32, 1, 128).transpose(0, 1)
    got, want = prism.prism_head_norm_quant(heads, w[:128]), prism.prism_head_norm_quant(x.reshape(1, 32, 128).contiguous(), w[:128])
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_empty():
    w = torch.ones(64, device="cuda")
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    q, s, h = prism.prism_norm_quant(x, w, delta=x)
    assert q.shape == (0, 64) and s.shape == (0,) and h.shape == (0, 64)
    assert prism.prism_glu_quant(x)[0].shape == (0, 32)
    assert prism.prism_head_norm_quant(x.view(0, 1, 64), w)[0].shape == (0, 64)


@pytest.mark.parametrize("call", [
    lambda x, w: prism.prism_norm_quant(x, w.half()),
    lambda x, w: prism.prism_norm_quant(x, w[:32]),
    lambda x, w: prism.prism_norm_quant(x, None),
    lambda x, w: prism.prism_norm_quant(x.float(), w),
    lambda x, w: prism.prism_norm_quant(x, w, delta=x[:2]),
    lambda x, w: prism.prism_norm_quant(x, w, h=x),                       # nothing is added
    lambda x, w: prism.prism_norm_quant(x, w, post_weight=w),
    lambda x, w: prism.prism_norm_quant(x, w, form="fp8"),
    lambda x, w: prism.prism_norm_quant(x, w, form=0),
    lambda x, w: prism.prism_norm_quant(x.t(), w[:4]),
    lambda x, w: prism.prism_glu_quant(x[:, :63]),
    lambda x, w: prism.prism_glu_quant(x, w),
    lambda x, w: prism.prism_head_norm_quant(x.view(4, 1, 64), w, gate=x),
    lambda x, w: prism.prism_head_norm_quant(torch.empty((4, 2, 128), dtype=torch.bfloat16, device="cuda")[:, :, :64], w),
    lambda x, w: prism.prism_norm_quant(x, w, eps=0.0),
])
def test_refusals(call):
    x, w = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises((TypeError, ValueError, prism.PrismError)):
        call(x, w)
