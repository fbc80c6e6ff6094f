"""Rows that are not finite, down to codes: the row's scale is NaN and its codes are 0
(bf16 values: not finite where they depend on what is not), as prism_quant_act_rows
marks its rows, so that the next linear's outputs are NaN; other rows are as they were."""
import math

import numpy as np
import pytest
import torch

import deterministic_w8a8_int8_gb300 as prism

pytestmark = pytest.mark.gpu

FORMS = ["int8", "f16", "bf16"]
BAD = [math.nan, -math.nan, math.inf, -math.inf]


def normal(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def compare(call, form, rows, spoilt, where):
    """``call()`` before and after ``spoilt()``; ``where`` the values of a bad row that are not finite."""
    before = [None if t is None else t.clone() for t in call()[:2]]
    spoilt()
    q, scale = call()[:2]
    good = [i for i in range(q.shape[0]) if i not in rows]
    assert torch.equal(q[good], before[0][good]) and (form == "bf16" or torch.equal(scale[good], before[1][good]))
    if form == "bf16":
        assert scale is None and not bool(q[rows][:, where].isfinite().any())
    else:
        assert bool(scale[rows].isnan().all()) and not q[rows].any() and bool(before[1].isfinite().all())


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bad", BAD, ids=str)
@pytest.mark.parametrize("m,k", [(3, 16), (5, 256), (7, 1040), (2500, 5120), (3, 20480), (3, 32768)])
def test_norm(m, k, bad, form):
    w = torch.rand(k, device="cuda") + 0.5
    rows = [0, m - 1]
    for post in (None, w):
        for at in ("x", "delta"):
            x, d = normal((m, k), 1), normal((m, k), 2)
            into = x if at == "x" else d

            def spoil():
                into[0, k - 1] = bad
                into[m - 1, 0] = bad

            compare(lambda: prism.prism_norm_quant(x, w, delta=d, post_weight=post, form=form), form, rows, spoil, slice(None))
    x = normal((m, k), 3)

    def spoil():
        x[rows, k // 2] = bad

    compare(lambda: prism.prism_norm_quant(x, w, form=form), form, rows, spoil, slice(None))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bad", BAD, ids=str)
@pytest.mark.parametrize("m,h,d", [(3, 1, 64), (5, 3, 128), (2500, 40, 128), (3, 70, 256), (3, 512, 64)])
def test_heads(m, h, d, bad, form):
    w, inv = torch.rand(d, device="cuda") + 0.5, torch.rand(h * d, device="cuda") + 0.5
    rows, head = [0, m - 1], slice((h - 1) * d, h * d)
    for gated in (False, True):
        x, z = normal((m, h, d), 4), normal((m, h, d), 5) if gated else None

        def spoil():
            x[rows, h - 1, 7] = bad

        compare(lambda: prism.prism_head_norm_quant(x, w, gate=z, inv_s=inv, form=form), form, rows, spoil, head)
    x, z = normal((m, h, d), 4), normal((m, h, d), 5)

    def spoil_gate():
        z[rows, h - 1, d - 1] = bad

    compare(lambda: prism.prism_head_norm_quant(x, w, gate=z, form=form), form, rows, spoil_gate, slice(h * d - 1, h * d))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bad", BAD, ids=str)
@pytest.mark.parametrize("m,f", [(3, 16), (5, 1040), (2500, 4096), (400, 17408), (3, 32768)])
def test_glu(m, f, bad, form):
    rows = [0, m - 1]
    for at in (f - 1, f):      # the last gate, the first value
        x = normal((m, 2 * f), 6)

        def spoil():
            x[rows, at] = bad

        compare(lambda: prism.prism_glu_quant(x, form=form), form, rows, spoil, slice(at % f, at % f + 1))


def test_a_malformed_sequence_reaches_the_next_linear():
    """Linear attention's NaN rows go through the heads' norm into a linear: its rows are NaN, the others as without them."""
    h, d, n = 2, 128, 64
    lens = [12, 3, 20]
    t = sum(lens)
    q, k, v, z = (normal((t, h, d), s) for s in range(4))
    g = torch.full((t, h), -0.1, device="cuda")
    state = torch.zeros((3, h, d, d), device="cuda")
    cu = torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32, device="cuda")
    w = torch.randint(-127, 128, (n, h * d), dtype=torch.int8, device="cuda")
    ws, weight = torch.rand(n, device="cuda") * 1e-3, torch.ones(d, device="cuda")

    def run(first, form):
        first = torch.tensor(first, dtype=torch.int32, device="cuda")
        y = prism.prism_linear_attention(q, k, v, g, state, first, cu=cu, max_len=20)
        codes, scale = prism.prism_head_norm_quant(y, weight, gate=z, form=form)
        if form == "int8":
            return prism.prism_w8a8_linear(codes, scale, w, ws)
        return prism.prism_w8a8_linear_f16(codes, scale, w.to(torch.float16), ws)

    for form in ("int8", "f16"):
        want = run([0, 1, 2], form)
        for i, (b, e) in enumerate(((0, 12), (12, 15), (15, 35))):
            got = run([9 if s == i else s for s in range(3)], form)
            good = [r for r in range(t) if not b <= r < e]
            assert bool(got[b:e].isnan().all()) and torch.equal(got[good], want[good]) and bool(want.isfinite().all())
