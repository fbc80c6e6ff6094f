"""Operands of more than 2^31 values: rows, tokens and slots at the far end, against calls on
those alone."""
import pytest
import torch

import deterministic_w8a8_int8_gb300 as prism

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def index(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def normal(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)


@pytest.mark.parametrize("lens", [(140000, 150), (140000, 7, 1, 60)], ids=str)
def test_tokens_and_slots(lens):
    """Values of 128 heads of 128 channels: the last sequences begin behind 2^31 of them; slots of
    2^21 values, the last behind 2^31."""
    t, h, d, slots = sum(lens), 128, 128, 1030
    q, k, v = normal((t, 2, d), 1), normal((t, 2, d), 2), normal((t, h, d), 3)
    g = -torch.rand((t, h), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda") * 0.1
    assert v.numel() > 1 << 31 and (slots - len(lens)) * h * d * d > 1 << 31
    state = torch.zeros((slots, h, d, d), device="cuda")
    own = [slots - 1 - i for i in range(len(lens))]
    for i in own:
        state[i].normal_(generator=torch.Generator(device="cuda").manual_seed(i))
    start = [state[i:i + 1].clone() for i in own]
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    out = prism.prism_linear_attention(q, k, v, g, state, index(*own), index(*own), cu=index(*cu), max_len=lens[0])
    for i, n in list(enumerate(lens))[1:]:
        b, e = cu[i], cu[i + 1]
        mine = start[i]
        one = prism.prism_linear_attention(q[b:e].clone(), k[b:e].clone(), v[b:e].clone(), g[b:e].clone(), mine, index(0), index(0),
                                           cu=index(0, n))
        assert torch.equal(one, out[b:e]) and torch.equal(mine[0], state[own[i]])
    assert bool(out[-1].isfinite().all()) and not state[:slots - len(lens)].any()


def test_rows():
    k, m = 32768, 70000
    x, d = normal((m, k), 5), normal((m, k), 6)
    w = torch.rand(k, device="cuda") + 0.5
    last = slice(m - 3, m)
    assert x.numel() > 1 << 31
    one = prism.prism_norm_quant(x[last].clone(), w, delta=d[last].clone(), post_weight=w)
    all_rows = prism.prism_norm_quant(x, w, delta=d, post_weight=w)
    assert all(torch.equal(a, b[last]) for a, b in zip(one, all_rows))
    del all_rows
    one = prism.prism_glu_quant(x[last].clone(), w[:k // 2], form="f16")
    all_rows = prism.prism_glu_quant(x, w[:k // 2], form="f16")
    assert all(torch.equal(a, b[last]) for a, b in zip(one, all_rows))
    del all_rows
    heads, gate = x.view(m, 256, 128), d.view(m, 256, 128)
    one = prism.prism_head_norm_quant(heads[last].clone(), w[:128], gate=gate[last].clone(), inv_s=w)
    all_rows = prism.prism_head_norm_quant(heads, w[:128], gate=gate, inv_s=w)
    assert all(torch.equal(a, b[last]) for a, b in zip(one, all_rows))
