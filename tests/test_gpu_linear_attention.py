"""Linear attention with a decay for each head against its recurrence in 64 bits."""
import math

import numpy as np
import pytest
import torch

import deterministic_w8a8_int8_gb300 as prism
from tests import layer_util as u

pytestmark = pytest.mark.gpu


def make(seed, lens, hk, hv, dk, dv, decay="token", rate=(2.0, 7.0), pad=0):
    """Packed inputs (float32 values of bf16) with ``pad`` rows of NaN behind the last sequence."""
    rng = np.random.default_rng(seed)
    t = sum(lens)
    q, k, v = (u.bf16(rng.standard_normal((t + pad, h, d))) for h, d in ((hk, dk), (hk, dk), (hv, dv)))
    g = -np.exp2(-rng.uniform(*rate, hv))
    if decay == "token":
        g = g * rng.exponential(1.0, (t + pad, hv))
    g = g.astype(np.float32)
    for x in (q, k, v) + ((g,) if decay == "token" else ()):
        x[t:] = np.nan
    return q, k, v, g


def dev(x, dtype=torch.bfloat16):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).cuda()


def offsets(lens):
    return torch.tensor(np.concatenate(([0], np.cumsum(lens))), dtype=torch.int32, device="cuda")


def index(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(data, lens, state, first, last, **kw):
    q, k, v, g = data
    out = torch.full(v.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    prism.prism_linear_attention(dev(q), dev(k), dev(v), dev(g, torch.float32), state, state_in=first, state_out=last,
                                 cu=offsets(lens), out=out, **{"max_len": max(max(lens), 1), **kw})
    return out


def check(data, lens, start, got, states, scale=None):
    q, k, v, g = data
    t, dk = sum(lens), q.shape[2]
    g = g[:t] if g.ndim == 2 else g
    want, bound, after, after_bound = u.linear_attention(q[:t], k[:t], v[:t], g, start, lens, dk ** -0.5 if scale is None else scale)
    off = np.abs(got[:t].double().cpu().numpy() - want)
    assert np.all(off <= bound), f"out: {np.max(off / bound)} of the bound"
    assert bool((got[t:] == 5).all())
    off = np.abs(states.double().cpu().numpy() - after)
    assert np.all(off <= after_bound), f"state: {np.max(off / after_bound)} of the bound"


LENS = [[1], [1, 1, 1], [2, 8, 7], [9], [2, 16, 15], [17], [63, 64, 65], [0, 1, 130, 0, 40, 16], [255, 3, 256, 257], [511], [512], [513, 1], [1100, 1023], [1024], [2600, 17, 1537], [1536], [384, 768, 767]]


@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("hk,hv,dk,dv,decay", [(1, 1, 128, 128, "token"), (2, 6, 64, 128, "head"), (2, 2, 128, 64, "token"), (1, 3, 64, 64, "token")])
def test_against_the_recurrence(lens, hk, hv, dk, dv, decay):
    """Sequences that go on from their own slots, from zeros, and keep nothing."""
    data = make(len(lens) * 7 + sum(lens), lens, hk, hv, dk, dv, decay, pad=5)
    rng = np.random.default_rng(1)
    n = len(lens)
    slots = rng.permutation(n + 2)[:n]
    state = rng.standard_normal((n + 2, hv, dk, dv)).astype(np.float32) * 3
    first = np.where(np.arange(n) % 3 == 2, -1, slots)
    start = np.where((first >= 0)[:, None, None, None], state[slots], 0)
    dstate = dev(state, torch.float32)
    got = run(data, lens, dstate, index(first), index(slots))
    check(data, lens, start, got, dstate[index(slots).long()])
    others = [i for i in range(n + 2) if i not in slots]
    assert np.array_equal(dstate[others].cpu().numpy(), state[others])
    again = run(data, lens, None, None, None)         # from zeros, nothing kept
    check(data, lens, np.zeros_like(start), again, torch.from_numpy(u.linear_attention(*(x[:sum(lens)] if x.ndim > 1 else x for x in data), np.zeros_like(start), lens, 1.0)[2]))


def test_one_token_each_without_offsets():
    data = make(3, [1] * 7, 2, 4, 128, 128)
    state = np.random.default_rng(2).standard_normal((7, 4, 128, 128)).astype(np.float32)
    dstate = dev(state, torch.float32)
    own = index(list(range(7)))
    out = prism.prism_linear_attention(*(dev(x) for x in data[:3]), dev(data[3], torch.float32), dstate, own, own)
    check(data, [1] * 7, state, torch.cat((out, torch.full_like(out[:1], 5.0))), dstate)


def test_branches_of_one_parent():
    """Several sequences start from one state and leave it as it is."""
    lens = [16, 48, 1, 300]
    data = make(4, lens, 2, 4, 128, 128)
    state = np.random.default_rng(3).standard_normal((6, 4, 128, 128)).astype(np.float32)
    dstate = dev(state, torch.float32)
    got = run(data, lens, dstate, index([5] * 4), index([0, 1, 2, -1]))
    start = np.repeat(state[5:], 4, 0)
    q, k, v, g = data
    after = u.linear_attention(q, k, v, g, start, lens, 1.0)[2]
    check(data, lens, start, got, torch.cat((dstate[:3].cpu(), torch.from_numpy(after[3:]).float())))
    assert np.array_equal(dstate[3:].cpu().numpy(), state[3:])


def test_a_text_in_pieces():
    """Pieces that hand the state on, against the whole text."""
    lens = [2300]
    data = make(5, lens, 1, 2, 128, 128)
    dstate = torch.zeros((1, 2, 128, 128), device="cuda")
    outs, at = [], 0
    for n in (1, 130, 16, 17, 1500, 636):
        piece = tuple(x[at:at + n] for x in data)
        outs.append(run(piece, [n], dstate, index([0]), index([0])))
        at += n
    assert at == 2300
    check(data, lens, np.zeros((1, 2, 128, 128)), torch.cat(outs), dstate)


@pytest.mark.parametrize("kind", ["-inf", "strong", "mixed", "growing", "none"])
@pytest.mark.parametrize("lens", [[9], [200], [1200]], ids=str)
@pytest.mark.parametrize("dim", [64, 128])
def test_decays(lens, kind, dim):
    data = list(make(6, lens, 1, 3, dim, dim))
    g = data[3]
    if kind == "-inf":
        g[::7] = -np.inf
    elif kind == "strong":
        g[:] = -30.0
    elif kind == "mixed":            # a long sum before small ones
        g[:20] = -200.0
        g[3] = -1e30
    elif kind == "growing":
        g[:] = 0.01
    else:
        g[:] = 0.0
    state = np.random.default_rng(4).standard_normal((1, 3, dim, dim)).astype(np.float32)
    dstate = dev(state, torch.float32)
    got = run(data, lens, dstate, index([0]), index([0]))
    check(data, lens, state, got, dstate)


@pytest.mark.parametrize("dk", [64, 128])
def test_strides_scale_and_rows_past_the_end(dk):
    lens = [70, 5]
    q, k, v, g = make(7, lens, 2, 4, dk, 128)
    t = sum(lens)
    buf = torch.full((t, 2, 3 * dk + 8), math.nan, dtype=torch.bfloat16, device="cuda")     # q and k of wider rows
    buf[..., :dk], buf[..., 2 * dk:3 * dk] = dev(q), dev(k)
    vb = torch.full((4, t, 136), math.nan, dtype=torch.bfloat16, device="cuda")              # heads outermost
    vb[..., :128] = dev(v).transpose(0, 1)
    gb = torch.full((t, 9), math.nan, device="cuda")
    gb[:, :4] = dev(g, torch.float32)
    ob = torch.full((t, 4, 160), 5.0, dtype=torch.bfloat16, device="cuda")
    out = prism.prism_linear_attention(buf[..., :dk], buf[..., 2 * dk:3 * dk], vb[..., :128].transpose(0, 1), gb[:, :4],
                                       cu=offsets(lens), max_len=70, scale=-0.3, out=ob[..., :128])
    assert bool((ob[..., 128:] == 5).all())
    want, bound, *_ = u.linear_attention(q, k, v, g, np.zeros((2, 4, dk, 128)), lens, -0.3)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= bound)


def test_bits_do_not_depend_on_the_batch():
    lens = [5, 1900, 17, 64, 300, 8, 0, 1, 9]
    data = make(8, lens, 2, 4, 128, 128)
    state = dev(np.random.default_rng(5).standard_normal((9, 4, 128, 128)), torch.float32)
    own = index(list(range(9)))
    all_state = state.clone()
    got = run(data, lens, all_state, own, own)
    at = 0
    for i, n in enumerate(lens):
        alone = state.clone()
        piece = tuple(x[at:at + n] for x in data)
        for most in {max(n, 1), 8 if n <= 8 else n, 1900}:
            alone = state.clone()
            one = run(piece, [n], alone, index([i]), index([i]), max_len=most)
            assert torch.equal(one, got[at:at + n]) and torch.equal(alone[i], all_state[i])
        at += n


def test_many_sequences_of_few_tokens():
    """Enough of them that a head is one CTA's, and few, in slices: the same bits."""
    lens = [1, 3, 8, 0] * 30
    data = make(9, lens, 4, 4, 128, 128)
    state = dev(np.random.default_rng(6).standard_normal((120, 4, 128, 128)), torch.float32)
    own = index(list(range(120)))
    many = state.clone()
    got = run(data, lens, many, own, own)
    few, n = state.clone(), sum(lens[:8])
    one = run(tuple(x[:n] for x in data), lens[:8], few, own[:8], own[:8])
    assert torch.equal(one, got[:n]) and torch.equal(few[:8], many[:8])
    check(data, lens, state.cpu().numpy(), got, many)


def test_more_work_than_places():
    """More items (sequence, head, segment) than SMs: each CTA has several, of several chunks."""
    lens = [2100, 70, 1100, 3]
    data = make(12, lens, 6, 48, 128, 128)
    state = np.random.default_rng(10).standard_normal((4, 48, 128, 128)).astype(np.float32)
    dstate = dev(state, torch.float32)
    own = index([3, 1, 0, 2])
    got = run(data, lens, dstate, own, own)
    check(data, lens, state[[3, 1, 0, 2]], got, dstate[own.long()])


@pytest.mark.parametrize("dim", [64, 128])
def test_errors(dim):
    lens = [20, 3, 40, 2, 300]
    data = make(10, lens, 1, 2, dim, dim)
    state = np.random.default_rng(7).standard_normal((5, 2, dim, dim)).astype(np.float32)
    for first, last, most, bit, bad in (
            ([0, 5, 2, 3, 4], [0, 1, 2, 3, 4], 300, 128, [1]), ([0, 1, -2, 3, 4], [0, 1, 2, 3, 4], 300, 128, [2]),
            ([0, 1, 2, 3, 4], [0, 1, 2, 3, 1 << 30], 300, 128, [4]), ([0, 1, 2, 3, 4], [-7, 1, 2, 3, 4], 300, 128, [0]),
            ([0, 1, 2, 3, 4], [0, 1, 2, 3, 4], 39, 64, [2, 4]), ([0, 1, 2, 3, 4], [0, 1, 2, 3, 4], 2, 64, [0, 1, 2, 4])):
        err = index([0])
        dstate = dev(state, torch.float32)
        got = run(data, lens, dstate, index(first), index(last), max_len=most, err=err)
        assert int(err) == bit
        at = 0
        for i, n in enumerate(lens):
            rows = got[at:at + n]
            assert bool(rows.isnan().all()) if i in bad else bool(rows.isfinite().all())
            assert torch.equal(dstate[i].cpu(), torch.from_numpy(state[i])) == (i in bad)
            at += n
    cu = index([0, 20, 10, 400, 65, 365])      # two that end before they begin or behind the rows
    err, dstate = index([0]), dev(state, torch.float32)
    out = torch.full((365, 2, dim), 5.0, dtype=torch.bfloat16, device="cuda")
    own = index([0, 1, 2, 3, 4])
    prism.prism_linear_attention(*(dev(x) for x in data[:3]), dev(data[3], torch.float32), dstate, own, own, cu=cu,
                                 max_len=300, out=out, err=err)
    assert int(err) == 64 and bool((out[20:65] == 5).all()) and bool(out[65:].isfinite().all())
    assert np.array_equal(dstate[1:4].cpu().numpy(), state[1:4])


def test_streams_graphs_and_given_workspaces():
    lens = [1600, 30]
    data = make(11, lens, 2, 4, 128, 128)
    args = [dev(x) for x in data[:3]] + [dev(data[3], torch.float32)]
    state = dev(np.random.default_rng(8).standard_normal((2, 4, 128, 128)), torch.float32)
    own, cu = index([0, 1]), offsets(lens)
    want_state = state.clone()
    want = prism.prism_linear_attention(*args, want_state, own, own, cu=cu, max_len=1600)
    size = prism.prism_linear_attention_workspace_bytes(2, 1630, 1600, 4, 128, 128)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")       # any contents
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mine = state.clone()
    side.wait_stream(torch.cuda.current_stream())
    got = prism.prism_linear_attention(*args, mine, own, own, cu=cu, max_len=1600, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(mine, want_state)
    graph = torch.cuda.CUDAGraph()
    buf = state.clone()
    with torch.cuda.graph(graph):
        out = prism.prism_linear_attention(*args, buf, own, own, cu=cu, max_len=1600)
    for _ in range(2):
        buf.copy_(state)
        graph.replay()
        assert torch.equal(out, want) and torch.equal(buf, want_state)


def test_no_wait_runs_out_beside_other_work():
    """Long sequences again and again, while copies on another stream take the memory's time."""
    g = torch.Generator(device="cuda").manual_seed(11)
    q, k, v = (torch.randn((16383, 8, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    decay = -torch.rand((16383, 8), generator=g, device="cuda") * 0.1
    state = torch.zeros((2, 8, 128, 128), device="cuda")
    out_to = torch.zeros((1,), dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 16383], dtype=torch.int32, device="cuda")
    big, side = torch.empty((1 << 28,), dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
    to = torch.empty_like(big)
    prism.prism_device_status()
    first = prism.prism_linear_attention(q, k, v, decay, state, state_out=out_to, cu=cu)
    for i in range(300):
        with torch.cuda.stream(side):
            to.copy_(big)
        last = prism.prism_linear_attention(q, k, v, decay, state, state_out=out_to, cu=cu)
    torch.cuda.synchronize()
    assert prism.prism_device_status() == 0 and torch.equal(first, last)


def test_states_without_tokens():
    state = dev(np.random.default_rng(9).standard_normal((3, 2, 64, 64)), torch.float32)
    keep = state.clone()
    empty = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    out = prism.prism_linear_attention(empty, empty, empty, torch.empty((0, 2), device="cuda"), state, index([0, -1]),
                                       index([2, 1]), cu=index([0, 0, 0]))
    assert out.shape == (0, 2, 64)
    assert torch.equal(state[2], keep[0]) and torch.equal(state[0], keep[0]) and not state[1].any()


@pytest.mark.parametrize("kw", [
    dict(state_in=index, state=None), dict(max_len=0), dict(log_decay="wide"), dict(cu="short"), dict(state="small"),
    dict(out="float"), dict(workspace="small"), dict(scale=math.nan), dict(k="short")])
def test_refusals(kw):
    q = torch.zeros((1600, 2, 64), dtype=torch.bfloat16, device="cuda")
    g = torch.zeros((1600, 2), device="cuda")
    d = dict(k=q, state=torch.zeros((2, 2, 64, 64), device="cuda"), state_in=None, state_out=None, cu=index([0, 1600]), max_len=1600)
    d.update(kw)
    if d.get("log_decay") == "wide":
        g = torch.zeros((1600, 3), device="cuda")
    d.pop("log_decay", None)
    if d["cu"] == "short" if isinstance(d["cu"], str) else False:
        d["cu"] = index([])
    if isinstance(d["state"], str):
        d["state"] = torch.zeros((2, 2, 64, 32), device="cuda")
    if isinstance(d.get("out"), str):
        d["out"] = q.float()
    if isinstance(d.get("workspace"), str):
        d["workspace"] = torch.zeros((512,), dtype=torch.uint8, device="cuda")
    if isinstance(d["k"], str):
        d["k"] = q[:5]
    if callable(d["state_in"]):
        d["state_in"] = index([0])
    k = d.pop("k")
    with pytest.raises((TypeError, ValueError, prism.PrismError)):
        prism.prism_linear_attention(q, k, q, g, d.pop("state"), **d)
