"""The operators between a layer's linears on two streams at once, in graphs that are
replayed side by side, and in calls of very many sequences: the bits of calls by themselves."""
import pytest
import torch

import deterministic_w8a8_int8_gb300 as prism

pytestmark = pytest.mark.gpu


def index(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Work:
    """A prompt in segments, one in a few chunks and single tokens in one call, and the rows' operators."""

    def __init__(self, seed, lens, hk, hv, d):
        g = torch.Generator(device="cuda").manual_seed(seed)
        t, n = sum(lens), len(lens)

        def normal(*shape):
            return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

        self.q, self.k, self.v, self.z = normal(t, hk, d), normal(t, hk, d), normal(t, hv, d), normal(t, hv, d)
        self.decay = -torch.rand((t, hv), generator=g, device="cuda")
        self.first = torch.randn((n, hv, d, d), generator=g, device="cuda")
        self.state, self.own, self.most = self.first.clone(), index(*range(n)), max(lens)
        self.cu = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda")
        self.w = torch.rand(hv * d, generator=g, device="cuda") + 0.5

    def run(self):
        out = prism.prism_linear_attention(self.q, self.k, self.v, self.decay, self.state, self.own, self.own, cu=self.cu, max_len=self.most)
        codes = prism.prism_head_norm_quant(out, self.w[:self.v.shape[2]], gate=self.z, inv_s=self.w)
        flat = out.flatten(1)
        h = prism.prism_norm_quant(flat, self.w, delta=self.z.flatten(1), form="f16")
        glu = prism.prism_glu_quant(flat, form="bf16")
        return out, *codes, *h, glu[0], self.state

    def alone(self):
        self.state.copy_(self.first)
        return [x.clone() for x in self.run()]


def works():
    return Work(1, [2500, 1, 70, 3], 2, 8, 128), Work(2, [1700, 9, 1, 200, 64], 4, 12, 64)


def test_two_streams_at_once():
    both = works()
    want = [w.alone() for w in both]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, w in enumerate(both):
            with torch.cuda.stream(streams[i]):
                w.state.copy_(w.first)
                got[i].append([x.clone() for x in w.run()])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for i in (0, 1) for run in got[i] for a, b in zip(run, want[i]))


def test_two_graphs_replayed_at_once():
    both = works()
    want = [w.alone() for w in both]
    graphs, outs = [], []
    for w in both:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            w.state.copy_(w.first)
            outs.append(w.run())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for i in (0, 1) for a, b in zip(outs[i], want[i]))


def test_very_many_sequences():
    """100000 sequences of no token or one, and one of 100 among them: single tokens as in a call of their own."""
    n, d, at, long = 100000, 64, 60001, 100
    lens = torch.ones(n, dtype=torch.int32)
    lens[::3] = 0
    lens[at] = long
    cu = torch.zeros(n + 1, dtype=torch.int32)
    cu[1:] = lens.cumsum(0)
    t = int(cu[-1])
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn((t, 1, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    decay = -torch.rand((t, 1), generator=g, device="cuda")
    first = torch.randn((n, 1, d, d), generator=g, device="cuda")
    own = torch.arange(n, dtype=torch.int32, device="cuda")
    state = first.clone()
    out = prism.prism_linear_attention(q, k, v, decay, state, own, own, cu=cu.cuda(), max_len=long)
    single = (lens == 1).nonzero()[:, 0].cuda()
    rows = cu.cuda()[single].long()
    alone = first[single]
    mine = torch.arange(len(single), dtype=torch.int32, device="cuda")
    one = prism.prism_linear_attention(q[rows], k[rows], v[rows], decay[rows], alone, mine, mine)
    assert torch.equal(one, out[rows]) and torch.equal(alone, state[single])
    none = (lens == 0).nonzero()[:, 0].cuda()
    assert torch.equal(state[none], first[none])
    b = int(cu[at])
    part = first[at:at + 1].clone()
    one = prism.prism_linear_attention(q[b:b + long], k[b:b + long], v[b:b + long], decay[b:b + long], part, index(0), index(0),
                                       cu=index(0, long))
    assert torch.equal(one, out[b:b + long]) and torch.equal(part[0], state[at])
