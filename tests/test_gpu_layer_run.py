"""The operators between a layer's linears run together, as a layer of linear
attention has them: the stream's norm, projections, linear attention over states
in slots, the gated norm of its heads, the output projection, the next norm,
gate/up, the activation, down.  An evidence text, then branches that start from its
state, then single tokens of each.  Every operator's result is compared with its
statement on the very inputs that it got."""
import numpy as np
import pytest
import torch

import deterministic_w8a8_int8_gb300 as prism
from tests import layer_util as u

pytestmark = pytest.mark.gpu

HIDDEN, HK, HV, D, FFN = 256, 2, 4, 128, 640
SLOTS = 4          # the evidence's state and three branches'


def host(t):
    return t.float().cpu().numpy()


class Layer:
    def __init__(self, check):
        g = torch.Generator().manual_seed(7)
        self.check = check

        def linear(n, k):
            w = torch.randint(-127, 128, (n, k), generator=g, dtype=torch.int8)
            return w.cuda(), (torch.rand(n, generator=g) * 0.02 * k ** -0.5).cuda()

        def gain(n):
            return (torch.rand(n, generator=g) + 0.5).cuda()

        self.qkv = linear((2 * HK + 2 * HV) * D, HIDDEN)     # q, k, v and the gate of the heads
        self.o, self.gate_up, self.down = linear(HIDDEN, HV * D), linear(2 * FFN, HIDDEN), linear(HIDDEN, FFN)
        self.norm1, self.norm2, self.post, self.head = gain(HIDDEN), gain(HIDDEN), gain(HIDDEN), gain(D)
        self.smooth_o, self.smooth_down = gain(HV * D), gain(FFN)
        self.rate = -torch.exp2(-1 - 4 * torch.rand(HV, generator=g)).cuda()
        self.state = torch.zeros((SLOTS, HV, D, D), device="cuda")

    def __call__(self, x, delta, first, last, cu, most):
        """(stream, the last block's output) of the rows ``x``, ``delta``."""
        T = x.shape[0]
        q8, s8, h = prism.prism_norm_quant(x, self.norm1, delta=delta, post_weight=self.post)
        rows = prism.prism_w8a8_linear(q8, s8, *self.qkv).view(T, -1, D)
        q, k, v, z = rows.split([HK, HK, HV, HV], dim=1)
        decay = self.rate * torch.sigmoid(v.float().mean(-1))
        before = self.state.clone() if self.check else None
        y = prism.prism_linear_attention(q, k, v, decay, self.state, first, last, cu=cu, max_len=most)
        oq, os = prism.prism_head_norm_quant(y, self.head, gate=z, inv_s=self.smooth_o)
        a = prism.prism_w8a8_linear(oq, os, *self.o)
        fq, fs, h2 = prism.prism_norm_quant(h, self.norm2, delta=a)
        gate_up = prism.prism_w8a8_linear(fq, fs, *self.gate_up)
        dq, ds = prism.prism_glu_quant(gate_up, self.smooth_down)
        b = prism.prism_w8a8_linear(dq, ds, *self.down)
        if self.check:
            self._compare(x, delta, (q8, s8, h), (q, k, v, z, decay, before, y), first, last, cu, (oq, os), a, (fq, fs, h2),
                          gate_up, (dq, ds))
        return h2, b

    def _compare(self, x, delta, n1, attn, first, last, cu, heads, a, n2, gate_up, glu):
        def codes(got, want):
            q, s = u.codes(want, "int8")
            assert np.array_equal(got[0].cpu().numpy(), q) and np.array_equal(got[1].cpu().numpy(), s)

        y, h = u.norm(host(x), host(self.norm1), delta=host(delta), post=host(self.post))
        codes(n1, y)
        assert np.array_equal(host(n1[2]), h)
        q, k, v, z, decay, before, out = attn
        lens = [1] * x.shape[0] if cu is None else cu.diff().tolist()
        at = first.long()
        start = torch.where((at >= 0)[:, None, None, None], before[at.clamp(min=0)], 0.0).cpu().numpy()
        want, bound, after, after_bound = u.linear_attention(host(q), host(k), host(v), host(decay), start, lens, D ** -0.5)
        assert np.all(np.abs(out.double().cpu().numpy() - want) <= bound)
        assert np.all(np.abs(self.state[last.long()].double().cpu().numpy() - after) <= after_bound)
        codes(heads, u.head_norm(host(out), host(self.head), gate=host(z), inv=host(self.smooth_o)))
        y, h = u.norm(h, host(self.norm2), delta=host(a))
        codes(n2, y)
        assert np.array_equal(host(n2[2]), h)
        codes(glu, u.glu(host(gate_up), inv=host(self.smooth_down)))


def index(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rows(n, seed):
    g = torch.Generator().manual_seed(seed)
    return tuple((torch.randn((n, HIDDEN), generator=g) * s).to(torch.bfloat16).cuda() for s in (2.0, 0.5))


def test_evidence_branches_and_tokens():
    layer = Layer(check=True)
    layer(*rows(150, 1), index(-1), index(0), index(0, 150), 150)                            # the evidence
    layer(*rows(16 + 40 + 7, 2), index(0, 0, 0), index(1, 2, 3), index(0, 16, 56, 63), 40)   # questions on it
    own = index(1, 2, 3)
    for step in range(2):
        layer(*rows(3, 3 + step), own, own, None, 1)                                         # a token of each


def test_a_branch_does_not_depend_on_the_others():
    alone, together = Layer(check=False), Layer(check=False)
    for layer in (alone, together):
        layer(*rows(150, 1), index(-1), index(0), index(0, 150), 150)
    x, d = rows(63, 2)
    got = together(x, d, index(0, 0, 0), index(1, 2, 3), index(0, 16, 56, 63), 40)
    one = alone(x[16:56], d[16:56], index(0), index(2), index(0, 40), 40)
    assert all(torch.equal(a[16:56], b) for a, b in zip(got, one))
    assert torch.equal(alone.state[2], together.state[2])


def test_a_captured_token():
    """A step captured in a graph and replayed: the same bits, and the states go on."""
    eager, replayed = Layer(check=False), Layer(check=False)
    own = index(0, 1, 2)
    x, d = rows(3, 9)
    buf_x, buf_d = torch.zeros_like(x), torch.zeros_like(d)
    replayed(buf_x, buf_d, own, own, None, 1)         # workspaces and the library are there
    replayed.state.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = replayed(buf_x, buf_d, own, own, None, 1)
    replayed.state.zero_()
    for step in range(3):
        x, d = rows(3, 10 + step)
        want = eager(x, d, own, own, None, 1)
        buf_x.copy_(x)
        buf_d.copy_(d)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(replayed.state, eager.state)
