"""The operators between a layer's linears and the work they are measured on.

  norm_quant        residual stream + block's output, RMS norm, int8 codes
  head_norm_quant   RMS norm of each head, gated, int8 codes of the token's row
  glu_quant         gated activation of the FFN, int8 codes
  linear_attention  linear attention with a decay for each head, states in slots

``run`` computes each in its plain form (elementary torch operations in 32 bits,
sums of squares and sums of decays in 64) or, where ``own`` is true, through the
package's entry points.  ``exact`` is the definition in 64 bits, written apart
from the plain form.
"""
import math

import numpy as np
import torch

own = False


# --------------------------------------------------------------------- cases
def listed():
    return [
        # One generated token between two blocks; latency counts.
        dict(name="norm_one", op="norm", m=1, k=5120, delta=True, post=False, alpha=1.0, form="int8"),
        # 64 clients x 32 tokens, the block's output normed before it is added, codes for the compute-bound linear.
        dict(name="norm_load_2048", op="norm", m=2048, k=5120, delta=True, post=True, alpha=1.0, form="f16"),
        # Long evidence.
        dict(name="norm_long_8192", op="norm", m=8192, k=5120, delta=True, post=False, alpha=0.25, form="int8"),
        # 64 clients' tokens of a decode step in the FFN.
        dict(name="glu_decode_64", op="glu", m=64, f=17408, smooth=False, form="int8"),
        # The FFN block of 64 clients x 32 tokens: gate/up's output to the down projection's input.
        dict(name="glu_load_2048", op="glu", m=2048, f=17408, smooth=True, form="f16"),
        # A short request's forest: 256 evidence tokens and 3 x 16 question tokens.
        dict(name="head_forest_304", op="head", m=304, h=40, d=128, gate=True, smooth=False, form="int8"),
        # Long evidence, with the smoothing of the output projection.
        dict(name="head_long_8192", op="head", m=8192, h=40, d=128, gate=True, smooth=True, form="int8"),
        # One client's generated token.
        dict(name="linear_one", op="lin", seqs=1, lo=1, hi=1, hk=40, hv=40, dk=128, dv=128, start="own", decay="token"),
        # 64 clients' generated tokens.
        dict(name="linear_decode_64", op="lin", seqs=64, lo=1, hi=1, hk=8, hv=40, dk=128, dv=128, start="own",
             decay="token"),
        # Three questions that start from the evidence's state.
        dict(name="linear_questions", op="lin", seqs=3, lo=13, hi=48, hk=40, hv=40, dk=128, dv=128, start="parent",
             decay="token"),
        # 64 clients' pieces of about 32 tokens, a decay of each head.
        dict(name="linear_clients_64", op="lin", seqs=64, lo=24, hi=41, hk=8, hv=40, dk=128, dv=128, start="own",
             decay="head"),
        # A long evidence text from its beginning.
        dict(name="linear_prompt_8191", op="lin", seqs=1, lo=8191, hi=8191, hk=40, hv=40, dk=128, dv=128, start="zero",
             decay="token"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "glu", "head", "lin", "lin"])
    form = rng.choice(["int8", "int8", "f16"])
    if op == "norm":
        k = 16 * _log_int(rng, 4, 1088)
        m = _log_int(rng, 1, min(8192, 8192 * 5120 // k))
        delta = rng.random() < 0.8
        return dict(op=op, m=m, k=k, delta=delta, post=delta and rng.random() < 0.4, alpha=rng.choice([1.0, 1.0, 0.22]),
                    form=rng.choice(["int8", "f16", "bf16"]))
    if op == "glu":
        f = 16 * _log_int(rng, 4, 1088)
        return dict(op=op, m=_log_int(rng, 1, min(8192, 2048 * 17408 // f)), f=f, smooth=rng.random() < 0.5, form=form)
    if op == "head":
        d = rng.choice([64, 128])
        h = _log_int(rng, 1, 64)
        return dict(op=op, m=_log_int(rng, 1, min(8192, 8192 * 5120 // (h * d))), h=h, d=d, gate=rng.random() < 0.7,
                    smooth=rng.random() < 0.5, form=form)
    hk = rng.choice([1, 2, 4, 8, 16])
    hv = hk * rng.choice([1, 1, 2, 3])
    dk, dv = rng.choice([64, 128, 128]), rng.choice([64, 128, 128])
    seqs = _log_int(rng, 1, 64)
    hi = 1 if rng.random() < 0.3 else _log_int(rng, 2, 32768)
    # the largest listed case bounds the rows, the one of 64 clients the states
    hi = max(1, min(hi, 8191 * 40 // (seqs * hv)))
    return dict(op=op, seqs=seqs, lo=rng.choice([1, 1 + hi // 3, hi]), hi=hi, hk=hk, hv=hv, dk=dk, dv=dv,
                start=rng.choice(["own", "parent", "zero"]), decay=rng.choice(["token", "head"]))


def _spread(i, lo, hi):
    """The i-th of a fixed ragged sequence of lengths in [lo, hi]."""
    return lo + int((hi - lo) * ((i * 0.6180339887498949 + 0.5) % 1.0) + 0.5)


def _lens(c):
    return [c["hi"] if i == 0 else _spread(i, c["lo"], c["hi"]) for i in range(c["seqs"])]


# -------------------------------------------------------------------- inputs
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _normal(shape, g, std=1.0):
    return torch.empty(shape, device="cuda").normal_(0.0, std, generator=g)


def _rows(shape, g, std):
    """Activations with a few channels of large values, as a residual stream has."""
    x = _normal(shape, g, std)
    hot = torch.randint(0, shape[-1], (max(1, shape[-1] // 100),), generator=g, device="cuda")
    x[..., hot] *= 20.0
    return x.to(torch.bfloat16)


def _positive(n, g):
    return torch.exp(_normal((n,), g, 0.3))


def prepare(case, seed):
    c = case
    g = _gen(seed, 1)
    if c["op"] == "norm":
        m, k = c["m"], c["k"]
        return dict(case=c, x=_rows((m, k), g, 2.0), delta=_rows((m, k), g, 0.7) if c["delta"] else None,
                    weight=_positive(k, g), post=_positive(k, g) if c["post"] else None)
    if c["op"] == "glu":
        m, f = c["m"], c["f"]
        return dict(case=c, x=_rows((m, 2 * f), g, 1.5), inv=1.0 / _positive(f, g) if c["smooth"] else None)
    if c["op"] == "head":
        m, h, d = c["m"], c["h"], c["d"]
        return dict(case=c, x=_normal((m, h, d), g, 0.5).to(torch.bfloat16), weight=_positive(d, g),
                    gate=_normal((m, h, d), g, 1.5).to(torch.bfloat16) if c["gate"] else None,
                    inv=1.0 / _positive(h * d, g) if c["smooth"] else None)
    lens = _lens(c)
    t, s = sum(lens), c["seqs"]
    q, k = (_normal((t, c["hk"], c["dk"]), g).to(torch.bfloat16) for _ in range(2))
    v = _normal((t, c["hv"], c["dv"]), g).to(torch.bfloat16)
    # heads that remember from about 4 to some thousand tokens
    rate = torch.exp2(-2.0 - 10.0 * torch.rand((c["hv"],), generator=g, device="cuda"))
    decay = -rate
    if c["decay"] == "token":
        decay = -rate * torch.empty((t, c["hv"]), device="cuda").exponential_(1.0, generator=g)
    # slots in a shuffled order: one for each sequence, and every third sequence's parent (the evidence) before them
    parents = -(-s // 3)
    slots = torch.from_numpy(np.random.RandomState(seed % (1 << 31)).permutation(s + parents).astype(np.int32)).cuda()
    state = _normal((s + parents, c["hv"], c["dk"], c["dv"]), g, 2.0)
    mine = slots[:s].contiguous()
    first = dict(own=mine, parent=slots[s + torch.arange(s, device="cuda") // 3].contiguous(),
                 zero=torch.full_like(mine, -1))[c["start"]]
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
    return dict(case=c, q=q, k=k, v=v, decay=decay, state=state, state_in=first, state_out=mine, cu=cu, max_len=max(lens))


# --------------------------------------------------------------- plain forms
def _divide(a, b):
    return torch.div(torch.full_like(b, a), b)


def _codes(y, form):
    """Codes and scales of rows: each step one operation in 32 bits."""
    if form == "bf16":
        return dict(y=y.to(torch.bfloat16))
    amax = y.abs().amax(dim=1)
    live = amax >= 2.0 ** -120
    inv = torch.where(live, _divide(127.0, amax), 0.0)
    q = torch.round(y * inv[:, None]).clamp_(-127, 127)
    scale = torch.where(live, torch.div(amax, torch.full_like(amax, 127.0)), 0.0)
    return dict(q=q.to(torch.int8 if form == "int8" else torch.float16), a_scale=scale)


def _fma(a, b, c):
    """a * b + c rounded once (the product of two 32-bit values is exact in 64)."""
    return (a.double() * b + c).float()


def _exp(x):
    """exp of x <= 0: x = n ln 2 + r, the series of e^r to r^7, times 2^n; each
    step one fused operation in 32 bits.  Below 2^-126: 0."""
    n = torch.round(x.double() * 1.44269502162933349609375).clamp_(min=-200.0).float()
    r = _fma(n, -0.693359375, x)
    r = _fma(n, 2.12194441701285541057586669921875e-4, r)
    p = torch.full_like(r, 1.98412701138295233249664306640625e-4)
    for a in (1.388888922519981861114501953125e-3, 8.333333767950534820556640625e-3, 4.16666679084300994873046875e-2,
              0.16666667163372039794921875, 0.5, 1.0, 1.0):
        p = _fma(p, r, a)
    two_n = ((n.clamp(min=-126.0).to(torch.int32) + 127) << 23).view(torch.float32)
    return torch.where(n >= -126.0, p * two_n, 0.0)


def _silu(z):
    e = _exp(-z.abs())
    return z * torch.div(torch.where(z >= 0, 1.0, e), e + 1.0)


def _rstd(x, eps=1e-6):
    """Of bf16 values, over the last dimension: the sum in 64 bits, the result rounded to 32."""
    mean = x.double().square().mean(dim=-1, keepdim=True)
    return (mean + float(np.float32(eps))).rsqrt().float()


def _plain_norm(s):
    c = s["case"]
    h, out = s["x"], {}
    if s["delta"] is not None:
        d = s["delta"].float()
        if s["post"] is not None:
            d = d * _rstd(s["delta"]) * s["post"]
        h = (h.float() + d * c["alpha"]).to(torch.bfloat16)
        out["h"] = h
    return out | _codes(h.float() * _rstd(h) * s["weight"], c["form"])


def _plain_glu(s):
    f = s["case"]["f"]
    y = _silu(s["x"][:, :f].float()) * s["x"][:, f:].float()
    return _codes(y if s["inv"] is None else y * s["inv"], s["case"]["form"])


def _plain_head(s):
    y = s["x"].float() * _rstd(s["x"]) * s["weight"]
    if s["gate"] is not None:
        y = y * _silu(s["gate"].float())
    y = y.reshape(y.shape[0], -1)
    return _codes(y if s["inv"] is None else y * s["inv"], s["case"]["form"])


def _plain_lin(s):
    """Chunks of 64 tokens: scores within a chunk, and the states that enter the
    chunks from the chunks' own sums and the products of decays between them."""
    c, size = s["case"], 64
    hk, hv, dk, dv, seqs = c["hk"], c["hv"], c["dk"], c["dv"], c["seqs"]
    cu = s["cu"].long()
    t = s["q"].shape[0]
    n = -(-s["max_len"] // size)
    seq = torch.repeat_interleave(torch.arange(seqs, device="cuda"), cu.diff(), output_size=t)
    at = torch.arange(t, device="cuda") - cu[seq]

    def padded(x, heads):                                                       # [S, Hv, N, C, ...], zeros past the end
        y = torch.zeros((seqs, n * size, *x.shape[1:]), dtype=torch.float32, device="cuda")
        y[seq, at] = x.float()
        y = y.transpose(1, 2).unflatten(2, (n, size))
        return y.repeat_interleave(hv // heads, dim=1)

    q, k, v = padded(s["q"], hk), padded(s["k"], hk), padded(s["v"], hv)
    g = torch.zeros((seqs, n * size, hv), dtype=torch.float64, device="cuda")
    g[seq, at] = s["decay"].double().expand(t, hv)
    g = g.transpose(1, 2).unflatten(2, (n, size)).cumsum(dim=3)                 # [S, Hv, N, C]: within the chunk
    total = g[..., -1].cumsum(dim=2)                                            # [S, Hv, N]: up to a chunk's end
    before = torch.nn.functional.pad(total, (1, 0))[..., :n + 1]                # up to its start, and of all
    after = (g.unsqueeze(4) - g.unsqueeze(3)).float()                           # [.., i, j]
    seen = torch.ones((size, size), dtype=torch.bool, device="cuda").tril()
    w = torch.exp(torch.where(seen, after, -math.inf))
    o = torch.matmul(torch.matmul(q, k.transpose(3, 4)) * w, v)
    sums = torch.matmul((k * torch.exp(g[..., -1:] - g).float()[..., None]).transpose(3, 4), v)   # of each chunk alone
    first = s["state"][s["state_in"].clamp(min=0).long()]
    first = torch.where((s["state_in"] >= 0)[:, None, None, None], first, 0.0)
    sums = torch.cat((first[:, :, None], sums), dim=2).flatten(3)               # [S, Hv, 1 + N, Dk Dv]
    rows = torch.arange(n + 1, device="cuda")
    link = before.unsqueeze(3) - before.unsqueeze(2)                            # from the end of source m - 1 (0: the start)
    link = torch.exp(torch.where(rows[None, :] <= rows[:, None], link, -math.inf)).float()
    states = torch.matmul(link, sums).unflatten(3, (dk, dv))                    # entering each chunk, and after all
    o = o + torch.matmul(q * torch.exp(g).float()[..., None], states[:, :, :n])
    s["state"][s["state_out"].long()] = states[:, :, n]
    o = (o * dk ** -0.5).flatten(2, 3).transpose(1, 2)[seq, at]
    return dict(out=o.to(torch.bfloat16), state=s["state"])


def run(state):
    s = state
    c = s["case"]
    if not own:
        return dict(norm=_plain_norm, glu=_plain_glu, head=_plain_head, lin=_plain_lin)[c["op"]](s)
    import deterministic_w8a8_int8_gb300 as prism
    if c["op"] == "lin":
        out = prism.prism_linear_attention(s["q"], s["k"], s["v"], s["decay"], s["state"], state_in=s["state_in"],
                                           state_out=s["state_out"], cu=s["cu"], max_len=s["max_len"])
        return dict(out=out, state=s["state"])
    if c["op"] == "norm":
        q, scale, h = prism.prism_norm_quant(s["x"], s["weight"], delta=s["delta"], alpha=c["alpha"],
                                             post_weight=s["post"], form=c["form"])
        out = dict(h=h) if c["delta"] else {}
        return out | (dict(y=q) if c["form"] == "bf16" else dict(q=q, a_scale=scale))
    if c["op"] == "glu":
        return dict(zip(("q", "a_scale"), prism.prism_glu_quant(s["x"], s["inv"], form=c["form"])))
    return dict(zip(("q", "a_scale"), prism.prism_head_norm_quant(s["x"], s["weight"], gate=s["gate"], inv_s=s["inv"],
                                                                  form=c["form"])))


# ---------------------------------------------------------------------- work
def work(case):
    c = case
    size = dict(int8=1, f16=2, bf16=2).get(c.get("form"), 0)
    if c["op"] == "norm":
        m, k = c["m"], c["k"]
        return dict(bytes=m * (k * (2 + size + 4 * c["delta"]) + 4) + 4 * k * (1 + c["post"]), flops=8.0 * m * k)
    if c["op"] == "glu":
        m, f = c["m"], c["f"]
        return dict(bytes=m * (f * (4 + size) + 4) + 4 * f * c["smooth"], flops=25.0 * m * f)
    if c["op"] == "head":
        m, k = c["m"], c["h"] * c["d"]
        return dict(bytes=m * (k * (2 + 2 * c["gate"] + size) + 4) + 4 * (c["d"] + k * c["smooth"]),
                    flops=(8.0 + 22 * c["gate"]) * m * k)
    t, s, hv = sum(_lens(c)), c["seqs"], c["hv"]
    read = dict(own=s, parent=-(-s // 3), zero=0)[c["start"]]
    return dict(bytes=4.0 * t * (c["hk"] * c["dk"] + hv * c["dv"]) + 4.0 * hv * (t if c["decay"] == "token" else 1)
                + 4.0 * (read + s) * hv * c["dk"] * c["dv"], flops=4.0 * t * hv * c["dk"] * c["dv"])


# --------------------------------------------------------------------- exact
def _exact_rows(y, form):
    if form == "bf16":
        return dict(y=y)
    return dict(q=None, a_scale=y.abs().amax(dim=1) / 127.0)


def _exact_norm(c, s):
    norm = lambda x: x / torch.sqrt((x * x).sum(dim=1, keepdim=True) / x.shape[1] + 1e-6)  # noqa: E731
    h, out = s["x"].double(), {}
    if c["delta"]:
        d = s["delta"].double()
        h = h + c["alpha"] * (norm(d) * s["post"].double() if c["post"] else d)
        out["h"] = h
        h = h.to(torch.bfloat16).double()     # the stream is what is kept of it
    return out | _exact_rows(norm(h) * s["weight"].double(), c["form"])


def _exact_glu(c, s):
    gate, up = s["x"].double().chunk(2, dim=1)
    y = gate * torch.sigmoid(gate) * up
    return _exact_rows(y if s["inv"] is None else y * s["inv"].double(), c["form"])


def _exact_head(c, s):
    x = s["x"].double()
    y = x / torch.sqrt((x * x).sum(dim=2, keepdim=True) / c["d"] + 1e-6) * s["weight"].double()
    if c["gate"]:
        z = s["gate"].double()
        y = y * (z * torch.sigmoid(z))
    y = y.flatten(1)
    return _exact_rows(y if s["inv"] is None else y * s["inv"].double(), c["form"])


def _exact_lin(c, s):
    """One token after the other, all sequences side by side."""
    lens, cu = _lens(c), s["cu"].tolist()
    rep = c["hv"] // c["hk"]
    state = s["state"].double()
    now = torch.zeros((c["seqs"], *state.shape[1:]), dtype=torch.float64, device="cuda")
    if c["start"] != "zero":
        now = state[s["state_in"].long()]
    gain = torch.exp(s["decay"].double())
    out = torch.empty(s["v"].shape, dtype=torch.float64, device="cuda")
    order = sorted(range(c["seqs"]), key=lambda i: -lens[i])     # the live ones lie in front
    now = now[torch.tensor(order, device="cuda")]
    begins = torch.tensor([cu[i] for i in order], device="cuda")
    live = c["seqs"]
    for i in range(max(lens)):
        while lens[order[live - 1]] <= i:
            live -= 1
        rows = begins[:live] + i
        k, q = (s[x][rows].double().repeat_interleave(rep, dim=1) for x in ("k", "q"))
        part = now[:live]
        part *= (gain[rows] if c["decay"] == "token" else gain[None])[..., None, None]
        part += k[..., None] * s["v"][rows].double()[:, :, None, :]
        out[rows] = (q[..., None, :] @ part)[..., 0, :] * c["dk"] ** -0.5
    state[s["state_out"].long()[torch.tensor(order, device="cuda")]] = now
    return dict(out=out, state=state)


def exact(case, seed):
    s = prepare(case, seed)
    return dict(norm=_exact_norm, glu=_exact_glu, head=_exact_head, lin=_exact_lin)[case["op"]](case, s)
