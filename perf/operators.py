"""The decode-path operators and the work they are measured on.

Four operators of a generated ("thought") token's step, next to the W8A8 linear
and the candidate read-out:

  kv_append       new K/V rows into a paged int8 cache, one scale per (page, head)
  kv_attention    attention of queries over that cache (one token or many per sequence)
  w4g_linear      int8 activations times 4-bit weights with group scales
  token_logprobs  log probabilities of given tokens, entropy, top alternatives

``run`` computes each in its plain form (elementary torch operations in 32 bits)
or, where ``own`` is true, through the package's entry points.  ``exact`` is the
definition in 64 bits, written apart from the plain form.
"""
import math

import numpy as np
import torch

own = False


# --------------------------------------------------------------------- cases
def listed():
    return [
        # One client's thought token: a single new query over a short request
        # (256 evidence tokens and a question); latency counts.
        dict(name="attn_one_short", op="attn", seqs=1, lo=271, hi=271, nq=1, hq=40, hkv=8, d=128, block=64,
             shared=0, window=0),
        # 64 clients generating at once, ragged contexts.
        dict(name="attn_decode_64", op="attn", seqs=64, lo=300, hi=4096, nq=1, hq=40, hkv=8, d=128, block=64,
             shared=0, window=0),
        # One generated token over a very long evidence text.
        dict(name="attn_decode_long", op="attn", seqs=1, lo=131071, hi=131071, nq=1, hq=32, hkv=4, d=256, block=128,
             shared=0, window=0),
        # Three questions of 16 tokens each on shared long evidence: the page
        # tables share the evidence's pages.
        dict(name="attn_questions", op="attn", seqs=3, lo=8208, hi=8208, nq=16, hq=40, hkv=8, d=128, block=16,
             shared=8192, window=0),
        # A prompt's piece of 512 tokens at the end of a long context.
        dict(name="attn_prompt_512", op="attn", seqs=1, lo=8187, hi=8187, nq=512, hq=40, hkv=8, d=128, block=64,
             shared=0, window=0),
        # 64 clients' new K/V rows of one generated token.
        dict(name="append_decode_64", op="append", seqs=64, lo=37, hi=1500, nn=1, hkv=8, d=128, block=64),
        # A long evidence prompt and two others entering the cache.
        dict(name="append_prompt", op="append", seqs=3, lo=5, hi=200, nn=8192, hkv=8, d=128, block=64),
        # One token through the attention output projection, with its residual.
        dict(name="w4g_o_proj_1", op="w4g", m=1, k=5120, n=5120, g=128, offset=False, residual=True),
        # 8 clients' tokens through the FFN's down projection, asymmetric groups of 32.
        dict(name="w4g_down_8", op="w4g", m=8, k=17408, n=5120, g=32, offset=True, residual=True),
        # 37 rows (answer rows and generated tokens) through gate/up.
        dict(name="w4g_gateup_37", op="w4g", m=37, k=5120, n=34816, g=64, offset=False, residual=False),
        # One generated token: its log probability, entropy and 20 alternatives.
        dict(name="logprobs_one", op="logp", r=1, v=248000, dtype="bf16", n_ids=1, top_k=20, masked=0.0),
        # Scoring a prompt of 768 tokens over the whole vocabulary.
        dict(name="logprobs_prompt", op="logp", r=768, v=248000, dtype="bf16", n_ids=1, top_k=5, masked=0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "append", "w4g", "w4g", "logp"])
    if op == "attn":
        d = rng.choice([64, 128, 128, 256])
        hkv = rng.choice([1, 2, 4, 8, 16])
        g = rng.choice([1, 2, 4, 5, 8])
        block = rng.choice([16, 32, 64, 128])
        nq = 1 if rng.random() < 0.5 else _log_int(rng, 2, 512)
        seqs = _log_int(rng, 1, 64)
        # the largest listed cases bound the query rows, the cache bytes and the score products
        nq = max(1, min(nq, (1 << 21) // (seqs * hkv * g * d)))
        hi = _log_int(rng, 1, 131071)
        hi = max(1, min(hi, (1 << 28) // (seqs * hkv * d * 2), (1 << 34) // (seqs * nq * hkv * g * d)))
        lo = rng.choice([0, hi // 8, hi // 2, hi])
        shared = (lo // block // 2) * block if seqs > 1 and rng.random() < 0.3 else 0
        window = rng.choice([0, 0, 0, 1 + hi // 3])
        return dict(op=op, seqs=seqs, lo=lo, hi=hi, nq=nq, hq=hkv * g, hkv=hkv, d=d, block=block, shared=shared,
                    window=window)
    if op == "append":
        seqs = _log_int(rng, 1, 64)
        nn = rng.choice([1, 1, _log_int(rng, 2, 8192)])
        nn = max(1, min(nn, 8192 // seqs)) if nn > 1 else 1
        return dict(op=op, seqs=seqs, lo=rng.choice([0, 5]), hi=_log_int(rng, 5, 1500), nn=nn,
                    hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128, 256 if seqs * nn <= 4096 else 128]),
                    block=rng.choice([16, 32, 64, 128]))
    if op == "w4g":
        g = rng.choice([32, 64, 128])
        k = g * _log_int(rng, max(1, 256 // g), 17408 // g)
        n = _log_int(rng, 64, min(34816, 34816 * 5120 // k))
        return dict(op=op, m=_log_int(rng, 1, 37), k=k, n=n, g=g, offset=rng.random() < 0.5,
                    residual=rng.random() < 0.5)
    v = _log_int(rng, 1000, 248000)
    dtype = rng.choice(["bf16", "f32"])
    r = _log_int(rng, 1, max(1, min(768, 768 * 248000 // v // (2 if dtype == "f32" else 1))))
    return dict(op=op, r=r, v=v, dtype=dtype, n_ids=rng.choice([1, 1, 3]), top_k=rng.choice([0, 1, 5, 20, 32]),
                masked=rng.choice([0.0, 0.0, 0.9]))


def _spread(i, lo, hi):
    """The i-th of a fixed ragged sequence of lengths in [lo, hi]."""
    return lo + int((hi - lo) * ((i * 0.6180339887498949 + 0.5) % 1.0) + 0.5)


def _attn_lens(c):
    lens = [_spread(i, c["lo"], c["hi"]) for i in range(c["seqs"])]
    # ragged query counts where there are several sequences with several queries
    nq = [c["nq"] if c["lo"] == c["hi"] else max(1, _spread(3 * i + 1, (c["nq"] + 1) // 2, c["nq"]))
          for i in range(c["seqs"])]
    return [max(length, c["shared"]) for length in lens], nq


def _append_lens(c):
    before = [_spread(i, c["lo"], c["hi"]) for i in range(c["seqs"])]
    new = [c["nn"] if i == 0 or c["nn"] == 1 else _spread(i, 1, c["nn"] // 2 + 1) for i in range(c["seqs"])]
    return before, new


# -------------------------------------------------------------------- inputs
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _page_table(c, lens, seed):
    """Pages in a shuffled order; the first shared/block pages are the same for
    every sequence; entries past a sequence's pages are -1."""
    b = c["block"]
    counts = [-(-n // b) for n in lens]
    sh = c.get("shared", 0) // b
    total = sh + sum(max(0, n - sh) for n in counts)
    order = np.random.RandomState(seed % (1 << 31)).permutation(max(1, total)).astype(np.int32)
    table = np.full((len(lens), max(1, max(counts))), -1, np.int32)
    at = sh
    for i, n in enumerate(counts):
        table[i, :min(sh, n)] = order[:min(sh, n)]
        own_pages = max(0, n - sh)
        table[i, sh:sh + own_pages] = order[at:at + own_pages]
        at += own_pages
    return torch.from_numpy(table).cuda(), max(1, total)


def _offsets(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")


def _cache(c, pages, seqs, seed, open_rows):
    """Codes and scales as a cache of normal K/V rows holds them: block maxima of
    about 3.5 standard deviations, a few channels of K with large values."""
    hkv, b, d = c["hkv"], c["block"], c["d"]
    g = _gen(seed, 1)
    codes, scales = [], []
    for _ in range(2):
        x = torch.empty((pages, hkv, b, d), dtype=torch.float16, device="cuda").normal_(0.0, 36.0, generator=g)
        codes.append(x.round_().clamp_(-127, 127).to(torch.int8))
        del x
        scales.append((torch.rand((pages, hkv), generator=g, device="cuda") * 0.5 + 0.75) / 36.0)
    shape = (seqs, hkv, b, d) if open_rows else (0, hkv, b, d)
    opens = [torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    return (codes[0], codes[1], scales[0], scales[1], opens[0], opens[1])


def prepare(case, seed):
    c = case
    if c["op"] == "attn":
        lens, nq = _attn_lens(c)
        table, pages = _page_table(c, lens, seed)
        q = torch.randn((sum(nq), c["hq"], c["d"]), generator=_gen(seed, 2), device="cuda").to(torch.bfloat16)
        return dict(case=c, q=q, cache=_cache(c, pages, c["seqs"], seed, False), table=table,
                    lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), cu_q=_offsets(nq),
                    max_q=max(nq), max_len=max(lens))
    if c["op"] == "append":
        before, new = _append_lens(c)
        table, pages = _page_table(c, [a + n for a, n in zip(before, new)], seed)
        cache = _cache(c, pages, c["seqs"], seed, True)
        # the blocks that are open before the call hold their rows' codes and scales
        b = c["block"]
        g = _gen(seed, 3)
        k, v = (torch.randn((sum(new), c["hkv"], c["d"]), generator=g, device="cuda").to(torch.bfloat16)
                for _ in range(2))
        filled = torch.tensor([n % b for n in before], device="cuda")
        live = torch.arange(b, device="cuda")[None, :] < filled[:, None]                        # [S, B]
        held = (filled > 0).nonzero()[:, 0]
        page = table[held, torch.tensor([n // b for n in before], device="cuda")[held]].long()
        for codes, scales, rows in ((cache[0], cache[2], cache[4]), (cache[1], cache[3], cache[5])):
            x = rows.float() * live[:, None, :, None]
            amax = x.abs().amax(dim=(2, 3))
            y = torch.round(x * torch.where(amax > 0, 127.0 / amax, 0.0)[:, :, None, None]).to(torch.int8)
            codes[page] = y[held]
            scales[page] = (amax / 127.0)[held]
        return dict(case=c, k=k, v=v, cache=cache, table=table, cu_new=_offsets(new), max_new=max(new),
                    lens=torch.tensor(before, dtype=torch.int32, device="cuda"))
    if c["op"] == "w4g":
        m, n, k, g = c["m"], c["n"], c["k"], c["g"]
        r = _gen(seed, 4)
        x = torch.randn((m, k), generator=r, device="cuda")
        a = x.abs().amax(dim=1) / 127.0
        q = torch.round(x / a[:, None]).clamp_(-127, 127).to(torch.int8)
        w4 = torch.randint(0, 256, (n, k // 2), generator=r, device="cuda", dtype=torch.int32).to(torch.uint8)
        scale = ((torch.rand((n, k // g), generator=r, device="cuda") + 0.5) * 0.004).to(torch.float16)
        offset = (torch.randn((n, k // g), generator=r, device="cuda") * 0.004).to(torch.float16) if c["offset"] else None
        residual = torch.randn((m, n), generator=r, device="cuda").to(torch.bfloat16) if c["residual"] else None
        return dict(case=c, q=q, a=a, w4=w4, scale=scale, offset=offset, residual=residual)
    r, v = c["r"], c["v"]
    g = _gen(seed, 5)
    x = torch.randn((r, v), generator=g, device="cuda") * 2.0
    hot = torch.randint(0, v, (r, 8), generator=g, device="cuda")
    x.scatter_add_(1, hot, torch.rand((r, 8), generator=g, device="cuda") * 12.0)
    if c["masked"]:
        x.masked_fill_(torch.rand((r, v), generator=g, device="cuda") < c["masked"], -math.inf)
    x = x.to(torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)
    ids = torch.randint(0, v, (r, c["n_ids"]), generator=g, device="cuda").to(torch.int32)
    return dict(case=c, logits=x, ids=ids)


# --------------------------------------------------------------- plain forms
def _plain_attn(s):
    c = s["case"]
    hkv, d, b, window = c["hkv"], c["d"], c["block"], c["window"]
    g = c["hq"] // hkv
    kc, vc, ks, vs = s["cache"][:4]
    n = s["cu_q"].diff().long()
    lens = s["lens"].long()
    seqs, mq = lens.numel(), s["max_q"]
    pages = s["table"].clamp(min=0).long()
    length = pages.shape[1] * b
    k = (kc[pages].float() * ks[pages][..., None, None]).transpose(1, 2).reshape(seqs, hkv, length, d)
    v = (vc[pages].float() * vs[pages][..., None, None]).transpose(1, 2).reshape(seqs, hkv, length, d)
    i = torch.arange(mq, device="cuda")
    token = (s["cu_q"][:-1].long()[:, None] + i).clamp(max=s["q"].shape[0] - 1)                  # [S, mq]
    q = s["q"][token].float().view(seqs, mq, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(seqs, hkv, g * mq, d)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(d ** -0.5).view(seqs, hkv, g, mq, length)
    pos = (lens - n)[:, None] + i                                                                # [S, mq]
    j = torch.arange(length, device="cuda")
    hidden = (j > pos[..., None]) | (j >= lens[:, None, None])
    if window:
        hidden |= j <= pos[..., None] - window
    x = x.masked_fill_(hidden[:, None, None], -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x.sub_(torch.where(top == -math.inf, 0.0, top)))
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p.view(seqs, hkv, g * mq, length), v).view(seqs, hkv, g, mq, d)
    o = torch.where(total > 0, o / total, 0.0)
    seq_of = torch.repeat_interleave(torch.arange(seqs, device="cuda"), n, output_size=s["q"].shape[0])
    at = torch.arange(s["q"].shape[0], device="cuda") - s["cu_q"][:-1].long()[seq_of]
    return o.permute(0, 3, 1, 2, 4).reshape(seqs, mq, c["hq"], d)[seq_of, at].to(torch.bfloat16)


def _plain_append(s):
    """Every block that gets rows is quantised from its 16-bit rows: those held in
    the open buffer and the new ones."""
    c = s["case"]
    b = c["block"]
    kc, vc, ks, vs, ko, vo = s["cache"]
    before, n = s["lens"].long(), s["cu_new"].diff().long()
    after = before + n
    first, last = before // b, (after - 1) // b
    blocks = (s["max_new"] + 2 * b - 2) // b
    j = torch.arange(blocks, device="cuda")
    block = first[:, None] + j                                                                   # [S, J]
    seq, col = ((block <= last[:, None]) & (n > 0)[:, None]).nonzero(as_tuple=True)
    block = block[seq, col]
    page = s["table"][seq, block].long()
    pos = block[:, None] * b + torch.arange(b, device="cuda")                                    # [nb, B]
    old, live = pos < before[seq][:, None], pos < after[seq][:, None]
    token = (s["cu_new"][:-1].long()[seq][:, None] + pos - before[seq][:, None]).clamp(0, s["k"].shape[0] - 1)
    to_open = live & ((after // b)[seq] == block)[:, None]      # the block stays open: its rows are kept in 16 bits
    for new, codes, scales, rows in ((s["k"], kc, ks, ko), (s["v"], vc, vs, vo)):
        x = torch.where(old[:, :, None, None], rows.transpose(1, 2)[seq], new[token])            # [nb, B, H, D]
        y = x.float() * live[:, :, None, None]
        amax = y.abs().amax(dim=(1, 3))                                                          # [nb, H]
        inv = torch.where(amax >= 2.0 ** -120, 127.0 / amax, 0.0)
        y = torch.round(y * inv[:, None, :, None]).clamp_(-127, 127).to(torch.int8)
        at, row = live.nonzero(as_tuple=True)
        codes[page[at], :, row] = y[at, row]
        scales[page] = torch.where(amax >= 2.0 ** -120, amax / 127.0, 0.0)
        at, row = to_open.nonzero(as_tuple=True)
        rows[seq[at], :, row] = x[at, row]
    return dict(k_codes=kc, v_codes=vc, k_scale=ks, v_scale=vs, k_open=ko, v_open=vo)


def _plain_w4g(s):
    c = s["case"]
    m, n, k, g = c["m"], c["n"], c["k"], c["g"]
    low = (s["w4"] & 15).to(torch.int8)
    high = (s["w4"] >> 4).to(torch.int8)
    code = torch.stack((low, high), dim=-1).view(n, k // g, g)
    w = (code - 16 * (code > 7)).float() * s["scale"].float()[..., None]
    if s["offset"] is not None:
        w += s["offset"].float()[..., None]
    y = torch.matmul(s["q"].float(), w.view(n, k).T) * s["a"][:, None]
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(torch.bfloat16)


def _plain_logp(s):
    c = s["case"]
    x = s["logits"].float()
    top = x.amax(dim=1, keepdim=True)
    y = x - top
    e = torch.exp(y)
    total = e.sum(dim=1, keepdim=True)
    logz = torch.log(total)
    entropy = (logz - torch.where(e > 0, e * y, 0.0).sum(dim=1, keepdim=True) / total)[:, 0]
    out = dict(logprobs=y.gather(1, s["ids"].long()) - logz, entropy=entropy)
    if c["top_k"]:
        # ties go to the lowest id: a stable sort keeps their order
        value, place = torch.sort(x, dim=1, descending=True, stable=True)
        out.update(top_ids=place[:, :c["top_k"]].to(torch.int32), top_logprobs=value[:, :c["top_k"]] - top - logz)
    return out


def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"attn": _plain_attn, "append": _plain_append, "w4g": _plain_w4g, "logp": _plain_logp}[c["op"]](s)
    import deterministic_w8a8_int8_gb300 as prism
    if c["op"] == "attn":
        return prism.prism_kv_attention(s["q"], s["cache"], s["table"], s["lens"], cu_q=s["cu_q"], max_q=s["max_q"],
                                        window=c["window"])
    if c["op"] == "append":
        prism.prism_kv_append(s["k"], s["v"], s["cache"], s["table"], s["lens"], cu_new=s["cu_new"],
                              max_new=s["max_new"])
        return dict(zip(("k_codes", "v_codes", "k_scale", "v_scale", "k_open", "v_open"), s["cache"]))
    if c["op"] == "w4g":
        return prism.prism_w4g_linear(s["q"], s["a"], s["w4"], s["scale"], group_offset=s["offset"],
                                      residual=s["residual"])
    logprobs, entropy, top_ids, top_logprobs = prism.prism_token_logprobs(s["logits"], s["ids"], top_k=c["top_k"])
    out = dict(logprobs=logprobs, entropy=entropy)
    if c["top_k"]:
        out.update(top_ids=top_ids, top_logprobs=top_logprobs)
    return out


# ---------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "attn":
        lens, nq = _attn_lens(c)
        pairs = keys = 0
        for i, (length, n) in enumerate(zip(lens, nq)):
            seen = [(max(0, p + 1 - c["window"]) if c["window"] else 0, p + 1) for p in range(length - n, length)]
            pairs += sum(max(0, hi - max(0, lo)) for lo, hi in seen)
            low = max(0, min(lo for lo, _ in seen))
            keys += max(0, length - (max(low, c["shared"]) if i else low))
        return dict(bytes=2 * keys * c["hkv"] * (c["d"] + 4.0 / c["block"]) + 4 * sum(nq) * c["hq"] * c["d"],
                    flops=4.0 * pairs * c["hq"] * c["d"])
    if c["op"] == "append":
        t = sum(_append_lens(c)[1])
        # rows read in 16 bits, codes written; the rows of blocks that stay open are kept in 16 bits
        kept = sum(min(n, (a + n) % c["block"]) for a, n in zip(*_append_lens(c)))
        return dict(bytes=2 * c["hkv"] * (c["d"] * (3 * t + 2 * kept) + 4.0 * t / c["block"]),
                    flops=4.0 * t * c["hkv"] * c["d"])
    if c["op"] == "w4g":
        m, n, k, g = c["m"], c["n"], c["k"], c["g"]
        groups = n * (k // g)
        return dict(bytes=n * k / 2 + groups * (4 if c["offset"] else 2) + m * (k + 4) + m * n * (4 if c["residual"] else 2),
                    flops=2.0 * m * n * k)
    size = 2 if c["dtype"] == "bf16" else 4
    return dict(bytes=c["r"] * (c["v"] * size + 8 * c["n_ids"] + 4 + 8 * c["top_k"]), flops=4.0 * c["r"] * c["v"])


# --------------------------------------------------------------------- exact
def _exact_attn(c, s):
    lens, nq = _attn_lens(c)
    kc, vc, ks, vs = s["cache"][:4]
    b, d, hkv = c["block"], c["d"], c["hkv"]
    g = c["hq"] // hkv
    out = torch.zeros((sum(nq), c["hq"], d), dtype=torch.float64, device="cuda")
    at = 0
    for i, (length, n) in enumerate(zip(lens, nq)):
        if length:
            pages = s["table"][i, :-(-length // b)].long()
            j = torch.arange(length, device="cuda")
            for h in range(hkv):
                k = (kc[pages, h].double() * ks[pages, h].double()[:, None, None]).view(-1, d)[:length]
                v = (vc[pages, h].double() * vs[pages, h].double()[:, None, None]).view(-1, d)[:length]
                for a in range(0, n, 64):
                    z = min(n, a + 64)
                    pos = length - n + torch.arange(a, z, device="cuda")
                    seen = j[None, :] <= pos[:, None]
                    if c["window"]:
                        seen &= j[None, :] > pos[:, None] - c["window"]
                    q = s["q"][at + a:at + z, h * g:(h + 1) * g].double()                        # [z - a, g, d]
                    x = torch.einsum("igd,jd->igj", q, k) / math.sqrt(d)
                    x = torch.where(seen[:, None], x, -math.inf)
                    w = torch.softmax(x, dim=2).nan_to_num(0.0)
                    out[at + a:at + z, h * g:(h + 1) * g] = torch.einsum("igj,jd->igd", w, v)
        at += n
    return out


def _exact_append(c, s):
    before, new = _append_lens(c)
    table = s["table"].cpu().numpy()
    ks, vs, ko, vo = (x.clone() for x in s["cache"][2:])
    b, at = c["block"], 0
    for i, (a, n) in enumerate(zip(before, new)):
        for rows, scales, opens in ((s["k"], ks, ko), (s["v"], vs, vo)):
            everything = torch.cat((opens[i, :, :a % b].transpose(0, 1), rows[at:at + n]))       # from the open block's start
            for start in range(0, everything.shape[0], b):
                x = everything[start:start + b]
                scales[int(table[i, a // b + start // b])] = (x.double().abs().amax(dim=(0, 2)) / 127.0).float()
            tail = (a + n) % b
            if tail:
                opens[i, :, :tail] = everything[everything.shape[0] - tail:].transpose(0, 1)
        at += n
    return dict(k_codes=None, v_codes=None, k_scale=ks, v_scale=vs, k_open=ko, v_open=vo)


def _exact_w4g(c, s):
    m, n, k, g = c["m"], c["n"], c["k"], c["g"]
    out = torch.empty((m, n), dtype=torch.float64, device="cuda")
    x = s["q"].double() * s["a"].double()[:, None]
    for a in range(0, n, 1024):
        byte = s["w4"][a:a + 1024].int()
        w = torch.empty((byte.shape[0], k), dtype=torch.float64, device="cuda")
        w[:, 0::2] = ((byte & 15) ^ 8) - 8
        w[:, 1::2] = ((byte >> 4) ^ 8) - 8
        w *= s["scale"][a:a + 1024].double().repeat_interleave(g, dim=1)
        if s["offset"] is not None:
            w += s["offset"][a:a + 1024].double().repeat_interleave(g, dim=1)
        out[:, a:a + 1024] = x @ w.T
    return out if s["residual"] is None else out + s["residual"].double()


def _exact_logp(c, s):
    parts = dict(logprobs=[], entropy=[], top_logprobs=[])
    for a in range(0, c["r"], 64):
        lp = torch.log_softmax(s["logits"][a:a + 64].double(), dim=1)
        parts["logprobs"].append(lp.gather(1, s["ids"][a:a + 64].long()))
        parts["entropy"].append(torch.special.entr(lp.exp()).sum(dim=1))
        parts["top_logprobs"].append(lp.topk(c["top_k"], dim=1).values if c["top_k"] else lp[:, :0])
    out = {name: torch.cat(p) for name, p in parts.items()}
    if not c["top_k"]:
        del out["top_logprobs"]
        return out
    out["top_ids"] = None
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "append": _exact_append, "w4g": _exact_w4g, "logp": _exact_logp}[case["op"]](case, s)
