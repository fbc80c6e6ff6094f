"""Several clients' thoughts decoded together on the decode-step operators.

A small decoder with random 4-bit weights: per layer the 4-bit linear for
Q, K and V, the append to the paged int8 cache, the attention over it, and the
4-bit linears of the output projection and the FFN; at the end the LM head, and
of its logits the log probabilities that a client gets with its tokens.

    python examples/thought_decode.py [--clients 3] [--tokens 24]

A client's tokens and log probabilities do not depend on which others are in
the batch.
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import deterministic_w8a8_int8_gb300 as prism  # noqa: E402


@dataclass
class Config:
    hidden: int = 256
    heads: int = 8
    kv_heads: int = 2
    head_dim: int = 64
    ffn: int = 640
    layers: int = 2
    vocab: int = 1003
    group: int = 64
    block: int = 16        # tokens of a cache page
    max_tokens: int = 512  # of one client
    alternatives: int = 5  # returned with each token


class W4Linear:
    """Random weights, quantised by groups to 4 bits."""

    def __init__(self, n: int, k: int, group: int, rng: torch.Generator):
        w = torch.randn((n, k // group, group), generator=rng) * k ** -0.5
        scale = (w.abs().amax(-1) / 7).half()
        codes = (w / scale.float()[..., None]).round().clamp(-8, 7).to(torch.int32).reshape(n, k) & 15
        self.w4 = (codes[:, 0::2] | codes[:, 1::2] << 4).to(torch.uint8).cuda()
        self.scale = scale.cuda()

    def __call__(self, x, residual=None):
        q, a_scale = prism.prism_quant_act(x)
        return prism.prism_w4g_linear(q, a_scale, self.w4, self.scale, residual=residual)


def rms_norm(x):
    y = x.double()   # so that no order of the sum shows in the rounded result
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Decoder:
    """The model and the state of ``clients`` sequences."""

    def __init__(self, c: Config, clients: int, seed: int = 0):
        rng = torch.Generator().manual_seed(seed)
        self.c, self.clients = c, clients
        self.embedding = torch.randn((c.vocab, c.hidden), generator=rng).to(torch.bfloat16).cuda()
        attn = c.heads * c.head_dim
        self.layers = [
            (W4Linear(attn + 2 * c.kv_heads * c.head_dim, c.hidden, c.group, rng), W4Linear(c.hidden, attn, c.group, rng),
             W4Linear(2 * c.ffn, c.hidden, c.group, rng), W4Linear(c.hidden, c.ffn, c.group, rng))
            for _ in range(c.layers)
        ]
        self.head = W4Linear(c.vocab, c.hidden, c.group, rng)
        pages = -(-c.max_tokens // c.block)
        # the clients' pages lie mixed, as after a while of serving
        self.page_table = torch.randperm(clients * pages, generator=rng).to(torch.int32).reshape(clients, pages).cuda()
        self.caches = [prism.new_kv_cache(clients * pages, c.kv_heads, c.head_dim, c.block, clients) for _ in range(c.layers)]
        self.lens = torch.zeros(clients, dtype=torch.int32, device="cuda")       # tokens in the cache
        self.tokens = torch.zeros(clients, dtype=torch.int32, device="cuda")     # the last token of each, not yet in it
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def hidden_states(self, tokens, cu=None, most=1):
        """Appends ``tokens`` (``cu``: each client's, None for one each) and returns their last hidden states."""
        c = self.c
        new = 1 if cu is None else cu[1:] - cu[:-1]
        lens = (self.lens + new).to(torch.int32)
        x = self.embedding[tokens]
        for (qkv, o, gate_up, down), cache in zip(self.layers, self.caches):
            heads = qkv(rms_norm(x)).view(len(tokens), -1, c.head_dim)
            q, k, v = heads.split([c.heads, c.kv_heads, c.kv_heads], dim=1)
            prism.prism_kv_append(k, v, cache, self.page_table, self.lens, cu_new=cu, max_new=most, err=self.err)
            y = prism.prism_kv_attention(q, cache, self.page_table, lens, cu_q=cu, max_q=most, err=self.err)
            x = o(y.view(len(tokens), -1), residual=x)
            gate, up = gate_up(rms_norm(x)).float().chunk(2, dim=1)
            x = down((torch.nn.functional.silu(gate) * up).to(torch.bfloat16), residual=x)
        self.lens.copy_(lens)
        return x

    def choose(self, x):
        """The most probable next token of each row of ``x``, its log probability, and the alternatives'."""
        logits = self.head(rms_norm(x))
        ids = logits.float().argmax(-1, keepdim=True).to(torch.int32)
        logprobs, entropy, top_ids, top_logprobs = prism.prism_token_logprobs(logits, ids, top_k=self.c.alternatives, err=self.err)
        self.tokens.copy_(ids[:, 0])
        return logprobs[:, 0], entropy, top_ids, top_logprobs

    def prefill(self, prompts):
        """All prompts (lists of token ids) at once; chooses each client's first token."""
        cu = torch.tensor([0] + [len(p) for p in prompts]).cumsum(0).to(torch.int32).cuda()
        tokens = torch.tensor([t for p in prompts for t in p], dtype=torch.int32, device="cuda")
        x = self.hidden_states(tokens, cu, max(len(p) for p in prompts))
        return self.choose(x[(cu[1:] - 1).long()])

    def step(self):
        """One token more for every client.  Nothing here waits for the device, so a step can be captured in a graph."""
        return self.choose(self.hidden_states(self.tokens))


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--clients", type=int, default=3)
    ap.add_argument("--tokens", type=int, default=24)
    args = ap.parse_args()
    c = Config()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(c.vocab, (7 + 23 * i,), generator=g).tolist() for i in range(args.clients)]
    d = Decoder(c, args.clients)
    d.prefill(prompts)
    tokens, logprobs = [d.tokens.clone()], []
    logprobs.append(d.step()[0])
    tokens.append(d.tokens.clone())
    graph = torch.cuda.CUDAGraph()   # the steps after the first
    with torch.cuda.graph(graph):
        out = d.step()
    for _ in range(args.tokens - 1):
        graph.replay()
        tokens.append(d.tokens.clone())
        logprobs.append(out[0].clone())
    if int(d.err):
        raise RuntimeError(f"device error word {int(d.err)}")
    for i in range(args.clients):
        print(f"client {i}: {len(prompts[i])} prompt tokens, then",
              " ".join(f"{int(t[i])}" for t in tokens[:8]), "...",
              f"mean log probability {torch.stack(logprobs)[:, i].mean().item():.4f}")


if __name__ == "__main__":
    main()
