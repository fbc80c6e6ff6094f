"""The Python side of the decode-step entry points (csrc/decode_py.cpp): what it
refuses, what it passes on, and that it keeps nothing."""
import gc
import sys

import pytest
import torch

import deterministic_w8a8_int8_gb300 as prism

pytestmark = pytest.mark.gpu


def _attn():
    cache = prism.new_kv_cache(6, 2, 64, 16, 2)
    q = torch.randn((2, 4, 64), device="cuda").to(torch.bfloat16)
    kv = torch.randn((2, 2, 64), device="cuda").to(torch.bfloat16)
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    lens = torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    return dict(q=q, cache=cache, page_table=table, seq_lens=lens), kv


def _w4g():
    return dict(q=torch.ones((2, 64), dtype=torch.int8, device="cuda"), a_scale=torch.ones(2, device="cuda"),
                w4=torch.zeros((5, 32), dtype=torch.uint8, device="cuda"),
                group_scale=torch.ones((5, 2), dtype=torch.float16, device="cuda"))


def _logp():
    return dict(logits=torch.randn((2, 50), device="cuda"), token_ids=torch.zeros((2, 1), dtype=torch.int32, device="cuda"))


def _wide(t):   # the same values with a last dimension that is not contiguous
    return torch.stack((t, t), dim=-1)[..., 0]


W4G = [("a_scale", lambda t: t.double(), TypeError), ("a_scale", lambda t: t[:1], ValueError),
       ("a_scale", lambda t: None, TypeError), ("w4", lambda t: t.to(torch.int8), TypeError),
       ("w4", _wide, ValueError), ("w4", lambda t: t.cpu(), ValueError), ("w4", lambda t: t[:, :31], ValueError),
       ("group_scale", lambda t: t.float(), TypeError), ("group_scale", lambda t: t[0], ValueError),
       ("group_scale", lambda t: t[:, :0], ValueError), ("q", lambda t: t[0], ValueError), ("q", lambda t: t.float(), TypeError),
       ("q", lambda t: t[:, :63], ValueError), ("q", lambda t: "q", TypeError),
       ("residual", lambda t: torch.zeros((2, 4), dtype=torch.bfloat16, device="cuda"), ValueError),
       ("out", lambda t: torch.zeros((2, 5), device="cuda"), TypeError),
       ("group_offset", lambda t: torch.zeros((5, 1), dtype=torch.float16, device="cuda"), ValueError),
       ("stream", lambda t: 5, AttributeError)]


@pytest.mark.parametrize("name,change,error", W4G)
def test_w4g_refusals(cuda_device, name, change, error):
    args = _w4g()
    args[name] = change(args.get(name))
    with pytest.raises(error):
        prism.prism_w4g_linear(**args)


ATTN = [("q", lambda t: t[0], ValueError), ("q", lambda t: t.float(), TypeError), ("q", lambda t: t[:, :3], ValueError),
        ("q", lambda t: t[..., :32], ValueError), ("q", lambda t: t[:1], ValueError), ("q", _wide, ValueError),
        ("page_table", lambda t: t.long(), TypeError), ("page_table", lambda t: t.view(-1), ValueError),
        ("seq_lens", lambda t: t[:1], ValueError), ("seq_lens", lambda t: t.cpu(), ValueError),
        ("cache", lambda t: t[:3], ValueError), ("cache", lambda t: 7, TypeError),
        ("cache", lambda t: t._replace(k_scale=t.k_scale[:5]), ValueError),
        ("cache", lambda t: t._replace(v_codes=t.v_codes.float()), TypeError),
        ("cache", lambda t: t._replace(k_codes=t.k_codes.transpose(0, 1).contiguous().transpose(0, 1)), ValueError),
        ("cu_q", lambda t: torch.zeros(2, dtype=torch.int32, device="cuda"), ValueError),
        ("lse", lambda t: torch.zeros((2, 3), device="cuda"), ValueError),
        ("out", lambda t: torch.zeros((2, 4, 32), dtype=torch.bfloat16, device="cuda"), ValueError),
        ("workspace", lambda t: torch.zeros(8, dtype=torch.uint8), ValueError),
        ("workspace", lambda t: torch.zeros(8, dtype=torch.uint8, device="cuda")[::2], ValueError),
        ("max_q", lambda t: "one", TypeError), ("scale", lambda t: "one", TypeError),
        ("scale", lambda t: -1.0, prism.PrismError), ("window", lambda t: -1, prism.PrismError),
        ("max_q", lambda t: 0, prism.PrismError)]


@pytest.mark.parametrize("name,change,error", ATTN)
def test_attention_refusals(cuda_device, name, change, error):
    args, _ = _attn()
    args[name] = change(args.get(name))
    with pytest.raises(error):
        prism.prism_kv_attention(**args)


@pytest.mark.parametrize("name,change,error", [
    ("k", lambda t: t[0], ValueError), ("v", lambda t: t.float(), TypeError), ("v", lambda t: t[:1], ValueError),
    ("cache", lambda t: t[:4], ValueError), ("cache", lambda t: t._replace(k_open=t.k_open[:1]), ValueError),
    ("cu_new", lambda t: torch.zeros(3, dtype=torch.int64, device="cuda"), TypeError),
    ("max_new", lambda t: 0, prism.PrismError), ("err", lambda t: torch.zeros(2, dtype=torch.int32, device="cuda"), ValueError)])
def test_append_refusals(cuda_device, name, change, error):
    args, kv = _attn()
    del args["q"]
    args.update(k=kv, v=kv)
    args[name] = change(args.get(name))
    with pytest.raises(error):
        prism.prism_kv_append(**args)


@pytest.mark.parametrize("name,change,error", [
    ("logits", lambda t: t.half(), TypeError), ("logits", lambda t: t[0], ValueError), ("logits", _wide, ValueError),
    ("token_ids", lambda t: t.long(), TypeError), ("token_ids", lambda t: t[:1], ValueError),
    ("top_k", lambda t: -1, prism.PrismError), ("top_k", lambda t: 33, prism.PrismError), ("top_k", lambda t: 1.5, TypeError)])
def test_logprobs_refusals(cuda_device, name, change, error):
    args = _logp()
    args[name] = change(args.get(name))
    with pytest.raises(error):
        prism.prism_token_logprobs(**args)


def test_outputs_and_streams(cuda_device):
    args = _w4g()
    out = torch.empty((2, 5), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert prism.prism_w4g_linear(**args, out=out, stream=side) is out
    side.synchronize()
    with torch.cuda.stream(side):
        again = prism.prism_w4g_linear(**args)
    side.synchronize()
    assert torch.equal(out, again) and again.shape == (2, 5) and again.dtype == torch.bfloat16
    lp, ent, ids, top = prism.prism_token_logprobs(**_logp(), top_k=3)
    assert lp.shape == (2, 1) and ent.shape == (2,) and ids.shape == (2, 3) and ids.dtype == torch.int32 and top.shape == (2, 3)
    lp, ent, ids, top = prism.prism_token_logprobs(**_logp(), entropy=False)
    assert ent is None and ids is None and top is None
    a, kv = _attn()
    assert prism.prism_kv_append(kv, kv, list(a["cache"]), a["page_table"], a["seq_lens"] - 1) is None
    y = prism.prism_kv_attention(**a)
    assert y.shape == (2, 4, 64) and y.is_contiguous()
    ws = torch.empty(max(1, prism.prism_kv_attention_workspace_bytes(2, 2, 1, 3, 4, 2, 64, 16)), dtype=torch.uint8, device="cuda")
    assert torch.equal(prism.prism_kv_attention(**a, workspace=ws, scale=64 ** -0.5, max_q=1), y)


def test_nothing_is_kept(cuda_device):
    (a, kv), w, x = _attn(), _w4g(), _logp()
    held = [*a["cache"], a["q"], a["page_table"], a["seq_lens"], kv, *w.values(), *x.values(), torch.bfloat16, torch.empty]

    def calls():
        prism.prism_kv_append(kv, kv, a["cache"], a["page_table"], a["seq_lens"] - 1)
        prism.prism_kv_attention(**a)
        prism.prism_w4g_linear(**w)
        prism.prism_token_logprobs(**x, top_k=2)
        for bad in (lambda: prism.prism_w4g_linear(**{**w, "a_scale": None}),
                    lambda: prism.prism_kv_attention(**{**a, "window": -1}),
                    lambda: prism.prism_token_logprobs(**x, top_k=40)):
            with pytest.raises((TypeError, prism.PrismError)):
                bad()

    calls()
    torch.cuda.synchronize()
    gc.collect()
    refs, memory = [sys.getrefcount(t) for t in held], torch.cuda.memory_allocated()
    for _ in range(50):
        calls()
    torch.cuda.synchronize()
    gc.collect()
    assert torch.cuda.memory_allocated() == memory
    assert all(abs(sys.getrefcount(t) - n) < 10 for t, n in zip(held, refs))
