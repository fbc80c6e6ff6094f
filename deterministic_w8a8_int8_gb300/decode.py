"""Binding of the decode-step operators: the paged int8 K/V cache and the
attention over it, the 4-bit linear with group scales, and the token log
probabilities (contracts in ``include/prism.h``).

Entry points (same names as the C ABI):
  KvCache, new_kv_cache(...)                       the cache's six buffers
  prism_kv_append(k, v, cache, page_table, seq_lens, ...)
  prism_kv_attention(q, cache, page_table, seq_lens, ...)        -> out
  prism_w4g_linear(q, a_scale, w4, group_scale, ...)             -> out
  prism_token_logprobs(logits, token_ids, top_k=...)             -> (logprobs, entropy, top_ids, top_logprobs)
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _check, lib

_BF16, _F16, _F32, _I8, _U8, _I32 = (torch.bfloat16, torch.float16, torch.float32, torch.int8, torch.uint8, torch.int32)
_Tensor = torch.Tensor
_raw_stream = torch._C._cuda_getCurrentRawStream   # the current stream's handle without a Stream object around it


class KvCache(NamedTuple):
    """The buffers of a paged int8 K/V cache (``include/prism.h``); the entry
    points take any sequence of these six tensors."""
    k_codes: torch.Tensor   # int8 [num_pages, H_kv, block, D]
    v_codes: torch.Tensor
    k_scale: torch.Tensor   # float32 [num_pages, H_kv]
    v_scale: torch.Tensor
    k_open: torch.Tensor    # bf16 [S, H_kv, block, D]: the rows of each sequence's open page
    v_open: torch.Tensor


def new_kv_cache(num_pages: int, heads: int, head_dim: int, block: int, num_seqs: int, device="cuda") -> KvCache:
    """A zeroed cache of ``num_pages`` pages of ``block`` tokens for ``num_seqs`` sequences."""
    codes = [torch.zeros((num_pages, heads, block, head_dim), dtype=_I8, device=device) for _ in range(2)]
    scales = [torch.zeros((num_pages, heads), dtype=_F32, device=device) for _ in range(2)]
    opens = [torch.zeros((num_seqs, heads, block, head_dim), dtype=_BF16, device=device) for _ in range(2)]
    return KvCache(codes[0], codes[1], scales[0], scales[1], opens[0], opens[1])


# A decode step is a chain of short kernels: the checks below are plain
# comparisons in the order of their cost, so that a call's host time stays
# near its launch's.

def _device(t, name):
    """The CUDA device index of the first operand."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    return t.get_device()


def _tensor(t, name, dtype, shape, device):
    """A tensor of this dtype and shape on CUDA device ``device``, its last
    dimension contiguous; returns its address."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must be of shape {list(shape)}, got {list(t.shape)}")
    if t.stride(-1) != 1 and shape[-1] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t.data_ptr()


def _dense(t, name, dtype, shape, device):
    if isinstance(t, _Tensor) and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _tensor(t, name, dtype, shape, device)


def _rank(t, name, n):
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dims")
    return t.shape


def _cache(cache, page_table, seq_lens, device):
    """Checks the cache's own tensors: its geometry and the addresses of codes,
    scales, page table and lengths."""
    num_pages, heads, block, d = shape = _rank(cache[0], "k_codes", 4)
    seqs, max_pages = _rank(page_table, "page_table", 2)
    return (num_pages, heads, block, d, seqs, max_pages,
            _dense(cache[0], "k_codes", _I8, shape, device), _dense(cache[1], "v_codes", _I8, shape, device),
            _dense(cache[2], "k_scale", _F32, (num_pages, heads), device),
            _dense(cache[3], "v_scale", _F32, (num_pages, heads), device),
            _tensor(page_table, "page_table", _I32, (seqs, max_pages), device),
            _tensor(seq_lens, "seq_lens", _I32, (seqs,), device))


def _offsets(cu, name, seqs, rows, device):
    if cu is not None:
        return _tensor(cu, name, _I32, (seqs + 1,), device)
    if rows != seqs:
        raise ValueError(f"without {name} there is one row for each sequence")
    return None


def _stream(stream, device):
    return _raw_stream(device) if stream is None else stream.cuda_stream


def prism_kv_append(k, v, cache, page_table, seq_lens, cu_new=None, max_new=None, err=None, stream=None):
    """Append the rows ``k``, ``v`` bf16 [T, H_kv, D] to the sequences of
    ``cache`` (a KvCache).  ``seq_lens`` int32 [S]: tokens before the call
    (not changed); ``cu_new`` int32 [S + 1]: each sequence's rows, None for one
    row each; ``max_new``: a launch hint, the most rows of one sequence;
    ``err``: optional int32 [1] device error word."""
    device = _device(k, "k")
    num_pages, heads, block, d, seqs, max_pages, kc, vc, ks, vs, table, lens = _cache(cache, page_table, seq_lens, device)
    rows = _rank(k, "k", 3)[0]
    shape, open_shape = (rows, heads, d), (seqs, heads, block, d)
    k_ptr, v_ptr = _tensor(k, "k", _BF16, shape, device), _tensor(v, "v", _BF16, shape, device)
    ko = _dense(cache[4], "k_open", _BF16, open_shape, device)
    vo = _dense(cache[5], "v_open", _BF16, open_shape, device)
    cu = _offsets(cu_new, "cu_new", seqs, rows, device)
    if max_new is None:
        max_new = 1 if cu is None else max(1, rows)
    k_t, k_h, _ = k.stride()
    v_t, v_h, _ = v.stride()
    _check("prism_kv_append", lib().prism_kv_append(
        k_ptr, k_t, k_h, v_ptr, v_t, v_h, kc, vc, ks, vs, ko, vo, table, page_table.stride(0), lens, cu, seqs, rows,
        max_new, num_pages, max_pages, heads, d, block,
        None if err is None else _tensor(err, "err", _I32, (1,), device), _stream(stream, device)))


def prism_kv_attention_workspace_bytes(seqs: int, rows: int, max_q: int, max_pages: int, q_heads: int, heads: int,
                                       head_dim: int, block: int) -> int:
    return int(lib().prism_kv_attention_workspace_bytes(seqs, rows, max_q, max_pages, q_heads, heads, head_dim, block))


def prism_kv_attention(q, cache, page_table, seq_lens, cu_q=None, max_q=None, scale=None, causal=True, window=0,
                       out=None, lse=None, workspace=None, err=None, stream=None):
    """Attention of the queries ``q`` bf16 [T, H_q, D] over ``cache`` (its
    first four tensors) -> bf16 [T, H_q, D].

    ``seq_lens`` int32 [S]: tokens in the cache, the queries' own included;
    ``cu_q`` int32 [S + 1]: each sequence's queries, None for one each;
    ``max_q``: the most queries of one sequence (default: T, or 1 without
    cu_q); ``scale``: default D ** -0.5; ``window``: keys a query sees at most
    (0: all); ``lse``: optional float32 [T, H_q] output; ``workspace``: a uint8
    tensor of prism_kv_attention_workspace_bytes bytes (allocated when None);
    ``err``: optional int32 [1] device error word."""
    device = _device(q, "q")
    num_pages, heads, block, d, seqs, max_pages, kc, vc, ks, vs, table, lens = _cache(cache, page_table, seq_lens, device)
    shape = rows, q_heads, q_d = _rank(q, "q", 3)
    if q_d != d or q_heads == 0 or heads == 0 or q_heads % heads:
        raise ValueError("q must be [T, H_q, D] with H_q a multiple of H_kv")
    q_ptr = _tensor(q, "q", _BF16, shape, device)
    cu = _offsets(cu_q, "cu_q", seqs, rows, device)
    if max_q is None:
        max_q = 1 if cu is None else max(1, rows)
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=q.device)
    out_ptr = _tensor(out, "out", _BF16, shape, device)
    lse_ptr = None if lse is None else _dense(lse, "lse", _F32, (rows, q_heads), device)
    handle = lib()
    if workspace is None:
        ws, ws_bytes = None, handle.prism_kv_attention_workspace_bytes(seqs, rows, max_q, max_pages, q_heads, heads, d, block)
        if ws_bytes:
            workspace = torch.empty(ws_bytes, dtype=_U8, device=q.device)
            ws = workspace.data_ptr()
    else:
        if workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on cuda:{device}")
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    q_t, q_h, _ = q.stride()
    o_t, o_h, _ = out.stride()
    _check("prism_kv_attention", handle.prism_kv_attention(
        q_ptr, q_t, q_h, kc, vc, ks, vs, table, page_table.stride(0), lens, cu, out_ptr, o_t, o_h, lse_ptr,
        d ** -0.5 if scale is None else scale, 1 if causal else 0, window, seqs, rows, max_q, num_pages, max_pages,
        q_heads, heads, d, block, ws, ws_bytes, None if err is None else _tensor(err, "err", _I32, (1,), device),
        _stream(stream, device)))
    return out


def prism_w4g_linear(q, a_scale, w4, group_scale, group_offset=None, residual=None, out=None, stream=None):
    """out bf16 [M, N] = a_scale * (q @ w^T) + residual with 4-bit weights
    w[n, k] = group_scale[n, k / g] * code[n, k] + group_offset[n, k / g].

    ``q`` int8 [M, K], ``a_scale`` float32 [M] (prism_quant_act); ``w4`` uint8
    [N, K/2] (code 2j in the low nibble of byte j); ``group_scale`` and the
    optional ``group_offset`` float16 [N, K/g], g = 32, 64 or 128; ``residual``
    bf16 [M, N] or None, may be ``out`` itself."""
    device = _device(q, "q")
    m, k = _rank(q, "q", 2)
    n, groups = _rank(group_scale, "group_scale", 2)
    if groups == 0 or k % groups or k % 2:
        raise ValueError("q [M, K] and group_scale [N, K/g] do not agree")
    q_ptr, a_ptr = _tensor(q, "q", _I8, (m, k), device), _tensor(a_scale, "a_scale", _F32, (m,), device)
    w_ptr = _tensor(w4, "w4", _U8, (n, k // 2), device)
    s_ptr = _tensor(group_scale, "group_scale", _F16, (n, groups), device)
    if group_offset is None:
        b_ptr = ldb = 0
    else:
        b_ptr, ldb = _tensor(group_offset, "group_offset", _F16, (n, groups), device), group_offset.stride(0)
    if residual is None:
        r_ptr = ldr = 0
    else:
        r_ptr, ldr = _tensor(residual, "residual", _BF16, (m, n), device), residual.stride(0)
    if out is None:
        out = torch.empty((m, n), dtype=_BF16, device=q.device)
    _check("prism_w4g_linear", lib().prism_w4g_linear(
        q_ptr, q.stride(0), a_ptr, w_ptr, w4.stride(0), s_ptr, group_scale.stride(0), b_ptr, ldb, r_ptr, ldr,
        _tensor(out, "out", _BF16, (m, n), device), out.stride(0), m, n, k, k // groups, _stream(stream, device)))
    return out


def prism_token_logprobs(logits, token_ids, top_k: int = 0, entropy=True, err=None, stream=None):
    """Log probabilities of ``token_ids`` int32 [R, n] under ``logits`` [R, V]
    (bf16 or float32) -> (logprobs float32 [R, n], entropy float32 [R] or None,
    top_ids int32 [R, top_k], top_logprobs float32 [R, top_k]; the last two
    None for top_k = 0).  ``err``: optional int32 [1] device error word."""
    device = _device(logits, "logits")
    rows, vocab = _rank(logits, "logits", 2)
    n = _rank(token_ids, "token_ids", 2)[1]
    dtype = logits.dtype
    if dtype is not _BF16 and dtype is not _F32:
        raise TypeError(f"logits must be bfloat16 or float32, got {dtype}")
    x_ptr = _tensor(logits, "logits", dtype, (rows, vocab), device)
    id_ptr = _tensor(token_ids, "token_ids", _I32, (rows, n), device)
    on = logits.device
    logprobs = torch.empty((rows, n), dtype=_F32, device=on)
    ent = ent_ptr = top_ids = top_lp = ids_out = lp_out = None
    if entropy:
        ent = torch.empty((rows,), dtype=_F32, device=on)
        ent_ptr = ent.data_ptr()
    if top_k:
        top_ids = torch.empty((rows, top_k), dtype=_I32, device=on)
        top_lp = torch.empty((rows, top_k), dtype=_F32, device=on)
        ids_out, lp_out = top_ids.data_ptr(), top_lp.data_ptr()
    _check("prism_token_logprobs", lib().prism_token_logprobs(
        x_ptr, 1 if dtype is _F32 else 0, logits.stride(0), id_ptr, token_ids.stride(0), n, rows, vocab, top_k,
        logprobs.data_ptr(), ent_ptr, ids_out, lp_out,
        None if err is None else _tensor(err, "err", _I32, (1,), device), _stream(stream, device)))
    return logprobs, ent, top_ids, top_lp
