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

from . import _check, _stream, lib

_BF16, _F16, _F32, _I8, _U8, _I32 = (torch.bfloat16, torch.float16, torch.float32, torch.int8, torch.uint8, torch.int32)


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


def _tensor(t, name, dtype, ndim, device):
    """A CUDA tensor on ``device`` of this dtype and rank, whose last dimension is contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")
    if t.stride(-1) != 1 and t.size(-1) > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")


def _device(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    return t.device


def _cache(cache, page_table, seq_lens, device):
    """Checks the cache's own tensors; (num_pages, heads, block, D, sequences, pages a sequence)."""
    kc, vc, ks, vs = cache[0], cache[1], cache[2], cache[3]
    for t, name, dtype, ndim in ((kc, "k_codes", _I8, 4), (vc, "v_codes", _I8, 4), (ks, "k_scale", _F32, 2),
                                 (vs, "v_scale", _F32, 2)):
        _tensor(t, name, dtype, ndim, device)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    _tensor(page_table, "page_table", _I32, 2, device)
    _tensor(seq_lens, "seq_lens", _I32, 1, device)
    num_pages, heads, block, d = kc.shape
    if vc.shape != kc.shape or ks.shape != (num_pages, heads) or vs.shape != ks.shape:
        raise ValueError("the cache's shapes do not agree")
    seqs, max_pages = page_table.shape
    if seq_lens.numel() != seqs:
        raise ValueError("seq_lens must hold one length for each row of page_table")
    return num_pages, heads, block, d, seqs, max_pages


def _offsets(cu, name, seqs, rows, device):
    if cu is not None:
        _tensor(cu, name, _I32, 1, device)
        if cu.numel() != seqs + 1:
            raise ValueError(f"{name} must hold one offset more than sequences")
        return cu.data_ptr()
    if rows != seqs:
        raise ValueError(f"without {name} there is one row for each sequence")
    return None


def _err(err, device):
    if err is None:
        return None
    _tensor(err, "err", _I32, 1, device)
    if err.numel() < 1:
        raise ValueError("err must hold one word")
    return err.data_ptr()


def prism_kv_append(k, v, cache, page_table, seq_lens, cu_new=None, max_new=None, err=None, stream=None):
    """Append the rows ``k``, ``v`` bf16 [T, H_kv, D] to the sequences of
    ``cache`` (a KvCache).  ``seq_lens`` int32 [S]: tokens before the call
    (not changed); ``cu_new`` int32 [S + 1]: each sequence's rows, None for one
    row each; ``max_new``: a launch hint, the most rows of one sequence;
    ``err``: optional int32 [1] device error word."""
    device = _device(k, "k")
    num_pages, heads, block, d, seqs, max_pages = _cache(cache, page_table, seq_lens, device)
    _tensor(k, "k", _BF16, 3, device)
    _tensor(v, "v", _BF16, 3, device)
    rows = k.size(0)
    if k.shape != (rows, heads, d) or v.shape != k.shape:
        raise ValueError("k and v must be [T, H_kv, D]")
    ko, vo = cache[4], cache[5]
    for t, name in ((ko, "k_open"), (vo, "v_open")):
        _tensor(t, name, _BF16, 4, device)
        if t.shape != (seqs, heads, block, d) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [S, H_kv, block, D] tensor")
    cu = _offsets(cu_new, "cu_new", seqs, rows, device)
    if max_new is None:
        max_new = 1 if cu is None else max(1, rows)
    _check("prism_kv_append", lib().prism_kv_append(
        k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1), cache[0].data_ptr(),
        cache[1].data_ptr(), cache[2].data_ptr(), cache[3].data_ptr(), ko.data_ptr(), vo.data_ptr(),
        page_table.data_ptr(), page_table.stride(0), seq_lens.data_ptr(), cu, seqs, rows, max_new, num_pages,
        max_pages, heads, d, block, _err(err, device), _stream(stream)))


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
    num_pages, heads, block, d, seqs, max_pages = _cache(cache, page_table, seq_lens, device)
    _tensor(q, "q", _BF16, 3, device)
    rows, q_heads = q.size(0), q.size(1)
    if q.size(2) != d or q_heads == 0 or q_heads % heads:
        raise ValueError("q must be [T, H_q, D] with H_q a multiple of H_kv")
    cu = _offsets(cu_q, "cu_q", seqs, rows, device)
    if max_q is None:
        max_q = 1 if cu is None else max(1, rows)
    if out is None:
        out = torch.empty((rows, q_heads, d), dtype=_BF16, device=device)
    else:
        _tensor(out, "out", _BF16, 3, device)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if lse is not None:
        _tensor(lse, "lse", _F32, 2, device)
        if lse.shape != (rows, q_heads) or not lse.is_contiguous():
            raise ValueError("lse must be a contiguous [T, H_q] tensor")
    handle = lib()
    if workspace is None:
        need = handle.prism_kv_attention_workspace_bytes(seqs, rows, max_q, max_pages, q_heads, heads, d, block)
        if need:
            workspace = torch.empty(need, dtype=_U8, device=device)
    ws, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    _check("prism_kv_attention", handle.prism_kv_attention(
        q.data_ptr(), q.stride(0), q.stride(1), cache[0].data_ptr(), cache[1].data_ptr(), cache[2].data_ptr(),
        cache[3].data_ptr(), page_table.data_ptr(), page_table.stride(0), seq_lens.data_ptr(), cu, out.data_ptr(),
        out.stride(0), out.stride(1), None if lse is None else lse.data_ptr(), d ** -0.5 if scale is None else scale,
        1 if causal else 0, window, seqs, rows, max_q, num_pages, max_pages, q_heads, heads, d, block, ws, ws_bytes,
        _err(err, device), _stream(stream)))
    return out


def prism_w4g_linear(q, a_scale, w4, group_scale, group_offset=None, residual=None, out=None, stream=None):
    """out bf16 [M, N] = a_scale * (q @ w^T) + residual with 4-bit weights
    w[n, k] = group_scale[n, k / g] * code[n, k] + group_offset[n, k / g].

    ``q`` int8 [M, K], ``a_scale`` float32 [M] (prism_quant_act); ``w4`` uint8
    [N, K/2] (code 2j in the low nibble of byte j); ``group_scale`` and the
    optional ``group_offset`` float16 [N, K/g], g = 32, 64 or 128; ``residual``
    bf16 [M, N] or None, may be ``out`` itself."""
    device = _device(q, "q")
    _tensor(q, "q", _I8, 2, device)
    _tensor(a_scale, "a_scale", _F32, 1, device)
    _tensor(w4, "w4", _U8, 2, device)
    _tensor(group_scale, "group_scale", _F16, 2, device)
    m, k = q.shape
    n, groups = group_scale.shape
    if a_scale.numel() != m or w4.shape != (n, k // 2) or k % 2 or groups == 0 or k % groups:
        raise ValueError("q [M, K], a_scale [M], w4 [N, K/2] and group_scale [N, K/g] do not agree")
    if group_offset is not None:
        _tensor(group_offset, "group_offset", _F16, 2, device)
        if group_offset.shape != group_scale.shape:
            raise ValueError("group_offset must have group_scale's shape")
    if out is None:
        out = torch.empty((m, n), dtype=_BF16, device=device)
    else:
        _tensor(out, "out", _BF16, 2, device)
        if out.shape != (m, n):
            raise ValueError("out must be [M, N]")
    if residual is not None:
        _tensor(residual, "residual", _BF16, 2, device)
        if residual.shape != (m, n):
            raise ValueError("residual must be [M, N]")
    _check("prism_w4g_linear", lib().prism_w4g_linear(
        q.data_ptr(), q.stride(0), a_scale.data_ptr(), w4.data_ptr(), w4.stride(0), group_scale.data_ptr(),
        group_scale.stride(0), None if group_offset is None else group_offset.data_ptr(),
        0 if group_offset is None else group_offset.stride(0), None if residual is None else residual.data_ptr(),
        0 if residual is None else residual.stride(0), out.data_ptr(), out.stride(0), m, n, k, k // groups,
        _stream(stream)))
    return out


def prism_token_logprobs(logits, token_ids, top_k: int = 0, entropy=True, err=None, stream=None):
    """Log probabilities of ``token_ids`` int32 [R, n] under ``logits`` [R, V]
    (bf16 or float32) -> (logprobs float32 [R, n], entropy float32 [R] or None,
    top_ids int32 [R, top_k], top_logprobs float32 [R, top_k]; the last two
    None for top_k = 0).  ``err``: optional int32 [1] device error word."""
    device = _device(logits, "logits")
    if logits.dtype is not _BF16 and logits.dtype is not _F32:
        raise TypeError(f"logits must be bfloat16 or float32, got {logits.dtype}")
    _tensor(logits, "logits", logits.dtype, 2, device)
    _tensor(token_ids, "token_ids", _I32, 2, device)
    rows, vocab = logits.shape
    n = token_ids.size(1)
    if token_ids.size(0) != rows:
        raise ValueError("token_ids must have a row for each row of logits")
    logprobs = torch.empty((rows, n), dtype=_F32, device=device)
    ent = torch.empty((rows,), dtype=_F32, device=device) if entropy else None
    top_ids = torch.empty((rows, top_k), dtype=_I32, device=device) if top_k else None
    top_lp = torch.empty((rows, top_k), dtype=_F32, device=device) if top_k else None
    _check("prism_token_logprobs", lib().prism_token_logprobs(
        logits.data_ptr(), 1 if logits.dtype is _F32 else 0, logits.stride(0), token_ids.data_ptr(),
        token_ids.stride(0), n, rows, vocab, top_k, logprobs.data_ptr(), None if ent is None else ent.data_ptr(),
        None if top_ids is None else top_ids.data_ptr(), None if top_lp is None else top_lp.data_ptr(),
        _err(err, device), _stream(stream)))
    return logprobs, ent, top_ids, top_lp
