"""Binding of the decode-step operators: the paged int8 K/V cache and the
attention over it, the 4-bit linear with group scales, and the token log
probabilities (contracts in ``include/prism.h``).

Entry points (same names as the C ABI):
  KvCache, new_kv_cache(...)                       the cache's six buffers
  prism_kv_append(k, v, cache, page_table, seq_lens, ...)
  prism_kv_attention(q, cache, page_table, seq_lens, ...)        -> out
  prism_w4g_linear(q, a_scale, w4, group_scale, ...)             -> out
  prism_token_logprobs(logits, token_ids, top_k=...)             -> (logprobs, entropy, top_ids, top_logprobs)

Each takes ``stream`` (default: torch's current one); the outputs and the
workspace that a call allocates belong to that stream.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _check, lib

_BF16, _F32, _I8 = torch.bfloat16, torch.float32, torch.int8

lib()   # one loaded library for both bindings; says what to do where it is not built
try:
    from . import _decode  # (csrc/decode_py.cpp: checks, outputs and the calls)
except ImportError as e:
    raise ImportError("_decode.so is not built, or for another torch; run deterministic_w8a8_int8_gb300.build.build() "
                      "(needs nvcc, g++, and torch's and Python's headers)") from e

_decode.setup(_check)


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


def prism_kv_append(k, v, cache, page_table, seq_lens, cu_new=None, max_new=None, err=None, stream=None):
    """Append the rows ``k``, ``v`` bf16 [T, H_kv, D] to the sequences of
    ``cache`` (a KvCache).  ``seq_lens`` int32 [S]: tokens before the call
    (not changed); ``cu_new`` int32 [S + 1]: each sequence's rows, None for one
    row each; ``max_new``: a launch hint, the most rows of one sequence;
    ``err``: optional int32 [1] device error word."""
    _decode.append(k, v, cache, page_table, seq_lens, cu_new, max_new, err, stream)


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
    return _decode.attention(q, cache, page_table, seq_lens, cu_q, max_q, scale, causal, window, out, lse, workspace, err,
                             stream)


def prism_w4g_linear(q, a_scale, w4, group_scale, group_offset=None, residual=None, out=None, stream=None):
    """out bf16 [M, N] = a_scale * (q @ w^T) + residual with 4-bit weights
    w[n, k] = group_scale[n, k / g] * code[n, k] + group_offset[n, k / g].

    ``q`` int8 [M, K], ``a_scale`` float32 [M] (prism_quant_act); ``w4`` uint8
    [N, K/2] (code 2j in the low nibble of byte j); ``group_scale`` and the
    optional ``group_offset`` float16 [N, K/g], g = 32, 64 or 128; ``residual``
    bf16 [M, N] or None, may be ``out`` itself."""
    return _decode.w4g_linear(q, a_scale, w4, group_scale, group_offset, residual, out, stream)


def prism_token_logprobs(logits, token_ids, top_k: int = 0, entropy=True, err=None, stream=None):
    """Log probabilities of ``token_ids`` int32 [R, n] under ``logits`` [R, V]
    (bf16 or float32) -> (logprobs float32 [R, n], entropy float32 [R] or None,
    top_ids int32 [R, top_k], top_logprobs float32 [R, top_k]; the last two
    None for top_k = 0).  ``err``: optional int32 [1] device error word."""
    return _decode.token_logprobs(logits, token_ids, top_k, entropy, err, stream)
