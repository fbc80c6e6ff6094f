"""Binding of the operators between a layer's linears: norms and the gated
activation down to the codes of the next linear, and linear attention
(contracts in ``include/prism.h``).

Entry points (same names as the C ABI):
  prism_norm_quant(x, weight, delta=..., ...)       -> (q, a_scale, h)
  prism_head_norm_quant(x, weight, gate=..., ...)   -> (q, a_scale)
  prism_glu_quant(gate_up, inv_s=...)               -> (q, a_scale)
  prism_linear_attention(q, k, v, log_decay, state, ...) -> out

``form`` says what ``q`` is: "int8" (codes for prism_w8a8_linear and the other
int8 linears), "f16" (the same codes as float16, for prism_w8a8_linear_f16) or
"bf16" (the values themselves; ``a_scale`` is None).  A row that is not finite has
codes 0 and a NaN for its scale, which the next linear passes on.  Each takes ``stream``
(default: torch's current one); the outputs and the workspace that a call
allocates belong to that stream.
"""
from __future__ import annotations

from . import lib
from .decode import _decode   # the extension module of these entry points too


def prism_norm_quant(x, weight, delta=None, alpha: float = 1.0, post_weight=None, eps: float = 1e-6, h=None,
                     form: str = "int8", stream=None):
    """The residual stream ``x`` bf16 [M, K] and its RMS norm, as codes:
    h = x + alpha * delta (rounded to bf16), y = norm(h) * weight, quantised.

    ``weight`` float32 [K] (times the linear's inv_smooth where its input is
    smoothed); ``delta`` bf16 [M, K] or None (h is x then); ``post_weight``
    float32 [K]: delta is normed itself before it is added; ``h``: the stream
    after the addition, allocated when None, may be ``x`` or ``delta`` itself.
    Returns (q, a_scale, h)."""
    return _decode.norm_quant(x, weight, delta, alpha, post_weight, eps, h, form, stream)


def prism_head_norm_quant(x, weight, gate=None, inv_s=None, eps: float = 1e-6, form: str = "int8", stream=None):
    """The RMS norm of each head of ``x`` bf16 [M, H, D], times ``weight``
    float32 [D], silu(``gate``) (bf16 [M, H, D], or None) and ``inv_s`` (float32
    [H * D], or None), as codes [M, H * D].  The heads of a row lie side by side."""
    return _decode.head_norm_quant(x, weight, gate, inv_s, eps, form, stream)


def prism_glu_quant(gate_up, inv_s=None, form: str = "int8", stream=None):
    """silu(gate) * up of ``gate_up`` bf16 [M, 2 F] (gate first), times ``inv_s``
    float32 [F] (or None), as codes [M, F]."""
    return _decode.glu_quant(gate_up, inv_s, form, stream)


def prism_linear_attention_workspace_bytes(seqs: int, rows: int, max_len: int, heads: int, key_dim: int,
                                           value_dim: int) -> int:
    return int(lib().prism_linear_attention_workspace_bytes(seqs, rows, max_len, heads, key_dim, value_dim))


def prism_linear_attention(q, k, v, log_decay, state=None, state_in=None, state_out=None, cu=None, max_len=None,
                           scale=None, out=None, workspace=None, err=None, stream=None):
    """Linear attention with a decay for each head: S = e^g S + k v^T, out = scale * q S,
    over the states ``state`` float32 [slots, H_v, D_k, D_v] -> bf16 [T, H_v, D_v].

    ``q``, ``k`` bf16 [T, H_k, D_k], ``v`` bf16 [T, H_v, D_v]; ``log_decay``
    float32 [T, H_v], or [H_v]: g; ``state_in``, ``state_out`` int32 [S]: the slot
    that each sequence starts from (-1, or no tensor: zeros) and the one that its
    last state goes to (-1, or no tensor: none); ``cu`` int32 [S + 1]: each
    sequence's tokens, None for one each; ``max_len``: the most tokens of one
    sequence (default: T, or 1 without cu); ``scale``: default D_k ** -0.5;
    ``workspace``: a uint8 tensor of prism_linear_attention_workspace_bytes bytes
    (allocated when None); ``err``: optional int32 [1] device error word.  Single
    tokens beside long sequences are faster in a call of their own, which gives the
    same bits."""
    return _decode.linear_attention(q, k, v, log_decay, state, state_in, state_out, cu, max_len, scale, out, workspace, err,
                                    stream)
