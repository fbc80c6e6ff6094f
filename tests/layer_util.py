"""Plain statements of the operators between a layer's linears, shared by their
GPU tests.  Codes are restated step by step in binary32 (sums of squares in 64
bits), linear attention in 64 bits with the bound that its arithmetic allows."""
import numpy as np
import torch

F = np.float32
HALF_BF16 = 2.0 ** -8


def bf16(x):
    """float32 values rounded to bf16, as float32."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=F)).to(torch.bfloat16).float().numpy()


def rstd(x, eps):
    mean = np.square(x.astype(np.float64)).mean(axis=-1, keepdims=True)
    return (1.0 / np.sqrt(mean + float(F(eps)))).astype(F)


def fma(a, b, c):
    """a * b + c rounded once: the product of two binary32 values is exact in 64 bits."""
    return (a.astype(np.float64) * b + c).astype(F)


def exp_neg(x):
    """exp of x <= 0: n ln 2 + r, and the series of e^r to r^7 in fused steps."""
    n = np.maximum(np.rint(x.astype(np.float64) * float.fromhex("0x1.715476p+0")), -200).astype(F)
    r = fma(n, float.fromhex("0x1.bd0106p-13"), fma(n, -float.fromhex("0x1.63p-1"), x))
    p = np.full_like(r, float.fromhex("0x1.a01a02p-13"))
    for c in ("0x1.6c16c2p-10", "0x1.111112p-7", "0x1.555556p-5", "0x1.555556p-3", "0x1p-1", "0x1p+0", "0x1p+0"):
        p = fma(p, r, float.fromhex(c))
    return np.where(n < -126, F(0), p * np.exp2(np.maximum(n, -126)).astype(F)).astype(F)


def silu(z):
    with np.errstate(over="ignore", invalid="ignore"):
        e = exp_neg(-np.abs(z))
    return (z * (np.where(z >= 0, F(1), e) / (F(1) + e))).astype(F)


def codes(y, form):
    """(q, a_scale) of binary32 rows; form bf16: (values, None)."""
    if form == "bf16":
        return bf16(y), None
    amax = np.abs(y).max(axis=1).astype(F)
    live = amax >= F(2.0 ** -120)
    inv = np.where(live, F(127) / np.where(live, amax, F(1)), F(0)).astype(F)
    q = np.clip(np.rint(y * inv[:, None]), -127, 127)
    return q.astype(np.int8 if form == "int8" else np.float16), np.where(live, amax / F(127), F(0)).astype(F)


def norm(x, weight, delta=None, alpha=1.0, post=None, eps=1e-6):
    """(y, h) of float32 arrays of bf16 values."""
    h = x
    if delta is not None:
        d = delta if post is None else (delta * rstd(delta, eps)) * post
        h = bf16(x + F(alpha) * d)
    return (h * rstd(h, eps)) * weight, h


def head_norm(x, weight, gate=None, inv=None, eps=1e-6):
    y = (x * rstd(x, eps)) * weight
    if gate is not None:
        y = y * silu(gate)
    y = y.reshape(y.shape[0], -1)
    return y if inv is None else y * inv


def glu(x, inv=None):
    f = x.shape[1] // 2
    y = silu(x[:, :f]) * x[:, f:]
    return y if inv is None else y * inv


def linear_attention(q, k, v, decay, starts, lens, scale):
    """(out, bound, states, bounds): float64 of packed tokens; ``starts`` the states
    [S, H, Dk, Dv] that the sequences start from.

    With S' and A the state and the output of the absolute values: a state is the
    sum of products in binary32, 64 of them to a chunk, each addition off by
    2^-23 at most (2^-17 of S'), the parts of a value by 2^-25 and each further
    chunk's decay and addition by 2^-22.  An output's score and the state it reads
    are in parts to 2^-17 each, their sums of up to 128 products off by 2^-16
    each and those over 64 scores by 2^-17, besides the state's own error, the
    exponentials' 2^-21 and the rounding to bf16: under 2^-14 of A in all."""
    T, hv, dv = v.shape
    rep = hv // q.shape[1]
    q, k, v, decay, starts = (torch.from_numpy(np.ascontiguousarray(x)).double().cuda() for x in (q, k, v, decay, starts))
    gain = torch.exp(decay.clamp(-16384.0, 0.0)).expand(T, hv)[..., None, None]
    q, k = (x.repeat_interleave(rep, dim=1) for x in (q, k))
    out, size = torch.zeros((T, hv, dv)).double().cuda(), torch.zeros((T, hv, dv)).double().cuda()
    states, bounds = starts.clone(), torch.zeros_like(starts)
    at = 0
    for s, n in enumerate(lens):
        both = torch.stack((states[s], states[s].abs()))       # S and A
        for t in range(at, at + n):
            kv = k[t][:, :, None] * v[t][:, None, :]
            both = gain[t] * both + torch.stack((kv, kv.abs()))
            o = torch.stack((q[t], q[t].abs()))[:, :, None, :] @ both
            out[t], size[t] = o[0, :, 0] * scale, o[1, :, 0] * abs(scale)
        states[s] = both[0]
        bounds[s] = both[1] * (2.0 ** -17 + 2.0 ** -22 * (2 + n // 64))
        at += n
    bound = HALF_BF16 * out.abs() + 2.0 ** -14 * size + 1e-38
    return tuple(x.cpu().numpy() for x in (out, bound, states, bounds + 1e-38))
