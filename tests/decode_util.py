"""Plain 64-bit statements of the decode-step operators, shared by their GPU
tests.  Each returns the values and, where an output is rounded, the bound that
the arithmetic of the definition allows (counted in half steps of its types)."""
import numpy as np
import torch

HALF_BF16, HALF_F16, HALF_F32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24


def page_table(lens, block, rng, extra=2, shared=0):
    """Shuffled pages for the lengths (the first ``shared`` pages common to all);
    unused entries are far out of range."""
    counts = [-(-n // block) for n in lens]
    width = max(max(counts), 1) + extra
    total = shared + sum(max(0, c - shared) for c in counts)
    order = rng.permutation(total + 3).astype(np.int32)
    table = np.full((len(lens), width), 1 << 30, np.int32)
    at = shared
    for i, c in enumerate(counts):
        table[i, :min(c, shared)] = order[:min(c, shared)]
        n = max(0, c - shared)
        table[i, shared:shared + n] = order[at:at + n]
        at += n
    return table, total + 3


def random_cache(rng, pages, heads, block, d):
    codes = [rng.integers(-127, 128, (pages, heads, block, d)).astype(np.int8) for _ in range(2)]
    scales = [rng.uniform(0.004, 0.03, (pages, heads)).astype(np.float32) for _ in range(2)]
    return codes + scales


def rows_of(codes, scales, table_row, length, head, block):
    """Values [length, D] float64 of one sequence and KV head."""
    pages = table_row[:-(-length // block)]
    x = codes[pages, head].astype(np.float64) * scales[pages, head].astype(np.float64)[:, None, None]
    return x.reshape(-1, codes.shape[-1])[:length]


def attention(q, cache, table, lens, counts, block, scale, causal=True, window=0):
    """(out, bound, lse, lse_bound) in float64 for q [T, Hq, D] (float64 values of bf16).

    The bound of an output: half a bf16 step of the value, and A = sum p |v|
    times the relative error of a probability -- half a binary16 step, twice
    the error of its score (D binary32 additions of sum |q k|, one step each)
    and 2^-19 for the exponential and the sums (up to 64 pieces joined)."""
    T, hq, d = q.shape
    hkv = cache[0].shape[1]
    g = hq // hkv
    out, bound = np.zeros((T, hq, d)), np.zeros((T, hq, d))
    lse, lse_bound = np.full((T, hq), -np.inf), np.zeros((T, hq))
    at = 0
    for s, (length, n) in enumerate(zip(lens, counts)):
        for h in range(hkv):
            if length == 0 or n == 0:
                continue
            k = rows_of(cache[0], cache[2], table[s], length, h, block)
            v = rows_of(cache[1], cache[3], table[s], length, h, block)
            for i in range(n):
                p = length - n + i
                hi = min(length, p + 1) if causal else length
                lo = max(0, p + 1 - window) if window else 0
                if hi <= lo:
                    continue
                for j in range(h * g, (h + 1) * g):
                    x = k[lo:hi] @ q[at + i, j] * scale
                    size = (np.abs(k[lo:hi]) @ np.abs(q[at + i, j]) * scale).max()
                    m = x.max()
                    e = np.exp(x - m)
                    w = e / e.sum()
                    out[at + i, j] = w @ v[lo:hi]
                    score = d * 2 * HALF_F32 * size
                    rel = HALF_F16 + 2 * score + 2.0 ** -19
                    bound[at + i, j] = HALF_BF16 * np.abs(out[at + i, j]) + rel * (w @ np.abs(v[lo:hi])) \
                        + (hi - lo) * 2.0 ** -37 * np.abs(v[lo:hi]).max()
                    lse[at + i, j] = m + np.log(e.sum())
                    lse_bound[at + i, j] = 2 * score + 2.0 ** -19 + 4 * HALF_F32 * abs(lse[at + i, j])
        at += n
    return out, bound, lse, lse_bound


def quantise_block(x):
    """(codes, scales) of one page: x float32 [rows, H, D]; each step binary32."""
    amax = np.abs(x).max(axis=(0, 2)).astype(np.float32)
    live = amax >= np.float32(2.0 ** -120)
    safe = np.where(live, amax, np.float32(1.0))
    f = np.where(live, (np.float32(1.0) / safe) * np.float32(127.0), np.float32(0.0)).astype(np.float32)
    codes = np.clip(np.rint(x * f[None, :, None]), -127, 127).astype(np.int8)
    scale = np.where(live, amax * (np.float32(1.0) / np.float32(127.0)), np.float32(0.0)).astype(np.float32)
    return codes, scale


def bf16(rng, shape, scale=1.0):
    """(torch bf16 tensor, its float32 values)."""
    t = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)
    return t, t.float().numpy()
