// kv_plan.cuh -- how a call of the cache's attention is cut into items, and what
// its kernels share.
//
// A sequence's n queries times its G query heads per KV head are rows.  Up to
// kFewRows rows (decode steps, a few drafted tokens) go to the kernel that
// streams keys through the warp-level tensor instructions, more rows to the
// one on the tcgen05 tensor cores.  The keys of either are cut into pieces of
// at least kMinChunk; the choice and the cut depend on the sequence's own rows
// and length (and the number of KV heads) alone, so that its result does not
// depend on the rest of the batch.  The pieces of a row are joined in piece
// order.
#pragma once

#include "decode.cuh"

namespace prism {
namespace kv {

constexpr int kFewRows = 32;
constexpr int kWideRows = 128;         // rows of a tile of the tcgen05 kernel: the lanes of tensor memory
constexpr int kMinChunk = 1024;        // keys of a piece at least
constexpr int kMaxSplit = 128;         // pieces of a row at most
constexpr int kFillFew = 456;          // items that one sequence is cut into where it has the keys: three on each of 152 SMs
constexpr int kSms = 152;              // one wide item on each at a time
constexpr float kPShift = 12.0f;       // pieces keep their maximum m with 2^(x - m + 12) as the weight of score x
constexpr float kLn2 = 0.69314718055994531f;

// Pieces of the keys of a sequence with so many rows, H KV heads: for few rows
// as many as fill the SMs, for more the fewest that leave at most a fifth of
// the SMs' turns empty (or the best of eight).
__host__ __device__ __forceinline__ int split_count(int64_t keys, int64_t rows, int64_t H) {
  const int64_t n = (keys + kMinChunk - 1) / kMinChunk, most = n < 1 ? 1 : n > kMaxSplit ? kMaxSplit : n;
  if (rows <= kFewRows) {
    const int64_t cap = kFillFew / H;
    return static_cast<int>(most > cap ? (cap < 1 ? 1 : cap) : most);
  }
  if ((rows + kWideRows - 1) / kWideRows * H >= 4 * kSms) return 1;   // one piece uses four fifths
  const int one = static_cast<int>((rows + kWideRows - 1) / kWideRows * H);   // items with one piece
  int best = 1, best_n = 0, best_d = 1;                                       // share of the turns in use, as a fraction
  for (int k = one >= kSms ? 1 : (kSms * 4 / 5 + one - 1) / one, i = 0; i < 8; ++k, ++i) {
    if (k > most) k = static_cast<int>(most), i = 8;
    const int items = k * one, d = (items + kSms - 1) / kSms * kSms;
    if (items * best_d > best_n * d) best = k, best_n = items, best_d = d;
    if (items * 5 >= d * 4) break;
  }
  return best;
}
// The most rows of one (sequence, KV head) that can be cut into pieces, and
// its most (row, piece) pairs.  Fewer keys never make more pieces.
inline int64_t max_split_rows(int64_t max_q, int64_t G, int64_t max_keys, int64_t H, int64_t* rows) {
  int64_t most = 0;
  *rows = 0;
  auto take = [&](int64_t r) {
    const int64_t splits = split_count(max_keys, r, H);
    if (splits <= 1) return;
    *rows = std::max(*rows, r);
    most = std::max(most, splits * r);
  };
  take(std::min<int64_t>(kFewRows, max_q * G));
  for (int64_t tiles = 1; max_q * G > kFewRows; ++tiles) {
    take(std::min(tiles * kWideRows, max_q * G));
    if (tiles * kWideRows >= max_q * G || tiles * H >= 4 * kSms) break;   // beyond: one piece uses four fifths
  }
  return most;
}

// A sequence's plan: its rows, key range and pieces.
struct SeqPlan {
  SeqSpan sp;
  int32_t rows, tiles, splits;
  int32_t lo, chunk;     // first key seen by any of its queries (rounded down to 64), keys of a piece
  bool bad;              // malformed length: its rows get NaN
};
// The sequence's items (tiles x pieces x KV heads) of the kernel that asks, 0
// where the other one has it; -1 for malformed offsets (no rows to answer
// for).  A malformed length is the few-row kernel's.
template <bool kWide, int kTileRows>
__device__ __forceinline__ int seq_items(const KvAttentionArgs& a, int s, SeqPlan& p) {
  const bool ok = seq_span(a.c, a.cu_q, a.T, s, true, p.sp);
  if (p.sp.b < 0 || p.sp.n < 0 || static_cast<int64_t>(p.sp.b) + p.sp.n > a.T) return -1;
  p.bad = !ok || p.sp.n > a.max_q;
  p.rows = p.sp.n * a.G;
  p.tiles = (p.rows + kTileRows - 1) / kTileRows;
  p.splits = 1;
  p.lo = p.chunk = 0;
  if (!p.bad && p.rows > 0) {
    const int64_t first = a.window > 0 ? p.sp.len - p.sp.n + 1 - a.window : 0;
    p.lo = first > 0 ? static_cast<int32_t>(first) & ~63 : 0;
    const int64_t keys = p.sp.len - p.lo;
    p.splits = split_count(keys, p.rows, a.c.H);
    p.chunk = static_cast<int32_t>((((keys + p.splits - 1) / p.splits) + 63) & ~63ll);
  }
  if (kWide ? p.bad || p.rows <= kFewRows : !p.bad && p.rows > kFewRows) return 0;
  return p.tiles * p.splits * a.c.H;
}

// Walks a CTA's items: sequences are counted a window of one a thread at a
// time, by a scan.
struct Walk {
  int s0, next;                // first sequence of the window, and of the one after
  int64_t base;                // items before it
  int items;                   // items in it
  int tile, split, hk, s;      // the item found
};
__device__ __forceinline__ Walk new_walk() { return Walk{0, 0, 0, 0, 0, 0, 0, -1}; }
// Finds `item`, and the plan of its sequence (p keeps the one of w.s); false past the last one.  All kThreads threads; s_scan
// [kThreads] and s_warp [kThreads / 32] are free again after the caller's next
// barrier.  kThreads <= 1023.
template <bool kWide, int kTileRows, int kThreads>
__device__ __forceinline__ bool find_item(const KvAttentionArgs& a, int64_t item, Walk& w, int* s_scan, int* s_warp,
                                          SeqPlan& p) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  while (item >= w.base + w.items) {
    w.base += w.items;
    if (w.next >= a.c.S) return false;
    w.s0 = w.next;
    w.next += kThreads;
    SeqPlan q;
    int n = w.s0 + tid < a.c.S ? seq_items<kWide, kTileRows>(a, w.s0 + tid, q) : 0;
    if (!kWide && blockIdx.x == 0 && w.s0 + tid < a.c.S && (n < 0 || (q.bad && n > 0)) && a.err != nullptr)
      atomicOr(a.err, PRISM_DEV_ERR_SEQ_RANGE);
    n = max(n, 0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += v;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = n;
    __syncthreads();
    for (int i = 0; i < warp; ++i) n += s_warp[i];
    s_scan[tid] = n;
    __syncthreads();
    w.items = s_scan[kThreads - 1];
  }
  const int local = static_cast<int>(item - w.base);
  int at = 0;
#pragma unroll
  for (int o = 512; o > 0; o >>= 1)
    if (at + o <= kThreads && s_scan[at + o - 1] <= local) at += o;
  if (w.s != w.s0 + at) {
    w.s = w.s0 + at;
    seq_items<kWide, kTileRows>(a, w.s, p);
  }
  int rest = local - (at > 0 ? s_scan[at - 1] : 0);
  w.tile = rest % p.tiles;
  rest /= p.tiles;
  w.split = rest % p.splits;
  w.hk = rest / p.splits;
  return true;
}

// The keys that a tile's rows see: row r of the tile stands at position
// first_pos + (row0 + r) / G.  Rows rise, so every row sees [a_lo, a_hi) and
// some row [t_lo, t_hi).
struct TileKeys {
  int32_t row0, n_rows, first_pos, len, G, window;
  bool causal, none;
  int32_t a_hi, t_hi, t_lo, a_lo, k_begin, k_end;
  TileKeys() = default;
  __device__ __forceinline__ TileKeys(const KvAttentionArgs& a, const SeqPlan& p, const Walk& w, int tile_rows) {
    row0 = w.tile * tile_rows;
    n_rows = min(tile_rows, p.rows - row0);
    len = static_cast<int32_t>(p.sp.len);
    first_pos = len - p.sp.n;
    G = a.G;
    window = static_cast<int32_t>(min(a.window, static_cast<int64_t>(INT32_MAX)));
    causal = a.causal != 0;
    none = p.bad;
    a_hi = hi(0);
    t_hi = hi(n_rows - 1);
    t_lo = lo(a_hi);
    a_lo = lo(t_hi);
    k_begin = max(p.lo + w.split * p.chunk, t_lo & ~63);
    const int64_t piece_end = static_cast<int64_t>(p.lo) + static_cast<int64_t>(w.split + 1) * p.chunk;
    k_end = static_cast<int32_t>(min(static_cast<int64_t>(t_hi), piece_end));
  }
  __device__ __forceinline__ int32_t hi(int r) const {
    return r >= n_rows || none ? 0 : causal ? max(0, first_pos + (row0 + r) / G + 1) : len;
  }
  __device__ __forceinline__ int32_t lo(int32_t hi) const { return window > 0 && hi > window ? hi - window : 0; }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Bytes 0, 1 (sel 0x4140) or 2, 3 (sel 0x4342) of codes ^ 0x80 as a binary16 pair, exact.
__device__ __forceinline__ uint32_t widen(uint32_t biased, uint32_t sel) {
  const uint32_t h = __byte_perm(biased, 0x64646464u, sel);
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(0x64806480u));   // 1024 + 128
  return r;
}
// The power of two that puts a row's largest |channel| at 2^13 in binary16, as
// a biased exponent (its inverse is 254 minus it).
__device__ __forceinline__ int query_exponent(float amax) {
  const int be = static_cast<int>(__float_as_uint(amax) >> 23);
  return be == 255 || be == 0 ? 127 : min(253, 127 + 13 + 127 - be);
}

}  // namespace kv

// The tcgen05 kernel (kv_attention_tc.cu): sequences of more than kv::kFewRows rows.
cudaError_t launch_kv_attention_wide(const KvAttentionArgs& a, int64_t part_stride, cudaStream_t stream);
}  // namespace prism
