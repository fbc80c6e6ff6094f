// kv_plan.cuh -- how a call of the cache's attention is cut into items, and what
// its kernels share.
//
// A sequence's n queries times its G query heads per KV head are rows.  Up to
// kFewRows rows (decode steps, a few drafted tokens) go to the kernel that
// streams keys through the warp-level tensor instructions: an item is a tile of
// rows and a piece of the keys.  More rows go to the one on the tcgen05 tensor
// cores: the blocks of keys of one tile of 128 rows after the other form a line,
// which is cut into ranges of equal length, an item each; a tile is in pieces
// where a cut falls into it.  The choice and the cuts depend on the sequence's
// own rows and length (and the number of KV heads) alone, so that its result
// does not depend on the rest of the batch.  The pieces of a row are joined in
// the order of their keys.
#pragma once

#include "decode.cuh"

namespace prism {
namespace kv {

constexpr int kFewRows = 32;
constexpr int kWideRows = 128;         // rows of a tile of the tcgen05 kernel: the lanes of tensor memory
// Keys of a piece at least.  With 512, 1024 and 2048, 40 heads on 8 of 128 and one
// query: 64 sequences of 300 to 4096 keys 67.3, 62.0 and 64.7 us, one of 4096 keys
// 12.4, 15.2 and 21.4, eight of them 26.0, 24.2 and 28.8, 16 of 2000 to 9000 50.8,
// 45.4 and 41.9.
constexpr int kMinChunk = 1024;
constexpr int kMaxSplit = 128;         // pieces of a row at most
constexpr int kFillFew = 3 * kSms;     // items that one sequence is cut into where it has the keys: three on each SM
// Blocks of a range at least, where a line has more ranges than tiles: a part of
// a tile costs about eight blocks' time besides its blocks (80 rows, 8 KV heads,
// 8208 keys, with 6, 10 and 16 at least: one sequence 37.8, 40.1 and 48.1 us,
// three 60.5, 44.4 and 52.5, eight 123, 99 and 92).
constexpr int kMinBlocks = 10;
__host__ __device__ constexpr int wide_shift(int D) { return D == 256 ? 6 : 7; }
__host__ __device__ constexpr int wide_keys(int D) { return 1 << wide_shift(D); }   // keys of a block of the tcgen05 kernel
constexpr float kPShift = 12.0f;       // pieces keep their maximum m with 2^(x - m + 12) as the weight of score x
constexpr float kLn2 = 0.69314718055994531f;

// Pieces of the keys of a sequence of few rows, H KV heads: as many as fill the SMs.
__host__ __device__ __forceinline__ int split_count(int64_t keys, int64_t H) {
  const int64_t n = (keys + kMinChunk - 1) / kMinChunk, most = n < 1 ? 1 : n > kMaxSplit ? kMaxSplit : n;
  const int cap = kFillFew / static_cast<int>(H);
  return most > cap ? (cap < 1 ? 1 : cap) : static_cast<int>(most);
}
// Ranges of each KV head's line of so many tiles and blocks: as many as fill the
// SMs in the fewest turns that leave at most a tenth of them empty (or the best
// of four).
__host__ __device__ __forceinline__ int range_count(int64_t tiles, int64_t blocks, int H) {
  int best = 1, best_turns = 0;
  for (int turns = (H + kSms - 1) / kSms, i = 0; i < 4; ++turns, ++i) {
    const int n = kSms * turns / H;
    if (best_turns == 0 || n * best_turns > best * turns) best = n, best_turns = turns;
    if (n * H * 10 >= kSms * turns * 9) break;
  }
  const int64_t most = tiles > blocks / kMinBlocks ? tiles : blocks / kMinBlocks;
  return most < best ? static_cast<int>(most) : best;
}
// Pieces of a wide sequence, in slots of as many rows as its tiles have: a range
// has at most two tiles in pieces, the one that it begins inside of and one that
// begins in it, and along the line a next piece has a next range or a next tile.
__host__ __device__ __forceinline__ int64_t wide_slots(int64_t tiles, int64_t ranges) {
  return tiles <= ranges ? ranges + tiles - 1 : 2 * ranges;
}
__host__ __device__ __forceinline__ int64_t wide_slot(int64_t tiles, int64_t ranges, int64_t range, int64_t tile, bool begins) {
  return tiles <= ranges ? range + tile : 2 * range + (begins ? 1 : 0);
}

// A call's workspace: (D + 4) floats for a (row, piece) pair.  Its place depends on
// the sequence or on its first query alone, whichever takes less for the call:
// where sequences are long and few, so many pairs as one has at most for each; in
// a batch of many, so many for each query as it has at most.
struct Parts {
  int64_t rows = 0;                      // pairs of one KV head
  int64_t per_seq = 0, per_query = 0;    // one of them is 0
  int64_t few = 0, ranges = 0;           // pairs of a sequence of few rows; ranges of a wide one: at most
};
// The most of everything; fewer rows or keys of a sequence never take more.  A
// wide sequence of t tiles has at least 128 (t - 1) + 1 rows (33), and at most
// max(t, t blocks / kMinBlocks) ranges: 1 + max(2, blocks / 5) pairs a row.
inline Parts parts_of(int64_t S, int64_t T, int64_t max_q, int64_t G, int64_t max_keys, int64_t H, int64_t D) {
  static_assert(kMinBlocks == 10, "the bound of a row's pairs");
  Parts p;
  const int64_t rows = max_q * G, splits = split_count(max_keys, H);
  int64_t of_seq = 0, of_row = 0;
  if (splits > 1) of_seq = p.few = splits * std::min<int64_t>(kFewRows, rows), of_row = splits;
  if (rows > kFewRows) {
    const int64_t tiles = (rows + kWideRows - 1) / kWideRows, blocks = (max_keys + wide_keys(static_cast<int>(D)) - 1) >> wide_shift(static_cast<int>(D));
    p.ranges = range_count(tiles, tiles * blocks, static_cast<int>(H));
    if (p.ranges > 1) {
      of_seq = std::max(of_seq, wide_slots(tiles, p.ranges) * std::min<int64_t>(kWideRows, rows));
      of_row = std::max(of_row, 1 + std::min(p.ranges, std::max<int64_t>(2, (blocks + 4) / 5)));
    }
  }
  if (S * of_seq <= T * G * of_row) {
    p.per_seq = of_seq;
    p.rows = S * of_seq;
  } else {
    p.per_query = G * of_row;
    p.rows = T * p.per_query;
  }
  return p;
}

// A sequence's plan: its rows, key range and pieces.
struct SeqPlan {
  SeqSpan sp;
  int32_t rows, tiles, splits;   // splits: pieces of a tile, or ranges
  int32_t lo, chunk;     // first key seen by any of its queries (rounded down to 64), keys of a piece
  bool bad;              // malformed length: its rows get NaN
};
// The sequence's items (tiles x pieces or ranges, x KV heads) of the kernel that asks, 0
// where the other one has it; -1 for malformed offsets (no rows to answer
// for).  A malformed length is the few-row kernel's.
template <bool kWide, int kTileRows, bool kJoin = false>   // kJoin: the plan of either kind
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
    if (p.rows <= kFewRows) {
      if constexpr (!kWide) {
        p.splits = split_count(keys, a.c.H);
        p.chunk = static_cast<int32_t>(((static_cast<uint32_t>(keys) + p.splits - 1) / p.splits + 63) & ~63u);
      }
    } else if constexpr (kWide || kJoin) {
      const int shift = wide_shift(a.c.D);
      const int64_t tiles = (static_cast<int64_t>(p.rows) + kWideRows - 1) / kWideRows;
      p.splits = range_count(tiles, tiles * ((keys + (1 << shift) - 1) >> shift), a.c.H);
    }
  }
  if (kWide ? p.bad || p.rows <= kFewRows : !p.bad && p.rows > kFewRows) return 0;
  return (kWide ? 1 : p.tiles) * p.splits * a.c.H;
}

// The sequence's first pair in the workspace, in pairs.
__device__ __forceinline__ int64_t first_part(const Parts& w, const SeqPlan& p, int s, int hk) {
  return hk * w.rows + s * w.per_seq + p.sp.b * w.per_query;
}
// The first row of a piece of tile `tile`, from there.
__device__ __forceinline__ int64_t wide_part(const SeqPlan& p, int range, int tile, bool begins) {
  return wide_slot((p.rows + kWideRows - 1) / kWideRows, p.splits, range, tile, begins) * min(p.rows, kWideRows);
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
  if (!kWide) {
    w.tile = rest % p.tiles;
    rest /= p.tiles;
  }
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
  int32_t k_first;             // no row sees a key of the 16-key units before it: their pages may be gone
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
    k_first = t_lo & ~15;
    const int64_t piece_end = static_cast<int64_t>(p.lo) + static_cast<int64_t>(w.split + 1) * p.chunk;
    k_end = static_cast<int32_t>(min(static_cast<int64_t>(t_hi), piece_end));
  }
  __device__ __forceinline__ int32_t hi(int r) const {
    return r >= n_rows || none ? 0 : causal ? max(0, first_pos + (row0 + r) / G + 1) : len;
  }
  __device__ __forceinline__ int32_t lo(int32_t hi) const { return window > 0 && hi > window ? hi - window : 0; }
};

// The lines of a wide sequence.  A tile's blocks: the first begins at the first
// key that any of its rows sees, rounded down to 64; at least one.
__device__ __forceinline__ int tile_blocks(const KvAttentionArgs& a, const SeqPlan& p, int tile) {
  Walk w = new_walk();
  w.tile = tile;
  const TileKeys k(a, p, w, kWideRows);
  const int shift = wide_shift(a.c.D);
  return max(1, (k.t_hi - (k.t_lo & ~63) + (1 << shift) - 1) >> shift);
}
// Blocks up to the end of each thread's tiles (tiles_a_thread of them) in s_line
// [kThreads]; s_warp64 [kThreads / 32].  All threads, ends with a barrier.
template <int kThreads>
__device__ __forceinline__ void lay_line(const KvAttentionArgs& a, const SeqPlan& p, int64_t* s_line, int64_t* s_warp64) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tiles = (p.rows + kWideRows - 1) / kWideRows, each = (tiles + kThreads - 1) / kThreads;
  int64_t n = 0;
  for (int t = tid * each; t < min(tiles, (tid + 1) * each); ++t) n += tile_blocks(a, p, t);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, n, o);
    if (lane >= o) n += v;
  }
  __syncthreads();
  if (lane == 31) s_warp64[warp] = n;
  __syncthreads();
  for (int i = 0; i < warp; ++i) n += s_warp64[i];
  s_line[tid] = n;
  __syncthreads();
}
// A tile's place in its line: its first block and its number of blocks.
struct TileSpan {
  int64_t x;
  int blocks;
};
template <int kThreads>
__device__ __forceinline__ TileSpan tile_span(const KvAttentionArgs& a, const SeqPlan& p, const int64_t* s_line, int tile) {
  const int tiles = (p.rows + kWideRows - 1) / kWideRows, each = (tiles + kThreads - 1) / kThreads, at = tile / each;
  TileSpan t{at > 0 ? s_line[at - 1] : 0, 0};
  if (each == 1) {
    t.blocks = static_cast<int>(s_line[at] - t.x);
    return t;
  }
  for (int i = at * each; i < tile; ++i) t.x += tile_blocks(a, p, i);
  t.blocks = tile_blocks(a, p, tile);
  return t;
}
// The tile that block x lies in.
template <int kThreads>
__device__ __forceinline__ int tile_at(const KvAttentionArgs& a, const SeqPlan& p, const int64_t* s_line, int64_t x) {
  const int tiles = (p.rows + kWideRows - 1) / kWideRows, each = (tiles + kThreads - 1) / kThreads;
  int at = 0;
#pragma unroll
  for (int o = 512; o > 0; o >>= 1)
    if (at + o < kThreads && s_line[at + o - 1] <= x) at += o;
  int tile = at * each;
  if (each == 1) return tile;
  for (int64_t y = at > 0 ? s_line[at - 1] : 0;; ++tile) {
    y += tile_blocks(a, p, tile);
    if (y > x || tile + 1 >= tiles) return tile;
  }
}
// The line of `blocks` in `ranges`: range r is [cut(r), cut(r + 1)), none empty.
struct Cuts {
  int64_t blocks;
  int ranges;
  int64_t whole;
  int rest;              // blocks = whole * ranges + rest
  __device__ __forceinline__ Cuts(int64_t blocks, int most)
      : blocks(blocks), ranges(static_cast<int>(min(blocks, static_cast<int64_t>(most)))) {
    whole = blocks >> 31 == 0 ? static_cast<int>(blocks) / ranges : blocks / ranges;
    rest = static_cast<int>(blocks - whole * ranges);
  }
  __device__ __forceinline__ int64_t cut(int r) const {
    r = min(r, ranges);
    return whole * r + rest * r / ranges;   // ranges^2 stays below 2^31
  }
  __device__ __forceinline__ int range_of(int64_t x) const {
    const int64_t n = (x + 1) * ranges - 1;
    return static_cast<int>(blocks >> 20 == 0 ? static_cast<int>(n) / static_cast<int>(blocks) : n / blocks);   // ranges < 2^11
  }
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
cudaError_t launch_kv_attention_wide(const KvAttentionArgs& a, const kv::Parts& parts, cudaStream_t stream);
}  // namespace prism
