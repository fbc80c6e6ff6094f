// kv_attention.cu -- attention of new queries over the paged int8 K/V cache:
//   o = sum_j softmax_j(sm_scale * ks * (q . ck_j)) * vs * cv_j
// with codes ck, cv and one scale ks, vs per (page, head).
//
// Work: a sequence's n queries times its G query heads per KV head are rows;
// 16 rows make a tile, and the tile's keys are cut into pieces of at least
// kMinChunk keys (split_count below: a function of the sequence's own length
// and rows, so its result does not depend on the rest of the batch).  A
// persistent grid walks the items (sequence, KV head, piece, tile); pieces of
// one tile are joined by kv_combine_kernel in piece order.
//
// One item is one CTA of four warps; warp w takes every fourth step of 8 KB of
// K and V.  Each warp is on its own: its steps arrive through a private ring
// of cp.async copies, it keeps its own running maximum, sum and output, and
// the four are joined in shared memory at the end -- no barrier in the loop.
//   S = Q K^T and O += P V run on mma.sync m16n8k16 with binary16 operands and
// binary32 sums.  The codes widen exactly (byte ^ 0x80 under the exponent of
// 1024, minus 1152).  The order of channels inside S's contraction and of the
// output's columns is free, so lane (r, c) of a warp reads its operands as
// 16-byte pieces: channels 16c.. of key r for K; channels 16r.. of keys 2c,
// 2c+1, 2c+8, 2c+9 for V, whose two-key pairs a byte permute forms.  Queries
// become binary16 after an exact power-of-two scale that puts the row's
// largest channel at 2^13 (channels 2^27 below it lose bits: under 2^-38 of
// the row's maximum).  Probabilities are rounded to binary16 (half a step is
// 2^-11) with 2^12 as the value of the running maximum, so that keys down to
// 2^-26 of it stay normal numbers; a page's vs enters as its ratio to the
// largest vs seen so far.  Maxima, sums and outputs are binary32.
#include <cuda_fp16.h>

#include "decode.cuh"

namespace prism {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;
constexpr int kStages = 2;
constexpr int kStageBytes = 8192;      // K and V of one step of a warp
constexpr int kMinChunk = 512;         // keys of a piece at least
constexpr int kMaxSplit = 64;          // pieces x row tiles of a (sequence, KV head) at most
constexpr float kPShift = 12.0f;       // log2 of the probability of the running maximum
constexpr float kLn2 = 0.69314718055994531f;

template <int D>
constexpr int kUnits = kStageBytes / (2 * 16 * D);   // 16-key units of a step: 4, 2, 1 for D = 64, 128, 256
template <int D>
constexpr int kStepKeys = 16 * kUnits<D>;

__host__ __device__ __forceinline__ int split_count(int64_t keys, int64_t tiles) {
  const int64_t cap = tiles >= kMaxSplit ? 1 : kMaxSplit / tiles;
  const int64_t n = (keys + kMinChunk - 1) / kMinChunk;
  return static_cast<int>(n < 1 ? 1 : n > cap ? cap : n);
}
// Most (row, piece) pairs of one (sequence, KV head) that a call can split.
int64_t max_split_rows(int64_t max_q, int64_t G, int64_t max_keys) {
  int64_t most = 0;
  for (int64_t tiles = 1; tiles <= kMaxSplit / 2; ++tiles) {
    const int64_t splits = split_count(max_keys, tiles);
    if (splits > 1) most = std::max(most, splits * std::min(tiles * kRows, max_q * G));
    if (tiles * kRows >= max_q * G) break;
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
__device__ __forceinline__ int seq_items(const KvAttentionArgs& a, int s, SeqPlan& p) {
  const bool ok = seq_span(a.c, a.cu_q, a.T, s, true, p.sp);
  if (p.sp.b < 0 || p.sp.n < 0 || static_cast<int64_t>(p.sp.b) + p.sp.n > a.T) return -1;   // no rows to answer for
  p.bad = !ok || p.sp.n > a.max_q;
  p.rows = p.sp.n * a.G;
  p.tiles = (p.rows + kRows - 1) / kRows;
  p.splits = 1;
  p.lo = p.chunk = 0;
  if (!p.bad && p.rows > 0) {
    const int64_t first = a.window > 0 ? p.sp.len - p.sp.n + 1 - a.window : 0;
    p.lo = first > 0 ? static_cast<int32_t>(first) & ~63 : 0;
    const int64_t keys = p.sp.len - p.lo;
    p.splits = split_count(keys, p.tiles);
    p.chunk = static_cast<int32_t>((((keys + p.splits - 1) / p.splits) + 63) & ~63ll);
  }
  return p.tiles * p.splits * a.c.H;
}

__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src, int src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
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

// Shared-memory place of 16-byte piece `ch` of key `key` in a step's K (V):
// pieces of neighbouring keys are turned so that the eight lanes of a phase
// (keys r, r + 1 for K; keys 0, 2, 4, 6 for V) touch all banks once.
template <int D>
__device__ __forceinline__ int k_place(int key, int ch) {
  return key * D + ((D == 64 ? ch : ch ^ ((key & 1) << 2)) << 4);
}
template <int D>
__device__ __forceinline__ int v_place(int key, int ch) {
  return key * D + ((D == 64 ? ch ^ (key & 2) : ch ^ (key & 6)) << 4);
}

template <int D>
struct Smem {
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kJoin = kWarps * kRows * D * 4;   // reuses the ring
  static constexpr int kBody = kRing > kJoin ? kRing : kJoin;
  static constexpr int kQ = D == 256 ? kRows * D * 2 : 0;
  static constexpr int kBytes = kBody + kQ;
};

template <int D>
__global__ void __launch_bounds__(kThreads, D == 256 ? 2 : 3)
    kv_attention_kernel(const __grid_constant__ KvAttentionArgs a, int64_t part_stride) {
  constexpr int U = kUnits<D>;
  constexpr int kSteps16 = D / 16;       // k16 steps of S
  constexpr int kTiles = D / 8;          // n8 tiles of O
  constexpr bool kQSmem = D == 256;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_scan[kThreads];
  __shared__ int s_warp[kWarps];
  __shared__ float s_scale[kWarps][kStages][U][2];
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  pdl_trigger();
  pdl_wait();
  const KvPages& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lr = lane >> 2, lc = lane & 3;
  uint8_t* ring = smem + warp * kStages * kStageBytes;
  const uint32_t ring_u = smem_u32(ring);

  int s0 = -kThreads;                      // first sequence of the window in s_scan
  int64_t win_base = 0;                    // items before the window
  int win_items = 0;
  for (int64_t item = blockIdx.x;; item += gridDim.x) {
    // ---- the item's sequence: inclusive scan of the item counts, 128 sequences at a time
    while (item >= win_base + win_items) {
      win_base += win_items;
      s0 += kThreads;
      if (s0 >= c.S) return;
      SeqPlan p;
      int n = s0 + tid < c.S ? seq_items(a, s0 + tid, p) : 0;
      if (blockIdx.x == 0 && s0 + tid < c.S && (n < 0 || (p.bad && n > 0)) && a.err != nullptr)
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
      for (int w = 0; w < warp; ++w) n += s_warp[w];
      s_scan[tid] = n;
      __syncthreads();
      win_items = s_scan[kThreads - 1];
    }
    const int local = static_cast<int>(item - win_base);
    int at = 0;
#pragma unroll
    for (int o = kThreads / 2; o > 0; o >>= 1)
      if (s_scan[at + o - 1] <= local) at += o;
    const int s = s0 + at;
    SeqPlan p;
    seq_items(a, s, p);
    int rest = local - (at > 0 ? s_scan[at - 1] : 0);
    const int tile = rest % p.tiles;
    rest /= p.tiles;
    const int split = rest % p.splits, hk = rest / p.splits;

    // ---- rows of this lane, and the keys they see
    const int row0 = tile * kRows;
    int32_t r_lo[2], r_hi[2];
    const uint16_t* qp[2];
    int32_t t_lo = INT32_MAX, t_hi = 0;   // what any row of the tile sees
    const int32_t first_pos = static_cast<int32_t>(p.sp.len) - p.sp.n;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = row0 + lr + 8 * i;
      const int tok = r / a.G, g = r - tok * a.G;
      r_lo[i] = r_hi[i] = 0;
      qp[i] = nullptr;
      if (r < p.rows && !p.bad) {
        const int32_t pos = first_pos + tok;
        r_hi[i] = a.causal ? max(0, pos + 1) : static_cast<int32_t>(p.sp.len);
        r_lo[i] = a.window > 0 && pos + 1 > a.window ? static_cast<int32_t>(pos + 1 - a.window) : 0;
        qp[i] = a.q + static_cast<int64_t>(p.sp.b + tok) * a.ldq_t + static_cast<int64_t>(hk * a.G + g) * a.ldq_h;
        t_hi = max(t_hi, r_hi[i]);
        if (r_hi[i] > r_lo[i]) t_lo = min(t_lo, r_lo[i]);
      }
    }
    t_hi = __reduce_max_sync(0xffffffffu, t_hi);
    t_lo = __reduce_min_sync(0xffffffffu, t_lo);
    // every row sees [a_lo, a_hi): steps inside need no mask
    const int32_t a_hi = __reduce_min_sync(0xffffffffu, min(qp[0] ? r_hi[0] : INT32_MAX, qp[1] ? r_hi[1] : INT32_MAX));
    const int32_t a_lo = __reduce_max_sync(0xffffffffu, max(r_lo[0], r_lo[1]));
    const int32_t k_begin = max(p.lo + split * p.chunk, min(t_lo, t_hi) & ~63);
    const int64_t piece_end = static_cast<int64_t>(p.lo) + static_cast<int64_t>(split + 1) * p.chunk;
    const int32_t k_end = static_cast<int32_t>(min(static_cast<int64_t>(t_hi), piece_end));
    const int steps = k_end > k_begin ? (k_end - k_begin + kStepKeys<D> - 1) / kStepKeys<D> : 0;
    const int my_steps = (steps - warp + kWarps - 1) / kWarps;   // steps warp, warp + 4, ...

    // ---- page ids of the next 32 units of this warp, one a lane
    const int32_t* table = c.table + s * c.ld_table;
    int32_t page_l = 0;
    bool bad_page = false;
    auto load_pages = [&](int st) {      // units of steps st, st + 1, ... of this warp
      const int u = lane % U, j = st + lane / U;
      const int32_t key = k_begin + (warp + kWarps * j) * kStepKeys<D> + u * 16;
      page_l = 0;
      if (j < my_steps && key < k_end) {
        page_l = table[key >> c.block_shift];
        if (page_l < 0 || page_l >= c.num_pages) {
          bad_page = true;
          page_l = 0;
        }
      }
    };
    auto issue = [&](int st) {           // copy step st of this warp into its ring
      if (st < my_steps) {
        if (st % (32 / U) == 0) load_pages(st);
        const int stage = st % kStages;
        const uint32_t dst = ring_u + stage * kStageBytes;
        const int32_t key0 = k_begin + (warp + kWarps * st) * kStepKeys<D>;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int32_t page = __shfl_sync(0xffffffffu, page_l, (st % (32 / U)) * U + u);
          const int32_t key = key0 + u * 16;
          const int bytes = key < k_end ? 16 : 0;   // units past the end: zeros
          const int64_t ph = static_cast<int64_t>(page) * c.H + hk;
          const int64_t off = (ph * c.block + (key & (c.block - 1))) * D + lane * 16;
          const int8_t* ks = c.k_codes + off;
          const int8_t* vs = c.v_codes + off;
          constexpr int kCh = D / 16;    // 16-byte pieces of a key
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const int idx = i * 32 + lane, kk = idx / kCh, ch = idx % kCh;
            cp_async_16(dst + u * 16 * D + k_place<D>(kk, ch), ks + i * 512, bytes);
            cp_async_16(dst + kStageBytes / 2 + u * 16 * D + v_place<D>(kk, ch), vs + i * 512, bytes);
          }
          if (lane < 2)
            cp_async_4(smem_u32(&s_scale[warp][stage][u][lane]), (lane == 0 ? c.k_scale : c.v_scale) + ph, bytes / 4);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int st = 0; st < kStages - 1; ++st) issue(st);

    // ---- queries as binary16 fragments: lane (r, c) holds channels 64 i + 16 c .. + 15 of rows r, r + 8
    uint32_t qf[kQSmem ? 1 : kSteps16][4];
    float q_unit[2];
    uint4* sq = reinterpret_cast<uint4*>(smem + Smem<D>::kBody);
    {
      uint4 raw[2][D / 32];
      float amax[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          raw[i][j] = qp[i] != nullptr ? *reinterpret_cast<const uint4*>(qp[i] + (j >> 1) * 64 + lc * 16 + (j & 1) * 8)
                                       : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t w[4] = {raw[i][j].x, raw[i][j].y, raw[i][j].z, raw[i][j].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) amax[i] = fmaxf(amax[i], fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
        }
        amax[i] = fmaxf(amax[i], __shfl_xor_sync(0xffffffffu, amax[i], 1));
        amax[i] = fmaxf(amax[i], __shfl_xor_sync(0xffffffffu, amax[i], 2));
      }
      float f[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int e = static_cast<int>(__float_as_uint(amax[i]) >> 23);   // biased exponent of the row's maximum
        const int fe = e == 255 || e == 0 ? 127 : min(253, 127 + 13 + 127 - e);
        f[i] = __uint_as_float(static_cast<uint32_t>(fe) << 23);
        q_unit[i] = __uint_as_float(static_cast<uint32_t>(254 - fe) << 23) * a.scale_log2;
      }
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        const uint32_t w0[4] = {raw[0][j].x, raw[0][j].y, raw[0][j].z, raw[0][j].w};
        const uint32_t w1[4] = {raw[1][j].x, raw[1][j].y, raw[1][j].z, raw[1][j].w};
#pragma unroll
        for (int e = 0; e < 2; ++e) {   // k16 step 2 j + e: four channels of the lane
          const uint32_t f0 = half2_bits(bf16_lo(w0[2 * e]) * f[0], bf16_hi(w0[2 * e]) * f[0]);
          const uint32_t f1 = half2_bits(bf16_lo(w1[2 * e]) * f[1], bf16_hi(w1[2 * e]) * f[1]);
          const uint32_t f2 = half2_bits(bf16_lo(w0[2 * e + 1]) * f[0], bf16_hi(w0[2 * e + 1]) * f[0]);
          const uint32_t f3 = half2_bits(bf16_lo(w1[2 * e + 1]) * f[1], bf16_hi(w1[2 * e + 1]) * f[1]);
          if constexpr (kQSmem) {
            if (warp == 0) sq[(2 * j + e) * 32 + lane] = make_uint4(f0, f1, f2, f3);
          } else {
            qf[2 * j + e][0] = f0, qf[2 * j + e][1] = f1, qf[2 * j + e][2] = f2, qf[2 * j + e][3] = f3;
          }
        }
      }
      if constexpr (kQSmem) __syncthreads();
    }

    float o[kTiles][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, v_ref = 0.0f;
#pragma unroll
    for (int i = 0; i < kTiles; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;

    for (int st = 0; st < my_steps; ++st) {
      issue(st + kStages - 1);
      cp_async_wait<kStages - 1>();
      __syncwarp();
      const int stage = st % kStages;
      const uint8_t* kb = ring + stage * kStageBytes;
      const uint8_t* vb = kb + kStageBytes / 2;
      const int32_t key0 = k_begin + (warp + kWarps * st) * kStepKeys<D>;
      // ---- S: scores of 16 rows x step keys, in log2 units
      float x[2 * U][4];
      float vs[U], v_top = v_ref;
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int j = 0; j < 2; ++j) x[2 * u + j][0] = x[2 * u + j][1] = x[2 * u + j][2] = x[2 * u + j][3] = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          uint4 kw[2];
#pragma unroll
          for (int j = 0; j < 2; ++j)
            kw[j] = *reinterpret_cast<const uint4*>(kb + u * 16 * D + k_place<D>(j * 8 + lr, 4 * i + lc));
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint4 qv;
            if constexpr (kQSmem) {
              qv = sq[(4 * i + w) * 32 + lane];
            } else {
              qv = make_uint4(qf[4 * i + w][0], qf[4 * i + w][1], qf[4 * i + w][2], qf[4 * i + w][3]);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t b = (w == 0 ? kw[j].x : w == 1 ? kw[j].y : w == 2 ? kw[j].z : kw[j].w) ^ 0x80808080u;
              mma_f16_16816(x[2 * u + j], qv.x, qv.y, qv.z, qv.w, widen(b, 0x4140u), widen(b, 0x4342u));
            }
          }
        }
        const float ks = s_scale[warp][stage][u][0];
        vs[u] = s_scale[warp][stage][u][1];
        v_top = fmaxf(v_top, vs[u]);
        const float f0 = ks * q_unit[0], f1 = ks * q_unit[1];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          x[2 * u + j][0] *= f0;
          x[2 * u + j][1] *= f0;
          x[2 * u + j][2] *= f1;
          x[2 * u + j][3] *= f1;
        }
      }
      if (key0 < a_lo || key0 + kStepKeys<D> > a_hi) {   // the step's edge: keys a row does not see
#pragma unroll
        for (int j = 0; j < 2 * U; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int32_t key = key0 + j * 8 + lc * 2 + (e & 1);
            if (key < r_lo[e >> 1] || key >= r_hi[e >> 1]) x[j][e] = -INFINITY;
          }
      }
      // ---- running maximum; the output is rescaled when it (or the value scale) grows
      float al[2], base[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float t = x[0][2 * i];
#pragma unroll
        for (int j = 0; j < 2 * U; ++j) t = fmaxf(t, fmaxf(x[j][2 * i], x[j][2 * i + 1]));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
        const float mn = fmaxf(m[i], t);
        base[i] = mn == -INFINITY ? 0.0f : mn - kPShift;
        al[i] = m[i] == -INFINITY ? 0.0f : ex2(m[i] - mn);
        m[i] = mn;
        l[i] *= al[i];
      }
      const float v_inv = v_top >= 0x1p-126f ? __frcp_rn(v_top) : 0.0f;
      if (v_top != v_ref) {
        al[0] *= v_ref * v_inv;
        al[1] *= v_ref * v_inv;
        v_ref = v_top;
      }
      if (__any_sync(0xffffffffu, al[0] != 1.0f || al[1] != 1.0f)) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          o[i][0] *= al[0];
          o[i][1] *= al[0];
          o[i][2] *= al[1];
          o[i][3] *= al[1];
        }
      }
      // ---- P and O += P V, a unit at a time
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t pf[4];
        const float vr = vs[u] * v_inv;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float* xj = x[2 * u + j];
          const float p0 = ex2(xj[0] - base[0]), p1 = ex2(xj[1] - base[0]);
          const float p2 = ex2(xj[2] - base[1]), p3 = ex2(xj[3] - base[1]);
          l[0] += p0 + p1;
          l[1] += p2 + p3;
          pf[2 * j] = half2_bits(p0 * vr, p1 * vr);
          pf[2 * j + 1] = half2_bits(p2 * vr, p3 * vr);
        }
#pragma unroll
        for (int h = 0; h < (D + 127) / 128; ++h) {
          constexpr int W = D == 64 ? 2 : 4;   // words of a lane's piece
          uint32_t vw[4][W];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = 2 * lc + (e & 1) + 8 * (e >> 1);
            if constexpr (D == 64) {
              const uint2 t = *reinterpret_cast<const uint2*>(vb + u * 16 * D + v_place<D>(key, lr >> 1) + (lr & 1) * 8);
              vw[e][0] = t.x, vw[e][1] = t.y;
            } else {
              const uint4 t = *reinterpret_cast<const uint4*>(vb + u * 16 * D + v_place<D>(key, lr + 8 * h));
              vw[e][0] = t.x, vw[e][1] = t.y, vw[e][2] = t.z, vw[e][3] = t.w;
            }
          }
#pragma unroll
          for (int w = 0; w < W; ++w) {
            const uint32_t a0 = __byte_perm(vw[0][w], vw[1][w], 0x5140u) ^ 0x80808080u;
            const uint32_t a1 = __byte_perm(vw[0][w], vw[1][w], 0x7362u) ^ 0x80808080u;
            const uint32_t b0 = __byte_perm(vw[2][w], vw[3][w], 0x5140u) ^ 0x80808080u;
            const uint32_t b1 = __byte_perm(vw[2][w], vw[3][w], 0x7362u) ^ 0x80808080u;
            float(*ot)[4] = o + h * 16 + 4 * w;
            mma_f16_16816(ot[0], pf[0], pf[1], pf[2], pf[3], widen(a0, 0x4140u), widen(b0, 0x4140u));
            mma_f16_16816(ot[1], pf[0], pf[1], pf[2], pf[3], widen(a0, 0x4342u), widen(b0, 0x4342u));
            mma_f16_16816(ot[2], pf[0], pf[1], pf[2], pf[3], widen(a1, 0x4140u), widen(b1, 0x4140u));
            mma_f16_16816(ot[3], pf[0], pf[1], pf[2], pf[3], widen(a1, 0x4342u), widen(b1, 0x4342u));
          }
        }
      }
      __syncwarp();   // the stage is free for the copy that the next turn issues
    }

    // ---- join the four warps
    cp_async_wait<0>();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    }
    const bool bad = __syncthreads_or(bad_page) || p.bad;   // and every warp is done with the ring
    float* so = reinterpret_cast<float*>(smem) + warp * kRows * D;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = lr + 8 * i;
      if (lc == 0) s_m[warp][r] = m[i], s_l[warp][r] = l[i];
      constexpr int kPiece = D == 64 ? 8 : 16;   // consecutive channels of an output column
#pragma unroll
      for (int h = 0; h < (D + 127) / 128; ++h)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int t = 0; t < kPiece; t += 4) {
            float(*ot)[4] = o + h * 16 + t;
            *reinterpret_cast<float4*>(so + r * D + h * 128 + (2 * lc + n) * kPiece + t) =
                make_float4(ot[0][2 * i + n] * v_ref, ot[1][2 * i + n] * v_ref, ot[2][2 * i + n] * v_ref,
                            ot[3][2 * i + n] * v_ref);
          }
    }
    __syncthreads();
    if (bad && tid == 0 && !p.bad && a.err != nullptr) atomicOr(a.err, PRISM_DEV_ERR_PAGE_RANGE);
    const float nanf = __uint_as_float(0x7fc00000u);
    float* part = static_cast<float*>(a.ws);
    for (int i = tid; i < kRows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d = (i % (D / 4)) * 4;
      if (row0 + r >= p.rows) break;
      float mx = s_m[0][r];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][r]);
      float sum = 0.0f;
      float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = s_m[w][r] == -INFINITY ? 0.0f : ex2(s_m[w][r] - mx);
        const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<float*>(smem) + (w * kRows + r) * D + d);
        sum = fmaf(f, s_l[w][r], sum);
        y.x = fmaf(f, v.x, y.x);
        y.y = fmaf(f, v.y, y.y);
        y.z = fmaf(f, v.z, y.z);
        y.w = fmaf(f, v.w, y.w);
      }
      const int tok = (row0 + r) / a.G, h = hk * a.G + (row0 + r) % a.G;
      if (p.splits == 1) {
        const float inv = mx == -INFINITY ? 0.0f : 1.0f / sum;
        uint2 w = make_uint2(float_to_bf16_rne(y.x * inv) | float_to_bf16_rne(y.y * inv) << 16,
                             float_to_bf16_rne(y.z * inv) | float_to_bf16_rne(y.w * inv) << 16);
        if (bad) w = make_uint2(kBf16NaN * 0x10001u, kBf16NaN * 0x10001u);
        const int64_t t = p.sp.b + tok;
        *reinterpret_cast<uint2*>(a.out + t * a.ldo_t + h * a.ldo_h + d) = w;
        if (d == 0 && a.lse != nullptr)
          a.lse[t * a.Hq + h] = bad ? nanf : mx == -INFINITY ? mx : (mx - kPShift + log2f(sum)) * kLn2;
      } else {
        const int64_t slot = (static_cast<int64_t>(s) * c.H + hk) * part_stride + split * p.rows + row0 + r;
        float* ps = part + slot * (D + 4);
        *reinterpret_cast<float4*>(ps + 4 + d) = y;
        if (d == 0) ps[0] = bad ? nanf : mx, ps[1] = sum;
      }
    }
    __syncthreads();   // s_m, s_l, the ring and s_scan are free again
  }
}

// Joins a row's pieces in piece order: one CTA per (sequence, KV head, row),
// warp w takes every fourth piece.
template <int D>
__global__ void __launch_bounds__(kThreads)
    kv_combine_kernel(const __grid_constant__ KvAttentionArgs a, int64_t part_stride) {
  constexpr int E = D / 32;
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hk = blockIdx.y, r = blockIdx.z;
  const int s = blockIdx.x;
  SeqPlan p;
  if (seq_items(a, s, p) <= 0 || p.splits == 1 || r >= p.rows) return;
  const float* part = static_cast<const float*>(a.ws) +
                      ((static_cast<int64_t>(s) * a.c.H + hk) * part_stride + r) * (D + 4);
  const int64_t step = static_cast<int64_t>(p.rows) * (D + 4);
  float m = -INFINITY, l = 0.0f, o[E];
  bool nan = false;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.0f;
#pragma unroll 4
  for (int i = warp; i < p.splits; i += kWarps) {
    const float* ps = part + i * step;
    const float pm = ps[0], pl = ps[1];
    float v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = ps[4 + e * 32 + lane];
    nan |= pm != pm;
    if (pm > -INFINITY) {
      const float mn = fmaxf(m, pm), f0 = m == -INFINITY ? 0.0f : ex2(m - mn), f1 = ex2(pm - mn);
      l = fmaf(l, f0, pl * f1);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], f0, v[e] * f1);
      m = mn;
    }
  }
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][e * 32 + lane] = o[e];
  nan = __syncthreads_or(nan);
  float mx = s_m[0], sum = 0.0f, f[kWarps];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, s_m[w]);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    f[w] = s_m[w] == -INFINITY ? 0.0f : ex2(s_m[w] - mx);
    sum = fmaf(f[w], s_l[w], sum);
  }
  const float nanf = __uint_as_float(0x7fc00000u), inv = mx == -INFINITY ? 0.0f : 1.0f / sum;
  const int64_t t = p.sp.b + r / a.G;
  const int h = hk * a.G + r % a.G;
  for (int d = tid; d < D; d += kThreads) {
    float y = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) y = fmaf(f[w], s_o[w][d], y);
    a.out[t * a.ldo_t + h * a.ldo_h + d] = static_cast<uint16_t>(nan ? kBf16NaN : float_to_bf16_rne(y * inv));
  }
  if (tid == 0 && a.lse != nullptr)
    a.lse[t * a.Hq + h] = nan ? nanf : mx == -INFINITY ? mx : (mx - kPShift + log2f(sum)) * kLn2;
}

template <int D>
cudaError_t launch_d(const KvAttentionArgs& a, cudaStream_t stream) {
  const int64_t max_keys = a.c.max_pages << a.c.block_shift;
  const int64_t part_stride = max_split_rows(a.max_q, a.G, max_keys);
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kv_attention_kernel<D>), Smem<D>::kBytes);
  if (e != cudaSuccess) return e;
  // persistent: as many CTAs as the SMs hold, or as the call can have items
  const int64_t tiles = a.T * a.G / kRows + a.c.S;
  const int64_t items = std::max(tiles, static_cast<int64_t>(a.c.S) * split_count(max_keys, 1)) * a.c.H;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(items, sm_count() * (D == 256 ? 2 : 3)));
  e = launch_kernel(kv_attention_kernel<D>, dim3(grid), dim3(kThreads), Smem<D>::kBytes, stream, true, a, part_stride);
  if (e != cudaSuccess || part_stride == 0) return e;
  const int64_t rows = std::min<int64_t>(a.max_q * a.G, kMaxSplit / 2 * kRows);
  return launch_kernel(kv_combine_kernel<D>, dim3(a.c.S, a.c.H, static_cast<unsigned>(rows)), dim3(kThreads), 0, stream,
                       true, a, part_stride);
}

}  // namespace

size_t kv_attention_workspace_bytes(int64_t S, int64_t, int64_t max_q, int64_t max_pages, int64_t Hq, int64_t Hkv,
                                    int64_t D, int64_t block) {
  return static_cast<size_t>(S * Hkv * max_split_rows(max_q, Hq / Hkv, max_pages * block)) * (D + 4) * 4;
}

cudaError_t launch_kv_attention(const KvAttentionArgs& a, cudaStream_t stream) {
  return a.c.D == 64 ? launch_d<64>(a, stream) : a.c.D == 128 ? launch_d<128>(a, stream) : launch_d<256>(a, stream);
}

}  // namespace prism
