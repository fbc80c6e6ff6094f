// kv_attention.cu -- attention of new queries over the paged int8 K/V cache:
//   o = sum_j softmax_j(sm_scale * ks * (q . ck_j)) * vs * cv_j
// with codes ck, cv and one scale ks, vs per (page, head).
//
// This file: the kernel for up to kv::kFewRows rows of a sequence and KV head
// (kv_plan.cuh), 8 NQ rows a tile, and the join of pieces.  A persistent grid
// walks the items (sequence, KV head, piece, tile).
//
// One item is one CTA of four warps; warp w takes every fourth step of 8 KB of
// K and V.  Each warp is on its own: its steps arrive through a private ring
// of cp.async copies, it keeps its own running maximum, sum and output, and
// the four are joined in shared memory at the end -- no barrier in the loop.
//   S^T = K Q^T and O^T += V^T P^T run on mma.sync m16n8k16 with binary16
// operands and binary32 sums: 16 keys (channels) by 8 rows, so that the one to
// eight rows of a decode step fill the instruction, and P^T's operand is S^T's
// result transposed by movmatrix.  The order of channels inside S's
// contraction and of the output's rows is free, so lane (r, c) of a warp reads
// its operands as 16-byte pieces: channels 16c.. of keys r, r + 8 for K;
// channels 16r.. of keys 2c, 2c+1, 2c+8, 2c+9 for V, whose two-key pairs a
// byte permute forms.
//   Codes widen exactly.  K: byte ^ 0x80 as a binary16 subnormal, (code + 128)
// 2^-24, and the sums start at -128 * 2^-24 * sum q.  V: the same byte under
// the exponent of 1024, minus 1152 (a start value would cancel badly there:
// the weights are all positive).  Queries become binary16 after an exact
// power-of-two scale that puts the row's largest channel at 2^13 (channels
// 2^27 below it lose bits: under 2^-38 of the row's maximum).  Probabilities
// are rounded to binary16 (half a step is 2^-11) with 2^12 as the value of the
// running maximum, so that keys down to 2^-26 of it stay normal numbers; a
// page's vs enters as its ratio to the largest vs seen so far.  Maxima, sums
// and outputs are binary32.
//
// It reads the codes once: 64 sequences of 300 to 4096 tokens (289 MB, 40 heads
// on 8 of 128) take 61 us, 4.7 TB/s; a single one of 131071 tokens (32 heads on 4
// of 256) 59 us, 4.6 TB/s.  No unit is full then: HBM at 64 %, the ALU pipe
// (widening, byte permutes) and the issue slots at half their rate, and the copies
// under way (8 KB a warp, 12 warps an SM) are enough for more.  Within a warp a
// step is a chain -- scores, their maximum over lanes, exponentials, transposition,
// second product -- with two other warps of the scheduler beside it (three CTAs an
// SM, by registers).
#include <cuda_fp16.h>

#include "kv_plan.cuh"

namespace prism {
namespace {

using namespace kv;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kJoinThreads = 256;
constexpr int kStages = 2;
constexpr int kStageBytes = 8192;      // K and V of one step of a warp

template <int D>
constexpr int kUnits = kStageBytes / (2 * 16 * D);   // 16-key units of a step: 4, 2, 1 for D = 64, 128, 256
template <int D>
constexpr int kStepKeys = 16 * kUnits<D>;

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
// The 8x8 matrix of binary16 whose row r lies in lanes 4r .. 4r + 3, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// Shared-memory place of 16-byte piece `ch` of key `key` in a step's K (V):
// pieces of neighbouring keys are turned so that the eight lanes of a phase
// (keys r, r + 1 for K; keys 0, 2, 4, 6 for V) touch all banks once (D = 64:
// at most twice).
template <int D>
__device__ __forceinline__ int k_place(int key, int ch) {
  return key * D + ((D == 64 ? ch : ch ^ ((key & 1) << 2)) << 4);
}
template <int D>
__device__ __forceinline__ int v_place(int key, int ch) {
  return key * D + ((D == 64 ? ch ^ (key & 2) : ch ^ (key & 6)) << 4);
}

template <int D, int NQ>
struct Smem {
  static constexpr bool kQ = NQ > 1;          // the queries' fragments lie in shared memory
  static constexpr int kRows = 8 * NQ;
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kJoin = kWarps * kRows * D * 4;   // reuses the ring
  static constexpr int kBody = kRing > kJoin ? kRing : kJoin;
  static constexpr int kBytes = kBody + (kQ ? kRows * D * 2 : 0);
  // CTAs an SM holds, by registers and shared memory
  static constexpr int kCtas = D * NQ <= 256 && NQ < 4 ? 3 : 2;
};

template <int D, int NQ>
__global__ void __launch_bounds__(kThreads, Smem<D, NQ>::kCtas)
    kv_attention_kernel(const __grid_constant__ KvAttentionArgs a, const __grid_constant__ Parts parts) {
  constexpr int U = kUnits<D>;
  constexpr int kSteps16 = D / 16;       // k16 steps of S^T, m16 tiles of O^T
  constexpr bool kQSmem = Smem<D, NQ>::kQ;
  constexpr int kRows = 8 * NQ;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_scan[kThreads];
  __shared__ int s_warp[kWarps];
  __shared__ float s_scale[kWarps][kStages][U][2];
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ float2 s_q[kRows];          // unit and start value of a row's scores
  pdl_wait();
  const KvPages& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lr = lane >> 2, lc = lane & 3;
  uint8_t* ring = smem + warp * kStages * kStageBytes;
  const uint32_t ring_u = smem_u32(ring);

  Walk walk = new_walk();
  SeqPlan p;
  for (int64_t item = blockIdx.x; find_item<false, kRows, kThreads>(a, item, walk, s_scan, s_warp, p); item += gridDim.x) {
    const int s = walk.s, hk = walk.hk, split = walk.split;
    const TileKeys keys(a, p, walk, kRows);
    const int row0 = keys.row0, n_rows = keys.n_rows;
    const int32_t k_begin = keys.k_begin, k_first = keys.k_first, k_end = keys.k_end;
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
      if (j < my_steps && key >= k_first && key < k_end) {
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
          const int bytes = key >= k_first && key < k_end ? 16 : 0;   // units that no row sees: zeros
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

    // ---- queries as binary16 fragments: lane (r, c) holds channels 64 i + 16 c .. + 15 of row r
    uint2 qf[kQSmem ? 1 : kSteps16];
    float q_unit[NQ][2], q_start[NQ][2];
    uint2* sq = reinterpret_cast<uint2*>(smem + Smem<D, NQ>::kBody);   // [step][NQ][lane]
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
      if (kQSmem && (t & (kWarps - 1)) != warp) continue;   // fragments in shared memory: a tile of rows each
      const int r = 8 * t + lr;
      const uint16_t* qp = nullptr;
      if (r < n_rows) {
        const int tok = (row0 + r) / a.G, g = (row0 + r) - tok * a.G;
        qp = a.q + static_cast<int64_t>(p.sp.b + tok) * a.ldq_t + static_cast<int64_t>(hk * a.G + g) * a.ldq_h;
      }
      uint4 raw[D / 32];
      float amax = 0.0f;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        raw[j] = qp != nullptr ? *reinterpret_cast<const uint4*>(qp + (j >> 1) * 64 + lc * 16 + (j & 1) * 8)
                               : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int fe = query_exponent(amax);
      const float f = __uint_as_float(static_cast<uint32_t>(fe) << 23);
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
        for (int e = 0; e < 2; ++e) {   // k16 step 2 j + e: four channels of the lane
          const uint2 b = make_uint2(half2_bits(bf16_lo(w[2 * e]) * f, bf16_hi(w[2 * e]) * f),
                                     half2_bits(bf16_lo(w[2 * e + 1]) * f, bf16_hi(w[2 * e + 1]) * f));
          const float2 v0 = __half22float2(*reinterpret_cast<const __half2*>(&b.x));
          const float2 v1 = __half22float2(*reinterpret_cast<const __half2*>(&b.y));
          sum += (v0.x + v0.y) + (v1.x + v1.y);
          if constexpr (kQSmem) {
            sq[((2 * j + e) * NQ + t) * 32 + lane] = b;
          } else {
            qf[2 * j + e] = b;
          }
        }
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const float unit = __uint_as_float(static_cast<uint32_t>(254 - fe) << 23) * a.scale_log2;
      const float start = sum * -0x1p-17f;   // -128 * 2^-24
      if constexpr (kQSmem) {
        if (lc == 0) s_q[r] = make_float2(unit, start);
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          q_unit[t][i] = __shfl_sync(0xffffffffu, unit, (2 * lc + i) * 4);
          q_start[t][i] = __shfl_sync(0xffffffffu, start, (2 * lc + i) * 4);
        }
      }
    }
    if constexpr (kQSmem) {
      __syncthreads();
#pragma unroll
      for (int t = 0; t < NQ; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 v = s_q[8 * t + 2 * lc + i];
          q_unit[t][i] = v.x;
          q_start[t][i] = v.y;
        }
    }

    // lane (r, c) holds rows (queries) 2c, 2c + 1 of each tile of eight
    float o[kSteps16][NQ][4], m[NQ][2], l[NQ][2], v_ref = 0.0f;
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < kSteps16; ++i) o[i][t][0] = o[i][t][1] = o[i][t][2] = o[i][t][3] = 0.0f;
    }

    for (int st = 0; st < my_steps; ++st) {
      issue(st + kStages - 1);
      cp_async_wait<kStages - 1>();
      __syncwarp();
      const int stage = st % kStages;
      const uint8_t* kb = ring + stage * kStageBytes;
      const uint8_t* vb = kb + kStageBytes / 2;
      const int32_t key0 = k_begin + (warp + kWarps * st) * kStepKeys<D>;
      // ---- S^T: scores of the step's keys (rows r, r + 8 of a unit) and 8 NQ rows, in log2 units
      float x[U][NQ][4];
      float vs[U], v_top = v_ref;
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int t = 0; t < NQ; ++t) {
          x[u][t][0] = x[u][t][2] = q_start[t][0];
          x[u][t][1] = x[u][t][3] = q_start[t][1];
        }
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          uint4 kw[2];
#pragma unroll
          for (int j = 0; j < 2; ++j)
            kw[j] = *reinterpret_cast<const uint4*>(kb + u * 16 * D + k_place<D>(j * 8 + lr, 4 * i + lc));
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t k0 = (w == 0 ? kw[0].x : w == 1 ? kw[0].y : w == 2 ? kw[0].z : kw[0].w) ^ 0x80808080u;
            const uint32_t k1 = (w == 0 ? kw[1].x : w == 1 ? kw[1].y : w == 2 ? kw[1].z : kw[1].w) ^ 0x80808080u;
            const uint32_t a0 = __byte_perm(k0, 0u, 0x4140u), a2 = __byte_perm(k0, 0u, 0x4342u);
            const uint32_t a1 = __byte_perm(k1, 0u, 0x4140u), a3 = __byte_perm(k1, 0u, 0x4342u);
#pragma unroll
            for (int t = 0; t < NQ; ++t) {
              uint2 b;
              if constexpr (kQSmem) {
                b = sq[((4 * i + w) * NQ + t) * 32 + lane];
              } else {
                b = qf[4 * i + w];
              }
              mma_f16_16816(x[u][t], a0, a1, a2, a3, b.x, b.y);
            }
          }
        }
        const float ks = s_scale[warp][stage][u][0] * 0x1p24f;   // of code * 2^-24; beside q_unit it could leave binary32's range
        vs[u] = s_scale[warp][stage][u][1];
        v_top = fmaxf(v_top, vs[u]);
#pragma unroll
        for (int t = 0; t < NQ; ++t) {
          const float f0 = ks * q_unit[t][0], f1 = ks * q_unit[t][1];
          x[u][t][0] *= f0;
          x[u][t][1] *= f1;
          x[u][t][2] *= f0;
          x[u][t][3] *= f1;
        }
      }
      if (key0 < keys.a_lo || key0 + kStepKeys<D> > keys.a_hi) {   // keys that a row does not see
#pragma unroll
        for (int t = 0; t < NQ; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int32_t hi = keys.hi(8 * t + 2 * lc + i), lo = keys.lo(hi);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int32_t key = key0 + u * 16 + j * 8 + lr;
                if (key < lo || key >= hi) x[u][t][2 * j + i] = -INFINITY;
              }
          }
      }
      // ---- running maximum; the output is rescaled when it (or the value scale) grows
      const float v_inv = v_top >= 0x1p-126f ? __frcp_rn(v_top) : 0.0f;
      const float v_al = v_top != v_ref ? v_ref * v_inv : 1.0f;
      v_ref = v_top;
      float base[NQ][2];
#pragma unroll
      for (int t = 0; t < NQ; ++t) {
        float al[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float top = x[0][t][i];
#pragma unroll
          for (int u = 0; u < U; ++u) top = fmaxf(top, fmaxf(x[u][t][i], x[u][t][2 + i]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          const float mn = fmaxf(m[t][i], top);
          base[t][i] = mn == -INFINITY ? 0.0f : mn - kPShift;
          al[i] = m[t][i] == mn ? 1.0f : ex2(m[t][i] - mn);   // m = -inf: nothing to keep
          m[t][i] = mn;
          l[t][i] *= al[i];
          al[i] *= v_al;
        }
        if (__any_sync(0xffffffffu, al[0] != 1.0f || al[1] != 1.0f)) {
#pragma unroll
          for (int i = 0; i < kSteps16; ++i) {
            o[i][t][0] *= al[0];
            o[i][t][1] *= al[1];
            o[i][t][2] *= al[0];
            o[i][t][3] *= al[1];
          }
        }
      }
      // ---- P^T and O^T += V^T P^T, a unit at a time
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t pf[NQ][2];
        const float vr = vs[u] * v_inv;
#pragma unroll
        for (int t = 0; t < NQ; ++t)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float p0 = ex2(x[u][t][2 * j] - base[t][0]), p1 = ex2(x[u][t][2 * j + 1] - base[t][1]);
            l[t][0] += p0;
            l[t][1] += p1;
            pf[t][j] = transpose8(half2_bits(p0 * vr, p1 * vr));
          }
#pragma unroll
        for (int h = 0; h < (D + 127) / 128; ++h) {
          constexpr int W = D == 64 ? 2 : 4;   // words of a lane's piece
          uint32_t vw[4][W];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = 2 * lc + (e & 1) + 8 * (e >> 1);
            if constexpr (D == 64) {
              const uint2 v = *reinterpret_cast<const uint2*>(vb + u * 16 * D + v_place<D>(key, lr >> 1) + (lr & 1) * 8);
              vw[e][0] = v.x, vw[e][1] = v.y;
            } else {
              const uint4 v = *reinterpret_cast<const uint4*>(vb + u * 16 * D + v_place<D>(key, lr + 8 * h));
              vw[e][0] = v.x, vw[e][1] = v.y, vw[e][2] = v.z, vw[e][3] = v.w;
            }
          }
#pragma unroll
          for (int w = 0; w < W; ++w)
#pragma unroll
            for (int j = 0; j < 2; ++j) {      // channels 4 w + 2 j, + 1 of the lane's piece
              const uint32_t sel = j == 0 ? 0x5140u : 0x7362u;
              const uint32_t lo = __byte_perm(vw[0][w], vw[1][w], sel) ^ 0x80808080u;
              const uint32_t hi = __byte_perm(vw[2][w], vw[3][w], sel) ^ 0x80808080u;
              const uint32_t a0 = widen(lo, 0x4140u), a1 = widen(lo, 0x4342u);
              const uint32_t a2 = widen(hi, 0x4140u), a3 = widen(hi, 0x4342u);
#pragma unroll
              for (int t = 0; t < NQ; ++t) mma_f16_16816(o[h * 8 + 2 * w + j][t], a0, a1, a2, a3, pf[t][0], pf[t][1]);
            }
        }
      }
      __syncwarp();   // the stage is free for the copy that the next turn issues
    }

    // ---- join the four warps
    cp_async_wait<0>();
#pragma unroll
    for (int t = 0; t < NQ; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], 4);
        l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], 8);
        l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], 16);
      }
    const bool bad = __syncthreads_or(bad_page) || p.bad;   // and every warp is done with the ring
    float* so = reinterpret_cast<float*>(smem) + warp * kRows * D;
#pragma unroll
    for (int t = 0; t < NQ; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * t + 2 * lc + i;
        if (lr == 0) s_m[warp][r] = m[t][i], s_l[warp][r] = l[t][i];
        constexpr int kPiece = D == 64 ? 8 : 16;   // consecutive channels of a lane
#pragma unroll
        for (int h = 0; h < (D + 127) / 128; ++h)
#pragma unroll
          for (int e = 0; e < kPiece; e += 4) {
            const float* o0 = o[h * 8 + e / 2][t];
            const float* o1 = o[h * 8 + e / 2 + 1][t];
            if (r < n_rows)
              *reinterpret_cast<float4*>(so + r * D + h * 128 + lr * kPiece + e) =
                  make_float4(o0[i] * v_ref, o0[2 + i] * v_ref, o1[i] * v_ref, o1[2 + i] * v_ref);
          }
      }
    __syncthreads();
    if (bad && tid == 0 && !p.bad && a.err != nullptr) atomicOr(a.err, PRISM_DEV_ERR_PAGE_RANGE);
    const float nanf = __uint_as_float(0x7fc00000u);
    float* part = static_cast<float*>(a.ws);
    for (int i = tid; i < n_rows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d = (i % (D / 4)) * 4;
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
      const int tok = (row0 + r) / a.G, h = hk * a.G + (row0 + r) - tok * a.G;
      if (p.splits == 1) {
        const float inv = mx == -INFINITY ? 0.0f : 1.0f / sum;
        uint2 w = make_uint2(float_to_bf16_rne(y.x * inv) | float_to_bf16_rne(y.y * inv) << 16,
                             float_to_bf16_rne(y.z * inv) | float_to_bf16_rne(y.w * inv) << 16);
        if (bad) w = make_uint2(kBf16NaN * 0x10001u, kBf16NaN * 0x10001u);
        const int64_t t = p.sp.b + tok;
        *reinterpret_cast<uint2*>(a.out + t * a.ldo_t + h * a.ldo_h + d) = w;
        if (d == 0 && a.lse != nullptr)
          a.lse[t * a.Hq + h] = bad ? nanf : mx == -INFINITY ? mx + sum : (mx - kPShift + log2f(sum)) * kLn2;   // no key: sum 0; only NaN scores: NaN
      } else {
        const int64_t at = first_part(parts, p, s, hk) + static_cast<int64_t>(split) * p.rows + row0 + r;
        float* ps = part + at * (D + 4);
        *reinterpret_cast<float4*>(ps + 4 + d) = y;
        if (d == 0) ps[0] = bad ? nanf : mx, ps[1] = sum;
      }
    }
    __syncthreads();   // s_m, s_l, s_q, the ring and s_scan are free again
  }
  pdl_trigger();       // not before: a join that waits takes the places of CTAs that work
}

// A joined row's output and lse: y and sum against the reference mx.
template <int E>
__device__ __forceinline__ void store_row(const KvAttentionArgs& a, const SeqPlan& p, int hk, int r, int d, const float* y,
                                          float sum, float mx, bool nan) {
  const float inv = mx == -INFINITY ? 0.0f : 1.0f / sum;
  const int64_t t = p.sp.b + r / a.G;
  const int h = hk * a.G + r % a.G;
  uint32_t w[E / 2];
#pragma unroll
  for (int e = 0; e < E / 2; ++e)
    w[e] = nan ? kBf16NaN * 0x10001u : float_to_bf16_rne(y[2 * e] * inv) | float_to_bf16_rne(y[2 * e + 1] * inv) << 16;
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + t * a.ldo_t + h * a.ldo_h + d);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) dst[e] = w[e];
  if (d == 0 && a.lse != nullptr)
    a.lse[t * a.Hq + h] = nan ? __uint_as_float(0x7fc00000u) : mx == -INFINITY ? mx + sum : (mx - kPShift + log2f(sum)) * kLn2;
}

// Joins the pieces of rows of one (sequence, KV head).  Many rows: a row a
// warp, tiles in eighths.  Few rows, up to kWarpPieces
// pieces: a row a warp, each lane D / 32 channels.  More: a row a CTA; thread i
// weighs piece i, then D / 4 columns of threads by 1024 / D groups add every
// group-th piece in order, and the groups are added in order.
constexpr int kWarpPieces = 16;

template <int D, bool kMany>   // kMany: a sequence may have many rows
__global__ void __launch_bounds__(kJoinThreads)
    kv_combine_kernel(const __grid_constant__ KvAttentionArgs a, const __grid_constant__ Parts parts) {
  constexpr int kCols = D / 4, kGroups = kJoinThreads / kCols, kJoinWarps = kJoinThreads / 32, E = D / 32;
  __shared__ float s_f[kJoinThreads], s_red[kJoinWarps], s_sum[kJoinWarps];
  __shared__ float4 s_o[kJoinThreads];
  static_assert(kMaxSplit <= kJoinThreads, "a thread for each piece");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int s = blockIdx.x, hk = blockIdx.y;
  // the plan is made while the previous kernel ends: its inputs are older
  SeqPlan p;
  if (seq_items<false, 1, kMany>(a, s, p) < 0 || p.bad || p.splits == 1) {
    pdl_wait();   // this kernel ends no earlier than the one before it
    return;
  }
  if (!kMany || p.rows <= kFewRows) pdl_wait();
  const float* base = static_cast<const float*>(a.ws) + first_part(parts, p, s, hk) * (D + 4);
  if constexpr (kMany) if (p.rows > kFewRows) {
    __shared__ int64_t s_line[kJoinThreads], s_warp64[kJoinWarps];
    lay_line<kJoinThreads>(a, p, s_line, s_warp64);
    pdl_wait();
    const Cuts cuts(s_line[kJoinThreads - 1], p.splits);
    const int tiles = (p.rows + kWideRows - 1) / kWideRows;
    for (int u = blockIdx.z; u < tiles * 8; u += gridDim.z) {
      const TileSpan t = tile_span<kJoinThreads>(a, p, s_line, u >> 3);
      const int first = cuts.range_of(t.x), last = cuts.range_of(t.x + t.blocks - 1);
      if (first == last) continue;   // in one piece: answered
      for (int i = (u & 7) * (kWideRows / 8) + warp; i < (u & 7) * (kWideRows / 8) + kWideRows / 8; i += kJoinWarps) {
        const int r = (u >> 3) * kWideRows + i;
        if (r >= p.rows) break;
        auto piece = [&](int range) { return base + (wide_part(p, range, u >> 3, range == first) + i) * (D + 4); };
        float mx = -INFINITY;
        bool nan = false;
        for (int range = first + lane; range <= last; range += 32) {
          const float m = piece(range)[0];
          nan |= m != m;
          mx = fmaxf(mx, m);
        }
        nan = __any_sync(0xffffffffu, nan);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        float sum = 0.0f, y[E];
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = 0.0f;
#pragma unroll 4
        for (int range = first; range <= last; ++range) {
          const float* v = piece(range);
          const float w = v[0] == -INFINITY ? 0.0f : ex2(v[0] - mx);
          sum = fmaf(w, v[1], sum);
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const float2 x = *reinterpret_cast<const float2*>(v + 4 + lane * E + e);
            y[e] = fmaf(w, x.x, y[e]);
            y[e + 1] = fmaf(w, x.y, y[e + 1]);
          }
        }
        store_row<E>(a, p, hk, r, lane * E, y, sum, mx, nan);
      }
    }
    return;
  }
  const int64_t step = static_cast<int64_t>(p.rows) * (D + 4);
  if (p.splits <= kWarpPieces) {
    for (int r = blockIdx.z * kJoinWarps + warp; r < p.rows; r += gridDim.z * kJoinWarps) {
      const float* part = base + static_cast<int64_t>(r) * (D + 4);
      float pm = -INFINITY, pl = 0.0f;
      if (lane < p.splits) pm = part[lane * step], pl = part[lane * step + 1];
      const bool nan = __any_sync(0xffffffffu, pm != pm);
      float mx = pm;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      mx = __shfl_sync(0xffffffffu, mx, 0);
      const float f = pm == -INFINITY ? 0.0f : ex2(pm - mx);
      float sum = 0.0f, y[E];
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = 0.0f;
#pragma unroll 4
      for (int i = 0; i < p.splits; ++i) {
        const float w = __shfl_sync(0xffffffffu, f, i);
        sum = fmaf(w, __shfl_sync(0xffffffffu, pl, i), sum);
        const float* v = part + i * step + 4 + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += E < 4 ? 2 : 4) {
          if constexpr (E < 4) {
            const float2 x = *reinterpret_cast<const float2*>(v + e);
            y[e] = fmaf(w, x.x, y[e]);
            y[e + 1] = fmaf(w, x.y, y[e + 1]);
          } else {
            const float4 x = *reinterpret_cast<const float4*>(v + e);
            y[e] = fmaf(w, x.x, y[e]);
            y[e + 1] = fmaf(w, x.y, y[e + 1]);
            y[e + 2] = fmaf(w, x.z, y[e + 2]);
            y[e + 3] = fmaf(w, x.w, y[e + 3]);
          }
        }
      }
      store_row<E>(a, p, hk, r, lane * E, y, sum, mx, nan);
    }
    return;
  }
  for (int r = blockIdx.z; r < p.rows; r += gridDim.z) {
    const float* part = base + static_cast<int64_t>(r) * (D + 4);
    float pm = -INFINITY, pl = 0.0f;
    if (tid < p.splits) pm = part[tid * step], pl = part[tid * step + 1];
    const bool nan = __syncthreads_or(pm != pm);
    float mx = pm;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane == 0) s_red[warp] = mx;
    __syncthreads();
    mx = s_red[0];
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) mx = fmaxf(mx, s_red[w]);
    const float f = pm == -INFINITY ? 0.0f : ex2(pm - mx);
    s_f[tid] = f;
    float l = f * pl;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) s_sum[warp] = l;
    __syncthreads();
    const int col = tid % kCols, group = tid / kCols;
    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (int i = group; i < p.splits; i += kGroups) {
      const float4 v = *reinterpret_cast<const float4*>(part + i * step + 4 + col * 4);
      const float w = s_f[i];
      y[0] = fmaf(w, v.x, y[0]);
      y[1] = fmaf(w, v.y, y[1]);
      y[2] = fmaf(w, v.z, y[2]);
      y[3] = fmaf(w, v.w, y[3]);
    }
    s_o[tid] = make_float4(y[0], y[1], y[2], y[3]);
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int g = 1; g < kGroups; ++g) {
        const float4 v = s_o[g * kCols + col];
        y[0] += v.x, y[1] += v.y, y[2] += v.z, y[3] += v.w;
      }
      float sum = s_sum[0];
#pragma unroll
      for (int w = 1; w < kJoinWarps; ++w) sum += s_sum[w];
      store_row<4>(a, p, hk, r, col * 4, y, sum, mx, nan);
    }
    __syncthreads();   // the weights and sums are free again
  }
}

template <int D, int NQ>
cudaError_t launch_few(const KvAttentionArgs& a, const Parts& parts, cudaStream_t stream) {
  using M = Smem<D, NQ>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kv_attention_kernel<D, NQ>), M::kBytes);
  if (e != cudaSuccess) return e;
  // Persistent: as many CTAs as the SMs hold, or as the call can have items.
  // Each of a call's kernels is launched as the CTAs of the one before it end
  // (calls in a row, one query on 271 keys: 10.3 us without, 7.9 so; 131071 keys:
  // 65 and 59); allowed from their start, a join takes the places of CTAs that
  // work (64 sequences: 85 us), and the next call's CTAs those of a join (64
  // sequences of 500 to 3000 keys: 58.2 us, 53.2 so).
  const int64_t tiles = std::min<int64_t>(a.T * a.G, static_cast<int64_t>(a.c.S) * kFewRows) / M::kRows + a.c.S;
  const int64_t items = (tiles + (parts.few / M::kRows + kMaxSplit) * a.c.S) * a.c.H;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(items, sm_count() * M::kCtas));
  return launch_kernel(kv_attention_kernel<D, NQ>, dim3(grid), dim3(kThreads), M::kBytes, stream, true, a, parts);
}

// Rows of a tile: as many as a sequence of this kernel can have in this call
// (16 at most for D = 256, by the registers of the output).  A row's bits do
// not depend on the choice.
template <int D>
cudaError_t launch_d(const KvAttentionArgs& a, cudaStream_t stream) {
  const int64_t rows = a.max_q * a.G;
  const Parts parts = parts_of(a.c.S, a.T, a.max_q, a.G, a.c.max_pages << a.c.block_shift, a.c.H, D);
  cudaError_t e = rows <= 8                 ? launch_few<D, 1>(a, parts, stream)
                  : rows <= 16 || D == 256  ? launch_few<D, 2>(a, parts, stream)
                                            : launch_few<D, D == 256 ? 2 : 4>(a, parts, stream);
  if (e == cudaSuccess && rows > kFewRows) e = launch_kv_attention_wide(a, parts, stream);
  if (e != cudaSuccess || parts.rows == 0) return e;
  // CTAs of a (sequence, KV head): a row each of few, an eighth of a tile each
  // of many, in one turn of the four that an SM holds
  const int64_t want = rows <= kFewRows ? rows : (rows + kWideRows - 1) / kWideRows * 8;
  const int64_t most = rows <= kFewRows ? kFewRows : std::max<int64_t>(1, 4 * sm_count() / (static_cast<int64_t>(a.c.S) * a.c.H));
  const dim3 grid(a.c.S, a.c.H, static_cast<unsigned>(std::min<int64_t>(want, most)));
  return launch_kernel(rows <= kFewRows ? kv_combine_kernel<D, false> : kv_combine_kernel<D, true>, grid,
                       dim3(kJoinThreads), 0, stream, true, a, parts);
}

}  // namespace

size_t kv_attention_workspace_bytes(int64_t S, int64_t T, int64_t max_q, int64_t max_pages, int64_t Hq, int64_t Hkv,
                                    int64_t D, int64_t block) {
  return static_cast<size_t>(Hkv * parts_of(S, T, max_q, Hq / Hkv, max_pages * block, Hkv, D).rows) * (D + 4) * 4;
}

cudaError_t launch_kv_attention(const KvAttentionArgs& a, cudaStream_t stream) {
  return a.c.D == 64 ? launch_d<64>(a, stream) : a.c.D == 128 ? launch_d<128>(a, stream) : launch_d<256>(a, stream);
}

}  // namespace prism
