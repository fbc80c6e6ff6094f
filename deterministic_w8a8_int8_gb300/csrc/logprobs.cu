// logprobs.cu -- log probabilities of given tokens under full-vocabulary
// logits, with the entropy and the top alternatives:
//   m = max x, s = sum e^(x - m), lp(t) = (x_t - m) - ln s,
//   H = ln s - sum e^(x - m) (x - m) / s,
//   top k by (larger value, then lower id).
//
// Every logit is read once: V * 2 (4) bytes a row, HBM-bound for many rows and
// a chain of latencies for one.  A row is cut into 1 to 8 parts by V alone, and
// thread t of part c takes the 8-logit pieces (i * parts + c) * 512 + t as they
// arrive.  With few rows each part is a CTA of the row's cluster; with many, a
// CTA takes several parts or all of them in turn (a part's sums are the same
// either way, so a row's bits do not depend on the call): 768 rows of 248000
// took 185 us with eight CTAs a row, one row 7 us against 30 with one.  Now 96
// us (4.0 TB/s, 62 % of the issue slots, eleven instructions a logit, in 2.5 turns
// of the CTAs) and 7.4 us.  Rows off 16-byte boundaries (7 of 8 where V is odd) are
// read by single logits: 768 of 248001 take 248 us.  Rows whose maximum is beyond
// kFarRow are read twice: 178 us.
//   Sums: a thread adds 2^y and y 2^y, y = x L - r, L = log2 e, against a
// reference r = RN(L m), m the maximum of its first piece that has one -- one
// fused multiply-add and one ex2 a logit, x L itself being exact inside the
// former -- and takes a new reference only for a logit more than kSlack above
// it.  The references are joined over lanes, warps and CTAs by fixed trees.
// Everything is binary32.
//   Alternatives: one exchange of 128 group maxima through distributed shared
// memory gives every CTA, as the k-th largest of them, a bound that at least k
// logits reach: for logits in no order about 1.2 k do.  The pieces of threads whose
// maximum reaches it are read again (from L2) and these logits sent to the
// first CTA, which ranks them.  Where more than its list holds reach the bound
// (long ties, a row in rising order) every CTA extracts its own top k instead.
#include <cuda_bf16.h>

#include "decode.cuh"

namespace prism {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kVec = 8;                       // logits of a piece
constexpr int kLogTile = 12;
constexpr int kTile = 1 << kLogTile;          // logits of one piece of every thread
static_assert(kTile == kThreads * kVec, "tile");
constexpr int kMaxParts = 8;
constexpr int kGroups = 128;                  // group maxima of a row
constexpr int kList = 1024;                   // candidates the first CTA can take
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
// A thread's reference is RN(L m), so its terms are off by a common factor of 2^
// (half a step of L m), which the join takes back: below kFar that is 2^(1/16) at
// most (at 1e10 it would be 2^440).  Pieces at -kFar and below are masked ones,
// without a reference: their terms are zero.  That holds for rows whose maximum
// is well above -kFar; other rows, and those above kFarRow, are summed again by
// differences.
constexpr float kFar = 0x1p20f, kFarRow = 0x1p19f;
constexpr float kSlack = 27.0f;               // e^27 over the reference: far from binary32's limits

typedef unsigned long long u64;

// Larger keys come first: the value's order, then the lower id.
__device__ __forceinline__ u64 order_key(float x, uint32_t id) {
  const uint32_t u = __float_as_uint(__fadd_rn(x, 0.0f));   // -0 and +0 are equal
  const uint32_t o = u & 0x80000000u ? ~u : u | 0x80000000u;
  return (static_cast<u64>(o) << 32) | (0xffffffffu - id);
}
__device__ __forceinline__ float key_value(u64 k) {
  const uint32_t o = static_cast<uint32_t>(k >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
// The shared-memory address of `p` in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t at_rank(const void* p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_cluster(uint32_t a, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t a, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t add_cluster(uint32_t a, uint32_t v) {
  uint32_t r;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(r) : "r"(a), "r"(v) : "memory");
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}

// One piece: 8 bf16 in a uint4, or 8 float32 in two.
template <bool F32>
struct Piece {
  uint4 w[F32 ? 2 : 1];
  __device__ __forceinline__ float get(int i) const {
    const uint4& v = w[F32 ? i >> 2 : 0];
    if (F32) return __uint_as_float((i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w);
    const uint32_t u = (i >> 1) == 0 ? v.x : (i >> 1) == 1 ? v.y : (i >> 1) == 2 ? v.z : v.w;
    return i & 1 ? bf16_hi(u) : bf16_lo(u);
  }
  // Largest logit, NaN aside.
  __device__ __forceinline__ float top() const {
    if (F32) {
      float m = get(0);
#pragma unroll
      for (int i = 1; i < 8; ++i) m = fmaxf(m, get(i));
      return m;
    }
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(w);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&m);
    return fmaxf(bf16_lo(u), bf16_hi(u));
  }
  // Values at or below about -1e38 (masked ones) raised to it: their terms are
  // zero all the same, and 0 * inf does not arise.  NaN stays.
  __device__ __forceinline__ void lift() {
    uint32_t* u = reinterpret_cast<uint32_t*>(w);
#pragma unroll
    for (int i = 0; i < (F32 ? 8 : 4); ++i)
      u[i] = F32 ? __float_as_uint(max_nan(__uint_as_float(u[i]), -1e38f)) : max_nan_bf16x2(u[i], 0xfe96fe96u);
  }
};
// Logits [at, at + 8) of a row by plain loads; -inf from V on.
template <bool F32>
__device__ __forceinline__ Piece<F32> load_piece(const void* row, int64_t at, int64_t V) {
  Piece<F32> p;
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    if (F32) {
      u[i] = at + i < V ? __ldg(static_cast<const uint32_t*>(row) + at + i) : 0xff800000u;
    } else {
      u[i] = at + i < V ? __ldg(static_cast<const uint16_t*>(row) + at + i) : 0xff80u;
    }
  }
  if (F32) {
    p.w[0] = make_uint4(u[0], u[1], u[2], u[3]);
    p.w[F32 ? 1 : 0] = make_uint4(u[4], u[5], u[6], u[7]);
  } else {
    p.w[0] = make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
  }
  return p;
}

template <bool F32>
__global__ void __launch_bounds__(kThreads, 2)
    logprobs_kernel(const __grid_constant__ LogprobArgs a, int log_parts, int log_ctas) {
  __shared__ __align__(16) float s_max[kGroups];
  __shared__ __align__(16) u64 s_list[kList];
  __shared__ float s_part[kMaxParts * kWarps][3];   // each warp's reference, sum and weighted sum
  __shared__ float s_row_sum[4];
  __shared__ float s_top[kMaxParts][kThreads];        // each thread's maximum of the CTA's parts
  __shared__ u64 s_best[kWarps];
  __shared__ float s_far[kWarps][2];
  __shared__ uint32_t s_bound;
  __shared__ uint32_t s_count;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = 1 << log_ctas;
  const int rank = ctas > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int64_t r = blockIdx.x >> log_ctas;
  const void* row = F32 ? static_cast<const void*>(static_cast<const float*>(a.logits) + r * a.ldl)
                        : static_cast<const void*>(static_cast<const uint16_t*>(a.logits) + r * a.ldl);
  cluster_arrive();   // waited for before the first store into another CTA
  const bool aligned = (reinterpret_cast<uintptr_t>(row) & 15) == 0;
  const int tiles = static_cast<int>((a.V + kTile - 1) / kTile), parts = 1 << log_parts;
  const int64_t stride = static_cast<int64_t>(parts) * kTile;
  struct Range {
    int64_t first;     // the thread's first piece
    int mine, whole;   // its pieces; those that lie whole in an aligned row (at most one more is cut by V)
  };
  auto range = [&](int part) {
    Range g;
    g.first = static_cast<int64_t>(part) * kTile + tid * kVec;
    g.mine = (tiles - part + parts - 1) >> log_parts;
    g.whole = aligned && g.first + kVec <= a.V
                  ? min(g.mine, static_cast<int>((a.V - kVec - g.first) >> (kLogTile + log_parts)) + 1) : 0;
    return g;
  };
  // f(piece, number) over the thread's pieces, kAhead of them in flight
  auto each = [&](const Range& g, auto f) {
    constexpr int kWords = F32 ? 2 : 1, kAhead = F32 ? 4 : 8;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + g.first * (F32 ? 4 : 2));
    const int64_t step = stride * (F32 ? 4 : 2) / 16;
    for (int i0 = 0; i0 < g.whole; i0 += kAhead) {
      Piece<F32> p[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (i0 + i < g.whole) {
#pragma unroll
          for (int j = 0; j < kWords; ++j) p[i].w[j] = __ldg(src + i * step + j);
        }
      }
      src += kAhead * step;
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (i0 + i < g.whole) f(p[i], i0 + i);
    }
    for (int i = g.whole; i < g.mine; ++i) f(load_piece<F32>(row, g.first + i * stride, a.V), i);
  };
  if (tid == 0) s_count = 0, s_bound = 0xffffffffu;

  // ---- 1. a part at a time: the thread's maximum and sums
  for (int part = rank; part < parts; part += ctas) {
    float limit = -INFINITY, ref = 0.0f, p_max = -INFINITY;
    float2 s2 = make_float2(0.0f, 0.0f), e2 = s2;   // of the even and the odd logits
    each(range(part), [&](Piece<F32> p, int) {
      const float m = p.top();
      p_max = fmaxf(p_max, m);
      if (m > limit && fabsf(m) < kFar) {      // the first finite piece, or one far above the reference
        const float to = __fmul_rn(m, kLog2e), d = limit == -INFINITY ? 0.0f : ref - to, f = ex2(d);
        e2 = mul2(make_float2(f, f), fma2(s2, make_float2(d, d), e2));
        s2 = mul2(make_float2(f, f), s2);
        ref = to;
        limit = m + kSlack;
      }
      p.lift();
#pragma unroll
      for (int i = 0; i < kVec; i += 2) {
        const float2 y = fma2(make_float2(p.get(i), p.get(i + 1)), make_float2(kLog2e, kLog2e), make_float2(-ref, -ref));
        const float2 q = make_float2(ex2(y.x), ex2(y.y));
        s2 = add2(s2, q);
        e2 = fma2(q, y, e2);
      }
    });
    float s = __fadd_rn(s2.x, s2.y), e = __fadd_rn(e2.x, e2.y);
    s_top[part >> log_ctas][tid] = p_max;
    // the group's maximum (128 groups a row), and the warp's reference and sums
    const int g_lanes = 4 * parts;             // lanes of a group
    for (int o = 1; o < g_lanes; o <<= 1) p_max = fmaxf(p_max, __shfl_xor_sync(0xffffffffu, p_max, o));
    float w_ref = limit == -INFINITY ? -INFINITY : ref;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) w_ref = fmaxf(w_ref, __shfl_xor_sync(0xffffffffu, w_ref, o));
    {
      const float d = limit == -INFINITY ? 0.0f : ref - w_ref, f = ex2(d);   // without a reference the sums are 0 or NaN
      e = f * __fmaf_rn(s, d, e);
      s *= f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      e += __shfl_xor_sync(0xffffffffu, e, o);
    }
    if (part == rank) cluster_wait();          // every CTA of the cluster runs
    const int to = lane & (g_lanes - 1);       // lane j of a group writes rank j's copy
    if (to < ctas) st_cluster(at_rank(&s_max[(part * kThreads + tid) >> (2 + log_parts)], to), p_max);
    if (lane < 3) st_cluster(at_rank(&s_part[part * kWarps + warp][lane], 0), lane == 0 ? w_ref : lane == 1 ? s : e);
  }
  cluster_arrive();
  cluster_wait();

  // ---- 2. the k-th largest group maximum, the least one with fewer than k
  // above it: at least k logits reach it.  Four threads a maximum.
  if (a.top_k > 0) {
    const float v = s_max[tid >> 2];
    int above = 0;
#pragma unroll
    for (int j = 0; j < kGroups / 16; ++j) {
      const float4 w = *reinterpret_cast<const float4*>(&s_max[(j * 4 + (tid & 3)) * 4]);
      above += (w.x > v) + (w.y > v) + (w.z > v) + (w.w > v);
    }
    above += __shfl_xor_sync(0xffffffffu, above, 1);
    above += __shfl_xor_sync(0xffffffffu, above, 2);
    if (above < a.top_k) atomicMin(&s_bound, static_cast<uint32_t>(order_key(v, 0) >> 32));
    __syncthreads();
  }

  // ---- 3. the logits that reach the bound go to the first CTA: the pieces of a
  // thread whose maximum does are read again, two logits a lane of its warp
  const uint32_t count_at = at_rank(&s_count, 0);
  if (a.top_k > 0) {
    const float bound = key_value(static_cast<u64>(s_bound) << 32);
    for (int part = rank; part < parts; part += ctas) {
      uint32_t reach = __ballot_sync(0xffffffffu, s_top[part >> log_ctas][tid] >= bound);
      for (; reach != 0; reach &= reach - 1) {
        const int64_t at0 = static_cast<int64_t>(part) * kTile + (warp * 32 + __ffs(reach) - 1) * kVec + (lane & 3) * 2;
        for (int64_t at = at0 + (lane >> 2) * stride; at < a.V; at += 8 * stride) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (at + i >= a.V) break;
            const float x = F32 ? __ldg(static_cast<const float*>(row) + at + i)
                                : bf16_bits_to_float(__ldg(static_cast<const uint16_t*>(row) + at + i));
            if (x >= bound) {
              const uint32_t n = add_cluster(count_at, 1);
              if (n < kList) st_cluster(at_rank(&s_list[n], 0), order_key(x, static_cast<uint32_t>(at + i)));
            }
          }
        }
      }
    }
  }
  cluster_arrive();
  cluster_wait();
  uint32_t count = a.top_k > 0 ? ld_cluster_u32(count_at) : 0;
  if (count > kList) {
    // every CTA's own top k: a thread offers its best, the winner looks for its next
    auto next = [&](u64 below) {
      u64 best = 0;
      for (int part = rank; part < parts; part += ctas) {
      const Range g = range(part);
      each(g, [&](const Piece<F32>& p, int number) {
        const int64_t id = g.first + number * stride;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const u64 key = order_key(p.get(i), static_cast<uint32_t>(id + i));
          if (id + i < a.V && key < below && key > best) best = key;
        }
      });
      }
      return best;
    };
    u64 offer = next(~0ull);
    for (int k = 0; k < a.top_k; ++k) {
      u64 best = offer;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
      __syncthreads();
      if (lane == 0) s_best[warp] = best;
      __syncthreads();
      best = s_best[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) best = max(best, s_best[w]);
      if (tid == 0) st_cluster(at_rank(&s_list[rank * a.top_k + k], 0), best);   // 0: no logit left
      if (offer == best && best != 0) offer = next(best);
    }
    count = static_cast<uint32_t>(ctas * a.top_k);
    cluster_arrive();
    cluster_wait();
  }
  cluster_arrive();   // the first CTA's count has been read
  if (rank == 0) {
    // ---- 4. the row's maximum, reference and sums, and the outputs
    if (warp == 0) {
      const int n = parts * kWarps;
      float wr[4], top = -INFINITY, rr = -INFINITY, sum = 0.0f, ent = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        top = fmaxf(top, s_max[lane + 32 * i]);
        wr[i] = lane + 32 * i < n ? s_part[lane + 32 * i][0] : -INFINITY;
        rr = fmaxf(rr, wr[i]);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        rr = fmaxf(rr, __shfl_xor_sync(0xffffffffu, rr, o));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (lane + 32 * i < n) {
          const float ws = s_part[lane + 32 * i][1], we = s_part[lane + 32 * i][2];
          const float d = wr[i] == -INFINITY ? 0.0f : wr[i] - rr, f = ex2(d);
          sum += f * ws;
          ent += f * __fmaf_rn(ws, d, we);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        ent += __shfl_xor_sync(0xffffffffu, ent, o);
      }
      if (lane == 0) s_row_sum[0] = top, s_row_sum[1] = rr, s_row_sum[2] = sum, s_row_sum[3] = ent;
    }
    __syncthreads();
    const float top = s_row_sum[0];
    float rr = s_row_sum[1], sum = s_row_sum[2], ent = s_row_sum[3];
    const bool far = top > -INFINITY && top < INFINITY && !(fabsf(top) < kFarRow);
    if (far) {   // the row once more, differences first
      float fs = 0.0f, fe = 0.0f;
      for (int64_t v = tid; v < a.V; v += kThreads) {
        const float x = F32 ? static_cast<const float*>(row)[v] : bf16_bits_to_float(static_cast<const uint16_t*>(row)[v]);
        const float y = max_nan(__fmul_rn(__fsub_rn(x, top), kLog2e), -1000.0f), q = ex2(y);
        fs += q;
        fe = __fmaf_rn(q, y, fe);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        fs += __shfl_xor_sync(0xffffffffu, fs, o);
        fe += __shfl_xor_sync(0xffffffffu, fe, o);
      }
      if (lane == 0) s_far[warp][0] = fs, s_far[warp][1] = fe;
      __syncthreads();
      sum = ent = 0.0f;
      for (int w = 0; w < kWarps; ++w) sum += s_far[w][0], ent += s_far[w][1];
    }
    const bool ok = top > -INFINITY && top < INFINITY && sum == sum;
    const float nanf = __uint_as_float(0x7fc00000u), log_sum = log2f(sum);
    // ln of the sum of e^(x - top): the sum's reference against the maximum
    const float logz = (far ? log_sum : log_sum - __fmaf_rn(top, kLog2e, -rr)) * kLn2;
    auto log_prob = [&](float x) { return (x - top) - logz; };
    if (tid == 0 && a.entropy != nullptr) a.entropy[r] = ok ? (log_sum - ent / sum) * kLn2 : nanf;
    for (int i = tid; i < a.n_ids; i += kThreads) {
      const int32_t id = a.ids[r * a.ld_ids + i];
      const bool in = id >= 0 && id < a.V;
      if (!in && a.err != nullptr) atomicOr(a.err, PRISM_DEV_ERR_ID_RANGE);
      float x = 0.0f;
      if (in) x = F32 ? static_cast<const float*>(row)[id] : bf16_bits_to_float(static_cast<const uint16_t*>(row)[id]);
      a.logprobs[r * a.n_ids + i] = ok && in ? log_prob(x) : nanf;
    }
    if (ok) {
      for (uint32_t i = tid; i < count; i += kThreads) {
        const u64 key = s_list[i];
        int above = 0;
        for (uint32_t j = 0; j < count; ++j) above += s_list[j] > key;
        if (above < a.top_k && key != 0) {
          a.top_ids[r * a.top_k + above] = static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(key));
          a.top_logprobs[r * a.top_k + above] = log_prob(key_value(key));
        }
      }
    } else {
      for (int i = tid; i < a.top_k; i += kThreads) {
        a.top_ids[r * a.top_k + i] = -1;
        a.top_logprobs[r * a.top_k + i] = nanf;
      }
    }
  }
  cluster_wait();
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t stream) {
  // parts of a row: up to four pieces a thread, then up to eight parts; CTAs of
  // a row: one a part while they all run at once (two on an SM)
  const int64_t tiles = (a.V + kTile - 1) / kTile;
  int log_parts = 0;
  while ((1 << log_parts) < kMaxParts && tiles > (4 << log_parts)) ++log_parts;
  int log_ctas = log_parts;
  while (log_ctas > 0 && (a.R << log_ctas) > 2 * sm_count()) --log_ctas;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.R << log_ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1u << log_ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return a.f32 ? cudaLaunchKernelEx(&cfg, logprobs_kernel<true>, a, log_parts, log_ctas)
               : cudaLaunchKernelEx(&cfg, logprobs_kernel<false>, a, log_parts, log_ctas);
}

}  // namespace prism
