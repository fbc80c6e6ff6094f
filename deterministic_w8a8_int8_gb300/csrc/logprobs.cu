// logprobs.cu -- log probabilities of given tokens under full-vocabulary
// logits, with the entropy and the top alternatives:
//   m = max x, s = sum e^(x - m), lp(t) = (x_t - m) - ln s,
//   H = ln s - sum e^(x - m) (x - m) / s,
//   top k by (larger value, then lower id).
//
// Every logit is read once: V * 2 (4) bytes a row, HBM-bound for many rows and
// a chain of latencies for one.  A row is one thread-block cluster (1 to 8
// CTAs by V alone, so a row's bits do not depend on the call); thread t of
// rank c copies the 8-logit pieces (i * ranks + c) * 512 + t into shared memory
// (V up to 262144; longer rows are read again) and alone reads them there.
//   Sums: a warp takes its own maximum m and adds 2^(x L - r), L = log2 e,
// r = RN(m L) -- one fused multiply-add and one ex2 a logit, x L itself being
// exact inside the former -- so nothing waits for the row's maximum; the
// warps' (r, sum, weighted sum) are joined by the first CTA.  Sums are binary32
// per thread, then fixed trees over lanes and warps.
//   Alternatives: one exchange of 128 group maxima through distributed shared
// memory gives every CTA, as the k-th largest of them, a bound that at least k
// logits reach: for logits in no order about 1.2 k do, and these alone go to
// the first CTA, which ranks them.  Where more than its list holds reach it
// (long ties, a row in rising order) every CTA extracts its own top k instead.
#include <cuda_bf16.h>

#include "decode.cuh"

namespace prism {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kVec = 8;                       // logits of a piece
constexpr int kPieces = 8;                    // pieces of a thread that stay in shared memory
constexpr int kLogTile = 12;
constexpr int kTile = 1 << kLogTile;          // logits of one piece of every thread
static_assert(kTile == kThreads * kVec, "tile");
constexpr int kMaxCluster = 8;
constexpr int kGroups = 128;                  // group maxima of a row
constexpr int kList = 1024;                   // candidates the first CTA can take
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
constexpr float kFar = 1e37f;                 // beyond it x * log2(e) could leave binary32's range

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

// kHeld: the row fits the shared memory of its cluster.
template <bool F32, bool kHeld>
__global__ void __launch_bounds__(kThreads, F32 ? 1 : 3)
    logprobs_kernel(const __grid_constant__ LogprobArgs a, int log_ctas) {
  extern __shared__ __align__(16) uint4 s_row[];
  __shared__ __align__(16) float s_max[kGroups];
  __shared__ __align__(16) u64 s_list[kList];
  __shared__ float s_part[kMaxCluster * kWarps][3];   // each warp's reference, sum and weighted sum
  __shared__ float s_row_sum[3];
  __shared__ u64 s_best[kWarps];
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
  const int tiles = static_cast<int>((a.V + kTile - 1) / kTile);
  const int mine = (tiles - rank + ctas - 1) >> log_ctas;   // pieces of each thread
  const int64_t first = static_cast<int64_t>(rank) * kTile + tid * kVec, stride = static_cast<int64_t>(ctas) * kTile;
  // pieces that lie whole in an aligned row; at most one more is cut by V
  const int whole = aligned && first + kVec <= a.V ? min(mine, static_cast<int>((a.V - kVec - first) >> (kLogTile + log_ctas)) + 1) : 0;
  constexpr int kWords = F32 ? 2 : 1;        // 16-byte words of a piece
  constexpr int kBytes = F32 ? 4 : 2;
  uint4* held = s_row + tid;                 // word j of piece i: held[(i * kWords + j) * kThreads]
  if constexpr (kHeld) {
    const uint8_t* src = static_cast<const uint8_t*>(row) + first * kBytes;
    uint32_t dst = smem_u32(held);
    for (int i = 0; i < whole; ++i) {
#pragma unroll
      for (int j = 0; j < kWords; ++j) cp_async_16(dst + j * (kThreads * 16), src + j * 16, 16);
      src += stride * kBytes;
      dst += kWords * kThreads * 16;
    }
    cp_async_commit();
    for (int i = whole; i < mine; ++i) {
      const Piece<F32> p = load_piece<F32>(row, first + i * stride, a.V);
#pragma unroll
      for (int j = 0; j < kWords; ++j) held[(i * kWords + j) * kThreads] = p.w[j];
    }
    cp_async_wait<0>();
  }
  // f(piece, number) over the thread's pieces
  auto each = [&](auto f) {
    if constexpr (kHeld) {
      const uint4* src = held;
#pragma unroll 2
      for (int i = 0; i < mine; ++i) {
        Piece<F32> p;
#pragma unroll
        for (int j = 0; j < kWords; ++j) p.w[j] = src[j * kThreads];
        src += kWords * kThreads;
        f(p, i);
      }
    } else {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + first * kBytes);
#pragma unroll 2
      for (int i = 0; i < whole; ++i) {
        Piece<F32> p;
#pragma unroll
        for (int j = 0; j < kWords; ++j) p.w[j] = __ldg(src + j);
        src += stride * kBytes / 16;
        f(p, i);
      }
      for (int i = whole; i < mine; ++i) f(load_piece<F32>(row, first + i * stride, a.V), i);
    }
  };
  // ---- 1. maxima of the thread and its group (128 a row); the warp's sums of
  // 2^y and y 2^y, y = x L - r for the warp's reference r
  float t_max = -INFINITY;
  each([&](const Piece<F32>& p, int) { t_max = fmaxf(t_max, p.top()); });
  const int g_lanes = 4 * ctas;              // lanes of a group
  float g_max = t_max;
  for (int o = 1; o < g_lanes; o <<= 1) g_max = fmaxf(g_max, __shfl_xor_sync(0xffffffffu, g_max, o));
  float m = g_max;
  for (int o = g_lanes; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float ref = m == -INFINITY ? 0.0f : __fmul_rn(m, kLog2e);
  float s = 0.0f, e = 0.0f;
  if (m == -INFINITY || fabsf(m) < kFar) {
    float s2 = 0.0f, e2 = 0.0f;
    each([&](Piece<F32> p, int) {
      p.lift();
#pragma unroll
      for (int i = 0; i < kVec; i += 2) {
        const float y0 = __fmaf_rn(p.get(i), kLog2e, -ref), y1 = __fmaf_rn(p.get(i + 1), kLog2e, -ref);
        const float q0 = ex2(y0), q1 = ex2(y1);
        s = __fadd_rn(s, q0);
        s2 = __fadd_rn(s2, q1);
        e = __fmaf_rn(q0, y0, e);
        e2 = __fmaf_rn(q1, y1, e2);
      }
    });
    s = __fadd_rn(s, s2);
    e = __fadd_rn(e, e2);
  } else {   // a far maximum: differences first; the reference may be infinite, the row's join goes by m then
    each([&](const Piece<F32>& p, int) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const float y = max_nan(__fmul_rn(__fsub_rn(p.get(i), m), kLog2e), -1000.0f), q = ex2(y);
        s = __fadd_rn(s, q);
        e = __fmaf_rn(q, y, e);
      }
    });
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    e += __shfl_xor_sync(0xffffffffu, e, o);
  }
  if (tid == 0) s_count = 0, s_bound = 0xffffffffu;
  cluster_wait();   // every CTA of the cluster runs
  {
    const int to = lane & (g_lanes - 1);     // lane j of a group writes rank j's copy
    if (to < ctas) st_cluster(at_rank(&s_max[(rank * kThreads + tid) >> (2 + log_ctas)], to), g_max);
    if (lane < 3) st_cluster(at_rank(&s_part[rank * kWarps + warp][lane], 0), lane == 0 ? m : lane == 1 ? s : e);
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

  // ---- 3. the logits that reach the bound go to the first CTA
  const uint32_t count_at = at_rank(&s_count, 0);
  if (a.top_k > 0) {
    const float bound = key_value(static_cast<u64>(s_bound) << 32);
    if (t_max >= bound) {
      each([&](const Piece<F32>& p, int number) {
        if (!(p.top() >= bound)) return;
        const int64_t id = first + number * stride;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const float x = p.get(i);
          if (x >= bound && id + i < a.V) {
            const uint32_t at = add_cluster(count_at, 1);
            if (at < kList) st_cluster(at_rank(&s_list[at], 0), order_key(x, static_cast<uint32_t>(id + i)));
          }
        }
      });
    }
  }
  cluster_arrive();
  cluster_wait();
  uint32_t count = a.top_k > 0 ? ld_cluster_u32(count_at) : 0;
  if (count > kList) {
    // every CTA's own top k: a thread offers its best, the winner looks for its next
    auto next = [&](u64 below) {
      u64 best = 0;
      each([&](const Piece<F32>& p, int number) {
        const int64_t id = first + number * stride;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const u64 key = order_key(p.get(i), static_cast<uint32_t>(id + i));
          if (id + i < a.V && key < below && key > best) best = key;
        }
      });
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
    // ---- 4. the row's reference and sums, and the outputs
    if (warp == 0) {
      const int n = ctas * kWarps;
      float wm[4], top = -INFINITY, sum = 0.0f, ent = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        wm[i] = lane + 32 * i < n ? s_part[lane + 32 * i][0] : -INFINITY;
        top = fmaxf(top, wm[i]);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const bool far = !(fabsf(top) < kFar);
      const float r = __fmul_rn(top, kLog2e);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (lane + 32 * i < n) {
          const float ws = s_part[lane + 32 * i][1], we = s_part[lane + 32 * i][2];
          // the warp's reference against the row's, in log2 units; a warp with a
          // far maximum has it as it is (under a near one its terms are zero)
          float d = far ? (wm[i] - top) * kLog2e : fabsf(wm[i]) < kFar ? __fsub_rn(__fmul_rn(wm[i], kLog2e), r) : -1000.0f;
          d = max_nan(d, -1000.0f);
          const float f = ex2(d);
          sum += f * ws;
          ent += f * (we + d * ws);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        ent += __shfl_xor_sync(0xffffffffu, ent, o);
      }
      if (lane == 0) s_row_sum[0] = top, s_row_sum[1] = sum, s_row_sum[2] = ent;
    }
    __syncthreads();
    const float top = s_row_sum[0], sum = s_row_sum[1];
    const bool ok = top > -INFINITY && top < INFINITY && sum == sum, far = !(fabsf(top) < kFar);
    const float nanf = __uint_as_float(0x7fc00000u), log_sum = log2f(sum), ref_row = __fmul_rn(top, kLog2e);
    // ln of the sum against the maximum itself: the reference's rounding taken off
    const float logz = (far ? log_sum : log_sum - __fmaf_rn(top, kLog2e, -ref_row)) * kLn2;
    auto log_prob = [&](float x) { return (x - top) - logz; };
    if (tid == 0 && a.entropy != nullptr) a.entropy[r] = ok ? (log_sum - s_row_sum[2] / sum) * kLn2 : nanf;
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

template <bool F32, bool kHeld>
cudaError_t launch_kind(const LogprobArgs& a, int64_t tiles, int log_ctas, cudaStream_t stream) {
  const int ctas = 1 << log_ctas;
  constexpr int most = kPieces * kThreads * (F32 ? 32 : 16);
  if (kHeld) {
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(logprobs_kernel<F32, kHeld>), most);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.R * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kHeld ? static_cast<size_t>((tiles + ctas - 1) / ctas) * (most / kPieces) : 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<F32, kHeld>, a, log_ctas);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t stream) {
  // CTAs of a row: up to four pieces a thread, then up to eight CTAs
  const int64_t tiles = (a.V + kTile - 1) / kTile;
  int log_ctas = 0;
  while ((1 << log_ctas) < kMaxCluster && tiles > (4 << log_ctas)) ++log_ctas;
  const bool held = tiles <= kPieces << log_ctas;
  if (a.f32) return held ? launch_kind<true, true>(a, tiles, log_ctas, stream) : launch_kind<true, false>(a, tiles, log_ctas, stream);
  return held ? launch_kind<false, true>(a, tiles, log_ctas, stream) : launch_kind<false, false>(a, tiles, log_ctas, stream);
}

}  // namespace prism
