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
// (V up to 262144; longer rows are read again) and alone reads them there.  One exchange of 128 group
// maxima through distributed shared memory gives every CTA the row's maximum
// and, as the k-th largest of them, a bound that at least k logits reach: for
// logits in no order about 1.2 k do, and these alone go to the first CTA,
// which ranks them.  Where more than its list holds reach it (long ties, a row
// in rising order) every CTA extracts its own top k instead.
// Sums are binary32 per thread, then fixed trees over lanes, warps and CTAs.
#include "decode.cuh"

namespace prism {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kVec = 8;                       // logits of a piece
constexpr int kPieces = 8;                    // pieces of a thread that stay in shared memory
constexpr int kTile = kThreads * kVec;        // logits of one piece of every thread
constexpr int kMaxCluster = 8;
constexpr int kGroups = 128;                  // group maxima of a row
constexpr int kList = 1024;                   // candidates the first CTA can take
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

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
    logprobs_kernel(const __grid_constant__ LogprobArgs a, int ctas) {
  extern __shared__ __align__(16) uint4 s_row[];
  __shared__ __align__(16) float s_max[kGroups];
  __shared__ __align__(16) u64 s_list[kList];
  __shared__ float s_sum[kMaxCluster][2];
  __shared__ float s_red[kWarps][2];
  __shared__ u64 s_best[kWarps];
  __shared__ float s_bound;
  __shared__ uint32_t s_count;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = ctas > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int64_t r = blockIdx.x / ctas;
  const void* row = F32 ? static_cast<const void*>(static_cast<const float*>(a.logits) + r * a.ldl)
                        : static_cast<const void*>(static_cast<const uint16_t*>(a.logits) + r * a.ldl);
  const bool aligned = (reinterpret_cast<uintptr_t>(row) & 15) == 0;
  const int tiles = static_cast<int>((a.V + kTile - 1) / kTile);
  const int mine = (tiles - rank + ctas - 1) / ctas;   // pieces of each thread
  auto base = [&](int i) { return (static_cast<int64_t>(i) * ctas + rank) * kTile + tid * kVec; };
  constexpr int kWords = F32 ? 2 : 1;        // 16-byte words of a piece
  auto word = [&](int i, int j) { return &s_row[(i * kWords + j) * kThreads + tid]; };
  if constexpr (kHeld) {
    for (int i = 0; i < mine; ++i) {
      const int64_t at = base(i);
      if (aligned && at + kVec <= a.V) {
#pragma unroll
        for (int j = 0; j < kWords; ++j)
          cp_async_16(smem_u32(word(i, j)), static_cast<const uint8_t*>(row) + at * (F32 ? 4 : 2) + j * 16, 16);
      } else {
        const Piece<F32> p = load_piece<F32>(row, at, a.V);
#pragma unroll
        for (int j = 0; j < kWords; ++j) *word(i, j) = p.w[j];
      }
    }
    cp_async_commit();
    cp_async_wait<0>();
  }
  // f(piece, first id) over the thread's pieces
  auto each = [&](auto f) {
#pragma unroll 2
    for (int i = 0; i < mine; ++i) {
      Piece<F32> p;
      if constexpr (kHeld) {
#pragma unroll
        for (int j = 0; j < kWords; ++j) p.w[j] = *word(i, j);
      } else if (aligned && base(i) + kVec <= a.V) {
        const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + base(i) * (F32 ? 4 : 2));
#pragma unroll
        for (int j = 0; j < kWords; ++j) p.w[j] = __ldg(x + j);
      } else {
        p = load_piece<F32>(row, base(i), a.V);
      }
      f(p, base(i));
    }
  };
  if (tid == 0) s_count = 0;

  // ---- 1. maxima: of the thread, its group (128 a row), the row
  float t_max = -INFINITY;
  each([&](const Piece<F32>& p, int64_t) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) t_max = fmaxf(t_max, p.get(i));
  });
  float g_max = t_max;
  for (int o = 1; o < 4 * ctas; o <<= 1) g_max = fmaxf(g_max, __shfl_xor_sync(0xffffffffu, g_max, o));
  if (ctas > 1) {   // no store reaches a CTA that has not started
    cluster_arrive();
    cluster_wait();
  }
  const int g_lanes = 4 * ctas;              // lanes of a group
  const int g_cta = kThreads / g_lanes;      // groups of a CTA
  if ((lane & (g_lanes - 1)) < ctas) {       // lane j of the group writes rank j's copy
    const int to = lane & (g_lanes - 1);
    st_cluster(at_rank(&s_max[rank * g_cta + tid / g_lanes], to), g_max);
  }
  if (ctas > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  float m = s_max[lane];
#pragma unroll
  for (int i = 1; i < kGroups / 32; ++i) m = fmaxf(m, s_max[lane + 32 * i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  // the k-th largest group maximum: at least k logits reach it
  if (a.top_k > 0 && tid < kGroups) {
    const float v = s_max[tid];
    int above = 0;
#pragma unroll 4
    for (int j = 0; j < kGroups; j += 4) {
      const float4 w = *reinterpret_cast<const float4*>(&s_max[j]);
      above += (w.x > v || (w.x == v && j < tid)) + (w.y > v || (w.y == v && j + 1 < tid)) +
               (w.z > v || (w.z == v && j + 2 < tid)) + (w.w > v || (w.w == v && j + 3 < tid));
    }
    if (above == a.top_k - 1) s_bound = v;
  }

  // ---- 2. sums of e^(x - m) and of (x - m) e^(x - m), the latter in units of ln 2
  float s = 0.0f, e = 0.0f;
  each([&](const Piece<F32>& p, int64_t) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      // a floor far below ex2's zero keeps 0 * -inf out; NaN passes
      const float y = max_nan(__fmul_rn(__fsub_rn(p.get(i), m), kLog2e), -1000.0f), q = ex2(y);
      s = __fadd_rn(s, q);
      e = __fmaf_rn(q, y, e);
    }
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    e += __shfl_xor_sync(0xffffffffu, e, o);
  }
  if (lane == 0) s_red[warp][0] = s, s_red[warp][1] = e;
  __syncthreads();   // and s_bound
  if (tid < 2) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += s_red[w][tid];
    st_cluster(at_rank(&s_sum[rank][tid], 0), v);
  }

  // ---- 3. the logits that reach the bound go to the first CTA
  const uint32_t count_at = at_rank(&s_count, 0);
  if (a.top_k > 0) {
    const float bound = s_bound;
    if (t_max >= bound) {
      each([&](const Piece<F32>& p, int64_t id) {
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
      each([&](const Piece<F32>& p, int64_t id) {
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
    // ---- 4. outputs
    float sum = 0.0f, ent = 0.0f;
    for (int i = 0; i < ctas; ++i) sum += s_sum[i][0], ent += s_sum[i][1];
    const bool ok = m > -INFINITY && m < INFINITY && sum == sum;
    const float nanf = __uint_as_float(0x7fc00000u), logz = log2f(sum) * kLn2;
    if (tid == 0 && a.entropy != nullptr) a.entropy[r] = ok ? logz - ent / sum * kLn2 : nanf;
    for (int i = tid; i < a.n_ids; i += kThreads) {
      const int32_t id = a.ids[r * a.ld_ids + i];
      const bool in = id >= 0 && id < a.V;
      if (!in && a.err != nullptr) atomicOr(a.err, PRISM_DEV_ERR_ID_RANGE);
      float x = 0.0f;
      if (in) x = F32 ? static_cast<const float*>(row)[id] : bf16_bits_to_float(static_cast<const uint16_t*>(row)[id]);
      a.logprobs[r * a.n_ids + i] = ok && in ? (x - m) - logz : nanf;
    }
    if (ok) {
      for (uint32_t i = tid; i < count; i += kThreads) {
        const u64 key = s_list[i];
        int above = 0;
        for (uint32_t j = 0; j < count; ++j) above += s_list[j] > key;
        if (above < a.top_k && key != 0) {
          a.top_ids[r * a.top_k + above] = static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(key));
          a.top_logprobs[r * a.top_k + above] = (key_value(key) - m) - logz;
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
cudaError_t launch_kind(const LogprobArgs& a, int64_t tiles, int ctas, cudaStream_t stream) {
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
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<F32, kHeld>, a, ctas);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t stream) {
  // CTAs of a row: up to four pieces a thread, then up to eight CTAs
  const int64_t tiles = (a.V + kTile - 1) / kTile;
  int ctas = 1;
  while (ctas < kMaxCluster && tiles > 4 * ctas) ctas *= 2;
  const bool held = tiles <= static_cast<int64_t>(kPieces) * ctas;
  if (a.f32) return held ? launch_kind<true, true>(a, tiles, ctas, stream) : launch_kind<true, false>(a, tiles, ctas, stream);
  return held ? launch_kind<false, true>(a, tiles, ctas, stream) : launch_kind<false, false>(a, tiles, ctas, stream);
}

}  // namespace prism
