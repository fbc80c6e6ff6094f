// linear_w4g.cu -- int8 activations times 4-bit weights with group scales:
//   out[m,n] = bf16(a[m] * sum_g (s[n,g] * sum_{k in g} q[m,k] c[n,k]
//                                 + b[n,g] * sum_{k in g} q[m,k]) + res[m,n])
//
// With few token rows this is a stream of N K / 2 weight bytes (plus 2 or 4
// bytes a group).  The group sums run on mma.sync m16n8k16 with binary16
// operands: 16 output channels are the rows, 8 tokens the columns.  A weight
// word of 8 codes becomes four binary16 pairs by (w & mask) ^ magic alone:
//   (w & 0x000f000f) ^ 0x64086408  =  1024 + (code + 8)        codes 0, 4 (2, 6 of w >> 8)
//   (w & 0x00f000f0) ^ 0x64806480  =  1024 + 16 (code + 8)     codes 1, 5 (3, 7 of w >> 8)
// and the constants are taken off exactly by starting the sums at
// -1032 sum q_even and -1152 sum q_odd.  Every partial sum is an integer
// below 2^24 (1152 * 127 * 64 for a group of 128), so the binary32
// accumulators are exact: sum_{k in g} q c = even + odd / 16.  Only the sum
// over the groups rounds, in group order.
//
// A CTA owns 64 channels (4 warps x 16) and one slice of K; the CTAs of a
// cluster hold the slices of one channel tile and add their sums through
// distributed shared memory in slice order.  The activations of up to
// kPassUnits * 32 channels at a time are widened once per CTA, in the order
// that the weight words want; each warp streams its weight rows through a
// private ring of cp.async copies (128 bytes of a row a step).
#include "decode.cuh"

namespace prism {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kCh = kWarps * 16;          // output channels of a CTA
constexpr int kStageUnits = 8;            // a unit is 32 input channels: 16 bytes of a weight row
constexpr int kPitch = kStageUnits * 16 + 16;   // bytes between the rows of a stage: words r * 36 + c hit all banks once
constexpr int kStageBytes = 16 * kPitch;
constexpr int kStages = 4;
constexpr int kSlabRows = 64;             // token rows of one pass over the weights

// Units whose activations are held at a time: 16 to 48 KB of shared memory.
template <int NT>
constexpr int kPassUnits = NT <= 2 ? 32 : NT <= 6 ? 16 : 8;

template <int NT, int GU>
struct Layout {
  static constexpr int kUnits = kPassUnits<NT>;
  static constexpr int kGroups = kUnits / GU;
  static constexpr int kScalePitch = kGroups + 8;                 // binary16 elements
  static constexpr int kRing = kWarps * kStages * kStageBytes;    // and the sums of the CTA at the end
  static constexpr int kB = kUnits * NT * 512;
  static constexpr int kInit = kGroups * NT * 8 * 8;              // (even, odd) start values of 8 tokens
  static constexpr int kSum = kGroups * NT * 8 * 4;
  static constexpr int kScale = kCh * kScalePitch * 2;
  static constexpr int kBytes = kRing + kB + kInit + kSum + 2 * kScale;
  static_assert(kRing >= NT * 8 * kCh * 4, "the sums fit into the ring");
};

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Bytes 0, 1 (sel 0x4140) or 2, 3 (sel 0x4342) of codes ^ 0x80 as a binary16 pair, exact.
__device__ __forceinline__ uint32_t widen(uint32_t biased, uint32_t sel) {
  const uint32_t h = __byte_perm(biased, 0x64646464u, sel);
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(0x64806480u));   // 1024 + 128
  return r;
}
__device__ __forceinline__ float half_bits_to_float(uint16_t h) {
  float f;
  asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(h));
  return f;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr, uint32_t rank) {
  uint32_t remote;
  float v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
  return v;
}

// NT: tiles of 8 token rows.  GU: units of a group.
template <int NT, int GU>
__global__ void __launch_bounds__(kThreads) w4g_kernel(const __grid_constant__ W4gArgs a, int slices, int slice_units) {
  using L = Layout<NT, GU>;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* s_b = smem + L::kRing;
  float2* s_init = reinterpret_cast<float2*>(s_b + L::kB);
  float* s_sum = reinterpret_cast<float*>(s_b + L::kB + L::kInit);
  uint16_t* s_scale = reinterpret_cast<uint16_t*>(s_b + L::kB + L::kInit + L::kSum);
  uint16_t* s_off = s_scale + kCh * L::kScalePitch;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lr = lane >> 2, lc = lane & 3;
  const int rank = blockIdx.x % slices;
  const int64_t n_cta = static_cast<int64_t>(blockIdx.x / slices) * kCh, n0 = n_cta + warp * 16;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kSlabRows;
  const int all_units = static_cast<int>(a.K >> 5);
  const int u_begin = min(rank * slice_units, all_units);
  const int units = min(slice_units, all_units - u_begin);
  const bool has_off = a.offset != nullptr;

  // ---- this warp's weight ring: 16 rows x 8 units a stage, 16-byte piece i * 32 + lane
  const uint32_t ring = smem_u32(smem) + warp * kStages * kStageBytes;
  const uint8_t* wp = a.w4 + (n0 + (lane >> 3)) * a.ldw4 + (static_cast<int64_t>(u_begin) + (lane & 7)) * 16;
  auto issue = [&](int st) {
    if (st * kStageUnits < units) {
      const uint32_t dst = ring + (st % kStages) * kStageBytes + (lane >> 3) * kPitch + (lane & 7) * 16;
      const bool in = st * kStageUnits + (lane & 7) < units;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool live = in && n0 + (lane >> 3) + 4 * i < a.N;
        cp_async_16(dst + 4 * i * kPitch, live ? wp + 4 * i * a.ldw4 + st * (kStageUnits * 16) : a.w4, live ? 16 : 0);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int st = 0; st < kStages - 1; ++st) issue(st);

  float y[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) y[t][0] = y[t][1] = y[t][2] = y[t][3] = 0.0f;

  for (int p0 = 0; p0 < units; p0 += L::kUnits) {
    const int groups = min(L::kUnits, units - p0) / GU;
    if (p0 > 0) __syncthreads();
    // ---- activations of this pass as B fragments, and their sums by group
    for (int i = warp; i < groups * NT; i += kWarps) {
      const int g = i / NT, t = i - g * NT;
      const int64_t m = m0 + t * 8 + lr;
      const int8_t* qp = a.q + m * a.ldq + (static_cast<int64_t>(u_begin) + p0 + g * GU) * 32 + lc * 8;
      uint2 w[GU];
#pragma unroll
      for (int u = 0; u < GU; ++u) w[u] = m < a.M ? __ldg(reinterpret_cast<const uint2*>(qp + u * 32)) : make_uint2(0u, 0u);
      int even = 0, odd = 0;
#pragma unroll
      for (int u = 0; u < GU; ++u) {
        even = __dp4a(static_cast<int>(w[u].x), 0x00010001, __dp4a(static_cast<int>(w[u].y), 0x00010001, even));
        odd = __dp4a(static_cast<int>(w[u].x), 0x01000100, __dp4a(static_cast<int>(w[u].y), 0x01000100, odd));
        const uint32_t x0 = __byte_perm(w[u].x, w[u].y, 0x5140u) ^ 0x80808080u;   // codes 0, 4, 1, 5
        const uint32_t x1 = __byte_perm(w[u].x, w[u].y, 0x7362u) ^ 0x80808080u;   // codes 2, 6, 3, 7
        *reinterpret_cast<uint4*>(s_b + ((g * GU + u) * NT + t) * 512 + lane * 16) =
            make_uint4(widen(x0, 0x4140u), widen(x1, 0x4140u), widen(x0, 0x4342u), widen(x1, 0x4342u));
      }
      even += __shfl_xor_sync(0xffffffffu, even, 1);
      odd += __shfl_xor_sync(0xffffffffu, odd, 1);
      even += __shfl_xor_sync(0xffffffffu, even, 2);
      odd += __shfl_xor_sync(0xffffffffu, odd, 2);
      if (lc == 0) {
        s_init[i * 8 + lr] = make_float2(static_cast<float>(-1032 * even), static_cast<float>(-1152 * odd));
        s_sum[i * 8 + lr] = static_cast<float>(even + odd);
      }
    }
    // ---- this pass's scales and offsets of the CTA's channels
    {
      const int64_t g0 = (u_begin + p0) / GU;
      for (int i = tid; i < kCh * L::kGroups; i += kThreads) {
        const int ch = i / L::kGroups, g = i % L::kGroups;
        if (g < groups && n_cta + ch < a.N) {
          s_scale[ch * L::kScalePitch + g] = __ldg(a.scale + (n_cta + ch) * a.lds + g0 + g);
          if (has_off) s_off[ch * L::kScalePitch + g] = __ldg(a.offset + (n_cta + ch) * a.ldb + g0 + g);
        }
      }
    }
    __syncthreads();
    const int st_end = (p0 + groups * GU + kStageUnits - 1) / kStageUnits;
    for (int st = p0 / kStageUnits; st < st_end; ++st) {
      issue(st + kStages - 1);
      cp_async_wait<kStages - 1>();
      __syncwarp();
      const uint8_t* wb = smem + (warp * kStages + st % kStages) * kStageBytes + lr * kPitch + lc * 4;
      const int ul = st * kStageUnits - p0;      // the stage's first unit in this pass
      float acc_e[NT][4], acc_o[NT][4];
#pragma unroll
      for (int u = 0; u < kStageUnits; ++u) {
        if (ul + u >= groups * GU) break;
        const uint32_t w0 = *reinterpret_cast<const uint32_t*>(wb + u * 16);
        const uint32_t w1 = *reinterpret_cast<const uint32_t*>(wb + 8 * kPitch + u * 16);
        const uint32_t h0 = w0 >> 8, h1 = w1 >> 8;
        const uint32_t ae[4] = {(w0 & 0x000f000fu) ^ 0x64086408u, (w1 & 0x000f000fu) ^ 0x64086408u,
                                (h0 & 0x000f000fu) ^ 0x64086408u, (h1 & 0x000f000fu) ^ 0x64086408u};
        const uint32_t ao[4] = {(w0 & 0x00f000f0u) ^ 0x64806480u, (w1 & 0x00f000f0u) ^ 0x64806480u,
                                (h0 & 0x00f000f0u) ^ 0x64806480u, (h1 & 0x00f000f0u) ^ 0x64806480u};
        const int g = (ul + u) / GU;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint4 b = *reinterpret_cast<const uint4*>(s_b + ((ul + u) * NT + t) * 512 + lane * 16);
          if (u % GU == 0) {
            const float4 c = *reinterpret_cast<const float4*>(s_init + (g * NT + t) * 8 + 2 * lc);
            acc_e[t][0] = acc_e[t][2] = c.x;
            acc_o[t][0] = acc_o[t][2] = c.y;
            acc_e[t][1] = acc_e[t][3] = c.z;
            acc_o[t][1] = acc_o[t][3] = c.w;
          }
          mma_f16_16816(acc_e[t], ae, b.x, b.y);
          mma_f16_16816(acc_o[t], ao, b.z, b.w);
        }
        if (u % GU == GU - 1) {
          const uint16_t* sp = s_scale + (warp * 16 + lr) * L::kScalePitch + g;
          const float s0 = half_bits_to_float(sp[0]), s1 = half_bits_to_float(sp[8 * L::kScalePitch]);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            y[t][0] = __fmaf_rn(__fmaf_rn(acc_o[t][0], 0.0625f, acc_e[t][0]), s0, y[t][0]);
            y[t][1] = __fmaf_rn(__fmaf_rn(acc_o[t][1], 0.0625f, acc_e[t][1]), s0, y[t][1]);
            y[t][2] = __fmaf_rn(__fmaf_rn(acc_o[t][2], 0.0625f, acc_e[t][2]), s1, y[t][2]);
            y[t][3] = __fmaf_rn(__fmaf_rn(acc_o[t][3], 0.0625f, acc_e[t][3]), s1, y[t][3]);
          }
          if (has_off) {
            const uint16_t* op = s_off + (warp * 16 + lr) * L::kScalePitch + g;
            const float o0 = half_bits_to_float(op[0]), o1 = half_bits_to_float(op[8 * L::kScalePitch]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const float2 q = *reinterpret_cast<const float2*>(s_sum + (g * NT + t) * 8 + 2 * lc);
              y[t][0] = __fmaf_rn(q.x, o0, y[t][0]);
              y[t][1] = __fmaf_rn(q.y, o0, y[t][1]);
              y[t][2] = __fmaf_rn(q.x, o1, y[t][2]);
              y[t][3] = __fmaf_rn(q.y, o1, y[t][3]);
            }
          }
        }
      }
      __syncwarp();   // the stage is free for the copy that the next turn issues
    }
  }

  // ---- the slices' sums, added in slice order by the CTAs of the cluster
  cp_async_wait<0>();
  __syncthreads();
  float* s_y = reinterpret_cast<float*>(smem);   // [token][channel]
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) s_y[(t * 8 + 2 * lc + (e & 1)) * kCh + warp * 16 + lr + 8 * (e >> 1)] = y[t][e];
  cluster_sync();
  const int rows = static_cast<int>(min(static_cast<int64_t>(NT * 8), a.M - m0));
  for (int i = rank * kThreads + tid; i < rows * kCh; i += slices * kThreads) {
    const int64_t m = m0 + i / kCh, n = n_cta + i % kCh;
    const uint32_t at = smem_u32(s_y + i);
    float v = 0.0f;
    for (int r = 0; r < slices; ++r) v = __fadd_rn(v, ld_cluster(at, r));
    if (n < a.N) {
      v = __fmul_rn(v, __ldg(a.a_scale + m));
      if (a.residual != nullptr) v = __fadd_rn(v, bf16_bits_to_float(a.residual[m * a.ldr + n]));
      a.out[m * a.ldo + n] = static_cast<uint16_t>(float_to_bf16_rne(v));
    }
  }
  cluster_sync();   // no CTA leaves while its sums are read
}

template <int NT, int GU>
cudaError_t launch_nt(const W4gArgs& a, cudaStream_t stream) {
  constexpr int smem = Layout<NT, GU>::kBytes;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(w4g_kernel<NT, GU>), smem);
  if (e != cudaSuccess) return e;
  // Slices of K: eight where the channel tiles alone leave SMs idle, else
  // four; whole groups of any size (4 units) each.
  const int64_t tiles = (a.N + kCh - 1) / kCh;
  const int slices = tiles * 4 < 2 * sm_count() ? 8 : 4;
  const int units = static_cast<int>(a.K >> 5);
  const int slice_units = ((units + slices - 1) / slices + 3) & ~3;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * slices), static_cast<unsigned>((a.M + kSlabRows - 1) / kSlabRows));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(slices);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, w4g_kernel<NT, GU>, a, slices, slice_units);
}

template <int GU>
cudaError_t launch_gu(const W4gArgs& a, cudaStream_t stream) {
  if (a.M <= 8) return launch_nt<1, GU>(a, stream);
  if (a.M <= 16) return launch_nt<2, GU>(a, stream);
  if (a.M <= 24) return launch_nt<3, GU>(a, stream);
  if (a.M <= 32) return launch_nt<4, GU>(a, stream);
  if (a.M <= 48) return launch_nt<6, GU>(a, stream);
  return launch_nt<8, GU>(a, stream);
}

}  // namespace

cudaError_t launch_w4g(const W4gArgs& a, cudaStream_t stream) {
  return a.group == 32 ? launch_gu<1>(a, stream) : a.group == 64 ? launch_gu<2>(a, stream) : launch_gu<4>(a, stream);
}

}  // namespace prism
