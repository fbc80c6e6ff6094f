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
// distributed shared memory in slice order.  The activations and scales of up
// to pass_units * 32 input channels at a time are laid into shared memory, the
// activations widened once per CTA in the order that the weight words want;
// each warp streams its weight rows through a private ring of cp.async copies
// (128 bytes of a row a step).
#include <type_traits>

#include "decode.cuh"

namespace prism {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kCh = kWarps * 16;          // output channels of a CTA
constexpr int kStageUnits = 8;            // a unit is 32 input channels: 16 bytes of a weight row
constexpr int kPitch = kStageUnits * 16 + 16;   // bytes between the rows of a stage: words r * 36 + c hit all banks once
constexpr int kStageBytes = 16 * kPitch;
constexpr int kStages = 3;
constexpr int kSlabRows = 64;             // token rows of one pass over the weights
constexpr int kRing = kWarps * kStages * kStageBytes;
constexpr int kMaxPass = 40;              // units of a pass at most: four CTAs of up to 8 rows fit an SM
constexpr int kMaxSmem = 96 * 1024;       // of a CTA; layout() stays below

// Shared memory of a CTA.  T: token rows held (M itself up to 8, so that one
// token's activations take 64 bytes a unit).
struct Layout {
  int pass_units, b, init, sum, scale, pitch, offset, bytes;
};
template <int NT, int GU>
Layout layout(int64_t M, int units, bool has_offset) {
  const int T = NT == 1 ? static_cast<int>(M) : NT * 8;
  constexpr int kBudget = NT == 1 ? 12288 : NT <= 5 ? NT * 8192 : NT * 4096;   // bytes of activations
  Layout l;
  l.pass_units = std::max(kStageUnits, std::min({kBudget / (T * 64), kMaxPass, units + kStageUnits - 1}) & ~(kStageUnits - 1));
  const int groups = l.pass_units / GU;
  l.b = kRing;
  l.init = l.b + l.pass_units * T * 64;
  l.sum = l.init + groups * NT * 64;
  l.scale = l.sum + groups * NT * 32;
  // a row's scales start at an element whose index is a multiple of 8
  l.pitch = (groups + 7 + 7) / 8 * 8 + 8;
  l.offset = l.scale + kCh * l.pitch * 2;
  l.bytes = std::max(l.offset + (has_offset ? kCh * l.pitch * 2 : 0), NT * 8 * kCh * 4);   // and the CTA's sums at the end
  return l;
}

// d = a b + c, with c given per column pair (the same for both row halves) where first.
template <bool kFirst>
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                              float c1) {
  if (kFirst) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
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
__global__ void __launch_bounds__(kThreads, NT == 1 ? 4 : NT <= 3 ? 3 : 2)
    w4g_kernel(const __grid_constant__ W4gArgs a, const __grid_constant__ Layout l, int slices, int slice_units) {
  extern __shared__ __align__(128) uint8_t smem[];
  uint4* s_b = reinterpret_cast<uint4*>(smem + l.b);          // [unit][T][4]: the B fragments of a unit
  float2* s_init = reinterpret_cast<float2*>(smem + l.init);  // [group][NT * 8]: start values (even, odd)
  float* s_sum = reinterpret_cast<float*>(smem + l.sum);      // [group][NT * 8]: sum of q
  uint16_t* s_scale = reinterpret_cast<uint16_t*>(smem + l.scale);
  uint16_t* s_off = reinterpret_cast<uint16_t*>(smem + l.offset);
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lr = lane >> 2, lc = lane & 3;
  const int rank = blockIdx.x % slices;
  const int64_t n_cta = static_cast<int64_t>(blockIdx.x / slices) * kCh, n0 = n_cta + warp * 16;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kSlabRows;
  const int all_units = static_cast<int>(a.K >> 5), all_groups = all_units / GU;
  const int u_begin = min(rank * slice_units, all_units);
  const int units = min(slice_units, all_units - u_begin);
  const int T = NT == 1 ? static_cast<int>(a.M) : NT * 8;
  const bool has_off = a.offset != nullptr;
  const bool wide = a.lds % 8 == 0 && (reinterpret_cast<uintptr_t>(a.scale) & 15) == 0 &&
                    (!has_off || (a.ldb % 8 == 0 && (reinterpret_cast<uintptr_t>(a.offset) & 15) == 0));

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

  for (int p0 = 0; p0 < units; p0 += l.pass_units) {
    const int pu = min(l.pass_units, units - p0), groups = pu / GU;
    const int g0 = (u_begin + p0) / GU, shift = wide ? g0 & 7 : 0;
    if (p0 > 0) __syncthreads();
    // ---- this pass's scales and offsets of the CTA's channels
    if (wide) {
      const int per_row = (shift + groups + 7) >> 3;
      for (int i = tid; i < kCh * per_row; i += kThreads) {
        const int ch = i / per_row, g = (i - ch * per_row) * 8;
        const int bytes = n_cta + ch < a.N ? min(16, (all_groups - (g0 - shift) - g) * 2) : 0;
        const uint32_t at = ch * l.pitch + g;
        const int64_t row = bytes > 0 ? n_cta + ch : 0, col = bytes > 0 ? g0 - shift + g : 0;
        cp_async_16(smem_u32(s_scale + at), a.scale + row * a.lds + col, bytes);
        if (has_off) cp_async_16(smem_u32(s_off + at), a.offset + row * a.ldb + col, bytes);
      }
      cp_async_commit();
    } else {
      for (int i = tid; i < kCh * groups; i += kThreads) {
        const int ch = i / groups, g = i - ch * groups;
        if (n_cta + ch < a.N) {
          s_scale[ch * l.pitch + g] = __ldg(a.scale + (n_cta + ch) * a.lds + g0 + g);
          if (has_off) s_off[ch * l.pitch + g] = __ldg(a.offset + (n_cta + ch) * a.ldb + g0 + g);
        }
      }
    }
    // ---- activations of this pass as B fragments, four pieces of a thread in flight
    const int total = pu * T * 4;
    const int8_t* q0 = a.q + (static_cast<int64_t>(u_begin) + p0) * 32;
    for (int i0 = tid; i0 < total; i0 += 4 * kThreads) {
      uint2 w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + j * kThreads, unit = (i >> 2) / T, tok = (i >> 2) - unit * T;
        w[j] = i < total && m0 + tok < a.M
                   ? __ldg(reinterpret_cast<const uint2*>(q0 + (m0 + tok) * a.ldq + unit * 32 + lc * 8))
                   : make_uint2(0u, 0u);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + j * kThreads;
        const uint32_t x0 = __byte_perm(w[j].x, w[j].y, 0x5140u) ^ 0x80808080u;   // codes 0, 4, 1, 5
        const uint32_t x1 = __byte_perm(w[j].x, w[j].y, 0x7362u) ^ 0x80808080u;   // codes 2, 6, 3, 7
        if (i < total) s_b[i] = make_uint4(widen(x0, 0x4140u), widen(x1, 0x4140u), widen(x0, 0x4342u), widen(x1, 0x4342u));
      }
    }
    // ---- and their sums by group
    for (int i = tid; i < groups * T; i += kThreads) {
      const int g = i / T, tok = i - g * T;
      int even = 0, odd = 0;
      if (m0 + tok < a.M) {
        const uint4* qp = reinterpret_cast<const uint4*>(q0 + (m0 + tok) * a.ldq + g * (GU * 32));
#pragma unroll
        for (int j = 0; j < 2 * GU; ++j) {
          const uint4 v = __ldg(qp + j);
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            even = __dp4a(static_cast<int>(u[e]), 0x00010001, even);
            odd = __dp4a(static_cast<int>(u[e]), 0x01000100, odd);
          }
        }
      }
      s_init[g * (NT * 8) + tok] = make_float2(static_cast<float>(-1032 * even), static_cast<float>(-1152 * odd));
      s_sum[g * (NT * 8) + tok] = static_cast<float>(even + odd);
    }
    cp_async_wait<0>();
    __syncthreads();

    // ---- a unit: 2 weight words of a lane (rows r, r + 8), 2 NT instructions
    const int bl = NT == 1 ? min(lr, T - 1) : lr;   // a column past the tokens repeats the last one and is not stored
    const uint16_t* sp = s_scale + (warp * 16 + lr) * l.pitch + shift;
    const uint16_t* op = s_off + (warp * 16 + lr) * l.pitch + shift;
    float acc_e[NT][4], acc_o[NT][4];
    auto unit = [&](const uint8_t* wb, int ul, auto first, auto last) {   // ul: the unit in this pass
      const uint32_t w0 = *reinterpret_cast<const uint32_t*>(wb);
      const uint32_t w1 = *reinterpret_cast<const uint32_t*>(wb + 8 * kPitch);
      const uint32_t h0 = w0 >> 8, h1 = w1 >> 8;
      const uint32_t ae[4] = {(w0 & 0x000f000fu) ^ 0x64086408u, (w1 & 0x000f000fu) ^ 0x64086408u,
                              (h0 & 0x000f000fu) ^ 0x64086408u, (h1 & 0x000f000fu) ^ 0x64086408u};
      const uint32_t ao[4] = {(w0 & 0x00f000f0u) ^ 0x64806480u, (w1 & 0x00f000f0u) ^ 0x64806480u,
                              (h0 & 0x00f000f0u) ^ 0x64806480u, (h1 & 0x00f000f0u) ^ 0x64806480u};
      const int g = ul / GU;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint4 b = s_b[(ul * T + t * 8 + bl) * 4 + lc];
        float4 c = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if constexpr (decltype(first)::value) c = *reinterpret_cast<const float4*>(s_init + g * (NT * 8) + t * 8 + 2 * lc);
        mma_f16_16816<decltype(first)::value>(acc_e[t], ae, b.x, b.y, c.x, c.z);
        mma_f16_16816<decltype(first)::value>(acc_o[t], ao, b.z, b.w, c.y, c.w);
      }
      if constexpr (decltype(last)::value) {
        const float s0 = half_bits_to_float(sp[g]), s1 = half_bits_to_float(sp[8 * l.pitch + g]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          y[t][0] = __fmaf_rn(__fmaf_rn(acc_o[t][0], 0.0625f, acc_e[t][0]), s0, y[t][0]);
          y[t][1] = __fmaf_rn(__fmaf_rn(acc_o[t][1], 0.0625f, acc_e[t][1]), s0, y[t][1]);
          y[t][2] = __fmaf_rn(__fmaf_rn(acc_o[t][2], 0.0625f, acc_e[t][2]), s1, y[t][2]);
          y[t][3] = __fmaf_rn(__fmaf_rn(acc_o[t][3], 0.0625f, acc_e[t][3]), s1, y[t][3]);
        }
        if (has_off) {
          const float o0 = half_bits_to_float(op[g]), o1 = half_bits_to_float(op[8 * l.pitch + g]);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const float2 q = *reinterpret_cast<const float2*>(s_sum + g * (NT * 8) + t * 8 + 2 * lc);
            y[t][0] = __fmaf_rn(q.x, o0, y[t][0]);
            y[t][1] = __fmaf_rn(q.y, o0, y[t][1]);
            y[t][2] = __fmaf_rn(q.x, o1, y[t][2]);
            y[t][3] = __fmaf_rn(q.y, o1, y[t][3]);
          }
        }
      }
    };
    auto group = [&](const uint8_t* wb, int ul) {
#pragma unroll
      for (int u = 0; u < GU; ++u) {
        if constexpr (GU == 1) {
          unit(wb, ul, std::true_type{}, std::true_type{});
        } else if (u == 0) {
          unit(wb, ul, std::true_type{}, std::false_type{});
        } else if (u == GU - 1) {
          unit(wb + u * 16, ul + u, std::false_type{}, std::true_type{});
        } else {
          unit(wb + u * 16, ul + u, std::false_type{}, std::false_type{});
        }
      }
    };
    const int st0 = p0 / kStageUnits, st_end = (p0 + pu + kStageUnits - 1) / kStageUnits;
    for (int st = st0; st < st_end; ++st) {
      issue(st + kStages - 1);
      cp_async_wait<kStages - 1>();
      __syncwarp();
      const uint8_t* wb = smem + (warp * kStages + st % kStages) * kStageBytes + lr * kPitch + lc * 4;
      const int ul = (st - st0) * kStageUnits, n = pu - ul;
      if (n >= kStageUnits) {
#pragma unroll
        for (int u = 0; u < kStageUnits; u += GU) group(wb + u * 16, ul + u);
      } else {
        for (int u = 0; u < n; u += GU) group(wb + u * 16, ul + u);
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
  // Slices of K: as many as let every CTA run at once (four on an SM), at
  // most a cluster of eight; whole groups of any size (4 units) each.
  const int64_t tiles = (a.N + kCh - 1) / kCh;
  const int units = static_cast<int>(a.K >> 5);
  const int slices = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({4 * sm_count() / tiles, 8, (units + 3) / 4})));
  const int slice_units = ((units + slices - 1) / slices + 3) & ~3;
  const Layout l = layout<NT, GU>(a.M, slice_units, a.offset != nullptr);
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(w4g_kernel<NT, GU>), kMaxSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * slices), static_cast<unsigned>((a.M + kSlabRows - 1) / kSlabRows));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(l.bytes);
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
  return cudaLaunchKernelEx(&cfg, w4g_kernel<NT, GU>, a, l, slices, slice_units);
}

template <int GU>
cudaError_t launch_gu(const W4gArgs& a, cudaStream_t stream) {
  if (a.M <= 8) return launch_nt<1, GU>(a, stream);
  if (a.M <= 16) return launch_nt<2, GU>(a, stream);
  if (a.M <= 24) return launch_nt<3, GU>(a, stream);
  if (a.M <= 32) return launch_nt<4, GU>(a, stream);
  if (a.M <= 40) return launch_nt<5, GU>(a, stream);
  if (a.M <= 48) return launch_nt<6, GU>(a, stream);
  return launch_nt<8, GU>(a, stream);
}

}  // namespace

cudaError_t launch_w4g(const W4gArgs& a, cudaStream_t stream) {
  return a.group == 32 ? launch_gu<1>(a, stream) : a.group == 64 ? launch_gu<2>(a, stream) : launch_gu<4>(a, stream);
}

}  // namespace prism
