// linear_w4g.cu -- int8 activations times 4-bit weights with group scales:
//   out[m,n] = bf16(a[m] * sum_g (s[n,g] * sum_{k in g} q[m,k] c[n,k]
//                                 + b[n,g] * sum_{k in g} q[m,k]) + res[m,n])
//
// With few token rows this is a stream of N K / 2 weight bytes (plus 2 or 4
// bytes a group).  The group sums run on mma.sync m16n8k16 with binary16
// operands: 16 output channels are the rows, 8 tokens the columns.  A weight
// word of 8 codes becomes four binary16 pairs, exactly:
//   ((w & 0x000f000f) ^ 0x64086408) - 1032        codes 0, 4 (2, 6 of w >> 8)
//   ((w & 0x00f000f0) ^ 0x64806480) / 16 - 72     codes 1, 5 (3, 7 of w >> 8)
// (the nibble's top bit flipped under the exponent of 1024).  A group's sum is
// an integer below 2^18, so its binary32 accumulator is exact; only the sum
// over the groups rounds, in group order.
//
// A CTA owns 64 or 128 channels (4 or 8 warps x 16) and one slice of K; the CTAs of a
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

// Warps of a CTA: with more token rows each CTA has more activations to lay
// out, so more channels share them (37 rows of 5120 x 34816: four warps 202 us,
// eight 94 us; 8 rows of 17408 x 5120: 30 and 41 us).
template <int T>
constexpr int kWarps = T <= 8 ? 4 : 8;
constexpr int kStageUnits = 8;            // a unit is 32 input channels: 16 bytes of a weight row
constexpr int kPitch = kStageUnits * 16 + 16;   // bytes between the rows of a stage: words r * 36 + c hit all banks once
constexpr int kStageBytes = 16 * kPitch;
constexpr int kStages = 3;
constexpr int kSlabRows = 64;             // token rows of one pass over the weights
constexpr int kMaxPass = 40;              // units of a pass at most: four CTAs of up to 8 rows fit an SM, or two of up to 40
constexpr int kMaxSmem = 128 * 1024;      // of a CTA; layout() stays below

// Shared memory of a CTA.  T: token rows held (1, 2, 4 or a multiple of 8: one
// token's activations take 64 bytes a unit).
struct Layout {
  int pass_units, b, sum, scale, pitch, offset, bytes;
};
template <int T, int GU>
Layout layout(int units, bool has_offset) {
  constexpr int NT = (T + 7) / 8;
  constexpr int kBudget = NT == 1 ? 12288 : NT <= 5 ? NT * 8192 : NT * 4096;   // bytes of activations
  Layout l;
  l.pass_units = std::max(kStageUnits, std::min({kBudget / (T * 64), kMaxPass, units + kStageUnits - 1}) & ~(kStageUnits - 1));
  const int groups = l.pass_units / GU;
  constexpr int kCh = kWarps<T> * 16;
  l.b = kWarps<T> * kStages * kStageBytes;
  l.sum = l.b + l.pass_units * T * 64;
  l.scale = l.sum + (has_offset ? groups * NT * 32 : 0);
  // a row's scales start at an element whose index is a multiple of 8
  l.pitch = (groups + 7 + 7) / 8 * 8 + 8;
  l.offset = l.scale + kCh * l.pitch * 2;
  l.bytes = std::max(l.offset + (has_offset ? kCh * l.pitch * 2 : 0), NT * 8 * kCh * 4);   // and the CTA's sums at the end
  return l;
}

// d = a b where first, else d += a b.
template <bool kFirst>
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kFirst) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}
// The even (odd) codes' pair from a masked weight word.
__device__ __forceinline__ uint32_t even_codes(uint32_t w) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"((w & 0x000f000fu) ^ 0x64086408u), "r"(0x64086408u));   // 1032
  return r;
}
__device__ __forceinline__ uint32_t odd_codes(uint32_t w) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;"
      : "=r"(r)
      : "r"((w & 0x00f000f0u) ^ 0x64806480u), "r"(0x2c002c00u), "r"(0xd480d480u));   // 1/16, -72
  return r;
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

// T: token rows held, NT tiles of 8.  GU: units of a group.  kOff: with offsets.
template <int T, int GU, bool kOff>
__global__ void __launch_bounds__(kWarps<T> * 32, T <= 8 ? 4 : T <= 40 ? 2 : 1)
    w4g_kernel(const __grid_constant__ W4gArgs a, const __grid_constant__ Layout l, int slices, int slice_units) {
  constexpr int NT = (T + 7) / 8, kThreads = kWarps<T> * 32, kCh = kWarps<T> * 16;
  extern __shared__ __align__(128) uint8_t smem[];
  uint4* s_b = reinterpret_cast<uint4*>(smem + l.b);          // [unit][T][4]: the B fragments of a unit
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
  const bool wide = a.lds % 8 == 0 && (reinterpret_cast<uintptr_t>(a.scale) & 15) == 0 &&
                    (!kOff || (a.ldb % 8 == 0 && (reinterpret_cast<uintptr_t>(a.offset) & 15) == 0));

  // ---- this warp's weight ring: 16 rows x 8 units a stage, 16-byte piece
  // i * 32 + lane.  Rows past N repeat the last one and are not stored.
  const uint32_t ring = smem_u32(smem) + warp * kStages * kStageBytes + (lane >> 3) * kPitch + (lane & 7) * 16;
  const uint8_t* wp[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    wp[i] = a.w4 + min(n0 + (lane >> 3) + 4 * i, a.N - 1) * a.ldw4 + (static_cast<int64_t>(u_begin) + (lane & 7)) * 16;
  auto issue = [&](int st) {
    if (st * kStageUnits + (lane & 7) < units) {
      const uint32_t dst = ring + (st % kStages) * kStageBytes;
#pragma unroll
      for (int i = 0; i < 4; ++i) cp_async_16(dst + 4 * i * kPitch, wp[i] + st * (kStageUnits * 16), 16);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int st = 0; st < kStages - 1; ++st) issue(st);

  float y[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) y[t][0] = y[t][1] = y[t][2] = y[t][3] = 0.0f;

  // ---- activations as B fragments: 16 codes of a token are a piece, in the
  // order (group, token, unit, half); a thread's pieces of the next pass are
  // read ahead
  constexpr int kPieces = ((NT == 1 ? 12288 : NT <= 5 ? NT * 8192 : NT * 4096) / 32 + kThreads - 1) / kThreads;
  uint4 w[kPieces];
  auto load_q = [&](int p0) {
    const int total = min(l.pass_units, units - p0) * T * 2;
    const int8_t* q0 = a.q + (static_cast<int64_t>(u_begin) + p0) * 32;
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int i = tid + j * kThreads, half = i & 1, u = (i >> 1) % GU, tok = (i / (2 * GU)) % T, g = i / (2 * GU * T);
      w[j] = make_uint4(0u, 0u, 0u, 0u);
      if (i < total && m0 + tok < a.M)
        w[j] = __ldg(reinterpret_cast<const uint4*>(q0 + (m0 + tok) * a.ldq + (g * GU + u) * 32 + half * 16));
    }
  };
  load_q(0);

  for (int p0 = 0; p0 < units; p0 += l.pass_units) {
    const int pu = min(l.pass_units, units - p0), groups = pu / GU;
    const int g0 = (u_begin + p0) / GU, shift = wide ? g0 & 7 : 0;
    if (p0 > 0) __syncthreads();
    // ---- this pass's scales and offsets of the CTA's channels
    if (wide) {
      // two threads a channel take turns; rows past N repeat the last one
      const int ch = tid >> 1, gw = g0 - shift;
      const int64_t row = min(n_cta + ch, a.N - 1);
      for (int g = (tid & 1) * 8; g < shift + groups; g += 16) {
        const int bytes = min(16, (all_groups - gw - g) * 2);
        cp_async_16(smem_u32(s_scale + ch * l.pitch + g), a.scale + row * a.lds + gw + g, bytes);
        if (kOff) cp_async_16(smem_u32(s_off + ch * l.pitch + g), a.offset + row * a.ldb + gw + g, bytes);
      }
      cp_async_commit();
    } else {
      for (int i = tid; i < kCh * groups; i += kThreads) {
        const int ch = i / groups, g = i - ch * groups;
        if (n_cta + ch < a.N) {
          s_scale[ch * l.pitch + g] = __ldg(a.scale + (n_cta + ch) * a.lds + g0 + g);
          if (kOff) s_off[ch * l.pitch + g] = __ldg(a.offset + (n_cta + ch) * a.ldb + g0 + g);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int i = tid + j * kThreads, half = i & 1, u = (i >> 1) % GU, tok = (i / (2 * GU)) % T, g = i / (2 * GU * T);
      const bool live = i < pu * T * 2;
      if (live) {
        uint4* dst = s_b + ((g * GU + u) * T + tok) * 4 + half * 2;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t u0 = e == 0 ? w[j].x : w[j].z, u1 = e == 0 ? w[j].y : w[j].w;
          const uint32_t x0 = __byte_perm(u0, u1, 0x5140u) ^ 0x80808080u;   // codes 0, 4, 1, 5
          const uint32_t x1 = __byte_perm(u0, u1, 0x7362u) ^ 0x80808080u;   // codes 2, 6, 3, 7
          dst[e] = make_uint4(widen(x0, 0x4140u), widen(x1, 0x4140u), widen(x0, 0x4342u), widen(x1, 0x4342u));
        }
      }
      if constexpr (kOff) {   // the group's sum of q: its 2 GU pieces lie in neighbouring lanes
        int sum = __dp4a(static_cast<int>(w[j].x), 0x01010101, __dp4a(static_cast<int>(w[j].y), 0x01010101, 0));
        sum = __dp4a(static_cast<int>(w[j].z), 0x01010101, __dp4a(static_cast<int>(w[j].w), 0x01010101, sum));
#pragma unroll
        for (int o = 1; o < 2 * GU; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (live && half == 0 && u == 0) s_sum[g * (NT * 8) + tok] = static_cast<float>(sum);
      }
    }
    cp_async_wait<0>();
    __syncthreads();
    if (p0 + l.pass_units < units) load_q(p0 + l.pass_units);

    // ---- a unit: 2 weight words of a lane (rows r, r + 8), 2 NT instructions
    const int bl = T < 8 ? min(lr, T - 1) : lr;   // a column past the tokens repeats the last one and is not stored
    const uint16_t* sp = s_scale + (warp * 16 + lr) * l.pitch + shift;
    const uint16_t* op = s_off + (warp * 16 + lr) * l.pitch + shift;
    float acc[NT][4];
    auto unit = [&](const uint8_t* wb, int ul, int g, auto first, auto last) {   // unit ul of group g in this pass
      const uint32_t w0 = *reinterpret_cast<const uint32_t*>(wb);
      const uint32_t w1 = *reinterpret_cast<const uint32_t*>(wb + 8 * kPitch);
      const uint32_t ae[4] = {even_codes(w0), even_codes(w1), even_codes(w0 >> 8), even_codes(w1 >> 8)};
      const uint32_t ao[4] = {odd_codes(w0), odd_codes(w1), odd_codes(w0 >> 8), odd_codes(w1 >> 8)};
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint4 b = s_b[(ul * T + t * 8 + bl) * 4 + lc];
        mma_f16_16816<decltype(first)::value>(acc[t], ae, b.x, b.y);
        mma_f16_16816<false>(acc[t], ao, b.z, b.w);
      }
      if constexpr (decltype(last)::value) {
        const float s0 = half_bits_to_float(sp[g]), s1 = half_bits_to_float(sp[8 * l.pitch + g]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          y[t][0] = __fmaf_rn(acc[t][0], s0, y[t][0]);
          y[t][1] = __fmaf_rn(acc[t][1], s0, y[t][1]);
          y[t][2] = __fmaf_rn(acc[t][2], s1, y[t][2]);
          y[t][3] = __fmaf_rn(acc[t][3], s1, y[t][3]);
        }
        if constexpr (kOff) {
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
    auto group = [&](const uint8_t* wb, int ul, int g) {
#pragma unroll
      for (int u = 0; u < GU; ++u) {
        if constexpr (GU == 1) {
          unit(wb, ul, g, std::true_type{}, std::true_type{});
        } else if (u == 0) {
          unit(wb, ul, g, std::true_type{}, std::false_type{});
        } else if (u == GU - 1) {
          unit(wb + u * 16, ul + u, g, std::false_type{}, std::true_type{});
        } else {
          unit(wb + u * 16, ul + u, g, std::false_type{}, std::false_type{});
        }
      }
    };
    const int st0 = p0 / kStageUnits, st_end = (p0 + pu + kStageUnits - 1) / kStageUnits;
    for (int st = st0; st < st_end; ++st) {
      issue(st + kStages - 1);
      cp_async_wait<kStages - 1>();
      __syncwarp();
      const uint8_t* wb = smem + (warp * kStages + st % kStages) * kStageBytes + lr * kPitch + lc * 4;
      const int ul = (st - st0) * kStageUnits, gl = (st - st0) * (kStageUnits / GU), n = pu - ul;
      if (n >= kStageUnits) {
#pragma unroll
        for (int u = 0; u < kStageUnits; u += GU) group(wb + u * 16, ul + u, gl + u / GU);
      } else {
        for (int u = 0; u < n; u += GU) group(wb + u * 16, ul + u, gl + u / GU);
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

template <int T, int GU, bool kOff>
cudaError_t launch_t(const W4gArgs& a, cudaStream_t stream) {
  // Slices of K: as many as let four CTAs of 64 channels on every SM run at
  // once, at most a cluster of eight; whole groups of any size (4 units) each.
  // A rule on N, K and the group alone: a row's sums do not depend on M.
  constexpr int kCh = kWarps<T> * 16;
  const int64_t tiles = (a.N + kCh - 1) / kCh, tiles64 = (a.N + 63) / 64;
  const int units = static_cast<int>(a.K >> 5);
  const int slices = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({4 * sm_count() / tiles64, 8, (units + 3) / 4})));
  const int slice_units = ((units + slices - 1) / slices + 3) & ~3;
  const Layout l = layout<T, GU>(slice_units, kOff);
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(w4g_kernel<T, GU, kOff>), kMaxSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * slices), static_cast<unsigned>((a.M + kSlabRows - 1) / kSlabRows));
  cfg.blockDim = dim3(kWarps<T> * 32);
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
  return cudaLaunchKernelEx(&cfg, w4g_kernel<T, GU, kOff>, a, l, slices, slice_units);
}

template <int GU, bool kOff>
cudaError_t launch_gu(const W4gArgs& a, cudaStream_t stream) {
  if (a.M <= 1) return launch_t<1, GU, kOff>(a, stream);
  if (a.M <= 2) return launch_t<2, GU, kOff>(a, stream);
  if (a.M <= 4) return launch_t<4, GU, kOff>(a, stream);
  if (a.M <= 8) return launch_t<8, GU, kOff>(a, stream);
  if (a.M <= 16) return launch_t<16, GU, kOff>(a, stream);
  if (a.M <= 24) return launch_t<24, GU, kOff>(a, stream);
  if (a.M <= 40) return launch_t<40, GU, kOff>(a, stream);
  return launch_t<64, GU, kOff>(a, stream);
}

template <bool kOff>
cudaError_t launch_off(const W4gArgs& a, cudaStream_t stream) {
  return a.group == 32   ? launch_gu<1, kOff>(a, stream)
         : a.group == 64 ? launch_gu<2, kOff>(a, stream)
                         : launch_gu<4, kOff>(a, stream);
}

}  // namespace

cudaError_t launch_w4g(const W4gArgs& a, cudaStream_t stream) {
  return a.offset != nullptr ? launch_off<true>(a, stream) : launch_off<false>(a, stream);
}

}  // namespace prism
