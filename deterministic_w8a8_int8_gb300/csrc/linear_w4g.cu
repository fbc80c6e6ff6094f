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
// A CTA owns 64 channels (up to 8 rows) or 128 and one slice of K; the CTAs of a
// cluster hold the slices of one channel tile and add their sums through
// distributed shared memory in slice order.  The weights pass through a ring in
// shared memory (128 bytes of a row a step); the activations are widened once
// per CTA into shared memory, in the order that the weight words want.
//
// Up to 8 rows no unit is full: half of the issue slots are taken (a weight word
// costs nine instructions for eight codes), HBM is at 28 to 50 %, and the stalls
// are at barriers and on loads -- each pass waits for its own scales at its head
// and with them for all of the ring (8 rows of 17408 x 5120 21.8 us; 5120 x 34816,
// one row, rings of 3, 4, 5 stages: 25.4, 26.7, 27.6 us, 3.5 TB/s of weights).
// With more rows the instructions themselves (608 TFLOP/s at best) take 42 % of
// the time and the slots 48 %, the contracting warps (two a scheduler) waiting at
// barriers: 37 rows of 5120 x 34816 take 61 us.  More than 64 rows stream and widen
// the weights again for every 64 (256 rows 353 us).  The same on
// tcgen05 (weights widened into swizzled shared memory, group sums read back from
// tensor memory) took 75 us, and 50 us against 36 with 12 rows: every weight then
// passes through shared memory twice.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "decode.cuh"
#include "tc_common.cuh"

namespace prism {

__device__ uint32_t g_w4g_status = 0;
// Test mode (prism_debug_wait_expiry): the waits' limit, and whether a laying thread
// of each CTA withholds its arrival for the first chunk until the CTA has run out.
__device__ unsigned long long g_w4g_wait_limit_ns = 2000000000ull;
__device__ int g_w4g_withhold = 0;

namespace {

constexpr unsigned long long kDrainNs = 2000000000ull;

constexpr int kWarps = 4, kThreads = kWarps * 32, kCh = kWarps * 16;   // of a CTA with up to 8 rows; its channels
constexpr int kStageUnits = 8;            // a unit is 32 input channels: 16 bytes of a weight row
constexpr int kPitch = kStageUnits * 16 + 16;   // bytes between the rows of a stage: words r * 36 + c hit all banks once
constexpr int kStageBytes = 16 * kPitch;
constexpr int kStages = 3;
constexpr int kSlabRows = 64;             // token rows of one pass over the weights
constexpr int kMaxBytes = 56 * 1024;      // of a CTA of up to 8 rows: four fit an SM

constexpr int kActBytes = 12288;          // activations of a pass: 64 bytes a token and unit

// Shared memory of a CTA of up to 8 rows.  T: token rows held (1, 2, 4 or 8).
struct Layout {
  int pass_units, b, sum, scale, pitch, offset, bytes;
};
template <int T, int GU>
Layout layout(int units, bool has_offset) {
  Layout l;
  l.pass_units = std::min(kActBytes / (T * 64), units);   // both multiples of a stage
  for (;; l.pass_units -= kStageUnits) {
    const int groups = l.pass_units / GU;
    l.b = kWarps * kStages * kStageBytes;
    l.sum = l.b + l.pass_units * T * 64;
    l.scale = l.sum + (has_offset ? groups * 32 : 0);
    // a row's scales start at an element whose index is a multiple of 8
    l.pitch = (groups + 7 + 7) / 8 * 8 + 8;
    l.offset = l.scale + kCh * l.pitch * 2;
    l.bytes = std::max(l.offset + (has_offset ? kCh * l.pitch * 2 : 0), 8 * kCh * 4);   // and the CTA's sums at the end
    if (l.bytes <= kMaxBytes || l.pass_units <= kStageUnits) return l;
  }
}

// d = a b where first, else d += a b.
template <bool kFirst>
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kFirst) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
  } else {
    asm(
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
// The binary16 scales of N consecutive groups, read at once.
template <int N>
struct Scales {
  uint32_t w[(N + 1) / 2];
  __device__ __forceinline__ explicit Scales(const uint16_t* p) {
    if constexpr (N == 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (N == 4) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else if constexpr (N == 2) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *p;
    }
  }
  __device__ __forceinline__ float operator[](int i) const {
    return half_bits_to_float(static_cast<uint16_t>(w[i / 2] >> (i % 2 * 16)));
  }
};
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

// The slices' sums (s_y: [token][channel] in each CTA of the cluster), added in
// slice order; every CTA takes its share of the tile's outputs.
template <int kCh>
__device__ __forceinline__ void join_slices(const W4gArgs& a, uint32_t s_y, int rank, int slices, int64_t m0, int held,
                                            int64_t n_cta, int tid, int threads) {
  cluster_sync();
  const int rows = static_cast<int>(min(static_cast<int64_t>(held), a.M - m0));
  for (int i = rank * threads + tid; i < rows * kCh; i += slices * threads) {
    const int64_t m = m0 + i / kCh, n = n_cta + i % kCh;
    float v = 0.0f;
    for (int r = 0; r < slices; ++r) v = __fadd_rn(v, ld_cluster(s_y + i * 4, r));
    if (n < a.N) {
      v = __fmul_rn(v, __ldg(a.a_scale + m));
      if (a.residual != nullptr) v = __fadd_rn(v, bf16_bits_to_float(a.residual[m * a.ldr + n]));
      a.out[m * a.ldo + n] = static_cast<uint16_t>(float_to_bf16_rne(v));
    }
  }
  cluster_sync();   // no CTA leaves while its sums are read
}

// ---- up to 8 rows.  T: token rows held.  GU: units of a group.  kOff: with offsets.
template <int T, int GU, bool kOff>
__global__ void __launch_bounds__(kThreads, 4)
    w4g_kernel(const __grid_constant__ W4gArgs a, const __grid_constant__ Layout l, int slices, int slice_units) {
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

  float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};

  // ---- activations as B fragments: 16 codes of a token are a piece, in the
  // order (group, token, unit, half); a thread's pieces of the next pass are
  // read ahead
  constexpr int kPieces = kActBytes / 32 / kThreads;
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
        if (live && half == 0 && u == 0) s_sum[g * 8 + tok] = static_cast<float>(sum);
      }
    }
    cp_async_wait<0>();
    __syncthreads();
    if (p0 + l.pass_units < units) load_q(p0 + l.pass_units);

    // ---- a unit: 2 weight words of a lane (rows r, r + 8), 2 instructions
    const int bl = T < 8 ? min(lr, T - 1) : lr;   // a column past the tokens repeats the last one and is not stored
    const uint16_t* sp = s_scale + (warp * 16 + lr) * l.pitch + shift;
    const uint16_t* op = s_off + (warp * 16 + lr) * l.pitch + shift;
    float acc[4];
    auto unit = [&](const uint8_t* wb, int ul, auto first) {   // unit ul of this pass
      const uint32_t w0 = *reinterpret_cast<const uint32_t*>(wb);
      const uint32_t w1 = *reinterpret_cast<const uint32_t*>(wb + 8 * kPitch);
      const uint32_t ae[4] = {even_codes(w0), even_codes(w1), even_codes(w0 >> 8), even_codes(w1 >> 8)};
      const uint32_t ao[4] = {odd_codes(w0), odd_codes(w1), odd_codes(w0 >> 8), odd_codes(w1 >> 8)};
      const uint4 b = s_b[(ul * T + bl) * 4 + lc];
      mma_f16_16816<decltype(first)::value>(acc, ae, b.x, b.y);
      mma_f16_16816<false>(acc, ao, b.z, b.w);
    };
    const int st0 = p0 / kStageUnits, st_end = (p0 + pu + kStageUnits - 1) / kStageUnits;
    for (int st = st0; st < st_end; ++st) {
      issue(st + kStages - 1);
      cp_async_wait<kStages - 1>();
      __syncwarp();
      const uint8_t* wb = smem + (warp * kStages + st % kStages) * kStageBytes + lr * kPitch + lc * 4;
      constexpr int GV = kStageUnits / GU;   // groups of a stage
      const int ul = (st - st0) * kStageUnits, gl = (st - st0) * GV, n = pu - ul;
      const Scales<GV> s0(sp + gl), s1(sp + 8 * l.pitch + gl), o0(kOff ? op + gl : sp), o1(kOff ? op + 8 * l.pitch + gl : sp);
      auto group = [&](int g) {
        unit(wb + g * GU * 16, ul + g * GU, std::true_type{});
#pragma unroll
        for (int u = 1; u < GU; ++u) unit(wb + (g * GU + u) * 16, ul + g * GU + u, std::false_type{});
        y[0] = __fmaf_rn(acc[0], s0[g], y[0]);
        y[1] = __fmaf_rn(acc[1], s0[g], y[1]);
        y[2] = __fmaf_rn(acc[2], s1[g], y[2]);
        y[3] = __fmaf_rn(acc[3], s1[g], y[3]);
        if constexpr (kOff) {
          const float2 q = *reinterpret_cast<const float2*>(s_sum + (gl + g) * 8 + 2 * lc);
          y[0] = __fmaf_rn(q.x, o0[g], y[0]);
          y[1] = __fmaf_rn(q.y, o0[g], y[1]);
          y[2] = __fmaf_rn(q.x, o1[g], y[2]);
          y[3] = __fmaf_rn(q.y, o1[g], y[3]);
        }
      };
      if (n >= kStageUnits) {
#pragma unroll
        for (int g = 0; g < GV; ++g) group(g);
      } else {
#pragma unroll
        for (int g = 0; g < GV; ++g)
          if (g * GU < n) group(g);
      }
      __syncwarp();   // the stage is free for the copy that the next turn issues
    }
  }

  // ---- the slices' sums, added in slice order by the CTAs of the cluster
  cp_async_wait<0>();
  __syncthreads();
  float* s_y = reinterpret_cast<float*>(smem);   // [token][channel]
#pragma unroll
  for (int e = 0; e < 4; ++e) s_y[(2 * lc + (e & 1)) * kCh + warp * 16 + lr + 8 * (e >> 1)] = y[e];
  join_slices<kCh>(a, smem_u32(smem), rank, slices, m0, 8, n_cta, tid, kThreads);
}

// ---- 9 and more rows.  A CTA owns 128 channels: four warps of 32 channels, so
// that a B fragment read from shared memory serves two instructions' rows, and
// four warps that lay chunks of 8 units of activations (and their scales) into
// one of two buffers while the other is used.  A chunk's weights come as one
// tensor copy, a box of 128 rows by 128 bytes whose 16-byte pieces are swizzled
// (piece u of row r at u ^ (r & 7)); rows past N and units past K read as zero.
// Chunk c's mbarrier counts the box's bytes and the laying threads; the named
// barrier kEmpty + (c & 1) says that chunk c has been read.  (The weights as
// cp.async copies of the contracting lanes cost a fifth of their time: 37 rows of
// 5120 x 34816 69 us; a box of 32 rows for each warp 61, one for the CTA asked
// for by the laying warps 60.  With up to 8 rows boxes are no faster: one row
// 25.4 and 26.3 us.)
constexpr int kWideWarps = 4, kSideWarps = 4;       // a warpgroup each
constexpr int kWideThreads = (kWideWarps + kSideWarps) * 32, kSide = kSideWarps * 32;
constexpr int kWideCh = kWideWarps * 32;
constexpr int kWidePitch = kStageUnits * 16, kWideStage = kWideCh * kWidePitch;
enum : int { kEmpty = 1, kDone = 3 };

// The two warpgroups share the registers that the CTA was launched with: 128 a
// thread, by the launch bounds.  (Two warps laying out, 168 registers for all:
// 37 rows of 17408 x 5120 58.7 us, 64 rows of 5120 x 34816 100; four warps and
// 168 + 88: 55.4 and 96, with spills; 184 + 72: 51.3 and 90.)
constexpr int kLaunchRegs = 128, kWideRegs = 184, kSideRegs = 72;
static_assert(kWideWarps * kWideRegs + kSideWarps * kSideRegs <= (kWideWarps + kSideWarps) * kLaunchRegs, "the launch's registers");
static_assert(2 * kWideThreads * kLaunchRegs <= 65536, "two CTAs an SM");
template <int n>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(n)); }
template <int n>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(n)); }

__device__ __forceinline__ void named_sync(int id) { asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kWideThreads) : "memory"); }
__device__ __forceinline__ void named_arrive(int id) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(kWideThreads) : "memory");
}

template <int T, int GU, bool kOff>
struct Wide {
  static constexpr int NT = T / 8;
  static constexpr int CU = kStageUnits;                           // units of a chunk
  static constexpr int NS = T <= 40 ? 3 : 2;                       // chunks of weights held: two CTAs fit an SM
  static constexpr int GC = CU / GU;                               // its groups
  static constexpr int kB = CU * T * 64, kScale = kWideCh * GC * 2, kSum = GC * T * 4;
  static constexpr int kBuffer = kB + (kOff ? 2 * kScale + kSum : kScale);
  static constexpr int kRing = NS * kWideStage;
  static constexpr int kBytes = 1024 + kRing + 2 * kBuffer;
  static_assert(kBytes >= T * kWideCh * 4, "the CTA's sums at the end");
  static_assert(2 * (kBytes + 1024) <= 227 * 1024, "two CTAs an SM");
};

template <int T, int GU, bool kOff>
__global__ void __launch_bounds__(kWideThreads, 2) w4g_wide_kernel(const __grid_constant__ W4gArgs a, const __grid_constant__ CUtensorMap w_map, int slices,
                                                                   int slice_units) {
  using C = Wide<T, GU, kOff>;
  constexpr int NT = C::NT, CU = C::CU, GC = C::GC, NS = C::NS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[NS];
  __shared__ int s_abort;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);   // the ring's boxes start on 1024-byte boundaries
  const uint32_t bars = smem_u32(s_bar);
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) tc::mbar_init(bars + 8 * i, kSide + 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lr = lane >> 2, lc = lane & 3;
  const int rank = blockIdx.x % slices;
  const int64_t n_cta = static_cast<int64_t>(blockIdx.x / slices) * kWideCh;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kSlabRows;
  const int all_units = static_cast<int>(a.K >> 5);
  const int u_begin = min(rank * slice_units, all_units);
  const int units = min(slice_units, all_units - u_begin), chunks = (units + CU - 1) / CU;
  auto buffer = [&](int c) { return smem + C::kRing + (c & 1) * C::kBuffer; };   // B fragments, scales, offsets, sums of q
  if (warp >= kWideWarps) {
    fewer_registers<kSideRegs>();
    // ============ activations as B fragments, and the scales ============
    // 16 codes of a token are a piece, in the order (group, token, unit, half)
    const int st = tid - kWideWarps * 32, half = st & 1, u = (st >> 1) % GU, pair = st / (2 * GU);
    constexpr int kPieces = CU * T * 2 / kSide, kPairs = kSide / (2 * GU);
    static_assert(CU * T * 2 % kSide == 0, "whole turns");
    const int8_t* q0 = a.q + m0 * a.ldq + static_cast<int64_t>(u_begin + u) * 32 + half * 16;
    const int live = static_cast<int>(min(static_cast<int64_t>(T), a.M - m0));
    // scales of a channel's chunk in one access, where they lie on its boundary
    const bool wide = a.lds % GC == 0 && (reinterpret_cast<uintptr_t>(a.scale) & (GC * 2 - 1)) == 0 &&
                      (!kOff || (a.ldb % GC == 0 && (reinterpret_cast<uintptr_t>(a.offset) & (GC * 2 - 1)) == 0));
    using Vec = std::conditional_t<GC == 8, uint4, std::conditional_t<GC == 4, uint2, std::conditional_t<GC == 2, uint32_t, uint16_t>>>;
    constexpr int kRows = kWideCh / kSide;
    uint4 w[kPieces];
    Vec sc[kRows], of[kOff ? kRows : 1];
    auto load = [&](int c) {
      const int left = units - c * CU;
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const int i = pair + j * kPairs, g = i / T, tok = i - g * T;
        w[j] = make_uint4(0u, 0u, 0u, 0u);
        if (g * GU < left && tok < live)
          w[j] = __ldg(reinterpret_cast<const uint4*>(q0 + tok * a.ldq + (c * CU + g * GU) * 32));
      }
      const int g0 = (u_begin + c * CU) / GU;
      const bool whole = wide && left >= CU;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int64_t n = min(n_cta + st + r * kSide, a.N - 1);   // rows past N repeat the last one
        const uint16_t *sp = a.scale + n * a.lds + g0, *op = kOff ? a.offset + n * a.ldb + g0 : nullptr;
        if (whole) {
          sc[r] = __ldg(reinterpret_cast<const Vec*>(sp));
          if (kOff) of[r] = __ldg(reinterpret_cast<const Vec*>(op));
        } else {
          alignas(16) uint16_t e[GC], f[GC];
#pragma unroll
          for (int g = 0; g < GC; ++g) {
            e[g] = g * GU < left ? __ldg(sp + g) : static_cast<uint16_t>(0);
            f[g] = kOff && g * GU < left ? __ldg(op + g) : static_cast<uint16_t>(0);
          }
          memcpy(&sc[r], e, sizeof(Vec));
          if (kOff) memcpy(&of[r], f, sizeof(Vec));
        }
      }
    };
    // chunk c's weights, into the place of chunk c - NS
    auto ask = [&](int c) {
      if (st == 0 && c < chunks) {
        const uint32_t bar = bars + 8 * (c % NS);
        tc::mbar_expect_tx(bar, kWideStage);
        tc::tma_load_2d(smem_u32(smem) + (c % NS) * kWideStage, &w_map, u_begin * 16 + c * kWidePitch, static_cast<int32_t>(n_cta), bar);
      }
    };
    // Once a wait has run out no more is asked for, and only chunks that were
    // asked for are arrived for, so that no phase of an mbarrier gets another's
    // arrivals; the boxes still under way land before the CTA ends.
    auto withheld = [&] { return st == 0 && *static_cast<volatile int*>(&g_w4g_withhold) != 0; };
    auto aborted = [&] { return __any_sync(0xffffffffu, *static_cast<volatile int*>(&s_abort)) != 0; };   // one answer for the warp
    auto drain = [&](int asked) {
      if (withheld()) tc::mbar_arrive(bars);
      for (int c = max(0, asked - NS); c < min(asked, chunks) && st == 0; ++c)
        tc::mbar_wait_drain_bounded(bars + 8 * (c % NS), (c / NS) & 1, kDrainNs, &g_w4g_status, PRISM_DEVSTATUS_WAIT_TIMEOUT);
    };
#pragma unroll
    for (int c = 0; c < NS; ++c) ask(c);
    if (chunks > 0) load(0);
    int c = 0;
    for (; c < chunks; ++c) {
      if (c >= 2) {
        named_sync(kEmpty + (c & 1));   // chunk c - 2 was read
        if (aborted()) {
          for (int k = c; k < chunks; ++k) {
            if (k > c) named_sync(kEmpty + (k & 1));
            if (k < c - 2 + NS) tc::mbar_arrive(bars + 8 * (k % NS));
          }
          drain(c - 2 + NS);
          break;
        }
        ask(c - 2 + NS);
      }
      uint8_t* buf = buffer(c);
      Vec* s_scale = reinterpret_cast<Vec*>(buf + C::kB);
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        s_scale[st + r * kSide] = sc[r];
        if (kOff) s_scale[kWideCh + st + r * kSide] = of[r];
      }
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const int i = pair + j * kPairs, g = i / T, tok = i - g * T;
        // [unit][even, odd][token][4 pairs of words]: the even codes' words of two lanes, then the odd ones'
        uint4* dst = reinterpret_cast<uint4*>(buf) + ((g * GU + u) * 2 * T + tok) * 2 + half;
        const uint32_t x0 = __byte_perm(w[j].x, w[j].y, 0x5140u) ^ 0x80808080u;   // codes 0, 4, 1, 5
        const uint32_t x1 = __byte_perm(w[j].x, w[j].y, 0x7362u) ^ 0x80808080u;   // codes 2, 6, 3, 7
        const uint32_t z0 = __byte_perm(w[j].z, w[j].w, 0x5140u) ^ 0x80808080u;
        const uint32_t z1 = __byte_perm(w[j].z, w[j].w, 0x7362u) ^ 0x80808080u;
        dst[0] = make_uint4(widen(x0, 0x4140u), widen(x1, 0x4140u), widen(z0, 0x4140u), widen(z1, 0x4140u));
        dst[2 * T] = make_uint4(widen(x0, 0x4342u), widen(x1, 0x4342u), widen(z0, 0x4342u), widen(z1, 0x4342u));
        if constexpr (kOff) {   // the group's sum of q: its 2 GU pieces lie in neighbouring lanes
          int sum = __dp4a(static_cast<int>(w[j].x), 0x01010101, __dp4a(static_cast<int>(w[j].y), 0x01010101, 0));
          sum = __dp4a(static_cast<int>(w[j].z), 0x01010101, __dp4a(static_cast<int>(w[j].w), 0x01010101, sum));
#pragma unroll
          for (int o = 1; o < 2 * GU; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          if (half == 0 && u == 0) reinterpret_cast<float*>(buf + C::kB + 2 * C::kScale)[i] = static_cast<float>(sum);
        }
      }
      if (c != 0 || !withheld()) tc::mbar_arrive(bars + 8 * (c % NS));
      if (c + 1 < chunks) load(c + 1);
    }
    named_sync(kDone);
    if (c == chunks && chunks > 0 && aborted()) drain(chunks);   // after the last chunk was asked for
    __syncwarp();
    more_registers<kLaunchRegs>();
  } else {
    more_registers<kWideRegs>();
    // ============ contraction ============
    float y[2][NT][4];
#pragma unroll
    for (int i = 0; i < 2 * NT * 4; ++i) y[i / (NT * 4)][i / 4 % NT][i & 3] = 0.0f;
    float acc[2][NT][4];
    for (int c = 0; c < chunks; ++c) {
      // bounded: where it runs out, the status bit says that the outputs are not valid
      tc::mbar_wait_bounded(bars + 8 * (c % NS), (c / NS) & 1, &s_abort, &g_w4g_wait_limit_ns, &g_w4g_status, PRISM_DEVSTATUS_WAIT_TIMEOUT);
      __syncwarp();
      const uint8_t* wb = smem + (c % NS) * kWideStage + (warp * 32 + lr) * kWidePitch + lc * 4;
      const uint8_t* buf = buffer(c);
      const uint2* s_b = reinterpret_cast<const uint2*>(buf) + lr * 4 + lc;
      const uint16_t* sp = reinterpret_cast<const uint16_t*>(buf + C::kB) + (warp * 32 + lr) * GC;
      const float* qs = reinterpret_cast<const float*>(buf + C::kB + 2 * C::kScale) + 2 * lc;
      const uint16_t* op = kOff ? sp + kWideCh * GC : sp;
      const Scales<GC> sv[4] = {Scales<GC>(sp), Scales<GC>(sp + 8 * GC), Scales<GC>(sp + 16 * GC), Scales<GC>(sp + 24 * GC)};
      const Scales<GC> ov[4] = {Scales<GC>(op), Scales<GC>(op + 8 * GC), Scales<GC>(op + 16 * GC), Scales<GC>(op + 24 * GC)};
      auto unit = [&](int u, auto first) {
        uint32_t ae[2][4], ao[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint8_t* at = wb + i * 16 * kWidePitch + ((u * 16) ^ (lr * 16));
          const uint32_t w0 = *reinterpret_cast<const uint32_t*>(at);
          const uint32_t w1 = *reinterpret_cast<const uint32_t*>(at + 8 * kWidePitch);
          ae[i][0] = even_codes(w0), ae[i][1] = even_codes(w1), ae[i][2] = even_codes(w0 >> 8), ae[i][3] = even_codes(w1 >> 8);
          ao[i][0] = odd_codes(w0), ao[i][1] = odd_codes(w1), ao[i][2] = odd_codes(w0 >> 8), ao[i][3] = odd_codes(w1 >> 8);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint2 b = s_b[(u * 2 * T + t * 8) * 4];
          mma_f16_16816<decltype(first)::value>(acc[0][t], ae[0], b.x, b.y);
          mma_f16_16816<decltype(first)::value>(acc[1][t], ae[1], b.x, b.y);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {   // an accumulator's next instruction comes 2 NT later
          const uint2 b = s_b[((u * 2 + 1) * T + t * 8) * 4];
          mma_f16_16816<false>(acc[0][t], ao[0], b.x, b.y);
          mma_f16_16816<false>(acc[1][t], ao[1], b.x, b.y);
        }
      };
      auto group = [&](int g) {
        unit(g * GU, std::true_type{});
#pragma unroll
        for (int u = 1; u < GU; ++u) unit(g * GU + u, std::false_type{});
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            y[i][t][0] = __fmaf_rn(acc[i][t][0], sv[i * 2][g], y[i][t][0]);
            y[i][t][1] = __fmaf_rn(acc[i][t][1], sv[i * 2][g], y[i][t][1]);
            y[i][t][2] = __fmaf_rn(acc[i][t][2], sv[i * 2 + 1][g], y[i][t][2]);
            y[i][t][3] = __fmaf_rn(acc[i][t][3], sv[i * 2 + 1][g], y[i][t][3]);
          }
          if constexpr (kOff) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const float2 q = *reinterpret_cast<const float2*>(qs + g * T + t * 8);
              y[i][t][0] = __fmaf_rn(q.x, ov[i * 2][g], y[i][t][0]);
              y[i][t][1] = __fmaf_rn(q.y, ov[i * 2][g], y[i][t][1]);
              y[i][t][2] = __fmaf_rn(q.x, ov[i * 2 + 1][g], y[i][t][2]);
              y[i][t][3] = __fmaf_rn(q.y, ov[i * 2 + 1][g], y[i][t][3]);
            }
          }
        }
      };
      const int n = units - c * CU;
      if (n >= CU) {
#pragma unroll
        for (int g = 0; g < GC; ++g) group(g);
      } else {
#pragma unroll
        for (int g = 0; g < GC; ++g)
          if (g * GU < n) group(g);
      }
      if (c + 2 < chunks) named_arrive(kEmpty + (c & 1));
    }
    named_sync(kDone);
    float* s_y = reinterpret_cast<float*>(smem);   // [token][channel]
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          s_y[(t * 8 + 2 * lc + (e & 1)) * kWideCh + warp * 32 + i * 16 + lr + 8 * (e >> 1)] = y[i][t][e];
    fewer_registers<kLaunchRegs>();
  }
  join_slices<kWideCh>(a, smem_u32(smem), rank, slices, m0, T, n_cta, tid, kWideThreads);
}

// The packed weights in the wide kernel's boxes.
cudaError_t weight_map(CUtensorMap* m, const W4gArgs& a) {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q{};
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(e == cudaSuccess && q == cudaDriverEntryPointSuccess ? f : nullptr);
  }();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.K / 2), static_cast<cuuint64_t>(a.N)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.ldw4)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(kWidePitch), kWideCh}, step[2] = {1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(a.w4), dims, strides, box, step,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <class... P, class... A>
cudaError_t launch_slices(void (*kernel)(P...), int channels, int threads, int bytes, int slices, const W4gArgs& a,
                          cudaStream_t stream, const A&... rest) {
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), bytes);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (a.N + channels - 1) / channels;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * slices), static_cast<unsigned>((a.M + kSlabRows - 1) / kSlabRows));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = static_cast<size_t>(bytes);
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
  return cudaLaunchKernelEx(&cfg, kernel, a, rest...);
}

template <int GU, bool kOff>
cudaError_t launch_gu(const W4gArgs& a, cudaStream_t stream) {
  // Slices of K: as many as let four CTAs of 64 channels (two of 128) on each of
  // kSms SMs run at once, at most a cluster of eight; each a multiple of a stage.
  // A rule on N and K alone: a row's sums do not depend on M, or on the device.
  const int64_t tiles64 = (a.N + 63) / 64;
  const int units = static_cast<int>(a.K >> 5), stages = (units + kStageUnits - 1) / kStageUnits;
  const int slices = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({4 * kSms / tiles64, 8, stages})));
  const int slice_units = (stages + slices - 1) / slices * kStageUnits;
  auto few = [&](auto t) {
    constexpr int T = decltype(t)::value;
    const Layout l = layout<T, GU>(slice_units, kOff);
    return launch_slices(w4g_kernel<T, GU, kOff>, kCh, kThreads, l.bytes, slices, a, stream, l, slices, slice_units);
  };
  auto wide = [&](auto t) {
    constexpr int T = decltype(t)::value;
    CUtensorMap map;
    const cudaError_t e = weight_map(&map, a);
    if (e != cudaSuccess) return e;
    return launch_slices(w4g_wide_kernel<T, GU, kOff>, kWideCh, kWideThreads, Wide<T, GU, kOff>::kBytes, slices, a, stream,
                         map, slices, slice_units);
  };
  if (a.M <= 1) return few(std::integral_constant<int, 1>{});
  if (a.M <= 2) return few(std::integral_constant<int, 2>{});
  if (a.M <= 4) return few(std::integral_constant<int, 4>{});
  if (a.M <= 8) return few(std::integral_constant<int, 8>{});
  // The tile's rows go up by the instruction's 8 columns: activations are laid out
  // and multiplied for every row of the tile, live or not (5120 x 34816: 32 rows in
  // tiles of 32 and 40 take 49.9 and 59.3 us, 48 in tiles of 48 and 64 68.4 and 88.8).
  if (a.M <= 16) return wide(std::integral_constant<int, 16>{});
  if (a.M <= 24) return wide(std::integral_constant<int, 24>{});
  if (a.M <= 32) return wide(std::integral_constant<int, 32>{});
  if (a.M <= 40) return wide(std::integral_constant<int, 40>{});
  if (a.M <= 48) return wide(std::integral_constant<int, 48>{});
  if (a.M <= 56) return wide(std::integral_constant<int, 56>{});
  return wide(std::integral_constant<int, 64>{});
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

cudaError_t read_and_clear_w4g_status(uint32_t* out) {
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_w4g_status, sizeof v);
  if (e != cudaSuccess) return e;
  if (v != 0) {
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_w4g_status, &zero, sizeof zero);
  }
  *out = v;
  return e;
}

cudaError_t set_w4g_wait_expiry(unsigned long long limit_ns, int withhold) {
  cudaError_t e = cudaMemcpyToSymbol(g_w4g_wait_limit_ns, &limit_ns, sizeof limit_ns);
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_w4g_withhold, &withhold, sizeof withhold);
  return e;
}

}  // namespace prism
