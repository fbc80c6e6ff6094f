// norm_quant.cu -- what turns a layer's bf16 rows into the codes of its next
// linear: the residual stream's norm, the norm of each head with its gate, and
// the FFN's gated activation, each down to int8 codes with a scale for the row
// (prism_quant_act's definition), the codes as binary16, or bf16 values.
//
//   norm   h = bf16(x + alpha * d), d = delta or delta * r(delta) * post
//          y = h * r(h) * weight
//   heads  y = x * r(x's head) * weight * silu(gate) * inv_s
//   glu    y = silu(gate) * up * inv_s
// with r(v) = (sum v^2 / n + eps)^(-1/2).  Every step is one binary32 operation
// rounded to nearest even, so that codes are the same bits wherever they are
// computed; a sum alone would depend on its order.  The squares of bf16 values
// are exact in binary32, and they are added as pairs of binary32 numbers (sum
// and error of each addition), good to about 2^-40 of the sum; r is formed to
// as much and rounded once.  exp is a series of fused steps.  (The compiler merges
// paired products and sums into fused ones where they meet; where a sum follows a
// product and both are to be rounded, the sum is a scalar one.)
//
// A row is one CTA's: its values stay in registers from the first read to the
// codes, 8 to a 16-byte vector, C vectors a thread, the fewest that keep the row
// within 512 threads.  Two exchanges in shared memory (three with a post norm)
// stand in the way of a row, the sum's and the largest magnitude's; the next
// row's loads are under way across them, and the other CTAs of the SM work.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "decode.cuh"
#include "layer.cuh"

namespace prism {
namespace {

constexpr int kMaxTeam = 512;
constexpr int kWarps = kMaxTeam / 32;

// A sum of binary32 numbers as the rounded sum and its error.
struct Sum {
  float h, l;
};
__device__ __forceinline__ Sum join(Sum a, Sum b) {
  const float s = __fadd_rn(a.h, b.h), t = __fsub_rn(s, a.h);
  const float e = __fadd_rn(__fsub_rn(a.h, __fsub_rn(s, t)), __fsub_rn(b.h, t));
  return Sum{s, __fadd_rn(e, __fadd_rn(a.l, b.l))};
}
// Two sums side by side.
struct Sum2 {
  float2 h, l;
};
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }
__device__ __forceinline__ void add_square(Sum2& a, float2 v) {
  const float2 p = mul2(v, v);
  const float2 s = add2(a.h, p), t = add2(s, neg2(a.h));
  const float2 e = add2(add2(a.h, neg2(add2(s, neg2(t)))), add2(p, neg2(t)));
  a.h = s;
  a.l = add2(a.l, e);
}
__device__ __forceinline__ Sum both(const Sum2& a) { return join(Sum{a.h.x, a.l.x}, Sum{a.h.y, a.l.y}); }

// (s / n + eps)^(-1/2): the reciprocal root's approximation and one step of
// Newton's iteration whose residual is formed from the rounding errors too.
__device__ __forceinline__ float inverse_root(Sum s, float inv_n, float inv_n_low, float eps) {
  const float p = __fmul_rn(s.h, inv_n);
  float e = __fmaf_rn(s.h, inv_n, -p);
  e = __fmaf_rn(s.h, inv_n_low, e);
  e = __fmaf_rn(s.l, inv_n, e);
  const Sum a = join(Sum{p, e}, Sum{eps, 0.0f});
  const float ah = __fadd_rn(a.h, a.l), al = __fsub_rn(a.l, __fsub_rn(ah, a.h));
  const float r = rsqrtf(ah), t = __fmul_rn(r, r), tl = __fmaf_rn(r, r, -t);
  float d = __fmaf_rn(-ah, t, 1.0f);
  d = __fmaf_rn(-ah, tl, d);
  d = __fmaf_rn(-al, t, d);
  return __fmaf_rn(__fmul_rn(0.5f, r), d, r);
}

// silu of two values: z / (1 + exp(-z)) as z * ((1 or e) / (1 + e)), e = exp(-|z|)
// by n ln 2 + r (ln 2 in two parts), the series of e^r to r^7 in fused steps, times
// 2^n; e = 0 for n < -126.
__device__ __forceinline__ float2 silu2(float2 z) {
  constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: its unit is 1
  auto two = [](float v) { return make_float2(v, v); };
  const float2 x = make_float2(-fabsf(z.x), -fabsf(z.y));
  float2 t = fma2(x, two(0x1.715476p+0f), two(kMagic));
  t = make_float2(fmaxf(t.x, kMagic - 200.0f), fmaxf(t.y, kMagic - 200.0f));
  const float2 n = add2(t, two(-kMagic));
  float2 r = fma2(n, two(-0x1.63p-1f), x);
  r = fma2(n, two(0x1.bd0106p-13f), r);
  float2 p = two(0x1.a01a02p-13f);
  p = fma2(p, r, two(0x1.6c16c2p-10f));
  p = fma2(p, r, two(0x1.111112p-7f));
  p = fma2(p, r, two(0x1.555556p-5f));
  p = fma2(p, r, two(0x1.555556p-3f));
  p = fma2(p, r, two(0x1p-1f));
  p = fma2(p, r, two(1.0f));
  p = fma2(p, r, two(1.0f));
  const float2 scale = make_float2(__uint_as_float((__float_as_uint(t.x) + 127u) << 23),
                                   __uint_as_float((__float_as_uint(t.y) + 127u) << 23));
  p = mul2(p, scale);
  const float2 e = make_float2(n.x >= -126.0f ? p.x : 0.0f, n.y >= -126.0f ? p.y : 0.0f);
  const float2 d = add2(e, two(1.0f));
  const float2 s = make_float2(__fdiv_rn(z.x >= 0.0f ? 1.0f : e.x, d.x), __fdiv_rn(z.y >= 0.0f ? 1.0f : e.y, d.y));
  return mul2(z, s);
}

__device__ __forceinline__ float2 pair(uint32_t v) { return make_float2(bf16_lo(v), bf16_hi(v)); }
__device__ __forceinline__ uint32_t bf16x2(float2 v) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
// Weights of the four pairs of channels 8 j .. 8 j + 7.
struct Weights {
  float4 a, b;
  __device__ __forceinline__ Weights(const float* w, int j)
      : a(__ldg(reinterpret_cast<const float4*>(w) + 2 * j)), b(__ldg(reinterpret_cast<const float4*>(w) + 2 * j + 1)) {}
  __device__ __forceinline__ float2 operator[](int i) const {
    return i == 0 ? make_float2(a.x, a.y) : i == 1 ? make_float2(a.z, a.w) : i == 2 ? make_float2(b.x, b.y) : make_float2(b.z, b.w);
  }
};

// The CTA's sums, in every thread.
__device__ __forceinline__ Sum team_sum(Sum s, Sum* red) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    s = join(s, Sum{__shfl_xor_sync(0xffffffffu, s.h, o), __shfl_xor_sync(0xffffffffu, s.l, o)});
  if (lane == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  s = lane < warps ? red[lane] : Sum{0.0f, 0.0f};
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1)
    s = join(s, Sum{__shfl_xor_sync(0xffffffffu, s.h, o), __shfl_xor_sync(0xffffffffu, s.l, o)});
  return Sum{__shfl_sync(0xffffffffu, s.h, 0), __shfl_sync(0xffffffffu, s.l, 0)};
}

// The row's values y, 8 C a thread (0 past the row's end), as codes.
template <int C>
__device__ __forceinline__ void store_codes(const RowCodes& o, int64_t row, int nvec, const float2 (&y)[C][4], uint32_t* red) {
  const int team = blockDim.x, lt = threadIdx.x, lane = lt & 31;
  if (o.form == PRISM_FORM_BF16) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int j = lt + i * team;
      if (j < nvec)
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(o.q) + row * o.ldq)[j] =
            make_uint4(bf16x2(y[i][0]), bf16x2(y[i][1]), bf16x2(y[i][2]), bf16x2(y[i][3]));
    }
    return;
  }
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(y[i][e].x), fabsf(y[i][e].y)));
  // magnitudes are ordered as their bits are
  const uint32_t wm = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
  if (lane == 0) red[lt >> 5] = wm;
  __syncthreads();
  const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, lane < (team >> 5) ? red[lane] : 0u));
  const bool zero_row = !(amax >= 0x1p-120f);
  const float inv = zero_row ? 0.0f : __fdiv_rn(127.0f, amax);
  if (lt == 0) o.a_scale[row] = zero_row ? 0.0f : __fdiv_rn(amax, 127.0f);
  // t + 1.5 * 2^23 is t rounded to an integer, in the low bits
  constexpr float kMagic = 12582912.0f;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int j = lt + i * team;
    if (j >= nvec) continue;
    float2 t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      t[e] = mul2(y[i][e], make_float2(inv, inv));
      t[e] = make_float2(__fadd_rn(t[e].x, kMagic), __fadd_rn(t[e].y, kMagic));   // scalar: never merged into a multiply-add
    }
    if (o.form == PRISM_FORM_F16) {
      uint32_t h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __half2 v = __floats2half2_rn(__fsub_rn(t[e].x, kMagic), __fsub_rn(t[e].y, kMagic));
        h[e] = *reinterpret_cast<const uint32_t*>(&v);
      }
      reinterpret_cast<uint4*>(static_cast<uint16_t*>(o.q) + row * o.ldq)[j] = make_uint4(h[0], h[1], h[2], h[3]);
    } else {
      uint32_t b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = __byte_perm(__float_as_uint(t[e].x), __float_as_uint(t[e].y), 0x0040u);
      reinterpret_cast<uint2*>(static_cast<int8_t*>(o.q) + row * o.ldq)[j] =
          make_uint2(__byte_perm(b[0], b[1], 0x5410u), __byte_perm(b[2], b[3], 0x5410u));
    }
  }
}

// A row's values are read once.  Not through the read-only path: a row may be
// written back in place.
__device__ __forceinline__ uint4 load_once_16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <int C>
struct Row {
  uint4 v[C];
  // Vectors of the thread; zeros past the row's end.
  __device__ __forceinline__ void load(const uint16_t* row, int nvec) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int j = threadIdx.x + i * static_cast<int>(blockDim.x);
      v[i] = j < nvec ? load_once_16(reinterpret_cast<const uint4*>(row) + j) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
};

template <int C, bool kDelta>
__global__ void __launch_bounds__(kMaxTeam) norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ Sum s_sum[2][kWarps], s_post[2][kWarps];
  __shared__ uint32_t s_top[2][kWarps];
  pdl_trigger();
  pdl_wait();
  const int team = blockDim.x, lt = threadIdx.x, nvec = static_cast<int>(a.K >> 3);
  Row<C> x, d;
  int64_t row = blockIdx.x;
  x.load(a.x + row * a.ldx, nvec);
  if constexpr (kDelta) d.load(a.delta + row * a.ldd, nvec);
  for (int par = 0; row < a.M; row += gridDim.x, par ^= 1) {
    if constexpr (kDelta) {
      float r = 1.0f;
      if (a.post != nullptr) {
        Sum2 s{};
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) add_square(s, pair(word(d.v[i], e)));
        r = inverse_root(team_sum(both(s), s_post[par]), a.inv_n, a.inv_n_low, a.eps);
      }
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int j = lt + i * team;
        if (j >= nvec) continue;
        float2 w[4];
        if (a.post != nullptr) {
          const Weights p(a.post, j);
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = mul2(mul2(pair(word(d.v[i], e)), make_float2(r, r)), p[e]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = pair(word(d.v[i], e));
        }
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 add = mul2(w[e], make_float2(a.alpha, a.alpha)), v = pair(word(x.v[i], e));
          h[e] = bf16x2(make_float2(__fadd_rn(v.x, add.x), __fadd_rn(v.y, add.y)));   // scalar: not merged with the product
        }
        x.v[i] = make_uint4(h[0], h[1], h[2], h[3]);
        reinterpret_cast<uint4*>(a.h + row * a.ldh)[j] = x.v[i];
      }
    }
    float2 y[C][4];
    Sum2 s{};
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[i][e] = pair(word(x.v[i], e));
        add_square(s, y[i][e]);
      }
    const int64_t next = row + gridDim.x;
    if (next < a.M) {
      x.load(a.x + next * a.ldx, nvec);
      if constexpr (kDelta) d.load(a.delta + next * a.ldd, nvec);
    }
    const float r = inverse_root(team_sum(both(s), s_sum[par]), a.inv_n, a.inv_n_low, a.eps);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int j = lt + i * team;
      if (j >= nvec) continue;
      const Weights w(a.weight, j);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[i][e] = mul2(mul2(y[i][e], make_float2(r, r)), w[e]);
    }
    store_codes<C>(a.o, row, nvec, y, s_top[par]);
  }
}

// A head's channels lie in D / 8 neighbouring lanes, whose sums are exchanged by shuffles.
template <int C, bool kGate>
__global__ void __launch_bounds__(kMaxTeam) head_norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ uint32_t s_top[2][kWarps];
  pdl_trigger();
  pdl_wait();
  const int team = blockDim.x, lt = threadIdx.x, nvec = static_cast<int>(a.K >> 3), lanes = a.D >> 3;
  Row<C> x, z;
  int64_t row = blockIdx.x;
  x.load(a.x + row * a.ldx, nvec);
  if constexpr (kGate) z.load(a.gate + row * a.ldg, nvec);
  const Weights w(a.weight, lt & (lanes - 1));   // a team is whole heads wide, or the row is one turn
  for (int par = 0; row < a.M; row += gridDim.x, par ^= 1) {
    float2 y[C][4];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int j = lt + i * team;
      Sum2 s{};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[i][e] = pair(word(x.v[i], e));
        add_square(s, y[i][e]);
      }
      Sum t = both(s);
      for (int o = lanes >> 1; o > 0; o >>= 1)
        t = join(t, Sum{__shfl_xor_sync(0xffffffffu, t.h, o), __shfl_xor_sync(0xffffffffu, t.l, o)});
      const float r = inverse_root(t, a.inv_n, a.inv_n_low, a.eps);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[i][e] = mul2(mul2(y[i][e], make_float2(r, r)), w[e]);
        if constexpr (kGate) y[i][e] = mul2(y[i][e], silu2(pair(word(z.v[i], e))));
      }
      if (a.inv_s != nullptr && j < nvec) {
        const Weights p(a.inv_s, j);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[i][e] = mul2(y[i][e], p[e]);
      }
    }
    const int64_t next = row + gridDim.x;
    if (next < a.M) {
      x.load(a.x + next * a.ldx, nvec);
      if constexpr (kGate) z.load(a.gate + next * a.ldg, nvec);
    }
    store_codes<C>(a.o, row, nvec, y, s_top[par]);
  }
}

template <int C>
__global__ void __launch_bounds__(kMaxTeam) glu_kernel(const __grid_constant__ GluArgs a) {
  __shared__ uint32_t s_top[2][kWarps];
  pdl_trigger();
  pdl_wait();
  const int team = blockDim.x, lt = threadIdx.x, nvec = static_cast<int>(a.F >> 3);
  Row<C> g, u;
  int64_t row = blockIdx.x;
  g.load(a.x + row * a.ldx, nvec);
  u.load(a.x + row * a.ldx + a.F, nvec);
  for (int par = 0; row < a.M; row += gridDim.x, par ^= 1) {
    float2 y[C][4];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int j = lt + i * team;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[i][e] = mul2(silu2(pair(word(g.v[i], e))), pair(word(u.v[i], e)));
      if (a.inv_s != nullptr && j < nvec) {
        const Weights p(a.inv_s, j);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[i][e] = mul2(y[i][e], p[e]);
      }
    }
    const int64_t next = row + gridDim.x;
    if (next < a.M) {
      g.load(a.x + next * a.ldx, nvec);
      u.load(a.x + next * a.ldx + a.F, nvec);
    }
    store_codes<C>(a.o, row, nvec, y, s_top[par]);
  }
}

// The fewest vectors a thread that keep a row within kMaxTeam threads.  The team
// follows from the row's length alone, and with it the order of its sums.
constexpr int vectors_of(int64_t K) {
  return static_cast<int>((K / 8 + kMaxTeam - 1) / kMaxTeam);
}

template <class Args>
cudaError_t launch_rows(void (*kernel)(const Args), const Args& a, int64_t M, int64_t K, cudaStream_t stream) {
  const int c = vectors_of(K);
  const int team = static_cast<int>(32 * ((K / 8 + 32 * c - 1) / (32 * c)));
  int per_sm = 0;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, team, 0);
  if (e != cudaSuccess) return e;
  // as many rows for each CTA that the SMs hold
  const int64_t most = static_cast<int64_t>(sm_count()) * std::max(per_sm, 1), each = (M + most - 1) / most;
  return launch_kernel(kernel, dim3(static_cast<unsigned>((M + each - 1) / each)), dim3(team), 0, stream, true, a);
}

template <class Args, class F>
cudaError_t with_vectors(int64_t K, const Args& a, int64_t M, cudaStream_t stream, F kernel) {
  switch (vectors_of(K)) {
    case 1: return launch_rows<Args>(kernel.template of<1>(), a, M, K, stream);
    case 2: return launch_rows<Args>(kernel.template of<2>(), a, M, K, stream);
    case 3: return launch_rows<Args>(kernel.template of<3>(), a, M, K, stream);
    case 4: return launch_rows<Args>(kernel.template of<4>(), a, M, K, stream);
    case 5: return launch_rows<Args>(kernel.template of<5>(), a, M, K, stream);
    case 6: return launch_rows<Args>(kernel.template of<6>(), a, M, K, stream);
    case 7: return launch_rows<Args>(kernel.template of<7>(), a, M, K, stream);
    default: return launch_rows<Args>(kernel.template of<8>(), a, M, K, stream);
  }
}
static_assert(vectors_of(PRISM_MAX_ROW) == 8, "the longest row");

template <bool kDelta>
struct NormKernel {
  template <int C>
  auto of() const { return norm_kernel<C, kDelta>; }
};
template <bool kGate>
struct HeadKernel {
  template <int C>
  auto of() const { return head_norm_kernel<C, kGate>; }
};
struct GluKernel {
  template <int C>
  auto of() const { return glu_kernel<C>; }
};

}  // namespace

cudaError_t launch_norm_quant(const NormArgs& a, cudaStream_t stream) {
  return a.delta != nullptr ? with_vectors(a.K, a, a.M, stream, NormKernel<true>())
                            : with_vectors(a.K, a, a.M, stream, NormKernel<false>());
}
cudaError_t launch_head_norm_quant(const NormArgs& a, cudaStream_t stream) {
  return a.gate != nullptr ? with_vectors(a.K, a, a.M, stream, HeadKernel<true>())
                           : with_vectors(a.K, a, a.M, stream, HeadKernel<false>());
}
cudaError_t launch_glu_quant(const GluArgs& a, cudaStream_t stream) {
  return with_vectors(a.F, a, a.M, stream, GluKernel());
}

}  // namespace prism
