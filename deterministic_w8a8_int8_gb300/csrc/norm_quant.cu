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
// codes, 8 to a 16-byte vector, C vectors a thread (vectors_of).  Two exchanges in
// shared memory (three with a post norm) stand in the way of a row, the sum's and
// the largest magnitude's; the next row's loads are under way across them, and the
// other CTAs of the SM work.
//
// A call's bytes (each operand once) are its floor; rows of 5120 and 17408, at 6784 GB/s:
//   norm   8192 rows with a delta 48.8 us (89 % of that rate), 2048 rows with a delta's
//          norm 19.6 us (63 %: a fill and seven CTAs' rows an SM, two sums in a row's way)
//   heads  8192 rows of 40 heads of 128 with gates 57.2 us (54 %: 73 instructions for two
//          values, 70 % of the issue slots, the ALU and FMA pipes 49 and 43 %)
//   glu    2048 rows 43.6 us (72 %: issue slots 58 %, weights from L2, sigmoids from
//          shared memory)
// One row takes 3.2 us, 64 rows of 17408 4.9: a launch, a row's loads and two exchanges.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "decode.cuh"
#include "layer.cuh"

namespace prism {
namespace {

constexpr int kMaxTeam = 512;
constexpr int kWarps = kMaxTeam / 32;

__device__ __forceinline__ float2 twice(float v) { return make_float2(v, v); }

// Sums of squares of bf16 values, two side by side.  They begin at the largest
// square of the thread's, which is taken off again at the end: with no addend
// above the sum, the error of an addition is what its difference leaves of the
// addend, three operations instead of six (Dekker's form).
struct Squares {
  float2 h, l;
  float top;
  __device__ __forceinline__ explicit Squares(float largest) : l(make_float2(0.0f, 0.0f)), top(largest * largest) {
    h = make_float2(top, top);
  }
  __device__ __forceinline__ void add(float2 v) {
    const float2 s = fma2(v, v, h);
    l = add2(l, fma2(v, v, fma2(s, twice(-1.0f), h)));
    h = s;
  }
  __device__ __forceinline__ Sum sum() const {
    return join(join(Sum{h.x, l.x}, Sum{h.y, l.y}), Sum{-2.0f * top, 0.0f});
  }
};
// The largest magnitude of a vector's values, and of what was there: bf16 pairs,
// whose magnitudes are ordered as their bits are.
__device__ __forceinline__ uint32_t larger(uint32_t m, const uint4& v) {
  constexpr uint32_t kMagnitude = 0x7fff7fffu;
  return __vimax3_u16x2(__vimax3_u16x2(m, v.x & kMagnitude, v.y & kMagnitude), v.z & kMagnitude, v.w & kMagnitude);
}
__device__ __forceinline__ float largest(uint32_t m) { return fmaxf(bf16_lo(m), bf16_hi(m)); }

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

// n / d rounded to nearest for d = -minus, 1 <= d <= 2: Markstein's quotient
// (1990).  The reciprocal's approximation and one step of Newton's iteration, and
// the remainder, which one fused operation forms exactly, put back.  There are 2^16
// gates, and the tests compare each one's result.
__device__ __forceinline__ float2 divide2(float2 n, float2 minus) {
  float2 r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(-minus.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(-minus.y));
  r = fma2(fma2(minus, r, twice(1.0f)), r, r);
  const float2 q = mul2(n, r);
  return fma2(fma2(minus, q, n), r, q);
}

// 1 / (1 + exp(-z)) of two values as (1 or e) / (1 + e), e = exp(-|z|) by n ln 2 + r
// (ln 2 in two parts), the series of e^r to r^7 in fused steps, times 2^n.  From
// |z| = 88 on n would be -127 or less, and 2^n counts as 0.
__device__ __forceinline__ float2 sigmoid2(float2 z) {
  constexpr float kMagic = 12582912.0f + 127.0f;   // 1.5 * 2^23, whose unit is 1, and the exponent's bias
  const float2 x = make_float2(fmaxf(-fabsf(z.x), -88.0f), fmaxf(-fabsf(z.y), -88.0f));
  const float2 t = fma2(x, twice(0x1.715476p+0f), twice(kMagic)), n = add2(t, twice(-kMagic));
  float2 r = fma2(n, twice(-0x1.63p-1f), x);
  r = fma2(n, twice(0x1.bd0106p-13f), r);
  float2 p = fma2(twice(0x1.a01a02p-13f), r, twice(0x1.6c16c2p-10f));
  p = fma2(p, r, twice(0x1.111112p-7f));
  p = fma2(p, r, twice(0x1.555556p-5f));
  p = fma2(p, r, twice(0x1.555556p-3f));
  p = fma2(p, r, twice(0x1p-1f));
  p = fma2(p, r, twice(1.0f));
  p = fma2(p, r, twice(1.0f));
  const float2 e = mul2(p, make_float2(__uint_as_float(__float_as_uint(t.x) << 23), __uint_as_float(__float_as_uint(t.y) << 23)));
  const float2 top = make_float2(z.x >= 0.0f ? 1.0f : e.x, z.y >= 0.0f ? 1.0f : e.y);
  return divide2(top, fma2(e, twice(-1.0f), twice(-1.0f)));
}

__device__ __forceinline__ float2 pair(uint32_t v) { return make_float2(bf16_lo(v), bf16_hi(v)); }
__device__ __forceinline__ uint32_t bf16x2(float2 v) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
// z * sigmoid(z), rounded once more.
__device__ __forceinline__ float2 silu2(uint32_t gates) {
  const float2 z = pair(gates);
  return mul2(z, sigmoid2(z));
}
// The sigmoids of all gates in shared memory: bf16 values whose magnitudes lie from
// 2^-25, up to where exp(-|z|) rounds to 1, to 88, from where on it counts as 0.
// The magnitudes' bits are the places, those with the sign behind the others.
struct SigmoidTable {
  static constexpr uint32_t kFirst = 0x3300u, kLast = 0x42b0u, kNegative = 0x4000u;   // bits of 2^-25 and 88; bytes
  static constexpr int kBytes = 2 * kNegative;
  static_assert((kLast - kFirst + 1) * 4 <= kNegative, "places of one sign");
  const uint8_t* at;
  __device__ __forceinline__ void build(uint8_t* smem) {   // the caller's barrier follows
    at = smem;
    for (uint32_t i = threadIdx.x; i <= kLast - kFirst; i += blockDim.x) {
      const float z = bf16_lo(kFirst + i);
      const float2 v = sigmoid2(make_float2(z, -z));
      *reinterpret_cast<float*>(smem + 4 * i) = v.x;
      *reinterpret_cast<float*>(smem + kNegative + 4 * i) = v.y;
    }
  }
  __device__ __forceinline__ float2 silu2(uint32_t gates) const {
    // max(min(magnitude - kFirst, kLast - kFirst), 0) of both
    const uint32_t m = __viaddmin_s16x2_relu(gates & 0x7fff7fffu, (0x10000u - kFirst) * 0x10001u, (kLast - kFirst) * 0x10001u);
    const uint32_t place = (m | ((gates >> 3) & (kNegative / 4 * 0x10001u))) << 2;
    return mul2(pair(gates), make_float2(*reinterpret_cast<const float*>(at + (place & 0xffffu)),
                                         *reinterpret_cast<const float*>(at + (place >> 16))));
  }
};
// Weights of the four pairs of channels 8 j .. 8 j + 7.
struct Weights {
  float4 a, b;
  Weights() = default;
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
  if (warps == 1) return s;
  if (lane == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  s = red[0];
  for (int i = 1; i < warps; ++i) s = join(s, red[i]);
  return s;
}

__device__ __forceinline__ float max3(float a, float b, float c) {   // NaN where one of them is
  float v;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(v) : "f"(a), "f"(b), "f"(c));
  return v;
}

// The codes of the CTA's rows whose scale is NaN are 0 (0 * NaN is no code): after the last
// row, since in the rows' way this takes the kernels registers (8192 rows of 40 heads 35.6
// us without a gate instead of 34.6; as a call, 300 rows of 96 gated heads 7.8 instead of 7.4).
__device__ __forceinline__ void clear_marked(const RowCodes& o, int64_t M, int nvec) {
  __syncthreads();   // the scales were written
  for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
    if (!isnan(*static_cast<volatile float*>(o.a_scale + row))) continue;
#pragma unroll 1
    for (int j = threadIdx.x; j < nvec; j += blockDim.x) {   // what the thread itself has written
      if (o.form == PRISM_FORM_F16) {
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(o.q) + row * o.ldq)[j] = make_uint4(0u, 0u, 0u, 0u);
      } else {
        reinterpret_cast<uint2*>(static_cast<int8_t*>(o.q) + row * o.ldq)[j] = make_uint2(0u, 0u);
      }
    }
  }
}

// The row's values y, 8 C a thread (0 past the row's end), as codes.  Where they are not
// all finite the scale is NaN, which the next linear passes on, the codes are those of
// clear_marked, and the answer, one for the CTA, is true.
template <int C>
__device__ __forceinline__ bool store_codes(const RowCodes& o, int64_t row, int nvec, const float2 (&y)[C][4], uint32_t* red) {
  const int team = blockDim.x, lt = threadIdx.x, lane = lt & 31;
  if (o.form == PRISM_FORM_BF16) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int j = lt + i * team;
      if (j < nvec)
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(o.q) + row * o.ldq)[j] =
            make_uint4(bf16x2(y[i][0]), bf16x2(y[i][1]), bf16x2(y[i][2]), bf16x2(y[i][3]));
    }
    return false;
  }
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) top = max3(top, fabsf(y[i][e].x), fabsf(y[i][e].y));
  // magnitudes are ordered as their bits are, NaN above all
  const uint32_t wm = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
  if (lane == 0) red[lt >> 5] = wm;
  __syncthreads();
  const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, lane < (team >> 5) ? red[lane] : 0u));
  const bool marked = !(amax < __int_as_float(0x7f800000)), dead = marked || amax < 0x1p-120f;
  const float inv = dead ? 0.0f : __fdiv_rn(127.0f, amax);
  if (lt == 0) o.a_scale[row] = dead ? __fmul_rn(amax, 0.0f) : __fdiv_rn(amax, 127.0f);
  // t + 1.5 * 2^23 is t rounded to an integer, in the low bits
  constexpr float kMagic = 12582912.0f;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int j = lt + i * team;
    if (j >= nvec) continue;
    float2 t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      t[e] = mul2(y[i][e], twice(inv));
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
  return marked;
}

// A thread's vectors of one operand's next row, on their way through shared
// memory: each thread copies and reads its own, so that no barrier is needed, and
// refills a place as soon as it has read it.
struct Ahead {
  uint32_t at;             // of vector 0
  int nvec;
  __device__ __forceinline__ Ahead(const uint8_t* smem, int operand, int vectors, int nvec)
      : at(smem_u32(smem) + (operand * vectors * blockDim.x + threadIdx.x) * 16), nvec(nvec) {}
  __device__ __forceinline__ int index(int i) const { return threadIdx.x + i * static_cast<int>(blockDim.x); }
  __device__ __forceinline__ void fill(const uint16_t* row, int i) const {
    if (index(i) < nvec) cp_async_16(at + i * blockDim.x * 16, row + index(i) * 8, 16);
  }
  __device__ __forceinline__ uint4 read(int i) const {   // zeros past the row's end
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (index(i) < nvec)
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                   : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                   : "r"(at + i * blockDim.x * 16)
                   : "memory");
    return v;
  }
};

// CTAs of an SM at least, by registers.
constexpr int ctas_of(int C) { return C <= 5 ? 2 : 1; }

template <int C, bool kDelta>
__global__ void __maxnreg__(C <= 4 ? 56 : C <= 6 ? 80 : 128) norm_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Sum s_sum[2][kWarps], s_post[2][kWarps];
  __shared__ uint32_t s_top[2][kWarps];
  pdl_trigger();
  pdl_wait();
  const int team = blockDim.x, lt = threadIdx.x, nvec = static_cast<int>(a.K >> 3);
  const Ahead ax(smem, 0, C, nvec), ad(smem, 1, C, nvec);
  bool marked = false;
  int64_t row = blockIdx.x;
  auto fill = [&](int64_t r) {
    if (r < a.M) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        ax.fill(a.x + r * a.ldx, i);
        if constexpr (kDelta) ad.fill(a.delta + r * a.ldd, i);
      }
    }
    cp_async_commit();
  };
  fill(row);
  for (int par = 0; row < a.M; row += gridDim.x, par ^= 1) {
    cp_async_wait<0>();
    uint4 x[C], d[kDelta ? C : 1];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      x[i] = ax.read(i);
      if constexpr (kDelta) d[i] = ad.read(i);
    }
    fill(row + gridDim.x);
    uint32_t m = 0;
    if constexpr (kDelta) {
      float r = 1.0f;
      if (a.post != nullptr) {
#pragma unroll
        for (int i = 0; i < C; ++i) m = larger(m, d[i]);
        Squares s(largest(m));
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) s.add(pair(word(d[i], e)));
        r = inverse_root(team_sum(s.sum(), s_post[par]), a.inv_n, a.inv_n_low, a.eps);
        m = 0;
      }
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int j = lt + i * team;
        if (j >= nvec) continue;
        float2 w[4];
        if (a.post != nullptr) {
          const Weights p(a.post, j);
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = mul2(mul2(pair(word(d[i], e)), twice(r)), p[e]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = pair(word(d[i], e));
        }
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 add = mul2(w[e], twice(a.alpha)), v = pair(word(x[i], e));
          h[e] = bf16x2(make_float2(__fadd_rn(v.x, add.x), __fadd_rn(v.y, add.y)));   // scalar: not merged with the product
        }
        x[i] = make_uint4(h[0], h[1], h[2], h[3]);
        reinterpret_cast<uint4*>(a.h + row * a.ldh)[j] = x[i];
      }
    }
#pragma unroll
    for (int i = 0; i < C; ++i) m = larger(m, x[i]);
    Squares s(largest(m));
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) s.add(pair(word(x[i], e)));
    const float r = inverse_root(team_sum(s.sum(), s_sum[par]), a.inv_n, a.inv_n_low, a.eps);
    float2 y[C][4];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int j = lt + i * team;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[i][e] = mul2(pair(word(x[i], e)), twice(r));
      if (j >= nvec) continue;
      const Weights w(a.weight, j);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[i][e] = mul2(y[i][e], w[e]);
    }
    marked |= store_codes<C>(a.o, row, nvec, y, s_top[par]);
  }
  cp_async_wait<0>();
  if (marked) clear_marked(a.o, a.M, nvec);
}

// A head's channels lie in D / 8 = `lanes` neighbouring lanes, and the sums of a
// thread's N vectors belong to N heads: with each exchange the lanes of one half
// take over half of the sums and the others the rest, until each lane has one,
// whose root it forms, and the roots are handed round.
template <int N>
__device__ __forceinline__ void head_roots(const Sum (&t)[N], int lanes, const NormArgs& a, float (&r)[N]) {
  const int lane = threadIdx.x & 31;
  auto exchanged = [&](Sum s, int o) {
    return Sum{__shfl_xor_sync(0xffffffffu, s.h, o), __shfl_xor_sync(0xffffffffu, s.l, o)};
  };
  auto half = [&](Sum s, Sum other, int o) {   // s of the lanes without bit o, the other of those with it
    const bool upper = lane & o;
    return join(upper ? other : s, exchanged(upper ? s : other, o));
  };
  int o = lanes >> 1;
  Sum s;
  if constexpr (N == 4) {
    const Sum u = half(t[0], t[2], o), v = half(t[1], t[3], o);
    o >>= 1;
    s = half(u, v, o);
    o >>= 1;
  } else if constexpr (N == 2) {
    s = half(t[0], t[1], o);
    o >>= 1;
  } else {
    s = t[0];
  }
  for (; o > 0; o >>= 1) s = join(s, exchanged(s, o));
  const float root = inverse_root(s, a.inv_n, a.inv_n_low, a.eps);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int from = N == 4 ? (i >> 1) * (lanes >> 1) + (i & 1) * (lanes >> 2) : N == 2 ? i * (lanes >> 1) : 0;
    r[i] = N == 1 ? root : __shfl_sync(0xffffffffu, root, (lane & ~(lanes - 1)) + from);
  }
}

template <int C, bool kGate, bool kTable>
__global__ void __maxnreg__(C <= 2 ? 64 : C == 4 ? 80 : 128) head_norm_kernel(const __grid_constant__ NormArgs a) {
  constexpr int N = C < 4 ? C : 4;
  static_assert(C % N == 0, "vectors go by in groups");
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint32_t s_top[2][kWarps];
  pdl_trigger();
  SigmoidTable table;
  if constexpr (kTable) table.build(smem);
  pdl_wait();
  constexpr int kRows = kTable ? SigmoidTable::kBytes : 0;
  const int nvec = static_cast<int>(a.K >> 3), lanes = a.D >> 3;
  const Ahead ax(smem + kRows, 0, C, nvec), az(smem + kRows, 1, C, nvec);
  bool marked = false;
  int64_t row = blockIdx.x;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    ax.fill(a.x + row * a.ldx, i);
    if constexpr (kGate) az.fill(a.gate + row * a.ldg, i);
  }
  if constexpr (kTable) __syncthreads();
  const Weights w(a.weight, threadIdx.x & (lanes - 1));   // a team is whole heads wide, or the row is one turn
  for (int par = 0; row < a.M; row += gridDim.x, par ^= 1) {
    const int64_t next = row + gridDim.x;
    float2 y[C][4];
    cp_async_commit();
    cp_async_wait<0>();
#pragma unroll
    for (int g = 0; g < C; g += N) {
      Sum t[N];
      float r[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint4 x = ax.read(g + i);
        Squares s(largest(larger(0u, x)));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[g + i][e] = pair(word(x, e));
          s.add(y[g + i][e]);
        }
        t[i] = s.sum();
        if (next < a.M) ax.fill(a.x + next * a.ldx, g + i);
      }
      head_roots<N>(t, lanes, a, r);
#pragma unroll
      for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) y[g + i][e] = mul2(mul2(y[g + i][e], twice(r[i])), w[e]);
        const bool smooth = a.inv_s != nullptr && ax.index(g + i) < nvec;
        Weights p;
        if (smooth) p = Weights(a.inv_s, ax.index(g + i));
        if constexpr (kGate) {
          const uint4 z = az.read(g + i);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[g + i][e] = mul2(y[g + i][e], kTable ? table.silu2(word(z, e)) : silu2(word(z, e)));
          if (next < a.M) az.fill(a.gate + next * a.ldg, g + i);
        }
        if (smooth) {
#pragma unroll
          for (int e = 0; e < 4; ++e) y[g + i][e] = mul2(y[g + i][e], p[e]);
        }
      }
    }
    marked |= store_codes<C>(a.o, row, nvec, y, s_top[par]);
  }
  cp_async_wait<0>();
  if (marked) clear_marked(a.o, a.M, nvec);
}

template <int C, bool kTable>
__global__ void __launch_bounds__(kMaxTeam, ctas_of(C)) glu_kernel(const __grid_constant__ GluArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint32_t s_top[2][kWarps];
  pdl_trigger();
  SigmoidTable table;
  if constexpr (kTable) table.build(smem);
  pdl_wait();
  constexpr int kRows = kTable ? SigmoidTable::kBytes : 0;
  const int nvec = static_cast<int>(a.F >> 3);
  const Ahead ag(smem + kRows, 0, C, nvec), au(smem + kRows, 1, C, nvec);
  bool marked = false;
  int64_t row = blockIdx.x;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    ag.fill(a.x + row * a.ldx, i);
    au.fill(a.x + row * a.ldx + a.F, i);
  }
  if constexpr (kTable) __syncthreads();
  for (int par = 0; row < a.M; row += gridDim.x, par ^= 1) {
    const int64_t next = row + gridDim.x;
    float2 y[C][4];
    cp_async_commit();
    cp_async_wait<0>();
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const uint4 g = ag.read(i), u = au.read(i);
      const bool smooth = a.inv_s != nullptr && ag.index(i) < nvec;
      Weights p;
      if (smooth) p = Weights(a.inv_s, ag.index(i));   // on its way beside the sigmoids
#pragma unroll
      for (int e = 0; e < 4; ++e) y[i][e] = mul2(kTable ? table.silu2(word(g, e)) : silu2(word(g, e)), pair(word(u, e)));
      if (next < a.M) {
        ag.fill(a.x + next * a.ldx, i);
        au.fill(a.x + next * a.ldx + a.F, i);
      }
      if (smooth) {
#pragma unroll
        for (int e = 0; e < 4; ++e) y[i][e] = mul2(y[i][e], p[e]);
      }
    }
    marked |= store_codes<C>(a.o, row, nvec, y, s_top[par]);
  }
  cp_async_wait<0>();
  if (marked) clear_marked(a.o, a.M, nvec);
}

// Vectors of 8 values a thread.  Sums cost a thread some 100 instructions, which many
// vectors share (norm of 2048 rows of 5120: 24 us with 2, 19 with 4); more than 4 cost
// the SM warps, and only rows beyond kMaxTeam threads have them (heads 8, which go by in
// fours).  A gate's steps fill the time that sums leave: gated heads have 2 vectors up
// to 8192 channels (8192 rows of 5120: 55.8 us, with 4 56.4; 304 of them 4.1 and 4.8;
// without a gate 39.2 and 34.0, 3.3 and 2.75).  The team follows from the row's length
// alone, and with it the order of its sums.
enum Rows { kNormRows, kHeadRows, kGatedHeadRows };
constexpr int vectors_of(int64_t K, Rows rows) {
  const int64_t n = K / 8;
  return n <= 32                                            ? 1
         : n <= (rows == kGatedHeadRows ? 2 * kMaxTeam : 64) ? 2
         : n <= 4 * kMaxTeam                                 ? 4
         : rows != kNormRows                                 ? 8
                                                             : static_cast<int>((n + kMaxTeam - 1) / kMaxTeam);
}
constexpr int team_of(int64_t K, int c) { return static_cast<int>(32 * ((K / 8 + 32 * c - 1) / (32 * c))); }

// A launch with as many CTAs as the SMs hold, each with `operands` vectors' rows ahead
// and `more` bytes of shared memory in front of them.
template <class Args>
cudaError_t launch_rows(void (*kernel)(const Args), std::atomic<int>* held, const Args& a, int64_t M, int64_t K, int c, int operands,
                        int more, cudaStream_t stream) {
  const int team = team_of(K, c);
  const int bytes = operands * c * team * 16 + more;
  cudaError_t e = cudaSuccess;   // 48 KB need no attribute, the kernel's own arrays among them
  if (bytes > 40 * 1024) e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), operands * c * kMaxTeam * 16 + more);
  if (e != cudaSuccess) return e;
  int per_sm = held[team / 32].load(std::memory_order_relaxed);   // a property of the kernel and its team
  if (per_sm == 0) {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, team, bytes);
    if (e != cudaSuccess) return e;
    per_sm = std::max(per_sm, 1);
    held[team / 32].store(per_sm, std::memory_order_relaxed);
  }
  const int64_t most = static_cast<int64_t>(sm_count()) * per_sm;
  return launch_kernel(kernel, dim3(static_cast<unsigned>(std::min(M, most))), dim3(team), bytes, stream, true, a);
}

// Whether CTAs make themselves a table of sigmoids: it costs each as much as 8034
// gates, about 1 us behind another kernel, and its shared memory costs an SM CTAs
// where they are small.  glu without and with it, 304 rows of 8192 behind a copy 5.7
// and 6.1 us, of 17408 10.0 and 9.7, 2048 rows of 17408 52.9 and 43.4; heads, 304
// rows of 8192 6.3 and 6.6, 8192 rows of 5120 74 and 57, 1536 rows of 2048 (128
// threads) 7.5 and 8.1, 4096 of them 15.9 and 14.2.
inline bool worth_table(int64_t M, int64_t K, int team) {
  return team >= 128 && M >= (static_cast<int64_t>(sm_count()) * 32768 + K - 1) / K;
}

template <class F, int C, class Args>
cudaError_t launch_c(const Args& a, int64_t M, int64_t K, cudaStream_t stream) {
  static std::atomic<int> held[2][kWarps + 1];
  if constexpr (C >= F::kTables) {
    if (worth_table(M, K, team_of(K, C)))
      return launch_rows<Args>(F::template of<C, true>(), held[1], a, M, K, C, F::kOperands, SigmoidTable::kBytes, stream);
  }
  return launch_rows<Args>(F::template of<C, false>(), held[0], a, M, K, C, F::kOperands, 0, stream);
}
template <class F, class Args>
cudaError_t launch_any(const Args& a, int64_t M, int64_t K, cudaStream_t stream) {
  switch (vectors_of(K, F::kRows)) {
    case 1: return launch_c<F, 1>(a, M, K, stream);
    case 2: return launch_c<F, 2>(a, M, K, stream);
    case 4: return launch_c<F, 4>(a, M, K, stream);
    case 5: return launch_c<F, F::kRows != kNormRows ? 8 : 5>(a, M, K, stream);
    case 6: return launch_c<F, F::kRows != kNormRows ? 8 : 6>(a, M, K, stream);
    case 7: return launch_c<F, F::kRows != kNormRows ? 8 : 7>(a, M, K, stream);
    default: return launch_c<F, 8>(a, M, K, stream);
  }
}
static_assert(vectors_of(PRISM_MAX_ROW, kNormRows) == 8 && PRISM_MAX_ROW <= 64 * kMaxTeam, "the longest row");

// kTables: vectors a thread from which on a table may pay, where teams can have 128
// threads (rows of 2 vectors a thread have 32, but for gated heads); 9: none.
template <bool kDelta>
struct NormKernel {
  static constexpr int kOperands = kDelta ? 2 : 1;
  static constexpr Rows kRows = kNormRows;
  static constexpr int kTables = 9;
  template <int C, bool kTable>
  static auto of() { return norm_kernel<C, kDelta>; }
};
template <bool kGate>
struct HeadKernel {
  static constexpr int kOperands = kGate ? 2 : 1;
  static constexpr Rows kRows = kGate ? kGatedHeadRows : kHeadRows;
  static constexpr int kTables = kGate ? 2 : 9;
  template <int C, bool kTable>
  static auto of() { return head_norm_kernel<C, kGate, kTable>; }
};
struct GluKernel {
  static constexpr int kOperands = 2;
  static constexpr Rows kRows = kNormRows;
  static constexpr int kTables = 4;
  template <int C, bool kTable>
  static auto of() { return glu_kernel<C, kTable>; }
};

}  // namespace

cudaError_t launch_norm_quant(const NormArgs& a, cudaStream_t stream) {
  return a.delta != nullptr ? launch_any<NormKernel<true>>(a, a.M, a.K, stream) : launch_any<NormKernel<false>>(a, a.M, a.K, stream);
}
cudaError_t launch_head_norm_quant(const NormArgs& a, cudaStream_t stream) {
  return a.gate != nullptr ? launch_any<HeadKernel<true>>(a, a.M, a.K, stream) : launch_any<HeadKernel<false>>(a, a.M, a.K, stream);
}
cudaError_t launch_glu_quant(const GluArgs& a, cudaStream_t stream) { return launch_any<GluKernel>(a, a.M, a.F, stream); }

}  // namespace prism
