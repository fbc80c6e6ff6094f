// linear_plan.cuh -- how a call of linear attention is cut up, and what its
// kernels share.
//
// Up to kFewTokens tokens of a sequence take the recurrence as it stands, more
// go by in chunks.  A long sequence is cut into segments, by its length and the
// number of heads alone, so that a sequence's bits do not depend on the batch: a
// first kernel forms each segment's own state from zero, and the second starts
// each segment from the states and decays of those before it.
#pragma once

#include "decode.cuh"
#include "layer.cuh"

namespace prism {
namespace lin {

// Tokens that take the recurrence.  40 heads of 128 by 128, 2, 4, 8 and 16 tokens by the
// recurrence: one sequence 3.8, 4.5, 6.3 and 9.7 us, 64 of them 60, 70, 92 and 136;
// in chunks 9.6 and 81 whatever the number (heads of 64 by 64: 8.8 and 60).
constexpr int kFewTokens = 8;
constexpr int kChunk = 64;
constexpr float kMinDecay = -16384.0f;   // e^x = 0 from far above it; sums of 64 stay finite

// The segments of a long sequence: those with which its heads fill the SMs in the
// fewest turns for what each then has to do, and one where more do not save a third: keys
// and values are read twice.  One sequence of 32767 tokens, 2 heads of 128 by 128, cut
// into 24, 48, 76 and 152 at most: 85, 65, 64 and 64 us, of one head 84, 61, 58 and 61.
// Segments of fewer tokens pay where a few heads leave SMs empty, and cost a batch the
// work twice.  2048 tokens, heads of 128 by 128, in us:
//   chunks                       2      4      8
//   8 heads, one sequence       27.3   29.8   38.3
//            four sequences     57.5   50.3
//   40 heads, one                      56.5   61.3
//             four                    180.7  161.0
constexpr int64_t kMaxSegments = 76;
inline Cut cut_of(int64_t Hv) {
  const int64_t most = std::max<int64_t>(8, std::min<int64_t>(kMaxSegments, kSms / Hv));
  auto turns = [&](int64_t n) { return (n * Hv + kSms - 1) / kSms; };
  int64_t best = 1;
  for (int64_t n = 2; n <= most; ++n)
    if (turns(n) * best < turns(best) * n) best = n;
  if (turns(best) * 3 > turns(1) * best * 2) best = 1;
  return Cut{best, best > 8 ? 8 : 9};
}
// Segments that a sequence of n tokens is cut into at most (two as short as may be do not
// earn the first kernel: 512 tokens of 8 heads of 128 by 128 in one 23.6, in two 28 us, 1024
// of 40 heads 40.1 and 41.4), the chunks of each, and as many as that makes.
__host__ __device__ __forceinline__ int64_t most_segments(int64_t n, const Cut& cut) {
  const int64_t segs = n >> cut.shift;
  return segs < 3 ? 1 : segs > cut.most ? cut.most : segs;
}
__host__ __device__ __forceinline__ int64_t segment_chunks(int64_t n, const Cut& cut) {
  const int64_t chunks = (n + kChunk - 1) / kChunk, segs = most_segments(n, cut);
  return (chunks + segs - 1) / segs;
}
__host__ __device__ __forceinline__ int64_t segment_count(int64_t n, const Cut& cut) {
  const int64_t chunks = (n + kChunk - 1) / kChunk, each = segment_chunks(n, cut);
  return (chunks + each - 1) / each;
}
// A sequence in segments has a place in the workspace for each but the last, and
// one for the state that it starts from.  They are counted by tokens, 2^shift at least to
// each, or by the segments that every sequence may have, whichever makes fewer: one text
// of 131071 tokens and 40 heads has 7 (18 MB), by tokens 255 (669 MB).
struct Places {
  int64_t total, each;   // each: a sequence's own; 0 where they go by tokens
};
inline Places places_of(int64_t S, int64_t T, int64_t max_len, const Cut& cut) {
  const int64_t segs = most_segments(max_len, cut), by_tokens = T >> cut.shift;
  if (segs <= 1) return Places{0, 0};
  return S * segs < by_tokens ? Places{S * segs, segs} : Places{by_tokens, 0};
}
__device__ __forceinline__ int64_t first_place(const LinAttnArgs& a, int64_t s, int64_t first_token) {
  return a.places_each != 0 ? s * a.places_each : first_token >> a.cut.shift;
}

struct Span {
  int64_t b, n;
  int64_t in, out;     // states: -1 for none
  bool bad;            // its rows get NaN, its state is not written
};
// Sequence s; false where its offsets are malformed (no rows to answer for).
__device__ __forceinline__ bool span_of(const LinAttnArgs& a, int64_t s, bool report, Span& p) {
  const int64_t b = a.cu != nullptr ? a.cu[s] : s, e = a.cu != nullptr ? a.cu[s + 1] : s + 1;
  p.b = b;
  p.n = e - b;
  p.in = a.state_in != nullptr ? a.state_in[s] : -1;
  p.out = a.state_out != nullptr ? a.state_out[s] : -1;
  const bool offsets = b >= 0 && e >= b && e <= a.T;
  const bool states = p.in >= -1 && p.in < a.num_states && p.out >= -1 && p.out < a.num_states;
  const bool length = p.n <= a.max_len;
  if (report && a.err != nullptr) {
    if (!offsets || !length) atomicOr(a.err, PRISM_DEV_ERR_SEQ_RANGE);
    if (!states) atomicOr(a.err, PRISM_DEV_ERR_STATE_RANGE);
  }
  p.bad = !states || !length;
  return offsets;
}

__device__ __forceinline__ float bounded_decay(float g) { return g < kMinDecay ? kMinDecay : g > 0.0f ? 0.0f : g; }
__device__ __forceinline__ float decay_of(const LinAttnArgs& a, int64_t token, int h) {
  return bounded_decay(__ldg(a.decay + token * a.ldd_t + h));
}

// ------------------------------------------------------------- few tokens ---
// One (sequence, head) and `width` of its columns from c0 on: kGroups groups of
// threads, group g on rows [g R, (g + 1) R), a thread on 4 columns.  Column sums
// are added in the order of the rows, whatever the width.  All of the CTA's threads
// take part, those past the groups' (kGroups * width / 4) at the barriers alone.
// What the tokens bring lies in shared memory before the first.
constexpr int kGroups = 8;
template <int DK>
__device__ __forceinline__ void few_tokens(const LinAttnArgs& a, const Span& p, int hv, int c0, int width, float* smem) {
  constexpr int R = DK / kGroups;
  float* s_q = smem;                               // [kFewTokens][DK]
  float* s_k = s_q + kFewTokens * DK;
  float* s_v = s_k + kFewTokens * DK;              // [kFewTokens][width]
  float* s_o = s_v + kFewTokens * width;           // [2][kGroups][width]
  float* s_d = s_o + 2 * kGroups * width;          // [kFewTokens]
  const int lanes = width >> 2, tid = threadIdx.x, group = tid / lanes, col = (tid % lanes) * 4;
  const bool in = group < kGroups;
  const int n = static_cast<int>(p.n), hk = hv / a.G;
  const int64_t plane = static_cast<int64_t>(DK) * a.Dv;
  float2 st[R][2];
  if (p.in >= 0 && !p.bad && in) {
    const float* src = a.state + (p.in * a.Hv + hv) * plane + static_cast<int64_t>(group * R) * a.Dv + c0 + col;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float4 x = __ldcs(reinterpret_cast<const float4*>(src + static_cast<int64_t>(i) * a.Dv));
      st[i][0] = make_float2(x.x, x.y);
      st[i][1] = make_float2(x.z, x.w);
    }
  } else {
    const float x = p.bad ? __uint_as_float(0x7fc00000u) : 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) st[i][0] = st[i][1] = make_float2(x, x);
  }
  auto widen8 = [](float* dst, const uint16_t* src) {
    const uint4 v = *reinterpret_cast<const uint4*>(src);
    reinterpret_cast<float4*>(dst)[0] = make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y));
    reinterpret_cast<float4*>(dst)[1] = make_float4(bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w));
  };
  for (int i = tid; i < n * (DK / 8); i += blockDim.x) {
    const int t = i / (DK / 8), c = i % (DK / 8) * 8;
    widen8(s_q + t * DK + c, a.q + (p.b + t) * a.ldq_t + hk * a.ldq_h + c);
    widen8(s_k + t * DK + c, a.k + (p.b + t) * a.ldk_t + hk * a.ldk_h + c);
  }
  for (int i = tid; i < n * (width / 8); i += blockDim.x) {
    const int t = i / (width / 8), c = i % (width / 8) * 8;
    widen8(s_v + t * width + c, a.v + (p.b + t) * a.ldv_t + hv * a.ldv_h + c0 + c);
  }
  if (tid < n) s_d[tid] = expf(decay_of(a, p.b + tid, hv));
  __syncthreads();
  for (int t = 0; t < n; ++t) {
    float* red = s_o + (t & 1) * kGroups * width;
    if (in) {
      const float2 d = make_float2(s_d[t], s_d[t]);
      const float4 vv = *reinterpret_cast<const float4*>(s_v + t * width + col);
      const float2 v[2] = {make_float2(vv.x, vv.y), make_float2(vv.z, vv.w)};
      float2 o[2] = {};
#pragma unroll
      for (int i = 0; i < R; i += 4) {
        const float4 k4 = *reinterpret_cast<const float4*>(s_k + t * DK + group * R + i);
        const float4 q4 = *reinterpret_cast<const float4*>(s_q + t * DK + group * R + i);
        const float ks[4] = {k4.x, k4.y, k4.z, k4.w}, qs[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            float2& x = st[i + e][f];
            x = fma2(make_float2(ks[e], ks[e]), v[f], mul2(d, x));
            o[f] = fma2(make_float2(qs[e], qs[e]), x, o[f]);
          }
      }
      *reinterpret_cast<float4*>(red + group * width + col) = make_float4(o[0].x, o[0].y, o[1].x, o[1].y);
    }
    __syncthreads();   // the other half was read before the last barrier
    for (int c = tid; c < width; c += blockDim.x) {
      float sum = red[c];
#pragma unroll
      for (int g = 1; g < kGroups; ++g) sum += red[g * width + c];
      a.out[(p.b + t) * a.ldo_t + hv * a.ldo_h + c0 + c] = static_cast<uint16_t>(float_to_bf16_rne(sum * a.scale));
    }
  }
  if (p.out >= 0 && !p.bad && in) {
    float* dst = a.state + (p.out * a.Hv + hv) * plane + static_cast<int64_t>(group * R) * a.Dv + c0 + col;
#pragma unroll
    for (int i = 0; i < R; ++i)
      __stcs(reinterpret_cast<float4*>(dst + static_cast<int64_t>(i) * a.Dv),
             make_float4(st[i][0].x, st[i][0].y, st[i][1].x, st[i][1].y));
  }
}
constexpr int few_smem(int DK, int width) { return (kFewTokens * (2 * DK + width + 1) + 2 * kGroups * width) * 4; }

// The rows of a sequence that cannot be answered.
__device__ __forceinline__ void spoil(const LinAttnArgs& a, const Span& p, int hv, int c0, int width) {
  for (int64_t i = threadIdx.x; i < p.n * width; i += blockDim.x)
    a.out[(p.b + i / width) * a.ldo_t + hv * a.ldo_h + c0 + i % width] = static_cast<uint16_t>(kBf16NaN);
}

// ----------------------------------------------------------------- chunks ---
// Two values as a pair of bf16, and what that leaves of them.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t split_bf16(float2& v) {
  const uint32_t r = pack_bf16(v.x, v.y);
  v = fma2(make_float2(bf16_lo(r), bf16_hi(r)), make_float2(-1.0f, -1.0f), v);
  return r;
}
__device__ __forceinline__ float ex2(float x) {   // to about 2^-22
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The decays of a chunk's 64 tokens, two a lane (0 past the end), summed up to
// each token and over the chunk, in powers of two.  (In binary64 this took the
// warp some 2000 cycles.)
struct Decays {
  Sum g[2], total;
};
__device__ __forceinline__ Decays sum_decays(const float (&dec)[2]) {
  constexpr float kLog2e = 1.44269504f, kLog2eLow = 1.92596299e-8f;
  const int lane = threadIdx.x & 31;
  Sum d[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    d[e].h = __fmul_rn(dec[e], kLog2e);
    d[e].l = fmaf(dec[e], kLog2eLow, fmaf(dec[e], kLog2e, -d[e].h));
  }
  Sum sum = join(d[0], d[1]);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sum v{__shfl_up_sync(0xffffffffu, sum.h, o), __shfl_up_sync(0xffffffffu, sum.l, o)};
    if (lane >= o) sum = join(sum, v);
  }
  Decays r;
  r.total = Sum{__shfl_sync(0xffffffffu, sum.h, 31), __shfl_sync(0xffffffffu, sum.l, 31)};
  r.g[0] = join(sum, Sum{-d[1].h, -d[1].l});
  r.g[1] = sum;
  return r;
}
// What the chunk's end has left of a token.
__device__ __forceinline__ float left_of(const Decays& d, int e) {
  return ex2(__fadd_rn(__fsub_rn(d.total.h, d.g[e].h), __fsub_rn(d.total.l, d.g[e].l)));
}

}  // namespace lin

// Sequences of more than lin::kFewTokens tokens (linear_attention_tc.cu).
template <int DK, int DV>
cudaError_t launch_linear_chunks(const LinAttnArgs& a, cudaStream_t stream);
}  // namespace prism
