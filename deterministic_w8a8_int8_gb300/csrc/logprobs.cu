// logprobs.cu -- log probabilities of given tokens under full-vocabulary
// logits, with the entropy and the top alternatives.
#include "decode.cuh"

namespace prism {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

__device__ __forceinline__ float logit(const LogprobArgs& a, int64_t at) {
  return a.f32 ? static_cast<const float*>(a.logits)[at]
               : bf16_bits_to_float(static_cast<const uint16_t*>(a.logits)[at]);
}
// Larger keys come first: the value's order, then the lower id.
__device__ __forceinline__ unsigned long long order_key(float x, uint32_t id) {
  const uint32_t u = __float_as_uint(__fadd_rn(x, 0.0f));   // -0 and +0 are equal
  const uint32_t o = u & 0x80000000u ? ~u : u | 0x80000000u;
  return (static_cast<unsigned long long>(o) << 32) | (0xffffffffu - id);
}
__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t o = static_cast<uint32_t>(k >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}

// One CTA per row: the maximum, the sums, then top_k passes.
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const __grid_constant__ LogprobArgs a) {
  __shared__ float s_a[kWarps], s_b[kWarps];
  __shared__ unsigned long long s_k[kWarps];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r = blockIdx.x, row = r * a.ldl;
  float m = -INFINITY;
  bool nan = false;
  for (int64_t v = tid; v < a.V; v += kThreads) {
    const float x = logit(a, row + v);
    nan |= x != x;
    m = fmaxf(m, x);
  }
  if (nan) m = INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) s_a[warp] = m;
  __syncthreads();
  m = s_a[0];
  for (int w = 1; w < kWarps; ++w) m = fmaxf(m, s_a[w]);
  __syncthreads();
  const bool ok = m > -INFINITY && m < INFINITY;
  float s = 0.0f, e = 0.0f;
  for (int64_t v = tid; v < a.V; v += kThreads) {
    const float y = logit(a, row + v) - m, p = exp2f(y * kLog2e);
    s += p;
    if (p > 0.0f) e = fmaf(p, y, e);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    e += __shfl_xor_sync(0xffffffffu, e, o);
  }
  if (lane == 0) s_a[warp] = s, s_b[warp] = e;
  __syncthreads();
  s = e = 0.0f;
  for (int w = 0; w < kWarps; ++w) s += s_a[w], e += s_b[w];
  const float nanf = __uint_as_float(0x7fc00000u), logz = log2f(s) * kLn2;
  if (tid == 0 && a.entropy != nullptr) a.entropy[r] = ok ? logz - e / s : nanf;
  for (int i = tid; i < a.n_ids; i += kThreads) {
    const int32_t id = a.ids[r * a.ld_ids + i];
    const bool in = id >= 0 && id < a.V;
    if (!in && a.err != nullptr) atomicOr(a.err, PRISM_DEV_ERR_ID_RANGE);
    a.logprobs[r * a.n_ids + i] = ok && in ? (logit(a, row + id) - m) - logz : nanf;
  }
  unsigned long long last = ~0ull;
  for (int k = 0; k < a.top_k; ++k) {
    unsigned long long best = 0;
    for (int64_t v = tid; v < a.V; v += kThreads) {
      const unsigned long long key = order_key(logit(a, row + v), static_cast<uint32_t>(v));
      if (key < last && key > best) best = key;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    __syncthreads();
    if (lane == 0) s_k[warp] = best;
    __syncthreads();
    best = s_k[0];
    for (int w = 1; w < kWarps; ++w) best = max(best, s_k[w]);
    if (tid == 0) {
      a.top_ids[r * a.top_k + k] = ok ? static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(best)) : -1;
      a.top_logprobs[r * a.top_k + k] = ok ? (key_value(best) - m) - logz : nanf;
    }
    last = best;
  }
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t stream) {
  return launch_kernel(logprobs_kernel, dim3(static_cast<unsigned>(a.R)), dim3(kThreads), 0, stream, true, a);
}

}  // namespace prism
