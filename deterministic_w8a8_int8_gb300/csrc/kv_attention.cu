// kv_attention.cu -- attention of new queries over the paged int8 K/V cache.
#include "decode.cuh"

namespace prism {
namespace {

constexpr int kWarps = 4;

// One CTA per (query token, query head); its warps take every fourth key, a
// lane holds D / 32 channels.  Online softmax per warp, joined at the end.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) kv_attention_kernel(const __grid_constant__ KvAttentionArgs a) {
  constexpr int E = D / 32;
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  __shared__ int s_seq, s_bad;
  pdl_trigger();
  pdl_wait();
  const KvPages& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t t = blockIdx.x;
  const int h = blockIdx.y, hk = h / a.G;
  if (tid == 0) s_seq = -1, s_bad = 0;
  __syncthreads();
  for (int s = tid; s < c.S; s += kWarps * 32) {
    const int64_t b = a.cu_q != nullptr ? a.cu_q[s] : s, e = a.cu_q != nullptr ? a.cu_q[s + 1] : s + 1;
    if (b >= 0 && b <= t && t < e && e <= a.T) s_seq = s;
    if (t == 0 && h == 0 && (b < 0 || e < b || e > a.T) && a.err != nullptr) atomicOr(a.err, PRISM_DEV_ERR_SEQ_RANGE);
  }
  __syncthreads();
  const int s = s_seq;
  if (s < 0) return;
  SeqSpan sp;
  const bool ok = seq_span(c, a.cu_q, a.T, s, true, sp) && sp.n <= a.max_q;
  const int64_t pos = sp.len - sp.n + (t - sp.b);
  const int64_t hi = !ok ? 0 : a.causal ? min(sp.len, pos + 1) : sp.len;
  const int64_t lo = a.window > 0 ? max(static_cast<int64_t>(0), pos + 1 - a.window) : 0;
  float q[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = bf16_bits_to_float(a.q[t * a.ldq_t + h * a.ldq_h + lane * E + i]);
    o[i] = 0.0f;
  }
  for (int64_t j = lo + warp; j < hi; j += kWarps) {
    const int32_t page = c.table[s * c.ld_table + (j >> c.block_shift)];
    if (page < 0 || page >= c.num_pages) {
      s_bad = 1;
      break;
    }
    const int64_t ph = static_cast<int64_t>(page) * c.H + hk;
    const int64_t at = (ph * c.block + (j & (c.block - 1))) * D + lane * E;
    float x = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) x = fmaf(q[i], static_cast<float>(c.k_codes[at + i]), x);
#pragma unroll
    for (int r = 16; r > 0; r >>= 1) x += __shfl_xor_sync(0xffffffffu, x, r);
    x *= c.k_scale[ph] * a.scale_log2;
    const float mn = fmaxf(m, x), al = exp2f(m - mn), p = exp2f(x - mn);
    l = fmaf(l, al, p);
    const float pv = p * c.v_scale[ph];
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = fmaf(o[i], al, pv * static_cast<float>(c.v_codes[at + i]));
    m = mn;
  }
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
  for (int i = 0; i < E; ++i) s_o[warp][lane * E + i] = o[i];
  __syncthreads();
  const bool bad = !ok || s_bad;
  if (bad && tid == 0 && a.err != nullptr) atomicOr(a.err, ok ? PRISM_DEV_ERR_PAGE_RANGE : PRISM_DEV_ERR_SEQ_RANGE);
  float mx = -INFINITY;
  for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_m[w]);
  float f[kWarps], sum = 0.0f;
  for (int w = 0; w < kWarps; ++w) {
    f[w] = s_m[w] == -INFINITY ? 0.0f : exp2f(s_m[w] - mx);
    sum = fmaf(f[w], s_l[w], sum);
  }
  for (int d = tid; d < D; d += kWarps * 32) {
    float y = 0.0f;
    for (int w = 0; w < kWarps; ++w) y = fmaf(f[w], s_o[w][d], y);
    y = lo >= hi ? 0.0f : y / sum;
    a.out[t * a.ldo_t + h * a.ldo_h + d] = static_cast<uint16_t>(bad ? kBf16NaN : float_to_bf16_rne(y));
  }
  if (tid == 0 && a.lse != nullptr)
    a.lse[t * a.Hq + h] = bad ? __uint_as_float(0x7fc00000u) : lo >= hi ? -INFINITY : (mx + log2f(sum)) * 0.69314718f;
}

}  // namespace

size_t kv_attention_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) {
  return 0;
}

cudaError_t launch_kv_attention(const KvAttentionArgs& a, cudaStream_t stream) {
  auto kernel = a.c.D == 64 ? kv_attention_kernel<64> : a.c.D == 128 ? kv_attention_kernel<128> : kv_attention_kernel<256>;
  return launch_kernel(kernel, dim3(static_cast<unsigned>(a.T), a.Hq), dim3(kWarps * 32), 0, stream, true, a);
}

}  // namespace prism
