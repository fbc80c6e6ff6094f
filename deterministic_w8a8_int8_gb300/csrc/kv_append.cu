// kv_append.cu -- append K/V rows to the paged int8 cache, one scale per
// (page, head).
#include "decode.cuh"

namespace prism {
namespace {

constexpr int kThreads = 128;

// scale = amax * RN(1/127) and code = rint(x * (127 * RN(1/amax))): one
// reciprocal for a page instead of two divisions; every step binary32 RN, so
// a page's codes are a fixed function of its rows.
__device__ __forceinline__ float page_scale(float amax) { return __fmul_rn(amax, 1.0f / 127.0f); }
__device__ __forceinline__ float code_factor(float amax) { return __fmul_rn(__frcp_rn(amax), 127.0f); }

// One CTA per (sequence, head, K or V) walks the pages that get rows.
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ KvAppendArgs a) {
  __shared__ float s_red[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const KvPages& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int s = blockIdx.x, h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  SeqSpan sp;
  if (!seq_span(c, a.cu_new, a.T, s, false, sp)) {
    if (tid == 0 && a.err != nullptr) atomicOr(a.err, PRISM_DEV_ERR_SEQ_RANGE);
    return;
  }
  if (sp.n == 0) return;
  const uint16_t* rows = is_v ? a.v : a.k;
  const int64_t ld_t = is_v ? a.ldv_t : a.ldk_t, ld_h = is_v ? a.ldv_h : a.ldk_h;
  int8_t* codes = is_v ? c.v_codes : c.k_codes;
  float* scales = is_v ? c.v_scale : c.k_scale;
  uint16_t* open = (is_v ? a.v_open : a.k_open) + (static_cast<int64_t>(s) * c.H + h) * c.block * c.D;
  const int64_t before = sp.len, after = sp.len + sp.n;
  for (int64_t pb = before >> c.block_shift; (pb << c.block_shift) < after; ++pb) {
    const int64_t p0 = pb << c.block_shift;
    const int n_rows = static_cast<int>(min(static_cast<int64_t>(c.block), after - p0));
    auto value = [&](int r, int d) {
      const int64_t pos = p0 + r;
      const uint16_t* src = pos < before ? open + static_cast<int64_t>(r) * c.D
                                         : rows + (sp.b + pos - before) * ld_t + h * ld_h;
      return src[d];
    };
    float amax = 0.0f;
    for (int i = tid; i < n_rows * c.D; i += kThreads)
      amax = fmaxf(amax, fabsf(bf16_bits_to_float(value(i / c.D, i % c.D))));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (lane == 0) s_red[warp] = amax;
    __syncthreads();
    amax = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
    const bool zero = !(amax >= 0x1p-120f);
    const float inv = zero ? 0.0f : code_factor(amax);
    const int32_t page = c.table[s * c.ld_table + pb];
    if (page < 0 || page >= c.num_pages) {
      if (tid == 0 && a.err != nullptr) atomicOr(a.err, PRISM_DEV_ERR_PAGE_RANGE);
    } else {
      const int64_t ph = static_cast<int64_t>(page) * c.H + h;
      if (tid == 0) scales[ph] = zero ? 0.0f : page_scale(amax);
      int8_t* dst = codes + ph * c.block * c.D;
      for (int i = tid; i < n_rows * c.D; i += kThreads) {
        const float x = bf16_bits_to_float(value(i / c.D, i % c.D));
        dst[i] = static_cast<int8_t>(max(-127, min(127, __float2int_rn(__fmul_rn(x, inv)))));
      }
    }
    __syncthreads();   // the open rows and s_red have been read
    if (after - p0 < c.block) {
      for (int i = tid; i < n_rows * c.D; i += kThreads) open[i] = value(i / c.D, i % c.D);
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t stream) {
  return launch_kernel(kv_append_kernel, dim3(a.c.S, a.c.H, 2), dim3(kThreads), 0, stream, true, a);
}

}  // namespace prism
