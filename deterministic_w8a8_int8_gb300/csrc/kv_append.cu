// kv_append.cu -- append K/V rows to the paged int8 cache, one scale per
// (page, head).
//
// A page's codes and scale are a function of its rows: amax over the rows, one
// scale, codes by one factor.  The rows of a sequence's open page are kept in
// bf16 as well and looked at again whenever rows are added: a scale that differs
// from the one in place (amax raised, or its row dropped by a sequence set back)
// is followed by a fresh quantisation of the whole page, and so is the row that
// completes it.  Where the scale stays (all but ln(block) of a page's rows, for
// values in random order) the earlier codes do, and only the new rows' are written.
//
// Bytes: 2 in and 1 out per value, 2 more out for the rows of a page that
// stays open -- HBM-bound for prompts; one generated token is a chain of three
// dependent reads (offsets, page and rows, scale).  One CTA per (sequence, page,
// head, K or V): a page's rows stay in registers between the maximum and the
// codes.  64 clients' rows of one token take 5.2 us; prompts of 24 million values
// 19.8 us, 3.6 TB/s; 69 % of the issue slots are taken (magnitudes one by one and
// codes rounded by a conversion: 21.5 us).
// CTAs that walk several pages and read the next one ahead: 20.7 us, and 7.4 us
// for single tokens.
#include "decode.cuh"

namespace prism {
namespace {

constexpr int kThreads = 256;

// scale = amax * RN(1/127) and code = rint(x * (127 * RN(1/amax))): one
// reciprocal for a page instead of two divisions; every step binary32 RN, so
// a page's codes are a fixed function of its rows.
__device__ __forceinline__ float page_scale(float amax) {
  return amax >= 0x1p-120f ? __fmul_rn(amax, 1.0f / 127.0f) : 0.0f;
}
__device__ __forceinline__ float code_factor(float amax) {
  return amax >= 0x1p-120f ? __fmul_rn(__frcp_rn(amax), 127.0f) : 0.0f;
}
// The larger magnitudes of m's two bf16 halves and the even and odd channels of v.
__device__ __forceinline__ uint32_t max8(const uint4& v, uint32_t m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(w[i] & 0x7fff7fffu));
  return m;
}
// rint(x f) for |x f| < 2^22 by the addition of 1.5 * 2^23, whose low byte is
// then the code; |x f| <= 127 (1 + 2^-22), so nothing needs a clamp.
__device__ __forceinline__ uint32_t code_bits(float x, float f) {
  return __float_as_uint(__fadd_rn(__fmul_rn(x, f), 12582912.0f));
}
__device__ __forceinline__ uint2 codes8(const uint4& v, float f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = __byte_perm(code_bits(bf16_lo(w[i]), f), code_bits(bf16_hi(w[i]), f), 0x0040u);
  return make_uint2(__byte_perm(c[0], c[1], 0x5410u), __byte_perm(c[2], c[3], 0x5410u));
}

// NV: 16-byte pieces of a page's bf16 rows per thread.
template <int NV>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ KvAppendArgs a, int row_shift) {
  __shared__ float s_red[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  const KvPages& c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int s = blockIdx.x, h = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  SeqSpan sp;
  if (!seq_span(c, a.cu_new, a.T, s, false, sp)) {
    if (tid == 0 && blockIdx.y == 0 && blockIdx.z == 0 && a.err != nullptr) atomicOr(a.err, PRISM_DEV_ERR_SEQ_RANGE);
    return;
  }
  if (sp.n == 0) return;
  const int64_t ld_t = is_v ? a.ldv_t : a.ldk_t;
  // row of position p: rows + (p - before) * ld_t
  const uint16_t* rows = (is_v ? a.v : a.k) + sp.b * ld_t + h * (is_v ? a.ldv_h : a.ldk_h);
  float* scales = is_v ? c.v_scale : c.k_scale;
  uint16_t* open = (is_v ? a.v_open : a.k_open) + ((static_cast<int64_t>(s) * c.H + h) << c.block_shift) * c.D;
  const int64_t before = sp.len, after = sp.len + sp.n;
  const int64_t first = before >> c.block_shift, open_page = after >> c.block_shift;
  const int64_t pages = ((after - 1) >> c.block_shift) - first + 1;
  // piece i of a page: row i >> row_shift, channels 8 (i mod 2^row_shift) on
  const int col = (tid & ((1 << row_shift) - 1)) * 8;   // 2^row_shift divides kThreads: the same for a thread's pieces
  for (int64_t j = blockIdx.z; j < pages; j += gridDim.z) {
    const int64_t p0 = (first + j) << c.block_shift;
    const int n_old = static_cast<int>(max(static_cast<int64_t>(0), before - p0));
    const int n_rows = static_cast<int>(min(static_cast<int64_t>(c.block), after - p0));
    const int32_t page = c.table[s * c.ld_table + first + j];
    uint4 x[NV];
    uint32_t most = 0u;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int r = (i * kThreads + tid) >> row_shift;
      x[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r >= n_old && r < n_rows) x[i] = *reinterpret_cast<const uint4*>(rows + (p0 + r - before) * ld_t + col);
    }
    if (n_old > 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int r = (i * kThreads + tid) >> row_shift;
        if (r < n_old) x[i] = *reinterpret_cast<const uint4*>(open + r * c.D + col);
      }
    }
    const bool page_ok = page >= 0 && page < c.num_pages;
    const int64_t ph = static_cast<int64_t>(page) * c.H + h;
    const float old_scale = page_ok && n_old > 0 ? scales[ph] : 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) most = max8(x[i], most);
    float amax = fmaxf(bf16_lo(most), bf16_hi(most));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    __syncthreads();
    if (lane == 0) s_red[warp] = amax;
    __syncthreads();
    amax = s_red[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) amax = fmaxf(amax, s_red[w]);
    // first row whose codes are written: those of the same scale stand already
    const int from = n_old > 0 && open_page == first && page_scale(amax) == old_scale ? n_old : 0;
    if (page_ok) {
      const float f = code_factor(amax);
      if (tid == 0 && from == 0) scales[ph] = page_scale(amax);
      int8_t* dst = (is_v ? c.v_codes : c.k_codes) + (ph << c.block_shift) * c.D + col;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int r = (i * kThreads + tid) >> row_shift;
        if (r >= from && r < n_rows) *reinterpret_cast<uint2*>(dst + r * c.D) = codes8(x[i], f);
      }
    } else if (tid == 0 && a.err != nullptr) {
      atomicOr(a.err, PRISM_DEV_ERR_PAGE_RANGE);
    }
    // ---- the open page's rows, by the CTA of the first page: only it reads
    // the open buffer, and it has (the barriers come after its reads)
    if (j == 0) {
      const int64_t o0 = open_page << c.block_shift;
      const int begin = open_page == first ? n_old : 0, end = static_cast<int>(after - o0);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int r = (i * kThreads + tid) >> row_shift;
        if (r >= begin && r < end)
          *reinterpret_cast<uint4*>(open + r * c.D + col) =
              open_page == first ? x[i] : *reinterpret_cast<const uint4*>(rows + (o0 + r - before) * ld_t + col);
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t stream) {
  const int shift = a.c.D == 64 ? 3 : a.c.D == 128 ? 4 : 5;
  const int pieces = a.c.block * a.c.D / 8 / kThreads;
  auto kernel = pieces <= 1   ? kv_append_kernel<1>
                : pieces <= 2 ? kv_append_kernel<2>
                : pieces <= 4 ? kv_append_kernel<4>
                : pieces <= 8 ? kv_append_kernel<8>
                              : kv_append_kernel<16>;
  // pages that max_new rows can touch; a sequence with more is walked in turns
  const int64_t pages = std::min<int64_t>((a.max_new + 2 * a.c.block - 2) >> a.c.block_shift, 65535);
  return launch_kernel(kernel, dim3(a.c.S, a.c.H * 2, static_cast<unsigned>(pages)), dim3(kThreads), 0, stream, true, a,
                       shift);
}

}  // namespace prism
