// kv_attention_tc.cu -- attention over the paged int8 cache for many rows (a
// prompt's piece, questions of many tokens) on the tcgen05 tensor cores.
//
// A tile is 128 rows (queries x heads of a KV head), each a lane of tensor
// memory.  Two threads have a row, one for each half of a block's keys (and of
// the output's channels); they exchange their maxima.  Keys go by in blocks of
// KB:
//   S = Q K^T      D / 16 steps of kind::f16, M 128, N KB; into KB columns
//   O += P V       KB / 16 steps, M 128, N D; P as the A operand from tensor
//                  memory, each half over its own half of S
// Bound by issue slots: the codes of a block become binary16 once for the 128
// rows (exactly: byte ^ 0x80 under the exponent of 1024, minus 1152), K as its
// rows, V transposed (8 keys of a channel are one 16-byte piece), both into the
// 128-byte-swizzled K-major operand layout; and each score costs about six
// instructions.  Raw codes of the next block are read ahead into registers.
// Two CTAs on an SM (one for D = 256) overlap one's conversion and softmax with
// the other's instructions.
//
// Scores are scaled as in the few-row kernel (queries by a power of two, ks of
// the unit of 16 keys).  The reference of the exponents follows the row's
// maximum only when that grows by more than 2^kSlack: then the threads rescale
// the row's output in tensor memory.  Probabilities are binary16 with 2^kShift as the
// value of the reference (2^15 at most), times vs relative to the piece's
// largest; sums and outputs are binary32.
//
// Every wait is bounded: after 2 s the kernel sets the device status bit, lets
// its instructions in flight complete and returns.
#include "kv_plan.cuh"
#include "tc_common.cuh"

namespace prism {

__device__ uint32_t g_kv_status = 0;

namespace {

using namespace kv;

constexpr unsigned long long kWaitNs = 2000000000ull;
constexpr float kShift = 9.0f, kSlack = 6.0f;
constexpr int kThreads = 256;

template <int D>
struct Tc {
  static constexpr int kKeys = D == 256 ? 64 : 128;            // keys of a block
  static constexpr int kUnits = kKeys / 16;
  static constexpr int kCtas = D == 256 ? 1 : 2;               // on an SM: tensor memory has 512 columns
  static constexpr int kCols = kKeys + D <= 256 ? 256 : 512;
  static constexpr int kQ = kWideRows * D * 2, kK = kKeys * D * 2, kV = kKeys * D * 2;
  static constexpr int kBytes = kQ + kK + kV + 1024;           // operands start on 1024-byte boundaries
  static constexpr int kLoadsK = kKeys * D / 16 / kThreads;    // 16-byte pieces of K a thread converts
  static constexpr int kLoadsV = kKeys / 8 * (D / 4) / kThreads;   // 8 keys x 4 channels of V
};

// One answer for the warp, whose lanes are together again afterwards.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, tc::mbar_wait_bounded(bar, parity, abort_flag, kWaitNs, &g_kv_status,
                                                       PRISM_DEVSTATUS_WAIT_TIMEOUT));
}

template <int D>
__global__ void __launch_bounds__(kThreads, Tc<D>::kCtas)
    kv_attention_tc_kernel(const __grid_constant__ KvAttentionArgs a, int64_t part_stride) {
  using C = Tc<D>;
  constexpr int KB = C::kKeys, U = C::kUnits;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_scan[kThreads];
  __shared__ int s_warp[kThreads / 32];
  __shared__ float s_max[kThreads / 32];
  __shared__ float s_top[2][kWideRows], s_l[kWideRows];   // the halves' maxima; one half's sum
  __shared__ int32_t s_page[3][U];       // of block j in buffer j mod 3
  __shared__ float s_ks[3][U], s_vr[3][U];
  __shared__ __align__(8) uint64_t s_bar[3];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* s_q = smem;
  uint8_t* s_k = s_q + C::kQ;
  uint8_t* s_v = s_k + C::kK;
  const uint32_t bar_s = smem_u32(&s_bar[0]), bar_o = smem_u32(&s_bar[1]), bar_end = smem_u32(&s_bar[2]);
  if (tid == 0) {
    tc::mbar_init(bar_s, 1);
    tc::mbar_init(bar_o, 1);
    tc::mbar_init(bar_end, 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(C::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = s_tmem;
  // this warp's 32 lanes, and its half of the scores' and the output's columns
  const int half = warp >> 2, r = tid & (kWideRows - 1);
  const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp & 3) << 21);
  const uint32_t t_s = t_lane + half * (KB / 2), t_o = t_lane + KB + half * (D / 2);
  constexpr int UH = U / 2;         // units of a half
  pdl_trigger();
  pdl_wait();
  const KvPages& c = a.c;
  uint32_t ph_s = 0, ph_o = 0;      // parity of the next completion
  bool ok = true;

  Walk walk;
  SeqPlan p;
  for (int64_t item = blockIdx.x; ok && find_item<true, kWideRows, kThreads>(a, item, walk, s_scan, s_warp, p); item += gridDim.x) {
    const int hk = walk.hk;
    const TileKeys keys(a, p, walk, kWideRows);
    const int32_t k_begin = keys.k_begin, k_end = keys.k_end;
    const int blocks = k_end > k_begin ? (k_end - k_begin + KB - 1) / KB : 0;
    const int32_t* table = c.table + walk.s * c.ld_table;

    // ---- the piece's largest value scale, and its pages' validity
    bool bad_page = false;
    float v_top = 0.0f;
    if (blocks > 0) {
      for (int32_t i = (k_begin >> c.block_shift) + tid; i <= (k_end - 1) >> c.block_shift; i += kThreads) {
        const int32_t page = table[i];
        if (page < 0 || page >= c.num_pages) {
          bad_page = true;
        } else {
          v_top = fmaxf(v_top, c.v_scale[static_cast<int64_t>(page) * c.H + hk]);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v_top = fmaxf(v_top, __shfl_xor_sync(0xffffffffu, v_top, o));
    if (lane == 0) s_max[warp] = v_top;
    const bool bad = __syncthreads_or(bad_page);
    v_top = s_max[0];
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) v_top = fmaxf(v_top, s_max[i]);
    const float v_inv = v_top >= 0x1p-126f ? __frcp_rn(v_top) : 0.0f;

    // page ids and scales of block j's units (threads below U)
    auto unit_page = [&](int j) {
      const int32_t key = k_begin + j * KB + tid * 16;
      const int32_t page = key < k_end ? table[key >> c.block_shift] : 0;
      return page < 0 || page >= c.num_pages ? 0 : page;
    };
    auto unit_scales = [&](int j, int32_t page) {
      const int64_t at = static_cast<int64_t>(page) * c.H + hk;
      return k_begin + j * KB + tid * 16 < k_end ? make_float2(c.k_scale[at], c.v_scale[at] * v_inv) : make_float2(0.0f, 0.0f);
    };
    auto stage_units = [&](int j, int32_t page, float2 scales) {
      s_page[j % 3][tid] = page;
      s_ks[j % 3][tid] = scales.x;
      s_vr[j % 3][tid] = scales.y;
    };
    uint4 kr[C::kLoadsK];
    uint32_t vr[C::kLoadsV][8];
    auto row_ptr = [&](const int8_t* codes, int j, int key) {   // key of block j
      const int32_t pos = k_begin + j * KB + key;
      return codes + ((static_cast<int64_t>(s_page[j % 3][key >> 4]) * c.H + hk) * c.block + (pos & (c.block - 1))) * D;
    };
    auto load_k = [&](int j) {
#pragma unroll
      for (int i = 0; i < C::kLoadsK; ++i) {
        const int at = i * kThreads + tid;
        kr[i] = ld_stream_16(row_ptr(c.k_codes, j, at / (D / 16)) + at % (D / 16) * 16);
      }
    };
    // item i: keys 8 kg .. + 7, channels 4 dq .. + 3; a warp has 4 kg x 8 dq
    auto v_kg = [&](int i) { return (i * 8 + warp) / (D / 32) * 4 + (lane & 3); };
    auto v_dq = [&](int i) { return (i * 8 + warp) % (D / 32) * 8 + (lane >> 2); };
    auto load_v = [&](int j) {
#pragma unroll
      for (int i = 0; i < C::kLoadsV; ++i) {
        const int8_t* src = row_ptr(c.v_codes, j, v_kg(i) * 8) + v_dq(i) * 4;
#pragma unroll
        for (int k = 0; k < 8; ++k) vr[i][k] = __ldg(reinterpret_cast<const uint32_t*>(src + k * D));
      }
    };
    if (tid < U) {
      for (int j = 0; j < min(blocks, 2); ++j) {
        const int32_t page = unit_page(j);
        stage_units(j, page, unit_scales(j, page));
      }
    }
    __syncwarp();

    // ---- the tile's queries as binary16, K-major: row r, a half of its channels
    float unit;
    {
      const int tok = (keys.row0 + r) / a.G, g = keys.row0 + r - tok * a.G;
      const uint16_t* qp = a.q + static_cast<int64_t>(p.sp.b + tok) * a.ldq_t + static_cast<int64_t>(hk * a.G + g) * a.ldq_h;
      const bool live = r < keys.n_rows;
      float amax = 0.0f;
#pragma unroll 8
      for (int i = 0; i < D / 8; ++i) {
        if (live) {
          const uint4 v = *reinterpret_cast<const uint4*>(qp + i * 8);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
        }
      }
      const int fe = query_exponent(amax);
      const float f = __uint_as_float(static_cast<uint32_t>(fe) << 23);
      unit = __uint_as_float(static_cast<uint32_t>(254 - fe) << 23) * a.scale_log2;
#pragma unroll 8
      for (int i = half * (D / 16); i < (half + 1) * (D / 16); ++i) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (live) v = *reinterpret_cast<const uint4*>(qp + i * 8);
        const uint4 h = make_uint4(half2_bits(bf16_lo(v.x) * f, bf16_hi(v.x) * f), half2_bits(bf16_lo(v.y) * f, bf16_hi(v.y) * f),
                                   half2_bits(bf16_lo(v.z) * f, bf16_hi(v.z) * f), half2_bits(bf16_lo(v.w) * f, bf16_hi(v.w) * f));
        *reinterpret_cast<uint4*>(s_q + (i >> 3) * (kWideRows * 128) + r * 128 + (((i & 7) ^ (r & 7)) << 4)) = h;
      }
    }
    const int32_t row_hi = keys.hi(r), my_lo = keys.lo(row_hi), my_hi = min(row_hi, k_end);
    __syncthreads();   // pages and scales of blocks 0 and 1
    if (blocks > 0) {
      load_k(0);
      load_v(0);
    }
    float m = -INFINITY, l = 0.0f;

    for (int j = 0; j < blocks; ++j) {
      // ---- K: 16 codes of a key are two pieces of the operand
#pragma unroll
      for (int i = 0; i < C::kLoadsK; ++i) {
        const int at = i * kThreads + tid, key = at / (D / 16), ch = at % (D / 16);
        const uint32_t x = kr[i].x ^ 0x80808080u, y = kr[i].y ^ 0x80808080u, z = kr[i].z ^ 0x80808080u, w = kr[i].w ^ 0x80808080u;
        uint8_t* dst = s_k + (ch >> 2) * (KB * 128) + key * 128;
        const int piece = (ch & 3) * 2;
        *reinterpret_cast<uint4*>(dst + ((piece ^ (key & 7)) << 4)) =
            make_uint4(widen(x, 0x4140u), widen(x, 0x4342u), widen(y, 0x4140u), widen(y, 0x4342u));
        *reinterpret_cast<uint4*>(dst + (((piece + 1) ^ (key & 7)) << 4)) =
            make_uint4(widen(z, 0x4140u), widen(z, 0x4342u), widen(w, 0x4140u), widen(w, 0x4342u));
      }
      if (j + 1 < blocks) load_k(j + 1);
      const bool stage = tid < U && j + 2 < blocks;   // this thread reads a unit of block j + 2 ahead
      int32_t next_page = 0;
      float2 next_scales = make_float2(0.0f, 0.0f);
      if (stage) next_page = unit_page(j + 2);
      tc::fence_proxy_async();
      if (j > 0) {          // P V of the block before: it read P where S goes now, and V
        if (!wait(bar_o, ph_o, &s_abort)) ok = false;
        ph_o ^= 1;
        tc::tc_fence_after();
      }
      tc::tc_fence_before();
      __syncthreads();      // K (and the queries) in place, S's columns free
      if (tid == 0) {
        tc::tc_fence_after();
        const uint32_t idesc = tc::idesc_f16_f32(KB);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc::tc_mma(tmem, tc::smem_desc_sw128(smem_u32(s_q) + (k >> 2) * (kWideRows * 128)) + 2 * (k & 3),
                     tc::smem_desc_sw128(smem_u32(s_k) + (k >> 2) * (KB * 128)) + 2 * (k & 3), idesc, k != 0 ? 1u : 0u);
        tc::tc_commit(bar_s);
      }
      __syncwarp();
      // ---- V, transposed: 8 keys of a channel are one piece of the operand
#pragma unroll
      for (int i = 0; i < C::kLoadsV; ++i) {
        uint32_t h[4][4];   // [channel][key pair]
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t x = __byte_perm(vr[i][2 * k], vr[i][2 * k + 1], 0x5140u) ^ 0x80808080u;
          const uint32_t y = __byte_perm(vr[i][2 * k], vr[i][2 * k + 1], 0x7362u) ^ 0x80808080u;
          h[0][k] = widen(x, 0x4140u);
          h[1][k] = widen(x, 0x4342u);
          h[2][k] = widen(y, 0x4140u);
          h[3][k] = widen(y, 0x4342u);
        }
        const int kg = v_kg(i), d0 = v_dq(i) * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<uint4*>(s_v + (kg >> 3) * (D * 128) + (d0 + e) * 128 + (((kg & 7) ^ ((d0 + e) & 7)) << 4)) =
              make_uint4(h[e][0], h[e][1], h[e][2], h[e][3]);
      }
      if (j + 1 < blocks) load_v(j + 1);
      if (stage) next_scales = unit_scales(j + 2, next_page);
      tc::fence_proxy_async();

      // ---- softmax of the row's half: the block's maximum, then P over S
      if (!wait(bar_s, ph_s, &s_abort)) ok = false;
      ph_s ^= 1;
      tc::tc_fence_after();
      const int32_t key0 = k_begin + j * KB, my_key = key0 + half * (KB / 2);
      const bool edge = key0 < keys.a_lo || key0 + KB > min(keys.a_hi, k_end);   // some row does not see all of it, or the next piece has it
      const float* ks = s_ks[j % 3] + half * UH;
      const float* vs = s_vr[j % 3] + half * UH;
      float top = -INFINITY;
#pragma unroll
      for (int u = 0; u < UH; ++u) {
        uint32_t x[16];
        tc::tmem_ld16(t_s + u * 16, x);
        tc::tmem_wait_ld();
        float t = -INFINITY;
        if (edge) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int32_t key = my_key + u * 16 + e;
            if (key >= my_lo && key < my_hi) t = fmaxf(t, __uint_as_float(x[e]));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) t = fmaxf(t, __uint_as_float(x[e]));
        }
        if (t > -INFINITY) top = fmaxf(top, t * (ks[u] * unit));
      }
      s_top[half][r] = top;
      __syncthreads();
      top = fmaxf(top, s_top[half ^ 1][r]);
      const float old = m;
      if (top > m + kSlack || m == -INFINITY) m = top;
      const float al = old == m ? 1.0f : ex2(old - m);   // old = -inf: nothing to keep
      if (__any_sync(0xffffffffu, al != 1.0f) && j > 0) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint32_t o[16];
          tc::tmem_ld16(t_o + i * 16, o);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
          tc::tmem_st16(t_o + i * 16, o);
        }
      }
      l *= al;
      const float base = m == -INFINITY ? 0.0f : m - kShift;
#pragma unroll
      for (int u = 0; u < UH; u += 2) {
        uint32_t pk[16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t x[16];
          tc::tmem_ld16(t_s + (u + h) * 16, x);
          tc::tmem_wait_ld();
          const float f = ks[u + h] * unit, vf = vs[u + h];
          float q[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) q[e] = ex2(__fmaf_rn(__uint_as_float(x[e]), f, -base));
          if (edge) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int32_t key = my_key + (u + h) * 16 + e;
              if (key < my_lo || key >= my_hi) q[e] = 0.0f;
            }
          }
          float l0 = 0.0f, l1 = 0.0f;
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            l0 += q[e];
            l1 += q[e + 1];
            pk[h * 8 + e / 2] = half2_bits(q[e] * vf, q[e + 1] * vf);
          }
          l += l0 + l1;
        }
        tc::tmem_st16(t_s + u * 8, pk);   // over scores that this thread has read
      }
      tc::tmem_wait_st();
      if (stage) stage_units(j + 2, next_page, next_scales);
      tc::tc_fence_before();
      if (__syncthreads_or(!ok)) {        // P, V and the next block's units in place
        ok = false;
        break;
      }
      if (tid == 0) {
        tc::tc_fence_after();
        const uint32_t idesc = tc::idesc_f16_f32(D);
#pragma unroll
        for (int k = 0; k < KB / 16; ++k)
          tc::tc_mma_ta(tmem + KB, tmem + k / UH * (KB / 2) + k % UH * 8, tc::smem_desc_sw128(smem_u32(s_v) + (k >> 2) * (D * 128)) + 2 * (k & 3), idesc,
                        (j | k) != 0 ? 1u : 0u);
        tc::tc_commit(bar_o);
      }
      __syncwarp();
    }
    if (ok && blocks > 0) {
      if (!wait(bar_o, ph_o, &s_abort)) ok = false;
      ph_o ^= 1;
      tc::tc_fence_after();
    }
    if (__syncthreads_or(!ok)) {
      ok = false;
      break;
    }

    // ---- the row's output, or its piece
    if (half == 1) s_l[r] = l;
    __syncthreads();
    if (half == 0) s_l[r] = l + s_l[r];
    __syncthreads();
    l = s_l[r];
    if (bad && tid == 0 && a.err != nullptr) atomicOr(a.err, PRISM_DEV_ERR_PAGE_RANGE);
    const float nanf = __uint_as_float(0x7fc00000u);
    const int tok = (keys.row0 + r) / a.G, h = hk * a.G + keys.row0 + r - tok * a.G;
    const int64_t t = p.sp.b + tok;
    const bool live = r < keys.n_rows;
    const bool some = m > -INFINITY || l != l;   // saw a key (or a NaN score)
    float* ps = static_cast<float*>(a.ws) +
                ((static_cast<int64_t>(walk.s) * c.H + hk) * part_stride + walk.split * p.rows + keys.row0 + r) * (D + 4);
    const float scale = !some ? 0.0f : p.splits == 1 ? v_top / l : v_top;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint32_t o[16] = {};
      if (blocks > 0) {
        tc::tmem_ld16(t_o + i * 16, o);
        tc::tmem_wait_ld();
      }
      const int d = half * (D / 2) + i * 16;
      float y[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] = some ? __uint_as_float(o[e]) * scale : 0.0f;
      if (live && p.splits == 1) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[e] = bad ? kBf16NaN * 0x10001u : float_to_bf16_rne(y[2 * e]) | float_to_bf16_rne(y[2 * e + 1]) << 16;
        uint4* dst = reinterpret_cast<uint4*>(a.out + t * a.ldo_t + h * a.ldo_h + d);
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
      } else if (live) {
#pragma unroll
        for (int e = 0; e < 16; e += 4)
          *reinterpret_cast<float4*>(ps + 4 + d + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
      }
      __syncwarp();
    }
    if (live && half == 0) {
      const float mx = some ? m - kShift + kPShift : -INFINITY;   // the weights' common form
      if (p.splits > 1) {
        ps[0] = bad ? nanf : mx;
        ps[1] = l;
      } else if (a.lse != nullptr) {
        a.lse[t * a.Hq + h] = bad ? nanf : !some ? mx : (mx - kPShift + log2f(l)) * kLn2;
      }
    }
    tc::tc_fence_before();
    __syncthreads();   // the queries, s_scan and the output's columns are free again
    tc::tc_fence_after();
  }

  // ---- every instruction in flight completes before the columns are given back
  if (tid == 0) {
    tc::tc_commit(bar_end);
    tc::mbar_wait_drain_bounded(bar_end, 0, kWaitNs, &g_kv_status, PRISM_DEVSTATUS_WAIT_TIMEOUT);
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols) : "memory");
  }
}

template <int D>
cudaError_t launch_d(const KvAttentionArgs& a, int64_t part_stride, cudaStream_t stream) {
  using C = Tc<D>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kv_attention_tc_kernel<D>), C::kBytes);
  if (e != cudaSuccess) return e;
  const int64_t tiles = a.T * a.G / kWideRows + a.c.S;
  const int64_t items = (tiles + part_stride / kFewRows * a.c.S) * a.c.H;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(items, sm_count() * C::kCtas));
  return launch_kernel(kv_attention_tc_kernel<D>, dim3(grid), dim3(kThreads), C::kBytes, stream, false, a, part_stride);
}

}  // namespace

cudaError_t launch_kv_attention_wide(const KvAttentionArgs& a, int64_t part_stride, cudaStream_t stream) {
  return a.c.D == 64    ? launch_d<64>(a, part_stride, stream)
         : a.c.D == 128 ? launch_d<128>(a, part_stride, stream)
                        : launch_d<256>(a, part_stride, stream);
}

cudaError_t read_and_clear_kv_status(uint32_t* out) {
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_kv_status, sizeof v);
  if (e != cudaSuccess) return e;
  if (v != 0) {
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_kv_status, &zero, sizeof zero);
  }
  *out = v;
  return e;
}

}  // namespace prism
