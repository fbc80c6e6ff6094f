// kv_attention_tc.cu -- attention over the paged int8 cache for many rows (a
// prompt's piece, questions of many tokens) on the tcgen05 tensor cores.
//
// A tile is 128 rows (queries x heads of a KV head), each a lane of tensor
// memory.  Keys go by in blocks of KB:
//   S = Q K^T      D / 16 steps of kind::f16, M 128, N KB; into one of two buffers
//   O += P V       KB / 16 steps, M 128, N D; P as the A operand from tensor
//                  memory, in columns of its own, twice too
// An item is a range of the line of blocks (kv_plan.cuh), worked through a tile's
// part at a time.  One CTA an SM, with three kinds of warps that pass blocks on
// by mbarriers:
//   converters (4 warps for K, 4 for V)  read a block's codes ahead into
//     registers, 8 keys by 16 channels a thread, and widen them once for the 128
//     rows, exactly (byte ^ 0x80 under the exponent of 1024, minus 1152), into
//     two stages of the 128-byte-swizzled K-major operand layout: K as its rows,
//     V transposed (8 keys of a channel are one 16-byte piece);
//   the issuer (1 warp)   Q K^T of block j + 1 ahead of P V of block j;
//   softmax (8 warps)     two threads a row, one for each half of the block's
//     keys (and of the output's channels); they exchange their maxima.
//
// A block of 128 x 128 x 128 takes 2900 cycles: 512 of them the instructions
// could do with, and halving the softmax's work, either product's or either
// conversion takes 1 to 7 % off the whole -- the chain of signals between the
// warps bounds it.  A 512-token piece of 40 heads on 8 KV heads of 128 at 8187
// keys takes 138 us with its join (600 TFLOP/s), against 42.5 us of the
// instructions at bf16 peak.  Code that is unrolled further is slower: the
// instruction cache then misses (pieces of 16 keys unrolled and masked in place:
// 3760 cycles a block).
//
// Scores are scaled as in the few-row kernel (queries by a power of two, ks of
// the unit of 16 keys).  Probabilities are formed against the reference at hand
// in one pass over the scores; where a row's maximum stands more than 2^kSlack
// above it (always in a first block) the row's output in tensor memory is
// rescaled and the pass repeated against the new maximum.  Probabilities are
// binary16 with 2^kShift as the value of the reference (2^15 at most), times vs
// relative to the part's largest; sums and outputs are binary32.
//
// Every wait on an mbarrier is bounded: after 2 s (prism_debug_wait_expiry shortens
// that for tests) the kernel sets the device status bit; every warp then runs its loops out without waiting (so that the
// named barriers still meet), the instructions in flight complete, and the
// kernel returns.
#include <type_traits>

#include "kv_plan.cuh"
#include "tc_common.cuh"

namespace prism {

__device__ uint32_t g_kv_status = 0;
// Test mode (prism_debug_wait_expiry): the waits' limit, and whether each CTA's
// issuer withholds the signal that its first block's scores are formed.
__device__ unsigned long long g_kv_wait_limit_ns = 2000000000ull;
__device__ int g_kv_withhold = 0;

namespace {

using namespace kv;

constexpr unsigned long long kDrainNs = 2000000000ull;
constexpr float kShift = 9.0f, kSlack = 6.0f;
constexpr int kSoftWarps = 8, kConvWarps = 8;
constexpr int kThreads = (kSoftWarps + kConvWarps + 1) * 32;
constexpr int kSoft = kSoftWarps * 32, kConv = kConvWarps * 32, kSide = kConv / 2;   // half for K, half for V
constexpr int kUnitSlots = 4;     // blocks whose units' scales are held

template <int D>
struct Tc {
  static constexpr int kKeys = D == 256 ? 64 : 128;            // keys of a block
  static constexpr int kUnits = kKeys / 16;
  static constexpr int kCols = 512;                            // S twice, O, P twice
  static constexpr int kQ = kWideRows * D * 2, kK = kKeys * D * 2, kV = kKeys * D * 2;
  static constexpr int kBytes = kQ + 2 * (kK + kV) + 1024;     // operands start on 1024-byte boundaries
  static constexpr int kItems = kKeys / 8 * (D / 16);          // 8 keys x 16 channels, one a thread
  static_assert(kItems <= kSide, "an item a thread");
  static_assert(3 * kKeys + D <= kCols, "tensor memory");
};

// One answer for the warp, whose lanes are together again afterwards.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, tc::mbar_wait_bounded(bar, parity, abort_flag, &g_kv_wait_limit_ns, &g_kv_status,
                                                       PRISM_DEVSTATUS_WAIT_TIMEOUT));
}
// True in one lane of the warp, in a way that lets the compiler issue the
// tensor instructions of that lane from uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kv_attention_tc_kernel(const __grid_constant__ KvAttentionArgs a, const __grid_constant__ Parts parts) {
  using C = Tc<D>;
  constexpr int KB = C::kKeys, U = C::kUnits, UH = U / 2;
  extern __shared__ uint8_t smem_raw[];
  // the item in work lies in shared memory: no warp holds another's part of it
  __shared__ struct {
    Walk walk;
    SeqPlan plan;
    TileKeys keys;
    int64_t x, x_end, tile_x;    // the range's blocks not yet in work; the first of tile walk.tile
    int64_t part;                // the piece's first row among the sequence's pieces; -1: the whole tile
  } s_item;
  __shared__ int s_scan[kThreads];
  __shared__ int s_warp[kThreads / 32];
  __shared__ int64_t s_line[kThreads], s_warp64[kThreads / 32];   // of sequence walk.s
  __shared__ float s_max[kConvWarps];                        // largest value scale of a warp's pages
  __shared__ int s_bad[kConvWarps];                          // an invalid one among them
  __shared__ float s_unit[kWideRows];                        // a row's scale
  __shared__ float s_top[2][2][kWideRows], s_l[kWideRows];   // the halves' maxima, exchanged in turn; one half's sum
  __shared__ float s_ks[kUnitSlots][U], s_vr[kUnitSlots][U];
  // completions: K, V converted; scales in place; S formed (K free); P formed; O added to (V, P free); queries; the end
  __shared__ __align__(8) uint64_t s_bar[6 * 2 + kUnitSlots + 2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* s_q = smem;
  uint8_t* s_k = s_q + C::kQ;            // two stages
  uint8_t* s_v = s_k + 2 * C::kK;
  const uint32_t bars = smem_u32(s_bar);
  auto bar_k = [&](uint32_t g) { return bars + 8 * (g & 1); };
  auto bar_v = [&](uint32_t g) { return bars + 16 + 8 * (g & 1); };
  auto bar_s = [&](uint32_t g) { return bars + 32 + 8 * (g & 1); };
  auto bar_kfree = [&](uint32_t g) { return bars + 48 + 8 * (g & 1); };
  auto bar_p = [&](uint32_t g) { return bars + 64 + 8 * (g & 1); };
  auto bar_o = [&](uint32_t g) { return bars + 80 + 8 * (g & 1); };
  auto bar_u = [&](uint32_t g) { return bars + 96 + 8 * (g & (kUnitSlots - 1)); };
  const uint32_t bar_q = bars + 96 + 8 * kUnitSlots, bar_end = bar_q + 8;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(bar_k(i), kSide);
      tc::mbar_init(bar_v(i), kSide);
      tc::mbar_init(bar_s(i), 1);
      tc::mbar_init(bar_kfree(i), 1);
      tc::mbar_init(bar_p(i), kSoft);
      tc::mbar_init(bar_o(i), 1);
    }
    for (int i = 0; i < kUnitSlots; ++i) tc::mbar_init(bar_u(i), kSide);
    tc::mbar_init(bar_q, kSoft);
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
  pdl_trigger();
  // Launched ahead of the end of the few-row kernel, all of whose CTAs have waited
  // for what the inputs come from; neither needs the other's results.  The wait stands at the end,
  // so that this kernel's end is also the other's.
  const KvPages& c = a.c;
  uint32_t g0 = 0, items = 0;      // blocks and items before this item: the phases of the mbarriers
  if (tid == 0) {
    s_item.walk = new_walk();
    s_item.x = s_item.x_end = 0;
  }
  __syncthreads();

  for (int64_t item = blockIdx.x;; ++items) {   // one tile's part of a range a turn
    if (s_item.x >= s_item.x_end) {
      Walk walk = s_item.walk;
      SeqPlan plan = s_item.plan;
      const int before = walk.s;
      if (!find_item<true, kWideRows, kThreads>(a, item, walk, s_scan, s_warp, plan)) break;
      item += gridDim.x;
      if (walk.s != before) lay_line<kThreads>(a, plan, s_line, s_warp64);
      __syncthreads();               // everyone has read s_item
      if (tid == 0) {
        const Cuts cuts(s_line[kThreads - 1], plan.splits);
        s_item.x = cuts.cut(walk.split);
        s_item.x_end = cuts.cut(walk.split + 1);
        if (s_item.x < s_item.x_end) walk.tile = tile_at<kThreads>(a, plan, s_line, s_item.x);
        if (s_item.x < s_item.x_end) s_item.tile_x = tile_span<kThreads>(a, plan, s_line, walk.tile).x;
        s_item.walk = walk;
        s_item.plan = plan;
      }
    }
    if (tid == 0 && s_item.x < s_item.x_end) {
      TileKeys k(a, s_item.plan, s_item.walk, kWideRows);
      const int n = max(1, (k.t_hi - (k.t_lo & ~63) + KB - 1) / KB);   // the tile's blocks
      const int x = static_cast<int>(s_item.x - s_item.tile_x);
      const int end = static_cast<int>(min(static_cast<int64_t>(n), s_item.x_end - s_item.tile_x));
      k.k_begin = (k.t_lo & ~63) + x * KB;
      k.k_end = static_cast<int32_t>(min(static_cast<int64_t>(k.t_hi), static_cast<int64_t>(k.t_lo & ~63) + static_cast<int64_t>(end) * KB));
      s_item.part = end - x == n ? -1 : wide_part(s_item.plan, s_item.walk.split, s_item.walk.tile, x == 0);
      s_item.keys = k;
    }
    __syncthreads();
    if (s_item.x >= s_item.x_end) {   // fewer blocks than ranges
      --items;
      continue;
    }
    const int hk = s_item.walk.hk;
    const int32_t k_begin = s_item.keys.k_begin, k_end = s_item.keys.k_end;
    const int blocks = k_end > k_begin ? (k_end - k_begin + KB - 1) / KB : 0;
    const int32_t* table = c.table + s_item.walk.s * c.ld_table;

    if (warp >= kSoftWarps && warp < kSoftWarps + kConvWarps) {
      // ============================ converters ==============================
      const bool is_v = warp >= kSoftWarps + kConvWarps / 2;
      const int ct = (tid - kSoft) & (kSide - 1);
      const bool mine = ct < C::kItems;
      // the thread's item, keys 8 kg .. + 7 and channels 16 ch .. + 15.  K: the
      // pieces of a row side by side; V: eight key groups of a channel, whose
      // pieces fill all banks
      const int kg = is_v ? ct / (8 * (D / 16)) * 8 + (ct & 7) : ct / (D / 16);
      const int ch = is_v ? ct / 8 % (D / 16) : ct % (D / 16);
      const bool has_unit = !is_v && ct < U;            // passes on the scales of unit ct
      // a page id is read ahead and looked at when it is used
      const int32_t k_first = max(k_begin, s_item.keys.k_first);
      auto page_at = [&](int32_t key, bool live) { return live && key >= k_first && key < k_end ? table[key >> c.block_shift] : 0; };
      auto code_page = [&](int j) { return page_at(k_begin + j * KB + kg * 8, mine); };
      auto unit_page = [&](int j) { return page_at(k_begin + j * KB + ct * 16, has_unit); };
      auto row = [&](int32_t page) {          // an invalid page (the rows get NaN) or none: page 0, in its stead
        return static_cast<int64_t>(page < 0 || page >= c.num_pages ? 0 : page) * c.H + hk;
      };
      auto unit_scales = [&](int j, int32_t page) {     // vs not yet divided
        const int64_t at = row(page);
        const int32_t key = k_begin + j * KB + ct * 16;
        return has_unit && key >= k_first && key < k_end ? make_float2(c.k_scale[at], c.v_scale[at]) : make_float2(0.0f, 0.0f);
      };
      uint4 raw[8];
      auto load = [&](int j, int32_t page) {
        const int32_t key = k_begin + j * KB + kg * 8;
        const int8_t* src = (is_v ? c.v_codes : c.k_codes) + (row(page) * c.block + (key & (c.block - 1))) * D + ch * 16;
#pragma unroll
        for (int k = 0; k < 8; ++k) raw[k] = ld_stream_16(src + k * D);
      };
      // ahead: codes by one block, their page by two; scales by two, their page by three
      int32_t next_page = 0, next_unit = 0;
      float2 scales = make_float2(0.0f, 0.0f), next_scales = scales;
      if (blocks > 0) {
        const int32_t page = code_page(0), u0 = unit_page(0), u1 = unit_page(1);
        next_page = code_page(1);
        next_unit = unit_page(2);
        if (mine) load(0, page);
        scales = unit_scales(0, u0);
        next_scales = unit_scales(1, u1);
      }
      // ---- the piece's largest value scale, and its pages' validity
      bool bad = false;
      float v_top = 0.0f;
      if (blocks > 0) {
        for (int32_t i = (k_first >> c.block_shift) + tid - kSoft; i <= (k_end - 1) >> c.block_shift; i += kConv) {
          const int32_t page = table[i];
          if (page < 0 || page >= c.num_pages) {
            bad = true;
          } else {
            v_top = fmaxf(v_top, c.v_scale[static_cast<int64_t>(page) * c.H + hk]);
          }
        }
      }
      bad = __any_sync(0xffffffffu, bad);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v_top = fmaxf(v_top, __shfl_xor_sync(0xffffffffu, v_top, o));
      if (lane == 0) {
        s_max[warp - kSoftWarps] = v_top;
        s_bad[warp - kSoftWarps] = bad;
      }
      named_barrier(5, kConv);
      v_top = s_max[0];
#pragma unroll
      for (int i = 1; i < kConvWarps; ++i) v_top = fmaxf(v_top, s_max[i]);
      const float v_inv = v_top >= 0x1p-126f ? __frcp_rn(v_top) : 0.0f;
      for (int j = 0; j < blocks; ++j) {
        const uint32_t g = g0 + j, ph = (g >> 1) & 1;
        if (!is_v) {
          // Q K^T of block g - 2 is complete: it was issued after P of block
          // g - 4 was formed, so the units' slot is free
          wait(bar_kfree(g), ph ^ 1u, &s_abort);
          if (has_unit) {
            s_ks[g & (kUnitSlots - 1)][ct] = scales.x;
            s_vr[g & (kUnitSlots - 1)][ct] = scales.y * v_inv;
          }
          tc::mbar_arrive(bar_u(g));
          scales = next_scales;
          next_scales = unit_scales(j + 2, next_unit);
          next_unit = unit_page(j + 3);
          // ---- K: 16 codes of a key are two pieces of the operand
          if (mine) {
            uint8_t* dst = s_k + (g & 1) * C::kK + (ch >> 2) * (KB * 128) + kg * 1024;
            const int piece = (ch & 3) * 2;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint32_t x = raw[k].x ^ 0x80808080u, y = raw[k].y ^ 0x80808080u;
              const uint32_t z = raw[k].z ^ 0x80808080u, w = raw[k].w ^ 0x80808080u;
              *reinterpret_cast<uint4*>(dst + k * 128 + ((piece ^ k) << 4)) =
                  make_uint4(widen(x, 0x4140u), widen(x, 0x4342u), widen(y, 0x4140u), widen(y, 0x4342u));
              *reinterpret_cast<uint4*>(dst + k * 128 + (((piece + 1) ^ k) << 4)) =
                  make_uint4(widen(z, 0x4140u), widen(z, 0x4342u), widen(w, 0x4140u), widen(w, 0x4342u));
            }
          }
        } else {
          // ---- V, transposed: 8 keys of a channel are one piece of the operand
          wait(bar_o(g), ph ^ 1u, &s_abort);
          if (mine) {
            uint8_t* dst = s_v + (g & 1) * C::kV + (kg >> 3) * (D * 128) + ch * 16 * 128;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              uint32_t h[4][4];   // [channel][key pair]
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint4 r0 = raw[2 * k], r1 = raw[2 * k + 1];
                const uint32_t w0 = w == 0 ? r0.x : w == 1 ? r0.y : w == 2 ? r0.z : r0.w;
                const uint32_t w1 = w == 0 ? r1.x : w == 1 ? r1.y : w == 2 ? r1.z : r1.w;
                const uint32_t x = __byte_perm(w0, w1, 0x5140u) ^ 0x80808080u;
                const uint32_t y = __byte_perm(w0, w1, 0x7362u) ^ 0x80808080u;
                h[0][k] = widen(x, 0x4140u);
                h[1][k] = widen(x, 0x4342u);
                h[2][k] = widen(y, 0x4140u);
                h[3][k] = widen(y, 0x4342u);
              }
#pragma unroll
              for (int e = 0; e < 4; ++e)
                *reinterpret_cast<uint4*>(dst + (w * 4 + e) * 128 + (((kg & 7) ^ ((w * 4 + e) & 7)) << 4)) =
                    make_uint4(h[e][0], h[e][1], h[e][2], h[e][3]);
            }
          }
        }
        if (mine && j + 1 < blocks) load(j + 1, next_page);
        tc::fence_proxy_async();
        tc::mbar_arrive(is_v ? bar_v(g) : bar_k(g));
        next_page = code_page(j + 2);
      }
    } else if (warp == kSoftWarps + kConvWarps) {
      // ============================ issuer ==================================
      // the whole warp forms the descriptors, one lane issues
      const bool lead = elect_one();
      const uint32_t id_s = tc::idesc_f16_f32(KB), id_o = tc::idesc_f16_f32(D);
      const uint64_t qd = tc::smem_desc_sw128(smem_u32(s_q));
      bool ok = blocks == 0 || wait(bar_q, items & 1u, &s_abort);
      auto issue_scores = [&](uint32_t g) {       // S of block g; block g - 2's was read: its P was waited for
        ok = ok && wait(bar_k(g), (g >> 1) & 1, &s_abort);
        if (ok) {
          tc::tc_fence_after();
          const uint64_t kd = tc::smem_desc_sw128(smem_u32(s_k + (g & 1) * C::kK));
          const uint32_t dt = tmem + (g & 1) * KB;
          if (lead) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              tc::tc_mma(dt, qd + (k >> 2) * (kWideRows * 8) + 2 * (k & 3), kd + (k >> 2) * (KB * 8) + 2 * (k & 3), id_s,
                         k != 0 ? 1u : 0u);
            if (g != 0 || *static_cast<volatile int*>(&g_kv_withhold) == 0) tc::tc_commit(bar_s(g));
            tc::tc_commit(bar_kfree(g));
          }
        }
        __syncwarp();
      };
      if (blocks > 0) issue_scores(g0);
      for (int j = 0; j < blocks; ++j) {
        const uint32_t g = g0 + j;
        if (j + 1 < blocks) issue_scores(g + 1);
        ok = ok && wait(bar_v(g), (g >> 1) & 1, &s_abort);
        ok = ok && wait(bar_p(g), (g >> 1) & 1, &s_abort);
        if (ok) {
          tc::tc_fence_after();
          const uint64_t vd = tc::smem_desc_sw128(smem_u32(s_v + (g & 1) * C::kV));
          const uint32_t pt = tmem + 2 * KB + D + (g & 1) * (KB / 2);
          if (lead) {
#pragma unroll
            for (int k = 0; k < KB / 16; ++k)
              tc::tc_mma_ta(tmem + 2 * KB, pt + k * 8, vd + (k >> 2) * (D * 8) + 2 * (k & 3), id_o, (j | k) != 0 ? 1u : 0u);
            tc::tc_commit(bar_o(g));
          }
        }
        __syncwarp();
      }
    } else {
      // ============================ softmax =================================
      // this warp's 32 lanes, and its half of the scores' and the output's columns
      const int half = warp >> 2, r = tid & (kWideRows - 1);
      const SeqPlan& p = s_item.plan;
      const TileKeys& keys = s_item.keys;
      const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp & 3) << 21);
      const uint32_t t_o = t_lane + 2 * KB + half * (D / 2);
      const bool live = r < keys.n_rows;
      const int my_tok = (keys.row0 + r) / a.G, my_h = hk * a.G + keys.row0 + r - my_tok * a.G;   // the row's token and head
      auto of_row = [&](int lane_of, int64_t ld_t, int64_t ld_h) {   // a row of this warp's 32
        const int tok = __shfl_sync(0xffffffffu, my_tok, lane_of), h = __shfl_sync(0xffffffffu, my_h, lane_of);
        return (p.sp.b + tok) * ld_t + h * ld_h;
      };
      // ---- the tile's queries as binary16, K-major: a warp takes 16 of its
      // quarter's rows, a row's 16-byte pieces side by side
      constexpr int kRowLanes = D / 8, kTurnRows = 32 / kRowLanes, kTurns = 16 / kTurnRows, kAhead = kTurns < 8 ? kTurns : 8;
      const int q_row = (warp & 3) * 32 + half * 16 + lane / kRowLanes, q_piece = lane % kRowLanes;
      auto load_q = [&](int turn) {
        const int64_t at = of_row((q_row + turn * kTurnRows) & 31, a.ldq_t, a.ldq_h) + q_piece * 8;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (q_row + turn * kTurnRows < keys.n_rows) v = __ldg(reinterpret_cast<const uint4*>(a.q + at));
        return v;
      };
      uint4 qv[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) qv[i] = load_q(i);
#pragma unroll
      for (int t0 = 0; t0 < kTurns; t0 += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const uint4 v = qv[i];
          if (t0 + kAhead < kTurns) qv[i] = load_q(t0 + kAhead + i);
          const int row = q_row + (t0 + i) * kTurnRows;
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          float amax = 0.0f;
#pragma unroll
          for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
#pragma unroll
          for (int o = 1; o < kRowLanes; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          const int fe = query_exponent(amax);
          const float f = __uint_as_float(static_cast<uint32_t>(fe) << 23);
          if (q_piece == 0) s_unit[row] = __uint_as_float(static_cast<uint32_t>(254 - fe) << 23) * a.scale_log2;
          *reinterpret_cast<uint4*>(s_q + (q_piece >> 3) * (kWideRows * 128) + row * 128 + (((q_piece & 7) ^ (row & 7)) << 4)) =
              make_uint4(half2_bits(bf16_lo(v.x) * f, bf16_hi(v.x) * f), half2_bits(bf16_lo(v.y) * f, bf16_hi(v.y) * f),
                         half2_bits(bf16_lo(v.z) * f, bf16_hi(v.z) * f), half2_bits(bf16_lo(v.w) * f, bf16_hi(v.w) * f));
        }
      }
      tc::fence_proxy_async();
      if (blocks > 0) tc::mbar_arrive(bar_q);
      named_barrier(1 + (warp & 3), 64);
      const float unit = s_unit[r];
      const int32_t row_hi = keys.hi(r), my_lo = keys.lo(row_hi), my_hi = min(row_hi, k_end);
      const int32_t all_lo = keys.a_lo, all_hi = min(keys.a_hi, k_end);   // the keys that every row sees here
      float m = -INFINITY, l = 0.0f;
      int swaps = 0;
      for (int j = 0; j < blocks; ++j) {
        const uint32_t g = g0 + j;
        wait(bar_u(g), (g / kUnitSlots) & 1, &s_abort);
        wait(bar_s(g), (g >> 1) & 1, &s_abort);
        tc::tc_fence_after();
        const uint32_t t_s = t_lane + (g & 1) * KB + half * (KB / 2), t_p = t_lane + 2 * KB + D + (g & 1) * (KB / 2) + half * (KB / 4);
        const int32_t key0 = k_begin + j * KB, my_key = key0 + half * (KB / 2);
        // some row does not see all of the block, or the next piece has its end
        const bool edge = key0 < all_lo || key0 + KB > all_hi;
        const float* ks = s_ks[g & (kUnitSlots - 1)] + half * UH;
        const float* vs = s_vr[g & (kUnitSlots - 1)] + half * UH;
        wait(bar_o(g), ((g >> 1) & 1) ^ 1u, &s_abort);   // P of block g - 2 was read
        // Probabilities against the reference at hand; again against the row's
        // maximum where that stands too far above it (in a first block always)
        for (;;) {
          const float base = m == -INFINITY ? 0.0f : m - kShift;
          float top = -INFINITY;
          float2 sum = make_float2(0.0f, 0.0f);
          // rolled, and blocks with masked scores apart: three kinds of warps share the instruction cache
          auto pass = [&](auto masked) {
#pragma unroll 1
            for (int u = 0; u < UH; u += 2) {
              uint32_t x[2][16], pk[16];
              tc::tmem_ld16(t_s + u * 16, x[0]);
              tc::tmem_ld16(t_s + u * 16 + 16, x[1]);
              tc::tmem_wait_ld();
              if constexpr (decltype(masked)::value) {
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  const int32_t key = my_key + u * 16 + e;
                  if (key < my_lo || key >= my_hi) x[e >> 4][e & 15] = 0xff800000u;   // -inf
                }
              }
#pragma unroll
              for (int v = 0; v < 2; ++v) {
                const float f = ks[u + v] * unit, vf = vs[u + v];
                float t0 = __uint_as_float(x[v][0]), t1 = __uint_as_float(x[v][1]), q[16];
#pragma unroll
                for (int e = 2; e < 16; e += 2) {
                  t0 = fmaxf(t0, __uint_as_float(x[v][e]));
                  t1 = fmaxf(t1, __uint_as_float(x[v][e + 1]));
                }
                t0 = fmaxf(t0, t1);
                if (t0 > -INFINITY) top = fmaxf(top, t0 * f);
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                  const float2 y = fma2(make_float2(__uint_as_float(x[v][e]), __uint_as_float(x[v][e + 1])),
                                        make_float2(f, f), make_float2(-base, -base));
                  q[e] = ex2(y.x);
                  q[e + 1] = ex2(y.y);
                }
                if constexpr (decltype(masked)::value) {
#pragma unroll
                  for (int e = 0; e < 16; ++e)
                    if (x[v][e] == 0xff800000u) q[e] = 0.0f;   // with f = 0 too
                }
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                  const float2 two = make_float2(q[e], q[e + 1]), w = mul2(two, make_float2(vf, vf));
                  sum = add2(sum, two);
                  pk[v * 8 + e / 2] = half2_bits(w.x, w.y);
                }
              }
              tc::tmem_st16(t_p + u * 8, pk);
            }
          };
          if (edge) {
            pass(std::true_type{});
          } else {
            pass(std::false_type{});
          }
          s_top[swaps & 1][half][r] = top;
          named_barrier(1 + (warp & 3), 64);
          top = fmaxf(top, s_top[swaps & 1][half ^ 1][r]);
          ++swaps;
          const bool far = top > m + kSlack;    // m = -inf: nothing seen yet
          if (!__any_sync(0xffffffffu, far)) {
            l += sum.x + sum.y;
            break;
          }
          const float al = far ? ex2(m - top) : 1.0f;
          if (far) m = top;
          l *= al;
          if (j > 0) {
            wait(bar_o(g - 1), ((g - 1) >> 1) & 1, &s_abort);
            tc::tc_fence_after();
#pragma unroll 1
            for (int i = 0; i < D / 32; ++i) {
              uint32_t o[16];
              tc::tmem_ld16(t_o + i * 16, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
              tc::tmem_st16(t_o + i * 16, o);
            }
          }
        }
        tc::tmem_wait_st();
        tc::tc_fence_before();
        tc::mbar_arrive(bar_p(g));
      }
      if (blocks > 0) {
        const uint32_t g = g0 + blocks - 1;
        wait(bar_o(g), (g >> 1) & 1, &s_abort);
        tc::tc_fence_after();
      }

      // ---- the row's output, or its piece
      bool bad = false;
      float v_top = 0.0f;
      if (blocks > 0) {   // in place since the first block's scales are
#pragma unroll
        for (int i = 0; i < kConvWarps; ++i) {
          bad |= s_bad[i] != 0;
          v_top = fmaxf(v_top, s_max[i]);
        }
      }
      if (half == 1) s_l[r] = l;
      named_barrier(1 + (warp & 3), 64);
      if (half == 0) s_l[r] = l + s_l[r];
      named_barrier(1 + (warp & 3), 64);
      l = s_l[r];
      if (bad && tid == 0 && a.err != nullptr) atomicOr(a.err, PRISM_DEV_ERR_PAGE_RANGE);
      const float nanf = __uint_as_float(0x7fc00000u);
      const bool some = m > -INFINITY || l != l;   // saw a key (or a NaN score)
      float* ps = static_cast<float*>(a.ws) +
                  (first_part(parts, p, s_item.walk.s, hk) + max(s_item.part, static_cast<int64_t>(0)) + r) * (D + 4);
      const bool final = s_item.part < 0;
      const float scale = !some ? 0.0f : final ? v_top / l : v_top;
      // a warp's 32 rows, 32 channels at a time, pass through its 4 KB of the
      // (now unused) K stages, 16-byte pieces swizzled: rows are written whole
      float* turn = reinterpret_cast<float*>(s_k) + warp * 1024;
      const bool spoilt = bad && final;
#pragma unroll 1
      for (int i = 0; i < D / 64; ++i) {
        uint32_t o[2][16] = {};
        if (blocks > 0) {
          tc::tmem_ld16(t_o + i * 32, o[0]);
          tc::tmem_ld16(t_o + i * 32 + 16, o[1]);
          tc::tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          float y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            y[k] = spoilt ? nanf : some ? __uint_as_float(o[(e + k) >> 4][(e + k) & 15]) * scale : 0.0f;
          *reinterpret_cast<float4*>(turn + lane * 32 + (((e >> 2) ^ (lane & 7)) << 2)) = make_float4(y[0], y[1], y[2], y[3]);
        }
        __syncwarp();
#pragma unroll 4
        for (int k = 0; k < 8; ++k) {
          const int rl = k * 4 + (lane >> 3), piece = lane & 7, rr = (warp & 3) * 32 + rl;   // the row of the tile
          const float4 v = *reinterpret_cast<const float4*>(turn + rl * 32 + ((piece ^ (rl & 7)) << 2));
          const int d = half * (D / 2) + i * 32 + piece * 4;
          const int64_t at = of_row(rl, a.ldo_t, a.ldo_h) + d;
          if (rr < keys.n_rows) {
            if (final) {
              *reinterpret_cast<uint2*>(a.out + at) =
                  make_uint2(float_to_bf16_rne(v.x) | float_to_bf16_rne(v.y) << 16,
                             float_to_bf16_rne(v.z) | float_to_bf16_rne(v.w) << 16);
            } else {
              *reinterpret_cast<float4*>(ps + static_cast<int64_t>(rr - r) * (D + 4) + 4 + d) = v;
            }
          }
        }
        __syncwarp();
      }
      if (live && half == 0) {
        const float mx = some ? m - kShift + kPShift : -INFINITY;   // the weights' common form
        if (!final) {
          ps[0] = bad ? nanf : mx;
          ps[1] = l;
        } else if (a.lse != nullptr) {
          a.lse[(p.sp.b + my_tok) * static_cast<int64_t>(a.Hq) + my_h] = bad ? nanf : !some ? mx : (mx - kPShift + log2f(l)) * kLn2;
        }
      }
    }
    if (blocks == 0) --items;          // the queries' mbarrier did not turn
    g0 += blocks;
    tc::tc_fence_before();
    __syncthreads();   // the queries, s_scan, s_max and the output's columns are free again
    tc::tc_fence_after();
    if (tid == 0) {    // on to the range's next tile
      const int64_t n = max(1, (s_item.keys.t_hi - (s_item.keys.t_lo & ~63) + KB - 1) / KB);
      s_item.tile_x += n;
      s_item.x = s_item.tile_x;
      ++s_item.walk.tile;
    }
    __syncthreads();
  }

  pdl_wait();
  // ---- every instruction in flight completes before the columns are given back
  if (warp == kSoftWarps + kConvWarps && elect_one()) {   // the issuing thread
    tc::tc_commit(bar_end);
    tc::mbar_wait_drain_bounded(bar_end, 0, kDrainNs, &g_kv_status, PRISM_DEVSTATUS_WAIT_TIMEOUT);
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols) : "memory");
  }
}

template <int D>
cudaError_t launch_d(const KvAttentionArgs& a, const Parts& parts, cudaStream_t stream) {
  using C = Tc<D>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kv_attention_tc_kernel<D>), C::kBytes);
  if (e != cudaSuccess) return e;
  const int64_t items = (a.T * a.G / kWideRows + a.c.S + 2 * parts.ranges * a.c.S) * a.c.H;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(items, sm_count()));
  return launch_kernel(kv_attention_tc_kernel<D>, dim3(grid), dim3(kThreads), C::kBytes, stream, true, a, parts);
}

}  // namespace

cudaError_t launch_kv_attention_wide(const KvAttentionArgs& a, const kv::Parts& parts, cudaStream_t stream) {
  return a.c.D == 64    ? launch_d<64>(a, parts, stream)
         : a.c.D == 128 ? launch_d<128>(a, parts, stream)
                        : launch_d<256>(a, parts, stream);
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

cudaError_t set_kv_wait_expiry(unsigned long long limit_ns, int withhold) {
  cudaError_t e = cudaMemcpyToSymbol(g_kv_wait_limit_ns, &limit_ns, sizeof limit_ns);
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_kv_withhold, &withhold, sizeof withhold);
  return e;
}

}  // namespace prism
