// linear_attention_tc.cu -- the chunked form of linear attention (linear_attention.cu)
// on the tcgen05 tensor cores.  With G_i the sum of a chunk's decays up to token i,
// w_ij = e^{G_i - G_j} and S the state that enters,
//   o_i = scale * (e^{G_i} q_i S + sum_{j <= i} w_ij (q_i . k_j) v_j)
//   S   = e^{G_C} S + sum_j e^{G_C - G_j} k_j v_j^T
// What is not bf16 already is split into bf16 parts: scores and the state where it is
// read out into two (2^-17 of the value), the decayed values of the update into three
// (2^-25), so that states are as good as binary32 sums.  Sums of decays are kept as two
// binary32 numbers (and added as such): their differences decide.
//
// A long sequence is cut into segments (by its length and the number of heads alone, so
// that a sequence's bits do not depend on the batch): a first kernel forms each
// segment's own state from zero, a scan adds up what each then starts from, and the
// second kernel has the outputs.
//
// A chunk's 64 tokens against one head of 128 by 128 channels (decays in powers of
// two), each product with 128 rows in the lanes of tensor memory:
//   A  = Q K^T                   64 by 64 scores (the lower 64 lanes)       8 steps of 16
//   O  = S^T Q^T                 128 channels of v by 64 tokens, S in two bf16 parts  2 * 8
//      + V^T (2^{-G_j} A)^T      the scores in two parts                     2 * 4
//   U  = (2^{G_C - G_j} V)^T K   128 by 128, V's decayed values in three parts  3 * 4
// and out = scale * 2^{G_i} O^T, S = 2^{G_C} S + U^T.  The scores' weights are those
// of a column alone.  Where a chunk's decays go below 2^-80 (kDeep), G_i stops there
// for the outputs, and the scores of those rows make up for it: what 2^-80 is left
// of in the state that entered counts as 2^-80 of it.  So that weights of up to 2^80 take
// no sum out of binary32, S and the weights are held 2^-40 times as large, and the
// outputs' factor has the 2^40: exact, and free but at an item's ends (64 sequences of 24
// to 41 tokens 86.7 -> 87.8 us; as a factor of S for the chunks alone that need it, 8191
// tokens took 146 to 150).
//
// S^T is an operand in tensor memory, formed by the warps that have it.  Q, K and V are
// read as they lie, by tensor copies in the 128-byte-swizzled layout (K-major for Q and
// K; for K in U and V in O along the tokens, the operand's other major); the weighted
// scores and values lie in shared memory beside them.  S stays in the registers of eight
// warps (lane v channel, 64 key channels a thread) from a sequence's first chunk to its
// last.  With 64 key channels the first four of those warps have it, and products over key
// channels take half the steps; with 64 value channels the warps of the lower lanes, and
// likewise the values' warps.  The other lanes hold anything, and nothing is stored from
// them.  U is formed from zero for each chunk, its small parts first, and added to S
// rounded to nearest, since the tensor cores' additions cut off.
//
// One CTA an SM walks the items (sequence, head, segment).  Its warps pass chunks
// on by mbarriers:
//   producer (1)   finds items, copies Q, K and V of chunks ahead into a ring of stages;
//                  the chunks' decays and what is to be done, in a longer one:
//                  at most five chunks are in work when one is begun
//   issuer (1)     U and O of a chunk, A of the next
//   state (8)      S's two parts; S after the chunk
//   values (8)     the decayed values' three parts; outputs of the chunk before
//   scores (2)     the weighted scores
//
// A chunk takes an SM some 4000 cycles, 3100 of them in its 44 instructions (70 to 85
// each, whatever their columns: near the pipe's rate for the 12 with 128, under half of it
// for the 32 with 64), the rest between the kinds of warps; the segments'
// kernel 2200, 12 instructions and the splitting of V.  64 sequences of 24
// to 41 tokens, 40 heads: 87 us (bytes at 6784 GB/s: 57); 8191 tokens of 40 heads
// 143 us (50): 42 segments, 9 scan, 92 outputs; 3 sequences of 48 tokens at most 10 us.
// 8191 tokens of 40 heads of 64 by 64 126 us, 64 by 128 135, 128 by 64 136.
//
// Every wait on an mbarrier is bounded: after 2 s (prism_debug_wait_expiry
// shortens that for tests) the kernel sets the device status bit; every warp leaves
// its loop, the copies and instructions in flight complete, and the kernel returns.
#include <cudaTypedefs.h>

#include "linear_plan.cuh"
#include "tc_common.cuh"

namespace prism {

__device__ uint32_t g_lin_status = 0;
// Test mode (prism_debug_wait_expiry): the waits' limit, and whether each CTA's
// issuer withholds the signal that its first U is formed.
__device__ unsigned long long g_lin_wait_limit_ns = 2000000000ull;
__device__ int g_lin_withhold = 0;

namespace {

using namespace lin;

constexpr unsigned long long kDrainNs = 2000000000ull;
constexpr int D = 128;
constexpr int kInfo = 6;             // chunks whose decays and work are held
constexpr int kStateWarps = 8, kIssuer = 14, kProducer = 15;   // values 8 .. 11, 16 .. 19; scores 12, 13
constexpr int kThreads = 640;
constexpr int kStateThreads = kStateWarps * 32;
constexpr int kTile = kChunk * D * 2, kHalf = kTile / 2;     // of q, k or v: halves of 64 channels
constexpr int kScores = kChunk * kChunk * 2;
constexpr int kTurn = 16 * 16 * 2;                           // a warp's turn of outputs
template <bool kLocal>
constexpr int kStagesOf = kLocal ? 5 : 3;
template <bool kLocal>
constexpr int kSmemOf = kStagesOf<kLocal> * (kLocal ? 2 : 3) * kTile + (kLocal ? 0 : 3 * kTile + 2 * kScores + kStateWarps * kTurn) + 1024;
constexpr int kAhead = 4;                                    // chunks whose decays are held, three on their way
template <int DK, int DV>
constexpr int kPart = DK * DV + 4;                           // floats of a segment's state in the workspace
// columns of tensor memory
constexpr uint32_t kColU = 0, kColS = 128, kColA = 256, kColO = 320;   // O of two chunks in turn
constexpr uint32_t kColV = 128;      // kLocal: the decayed values, of two chunks in turn

constexpr float kDeepest = 80.0f;
constexpr float kUp = 0x1p40f, kDown = 0x1p-40f;            // half of it; the second kernel's S and weights
enum { kFirst = 1, kLast = 2, kEnd = 4, kDeep = 8 };
struct Step {          // a chunk's work
  int64_t row;         // its first token
  int64_t in, out;     // states: of the sequence's start (kFirst); to write to (kLast), -1 for none
  int64_t part;        // of the sequence's first place in the workspace and this head
  int32_t live, hv, flags, seg;   // seg: the place of the state that the segment starts from; -1: the state slot
  float left;          // what the segment leaves of the state before it (kLast)
};

struct Maps {
  CUtensorMap q, k, v;
};

// A CTA's waits: their limit in cycles, and whether one has run out.
struct Limit {
  long long cycles;
  int abort;
};
// Compact, since it stands in many places and the kinds of warps share the
// instruction cache.  One answer for the warp.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile Limit* limit) {
  bool ok = tc::mbar_try_wait(bar, parity);
  if (!__all_sync(0xffffffffu, ok)) {
    long long left = limit->cycles;
    uint32_t last = static_cast<uint32_t>(clock());
    while (!ok && limit->abort == 0) {
      ok = tc::mbar_try_wait(bar, parity);
      const uint32_t now = static_cast<uint32_t>(clock());
      left -= min(now - last, 1u << 20) + 1;   // where the SM's clock steps, 2^20 at most
      last = now;
      if (!ok && left < 0) {
        limit->abort = 1;
        atomicOr(&g_lin_status, PRISM_DEVSTATUS_WAIT_TIMEOUT);
      }
    }
    ok = __all_sync(0xffffffffu, ok);
  }
  return ok;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ void store_matrices(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
// Four 8 by 8 matrices, each written transposed.
__device__ __forceinline__ void store_transposed(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
// 16 lanes by 16 columns, in the fragments of an m16n8 result for each 8 columns.
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// 16 lanes by 16 columns in such fragments, lanes 0 .. 7 and 8 .. 15: lane c / 4, column c % 4 of each four.
__device__ __forceinline__ void tmem_st_16x128b(uint32_t taddr, const uint32_t (&a)[4], const uint32_t (&b)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(a[0]), "r"(b[0]),
               "r"(a[1]), "r"(b[1]), "r"(a[2]), "r"(b[2]), "r"(a[3]), "r"(b[3]));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]));
}
// Predicated, not branched: with a branch here the segments' kernel spills 620 bytes a thread.
__device__ __forceinline__ void store_if(bool there, float2* to, float2 v) {
  asm volatile("{\n .reg .pred p;\n setp.ne.s32 p, %0, 0;\n @p st.global.v2.f32 [%1], {%2, %3};\n}\n" ::"r"(
                   static_cast<int>(there)),
               "l"(to), "f"(v.x), "f"(v.y)
               : "memory");
}
// One arrival for the warp, after what all of its lanes did.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bar);
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void copy_4(uint32_t dst, const float* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// A tile of rows of 64 channels, 128-byte swizzled, as an operand whose rows are
// the contraction's: 64 channels in 128 bytes, eight rows to 1024, the other 64
// channels a half tile on.
__device__ __forceinline__ uint64_t desc_along_rows(uint32_t addr) {
  return (tc::smem_desc_sw128(addr) & ~(static_cast<uint64_t>(0x3fff) << 16)) | (static_cast<uint64_t>(kHalf >> 4) << 16);
}
// bf16 operands, binary32 sums, M = 128.
__device__ __forceinline__ constexpr uint32_t idesc(int n, bool a_along_rows, bool b_along_rows) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_along_rows ? 1u << 15 : 0u) | (b_along_rows ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}

// Sequences of few tokens, and malformed ones, after the chunks: found kThreads at a
// time, their heads dealt out to the CTAs.
template <int DK, int DV>
__device__ void few_sequences(const LinAttnArgs& a, uint8_t* smem, uint32_t (&found)[kThreads / 32]) {
  const int tid = threadIdx.x;
  int64_t item = 0;
  for (int64_t s0 = 0; s0 < a.S; s0 += kThreads) {
    Span p;
    const int64_t s = s0 + tid;
    const bool few = s < a.S && span_of(a, s, blockIdx.x == 0, p) && (p.bad || p.n <= kFewTokens);
    const uint32_t mask = __ballot_sync(0xffffffffu, few);
    __syncthreads();
    if ((tid & 31) == 0) found[tid >> 5] = mask;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w)
      for (uint32_t rest = found[w]; rest != 0; rest &= rest - 1) {
        // heads hv with (item + hv) % gridDim.x == blockIdx.x
        const int64_t first = (static_cast<int64_t>(blockIdx.x) + gridDim.x - item % gridDim.x) % gridDim.x;
        for (int64_t hv = first; hv < a.Hv; hv += gridDim.x) {
          span_of(a, s0 + w * 32 + __ffs(rest) - 1, false, p);
          if (p.n > kFewTokens) {
            spoil(a, p, static_cast<int>(hv), 0, DV);
          } else {
            __syncthreads();       // shared memory is free again
            few_tokens<DK>(a, p, static_cast<int>(hv), 0, DV, reinterpret_cast<float*>(smem));
          }
        }
        item += a.Hv;
      }
  }
}

template <bool kLocal, int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1)
    linear_chunk_kernel(const __grid_constant__ LinAttnArgs a, const __grid_constant__ Maps maps, int max_segs) {
  constexpr int kStages = kStagesOf<kLocal>, kTiles = kLocal ? 2 : 3;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Step s_step[kInfo];
  __shared__ __align__(16) float s_gh[kInfo][kChunk], s_gl[kInfo][kChunk];   // G, in two parts (kDeep)
  // 2^G times the scale, 2^-G, 2^{G_C - G}
  __shared__ __align__(16) float s_out[kInfo][kChunk], s_in[kInfo][kChunk], s_w[kInfo][kChunk];
  __shared__ __align__(8) float s_dec[kAhead][kChunk];
  __shared__ float s_tot[kInfo];
  __shared__ __align__(8) uint64_t s_bar[2 * kStages + 14];
  __shared__ uint32_t s_tmem;
  __shared__ Limit s_limit;
  __shared__ uint32_t s_few[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t base = smem_u32(smem);
  auto tile_k = [&](int st) { return base + st * kTiles * kTile; };
  auto tile_v = [&](int st) { return base + st * kTiles * kTile + kTile; };
  auto tile_q = [&](int st) { return base + st * kTiles * kTile + 2 * kTile; };
  auto values = [&](int part) { return base + (kStages * kTiles + part) * kTile; };   // [128 channels][64 tokens] a part
  const uint32_t scores = values(3), turns = scores + 2 * kScores;                    // high parts, then low ones
  const uint32_t bars = smem_u32(s_bar);
  auto bar_full = [&](int st) { return bars + 8 * st; };
  auto bar_free = [&](int st) { return bars + 8 * (kStages + st); };
  const uint32_t bar_a = bars + 16 * kStages, bar_p = bar_a + 8, bar_ufree = bar_a + 16,
                 bar_s = bar_a + 24, bar_q = bar_a + 32, bar_end = bar_a + 40;
  auto bar_u = [&](uint32_t g) { return bar_a + 48 + 8 * (g & 1); };
  auto bar_v = [&](uint32_t g) { return bar_a + 96 + 8 * (g & 1); };
  // two in turn: O of chunk g + 1 may be formed before a warp looks for that of g; kLocal: U
  // too, and a warp may have the values of g + 1 when another is still at those of g
  auto bar_o = [&](uint32_t g) { return bar_a + 64 + 8 * (g & 1); };
  auto bar_ofree = [&](uint32_t g) { return bar_a + 80 + 8 * (g & 1); };
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(bar_full(i), 2);   // the copies, and what the producer writes itself
      // the issuer's instructions, the warps of decayed values; kLocal: the state's warps,
      // which nothing else keeps from missing a stage's whole turn (else bar_s does)
      tc::mbar_init(bar_free(i), 1 + 8 + (kLocal ? kStateWarps : 0));
    }
    tc::mbar_init(bar_a, 1);
    tc::mbar_init(bar_p, 2);
    tc::mbar_init(bar_ufree, kStateWarps);
    tc::mbar_init(bar_s, kStateWarps);
    tc::mbar_init(bar_q, 1);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(bar_u(i), 1);
      tc::mbar_init(bar_v(i), 8);
      tc::mbar_init(bar_o(i), 1);
      tc::mbar_init(bar_ofree(i), 8);
    }
    tc::mbar_init(bar_end, 1);
    s_limit.abort = 0;
    s_limit.cycles = static_cast<long long>(*static_cast<volatile unsigned long long*>(&g_lin_wait_limit_ns)) * 2;   // of 2 GHz
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // the scores of tokens 0 .. 31 with tokens 32 .. 63 are 0 for good
  if (!kLocal && warp == 12)
    for (int p = 4; p < 8; ++p)
      for (int part = 0; part < 2; ++part)
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(scores + part * kScores + lane * 128 +
                                                                                   ((p ^ (lane & 7)) << 4)),
                     "r"(0)
                     : "memory");
  tc::fence_proxy_async();
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = s_tmem, t_lane = tmem + (static_cast<uint32_t>(warp & 3) << 21);
  pdl_wait();
  uint32_t in_flight = 0;          // stages that the producer filled, where it does not come to the end

  if (warp == kProducer) {
    // ============================ producer ================================
    const int64_t per_seq = static_cast<int64_t>(max_segs) * a.Hv, total = a.S * per_seq;
    bool ok = true;
    int st = 0, in_slot = 0;
    uint32_t round = 0, issued = 0;
    auto turn = [&] {
      ++issued;
      if (++in_slot == kInfo) in_slot = 0;
      if (++st == kStages) st = 0, ++round;
    };
    for (int64_t at = blockIdx.x; ok && at < total; at += 32 * static_cast<int64_t>(gridDim.x)) {
      // 32 items at a time, one a lane: heads go by fastest, sequences slowest
      const int64_t item = at + lane * static_cast<int64_t>(gridDim.x);
      Span p{};
      int hv = 0, seg = 0, segs = 0;
      int64_t each = 0, place = 0;
      bool mine = false;
      if (item < total) {
        const int64_t s = item / per_seq;
        const int rest = static_cast<int>(item - s * per_seq);
        seg = rest / a.Hv;
        hv = rest - seg * a.Hv;
        mine = span_of(a, s, false, p) && !p.bad && p.n > kFewTokens;
        if (mine) {
          each = segment_chunks(p.n, a.cut);
          place = first_place(a, s, p.b);
          segs = static_cast<int>(segment_count(p.n, a.cut));
          mine = seg < (kLocal ? segs - 1 : segs);   // nothing comes after the last one
        }
      }
      uint32_t todo = __ballot_sync(0xffffffffu, mine);
      while (ok && todo != 0) {
        const int from = __ffs(todo) - 1;
        todo &= todo - 1;
        const int64_t b = __shfl_sync(0xffffffffu, p.b, from), n = __shfl_sync(0xffffffffu, p.n, from);
        const int64_t in = __shfl_sync(0xffffffffu, p.in, from), out = __shfl_sync(0xffffffffu, p.out, from);
        const int64_t chunks_each = __shfl_sync(0xffffffffu, each, from);
        const int h = __shfl_sync(0xffffffffu, hv, from), sg = __shfl_sync(0xffffffffu, seg, from);
        const int sgs = __shfl_sync(0xffffffffu, segs, from);
        const int64_t t0 = sg * chunks_each * kChunk, t1 = min(n, t0 + chunks_each * kChunk);
        const int chunks = static_cast<int>((t1 - t0 + kChunk - 1) / kChunk), hk = h / a.G;
        // decays by way of shared memory, three chunks ahead
        auto copy_decays = [&](int c) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int64_t i = t0 + static_cast<int64_t>(c) * kChunk + 2 * lane + e;
            const bool there = c < chunks && i < t1;
            copy_4(smem_u32(&s_dec[c & (kAhead - 1)][2 * lane + e]), a.decay + (there ? (b + i) * a.ldd_t : 0) + h, there ? 4 : 0);
          }
          cp_async_commit();
        };
        cp_async_wait<0>();        // the copies of the item before
        if (lane == 0 && in >= 0 && (kLocal ? sg == 0 : sgs == 1))
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a.state + (in * a.Hv + h) * (DK * DV)), "r"(DK * DV * 4)
                       : "memory");
        for (int c = 0; c < kAhead - 1; ++c) copy_decays(c);
        const int64_t part = (__shfl_sync(0xffffffffu, place, from) * a.Hv + h) * kPart<DK, DV>;
        Sum log_total{0.0f, 0.0f};
        for (int c = 0; c < chunks; ++c) {
          ok = wait(bar_free(st), (round & 1) ^ 1u, &s_limit);
          if (!ok) break;
          const int32_t row = static_cast<int32_t>(b + t0 + static_cast<int64_t>(c) * kChunk);
          if (elect_one()) {
            const uint32_t bar = bar_full(st);
            tc::mbar_expect_tx(bar, ((kLocal ? 1 : 2) * (DK / 64) + DV / 64) * kHalf);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if (!kLocal && half < DK / 64) tma_load_3d(tile_q(st) + half * kHalf, &maps.q, half * 64, hk, row, bar);
              if (half < DK / 64) tma_load_3d(tile_k(st) + half * kHalf, &maps.k, half * 64, hk, row, bar);
              if (half < DV / 64) tma_load_3d(tile_v(st) + half * kHalf, &maps.v, half * 64, h, row, bar);
            }
          }
          __syncwarp();
          copy_decays(c + kAhead - 1);
          cp_async_wait<kAhead - 1>();
          const float2 g2 = *reinterpret_cast<const float2*>(&s_dec[c & (kAhead - 1)][2 * lane]);
          const float dec[2] = {bounded_decay(g2.x), bounded_decay(g2.y)};
          const Decays d = sum_decays(dec);
          log_total = join(log_total, d.total);
          const bool deep = d.total.h < -kDeepest;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int i = 2 * lane + e;
            const float G = __fadd_rn(d.g[e].h, d.g[e].l);
            if constexpr (!kLocal) {
              s_out[in_slot][i] = ex2(fmaxf(G, -kDeepest)) * (a.scale * kUp);
              s_in[in_slot][i] = ex2(fminf(-G, kDeepest)) * kDown;
              if (deep) s_gh[in_slot][i] = d.g[e].h, s_gl[in_slot][i] = d.g[e].l;
            }
            s_w[in_slot][i] = kLocal ? left_of(d, e) : left_of(d, e) * kDown;
          }
          if (lane == 0) s_tot[in_slot] = exp2f(__fadd_rn(d.total.h, d.total.l));
          if (lane == 0) {
            Step& w = s_step[in_slot];
            w.row = row;
            w.live = static_cast<int>(min(static_cast<int64_t>(kChunk), t1 - t0 - static_cast<int64_t>(c) * kChunk));
            w.hv = h;
            w.flags = (c == 0 ? kFirst : 0) | (c + 1 == chunks ? kLast : 0) | (deep ? kDeep : 0);
            w.in = in;
            w.out = kLocal ? sg + 1 : sg + 1 == sgs ? out : -1;
            w.part = part;
            w.seg = kLocal ? sg : sgs == 1 ? -1 : sg;
            w.left = exp2f(log_total.h + log_total.l);
          }
          warp_arrive(bar_full(st));
          turn();
        }
      }
    }
    cp_async_wait<0>();            // of decays, where it left early
    if (ok && wait(bar_free(st), (round & 1) ^ 1u, &s_limit)) {
      if (lane == 0) {
        s_step[in_slot].flags = kEnd;
        tc::mbar_arrive(bar_full(st));
        tc::mbar_arrive(bar_full(st));
      }
      __syncwarp();
    } else {
      in_flight = issued;
    }
  } else if (warp == kIssuer) {
    // ============================ issuer ==================================
    const bool lead = elect_one();
    int st = 0, info = 0;
    uint32_t round = 0;
    bool more = wait(bar_full(0), 0, &s_limit) && !(s_step[0].flags & kEnd);
    auto issue_scores = [&] {
      if (lead) {
        const uint64_t qd = tc::smem_desc_sw128(tile_q(st)), kd = tc::smem_desc_sw128(tile_k(st));
#pragma unroll
        for (int k = 0; k < DK / 16; ++k)   // rows 64 .. of Q's tile are not its: those lanes are not read
          tc::tc_mma(tmem + kColA, qd + (k >> 2) * (kHalf >> 4) + 2 * (k & 3), kd + (k >> 2) * (kHalf >> 4) + 2 * (k & 3),
                     idesc(kChunk, false, false), k != 0 ? 1u : 0u);
        tc::tc_commit(bar_a);
      }
      __syncwarp();
    };
    if (!kLocal && more) issue_scores();
    for (uint32_t g = 0; more; ++g) {
      if (!wait(bar_v(g), (g >> 1) & 1, &s_limit)) break;
      if (g > 0 && !wait(bar_ufree, (g - 1) & 1, &s_limit)) break;
      tc::tc_fence_after();
      if (lead) {
        const uint64_t kd = desc_along_rows(tile_k(st));
#pragma unroll 1
        for (int part = 2; part >= 0; --part) {   // the small parts first
          const uint64_t vd = tc::smem_desc_sw128(values(part));
#pragma unroll
          for (int k = 0; k < kChunk / 16; ++k) {
            const uint32_t more_of = part != 2 || k != 0 ? 1u : 0u;
            if constexpr (kLocal) {
              tc::tc_mma_ta(tmem + kColU, tmem + kColV + (g & 1) * 96 + part * 32 + k * 8, kd + k * (16 * 128 >> 4),
                            idesc(DK, false, true), more_of);
            } else {
              tc::tc_mma(tmem + kColU, vd + 2 * k, kd + k * (16 * 128 >> 4), idesc(DK, false, true), more_of);
            }
          }
        }
        if (g != 0 || *static_cast<volatile int*>(&g_lin_withhold) == 0) tc::tc_commit(bar_u(g));
      }
      __syncwarp();
      if constexpr (!kLocal) {
        if (!wait(bar_s, g & 1, &s_limit)) break;
        if (g > 1 && !wait(bar_ofree(g), ((g - 2) >> 1) & 1, &s_limit)) break;
        tc::tc_fence_after();
        if (lead) {
          const uint64_t qd = tc::smem_desc_sw128(tile_q(st));
#pragma unroll 1
          for (int part = 1; part >= 0; --part)
#pragma unroll
            for (int k = 0; k < DK / 16; ++k)
              tc::tc_mma_ta(tmem + kColO + (g & 1) * kChunk, tmem + kColS + part * 64 + k * 8, qd + (k >> 2) * (kHalf >> 4) + 2 * (k & 3),
                            idesc(kChunk, false, false), part != 1 || k != 0 ? 1u : 0u);
          tc::tc_commit(bar_q);
        }
        __syncwarp();
        if (!wait(bar_p, g & 1, &s_limit)) break;
        tc::tc_fence_after();
        if (lead) {
          const uint64_t vd = desc_along_rows(tile_v(st)), pd = tc::smem_desc_sw128(scores);
#pragma unroll 1
          for (int part = 1; part >= 0; --part)
#pragma unroll
            for (int k = 0; k < kChunk / 16; ++k)
              tc::tc_mma(tmem + kColO + (g & 1) * kChunk, vd + k * (16 * 128 >> 4), pd + part * (kScores >> 4) + 2 * k,
                         idesc(kChunk, true, false), 1u);
          tc::tc_commit(bar_o(g));
        }
        __syncwarp();
      }
      if (lead) tc::tc_commit(bar_free(st));
      __syncwarp();
      if (++st == kStages) st = 0, ++round;
      if (++info == kInfo) info = 0;
      more = wait(bar_full(st), round & 1, &s_limit) && !(s_step[info].flags & kEnd);
      if (!kLocal && more) issue_scores();   // A was read: w A of this chunk was waited for
    }
  } else if (warp < kStateWarps) {
    // ============================ state ===================================
    const int half = warp >> 2, dv = (warp & 3) * 32 + lane;
    // The others' warps go the same way with anything, which no one reads.
    const bool own = half < DK / 64 && (warp & 3) < DV / 32;          // of the head's channels
    constexpr int kOwners = DK * DV / 64;                              // threads that are
    const int id = own ? half * DV + dv : 0;                           // among them
    const int at = own ? half * 64 * DV + dv : 0;                      // of the state's values
    float2 S[32];      // key channels 64 half + 2 i, + 1
    int st = 0, info = 0;
    uint32_t round = 0;
    for (uint32_t g = 0;; ++g) {
      if (!wait(bar_full(st), round & 1, &s_limit)) break;
      const Step& w = s_step[info];
      const int flags = w.flags;
      if (flags & kEnd) break;
      if constexpr (kLocal) warp_arrive(bar_free(st));   // its turn was seen
      if (flags & kFirst) {
        const float* src = a.state + (w.in * a.Hv + w.hv) * (DK * DV) + at;
        const int64_t part_step = static_cast<int64_t>(a.Hv) * kPart<DK, DV>;
        const float2* place = reinterpret_cast<const float2*>(a.ws + w.part + w.seg * part_step) + id;
        const bool slot = w.in >= 0 && (kLocal ? w.seg == 0 : w.seg < 0);
        if (!kLocal && w.seg >= 0) {
#pragma unroll
          for (int i = 0; i < 32; ++i) S[i] = place[i * kOwners];
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) S[i] = slot ? make_float2(src[2 * i * DV], src[(2 * i + 1) * DV]) : make_float2(0.0f, 0.0f);
        }
        if constexpr (!kLocal) {
#pragma unroll
          for (int i = 0; i < 32; ++i) S[i] = mul2(S[i], make_float2(kDown, kDown));
        }
        if constexpr (kLocal) {
          // the sequence's start has a place of its own: the last segment may write
          // the state back before another begins
          if (w.seg == 0) {
            float2* ps = reinterpret_cast<float2*>(a.ws + w.part) + id;
#pragma unroll
            for (int i = 0; i < 32; ++i) store_if(own, ps + i * kOwners, S[i]);
#pragma unroll
            for (int i = 0; i < 32; ++i) S[i] = make_float2(0.0f, 0.0f);
          }
        }
      }
      if constexpr (!kLocal) {
        if (g > 0 && !wait(bar_q, (g - 1) & 1, &s_limit)) break;   // the parts were read
        tc::tc_fence_after();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float2 x = S[i * 8 + e];
            hi[e] = split_bf16(x);
            lo[e] = pack_bf16(x.x, x.y);
          }
          tmem_st8(t_lane + kColS + half * 32 + i * 8, hi);
          tmem_st8(t_lane + kColS + 64 + half * 32 + i * 8, lo);
        }
        tc::tmem_wait_st();
        tc::tc_fence_before();
        warp_arrive(bar_s);
      }
      const float tot = s_tot[info], left = w.left;
      const int64_t last_out = w.out, last_part = w.part;
      const int hv = w.hv;
      if (!wait(bar_u(g), (g >> 1) & 1, &s_limit)) break;
      tc::tc_fence_after();
#pragma unroll
      for (int i = 0; i < 4; ++i) {   // 16 at a time, by registers
        uint32_t u[16];
        tc::tmem_ld16(t_lane + kColU + half * 64 + i * 16, u);
        tc::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e)
          S[i * 8 + e] = fma2(make_float2(tot, tot), S[i * 8 + e], make_float2(__uint_as_float(u[2 * e]), __uint_as_float(u[2 * e + 1])));
      }
      tc::tc_fence_before();
      warp_arrive(bar_ufree);
      if (flags & kLast) {
        if constexpr (kLocal) {
          float* ps = a.ws + last_part + last_out * (static_cast<int64_t>(a.Hv) * kPart<DK, DV>);
          if (own)
#pragma unroll
            for (int i = 0; i < 32; ++i) reinterpret_cast<float2*>(ps)[i * kOwners + id] = S[i];
          if (tid == 0) ps[DK * DV] = left;
        } else if (own && last_out >= 0) {
          float* dst = a.state + (last_out * a.Hv + hv) * (DK * DV) + at;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 x = mul2(S[i], make_float2(kUp, kUp));
            dst[2 * i * DV] = x.x, dst[(2 * i + 1) * DV] = x.y;
          }
        }
      }
      if (++st == kStages) st = 0, ++round;
      if (++info == kInfo) info = 0;
    }
  } else if (warp < kStateWarps + 4 || warp >= 16) {
    // ========================= decayed values ==============================
    // 32 channels of v and half of the tokens a warp, in three parts, transposed
    const int t0 = warp >= 16 ? 32 : 0;
    const uint32_t half = (warp & 2) ? kHalf : 0, first = (warp & 1) * 4;   // of the row's pieces of 8 channels
    const int r8 = lane & 7;
    const bool own = (warp & 3) < DV / 32;        // of the head's channels
    // ---- outputs of chunk g (place `of`): the warp's 32 channels and half of the
    // tokens, 16 channels by 16 tokens at a time by way of its own shared memory
    auto outputs = [&](uint32_t g, int of) {
      const Step& w = s_step[of];
      if (!wait(bar_o(g), (g >> 1) & 1, &s_limit)) return false;
      tc::tc_fence_after();
      const uint32_t turn = turns + ((warp & 3) + (t0 >> 3)) * kTurn;
      // where the lane writes a row of its matrix, and reads a piece: rows of 32 bytes, a token's 16 channels
      const int row_w = ((lane >> 4) << 3) + (lane & 7), row_r = lane >> 1;
      const uint32_t to = turn + row_w * 32 + ((((lane >> 3) ^ (row_w >> 2)) & 1) << 4);
      const uint32_t from = turn + row_r * 32 + (((lane ^ (row_r >> 2)) & 1) << 4);
      const int live = w.live - t0 - row_r;
      uint16_t* dst = a.out + (w.row + t0 + row_r) * a.ldo_t + w.hv * a.ldo_h + (warp & 3) * 32 + (lane & 1) * 8;
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        const int t = i & 1, k = i >> 1;
        uint32_t o[8], y[4];      // for each 8 tokens: channels c / 4 and c / 4 + 8, tokens 2 (c % 4), + 1
        tmem_ld_16x256b(t_lane + (16u * k << 16) + kColO + (g & 1) * kChunk + t0 + t * 16, o);
        const float2 e0 = *reinterpret_cast<const float2*>(&s_out[of][t0 + t * 16 + (lane & 3) * 2]);
        const float2 e1 = *reinterpret_cast<const float2*>(&s_out[of][t0 + t * 16 + 8 + (lane & 3) * 2]);
        tc::tmem_wait_ld();
        if (i == 3) {
          tc::tc_fence_before();
          warp_arrive(bar_ofree(g));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x = mul2(e < 2 ? e0 : e1, make_float2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])));
          y[e] = pack_bf16(x.x, x.y);
        }
        store_transposed(to, y[0], y[1], y[2], y[3]);
        __syncwarp();
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(from) : "memory");
        if (own && t * 16 < live) *reinterpret_cast<uint4*>(dst + t * 16 * a.ldo_t + k * 16) = v;
        __syncwarp();
      }
      return true;
    };
    int st = 0, info = 0, before = 0;
    uint32_t round = 0;
    for (uint32_t g = 0;; ++g) {
      if (!wait(bar_full(st), round & 1, &s_limit)) break;
      const Step& s = s_step[info];
      if (s.flags & kEnd) {
        if (!kLocal && g > 0) outputs(g - 1, before);
        break;
      }
      // Behind the sequence's end lies another, or anything: zeros, the warp's own
      // channels and tokens of V, and as many of K.
      if (s.live < kChunk)
        for (int row = max(s.live, t0) + (lane >> 3); row < t0 + 32; row += 4) {
          const uint32_t to = ((lane & 4) ? tile_k(st) : tile_v(st)) + half + row * 128 + (((first + (lane & 3)) ^ (row & 7)) << 4);
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(to), "r"(0) : "memory");
        }
      __syncwarp();
      float2 w[4];                    // of the tokens 8 i + 2 c, + 1, c = lane % 4
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float2*>(&s_w[info][t0 + i * 8 + (lane & 3) * 2]);
      // 8 channels of them: lane c / 4 has a channel, c % 4 two tokens of each eight
      auto form = [&](int p, uint32_t (&parts)[3][4]) {
        uint32_t x[4];
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                     : "r"(tile_v(st) + half + (t0 + lane) * 128 + (((first + p) ^ r8) << 4))
                     : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 y = mul2(make_float2(bf16_lo(x[i]), bf16_hi(x[i])), w[i]);
          parts[0][i] = split_bf16(y);
          parts[1][i] = split_bf16(y);
          parts[2][i] = pack_bf16(y.x, y.y);
        }
      };
      if constexpr (kLocal) {      // in tensor memory, where there is room for two chunks'
        if (g > 1 && !wait(bar_u(g), ((g - 2) >> 1) & 1, &s_limit)) break;
        tc::tc_fence_after();
        if (own)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t lower[3][4], upper[3][4];
          form(2 * k, lower);
          form(2 * k + 1, upper);
#pragma unroll
          for (int i = 0; i < 3; ++i)
            tmem_st_16x128b(t_lane + (16u * k << 16) + kColV + (g & 1) * 96 + i * 32 + (t0 >> 1), lower[i], upper[i]);
        }
        tc::tmem_wait_st();
        tc::tc_fence_before();
      } else {
        if (g > 0 && !wait(bar_u(g - 1), ((g - 1) >> 1) & 1, &s_limit)) break;   // the parts of the chunk before were read
        // rolled: the kinds of warps share the instruction cache
        if (own)
#pragma unroll 1
        for (int p = 0; p < 4; ++p) {
          uint32_t parts[3][4];
          form(p, parts);
          const uint32_t to = ((warp & 3) * 32 + p * 8 + r8) * 128 + ((((t0 >> 3) + (lane >> 3)) ^ r8) << 4);
#pragma unroll
          for (int k = 0; k < 3; ++k) store_matrices(values(k) + to, parts[k]);
        }
      }
      tc::fence_proxy_async();
      warp_arrive(bar_v(g));
      warp_arrive(bar_free(st));
      if (!kLocal && g > 0 && !outputs(g - 1, before)) break;
      before = info;
      if (++st == kStages) st = 0, ++round;
      if (++info == kInfo) info = 0;
    }
  } else if constexpr (!kLocal) {
    // ============================ scores ==================================
    // rows 0 .. 31 (warp 12), 32 .. 63 (13)
    if (warp <= 13) {
      const int rows = warp & 1, i = rows * 32 + lane;
      int st = 0, info = 0;
      uint32_t round = 0;
      for (uint32_t g = 0;; ++g) {
        if (!wait(bar_full(st), round & 1, &s_limit) || (s_step[info].flags & kEnd)) break;
        const bool deep = s_step[info].flags & kDeep;
        // (kDeep) what the row's outputs are short of, in two parts
        const float under = deep ? s_gh[info][i] + kDeepest : 0.0f;
        const float2 dh = make_float2(fminf(under, 0.0f), fminf(under, 0.0f));
        const float dl1 = under < 0.0f ? s_gl[info][i] : 0.0f;
        if (!wait(bar_a, g & 1, &s_limit)) break;
        tc::tc_fence_after();
        // 16 columns at a time; rolled: the kinds of warps share the instruction cache
#pragma unroll 2
        for (int j0 = 0; j0 < (rows + 1) * 32; j0 += 16) {
          uint32_t x[16], hi[8], lo[8];
          tc::tmem_ld16(t_lane + kColA + j0, x);
          float2 w[8];
          if (!deep) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = *reinterpret_cast<const float2*>(&s_in[info][j0 + 2 * e]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 gh = *reinterpret_cast<const float2*>(&s_gh[info][j0 + 2 * e]);
              const float2 gl = *reinterpret_cast<const float2*>(&s_gl[info][j0 + 2 * e]);
              w[e] = make_float2(ex2((dh.x - gh.x) + (dl1 - gl.x)), ex2((dh.y - gh.y) + (dl1 - gl.y)));
              w[e] = mul2(w[e], make_float2(kDown, kDown));
            }
          }
          tc::tmem_wait_ld();
          const int ahead = i - j0;      // columns that the row sees, less one: the others' scores may be anything
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float2 y = mul2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), w[e]);
            if (j0 >= rows * 32) y = make_float2(2 * e <= ahead ? y.x : 0.0f, 2 * e + 1 <= ahead ? y.y : 0.0f);
            hi[e] = split_bf16(y);
            lo[e] = pack_bf16(y.x, y.y);
          }
          const uint32_t to = scores + i * 128;
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            const uint32_t piece = (((j0 >> 3) + (e >> 2)) ^ (i & 7)) * 16;
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + piece), "r"(hi[e]), "r"(hi[e + 1]), "r"(hi[e + 2]),
                         "r"(hi[e + 3])
                         : "memory");
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + piece + kScores), "r"(lo[e]), "r"(lo[e + 1]),
                         "r"(lo[e + 2]), "r"(lo[e + 3])
                         : "memory");
          }
        }
        tc::tc_fence_before();
        tc::fence_proxy_async();
        warp_arrive(bar_p);
        if (++st == kStages) st = 0, ++round;
        if (++info == kInfo) info = 0;
      }
    }
  }

  // ---- every copy and instruction in flight completes before memory is given back
  // (copies: at the end, every one was waited for)
  if (lane == 0)
    for (uint32_t i = in_flight > kStages ? in_flight - kStages : 0; i < in_flight; ++i)
      tc::mbar_wait_drain_bounded(bar_full(i % kStages), (i / kStages) & 1, kDrainNs, &g_lin_status, PRISM_DEVSTATUS_WAIT_TIMEOUT);
  __syncwarp();
  if (warp == kIssuer && elect_one()) {
    tc::tc_commit(bar_end);
    tc::mbar_wait_drain_bounded(bar_end, 0, kDrainNs, &g_lin_status, PRISM_DEVSTATUS_WAIT_TIMEOUT);
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
  if constexpr (!kLocal) few_sequences<DK, DV>(a, smem, s_few);
  pdl_trigger();
}

// The states that the segments start from, place by place: place 0 holds the
// sequence's, place k + 1 what segment k makes of none.  A CTA for 1024 values.
constexpr int kScanThreads = 256;
template <int DK, int DV>
constexpr int kSlices = DK * DV / (4 * kScanThreads);
template <int DK, int DV>
__global__ void __launch_bounds__(kScanThreads) linear_scan_kernel(const __grid_constant__ LinAttnArgs a) {
  pdl_wait();
  const int64_t s = blockIdx.x / kSlices<DK, DV>;
  const int hv = blockIdx.y;
  Span p;
  if (span_of(a, s, false, p) && !p.bad && p.n > kFewTokens) {
    const int segs = static_cast<int>(segment_count(p.n, a.cut));
    const int64_t step = static_cast<int64_t>(a.Hv) * kPart<DK, DV>;
    float* place = a.ws + (first_place(a, s, p.b) * a.Hv + hv) * kPart<DK, DV>;
    const int at = static_cast<int>(blockIdx.x % kSlices<DK, DV>) * 4 * kScanThreads + threadIdx.x * 4;
    if (segs > 1) {
      float4 x = *reinterpret_cast<const float4*>(place + at);
#pragma unroll 4
      for (int k = 1; k < segs; ++k) {
        float4* here = reinterpret_cast<float4*>(place + k * step + at);
        const float left = place[k * step + DK * DV];
        const float4 y = *here;
        x = make_float4(fmaf(left, x.x, y.x), fmaf(left, x.y, y.y), fmaf(left, x.z, y.z), fmaf(left, x.w, y.w));
        *here = x;
      }
    }
  }
  pdl_trigger();
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const auto fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q{};
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f) : nullptr;
  }();
  return fn;
}

// [T, H, channels] bf16 in boxes of 64 tokens of a head by 64 channels; rows past T read 0.
cudaError_t make_map(CUtensorMap* m, const uint16_t* ptr, int64_t T, int64_t H, int64_t channels, int64_t ld_t, int64_t ld_h) {
  const auto fn = encode_fn();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(channels), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(H > 1 ? ld_h : channels) * 2, static_cast<cuuint64_t>(ld_t) * 2};
  const cuuint32_t box[3] = {64, 1, kChunk}, steps[3] = {1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(ptr), dims, strides, box, steps,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

template <int DK, int DV>
cudaError_t launch_linear_chunks(const LinAttnArgs& a, cudaStream_t stream) {
  Maps maps;
  cudaError_t e = make_map(&maps.q, a.q, a.T, a.Hk, DK, a.ldq_t, a.ldq_h);
  if (e == cudaSuccess) e = make_map(&maps.k, a.k, a.T, a.Hk, DK, a.ldk_t, a.ldk_h);
  if (e == cudaSuccess) e = make_map(&maps.v, a.v, a.T, a.Hv, DV, a.ldv_t, a.ldv_h);
  if (e != cudaSuccess) return e;
  const int segs = static_cast<int>(most_segments(a.max_len, a.cut));
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.S * segs * a.Hv, sm_count()));
  const auto first = linear_chunk_kernel<true, DK, DV>, second = linear_chunk_kernel<false, DK, DV>;
  if (segs > 1) {
    e = ensure_smem_attr(reinterpret_cast<const void*>(first), kSmemOf<true>);
    if (e == cudaSuccess) e = launch_kernel(first, dim3(grid), dim3(kThreads), kSmemOf<true>, stream, true, a, maps, segs);
    if (e == cudaSuccess)
      e = launch_kernel(linear_scan_kernel<DK, DV>, dim3(static_cast<unsigned>(a.S * kSlices<DK, DV>), a.Hv), dim3(kScanThreads), 0,
                        stream, true, a);
  }
  if (e == cudaSuccess) e = ensure_smem_attr(reinterpret_cast<const void*>(second), kSmemOf<false>);
  if (e != cudaSuccess) return e;
  return launch_kernel(second, dim3(grid), dim3(kThreads), kSmemOf<false>, stream, true, a, maps, segs);
}
template cudaError_t launch_linear_chunks<64, 64>(const LinAttnArgs&, cudaStream_t);
template cudaError_t launch_linear_chunks<64, 128>(const LinAttnArgs&, cudaStream_t);
template cudaError_t launch_linear_chunks<128, 64>(const LinAttnArgs&, cudaStream_t);
template cudaError_t launch_linear_chunks<128, 128>(const LinAttnArgs&, cudaStream_t);

cudaError_t read_and_clear_linear_status(uint32_t* out) {
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_lin_status, sizeof v);
  if (e != cudaSuccess) return e;
  if (v != 0) {
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_lin_status, &zero, sizeof zero);
  }
  *out = v;
  return e;
}

cudaError_t set_linear_wait_expiry(unsigned long long limit_ns, int withhold) {
  cudaError_t e = cudaMemcpyToSymbol(g_lin_wait_limit_ns, &limit_ns, sizeof limit_ns);
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_lin_withhold, &withhold, sizeof withhold);
  return e;
}

}  // namespace prism
