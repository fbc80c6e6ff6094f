// linear_attention.cu -- linear attention with a decay for each head:
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale * q_t S_t
// with a state S [Dk, Dv] in binary32 for each (sequence, value head).
//
// Up to kFewTokens tokens of a sequence (decode steps, drafted tokens): the
// recurrence as it stands.  The state is read once into registers, every token
// updates it and reads it out, and it is written once: bytes, 8 Dk Dv a head,
// bound it (64 sequences of a token, 40 heads of 128 by 128: 54.5 us, 6.2 TB/s of
// states; one sequence 3.3 us, a launch and a state's way to the SM and back).
//
// More tokens: chunks of 64.  With G_i the sum of the chunk's decays up to token
// i, w_ij = e^{G_i - G_j} and S the state that enters,
//   o_i = scale * (e^{G_i} q_i S + sum_{j <= i} w_ij (q_i . k_j) v_j)
//   S   = e^{G_C} S + sum_j e^{G_C - G_j} k_j v_j^T
// on the tensor cores (mma.sync m16n8k16, bf16 operands, binary32 sums; heads of 128
// by 128 on tcgen05, linear_attention_tc.cu).  Each warp
// keeps 16 columns of the state in registers, transposed: the result of its
// update, S^T += (w v)^T k, is laid out among the lanes as the operand that q S
// wants.  What is not bf16 already is split into bf16 parts: scores and the state
// where it is read out into two (2^-17 of the value), the decayed values of the
// update into three (2^-25), so that states are as good as binary32 sums.  Sums
// of decays are kept as two binary32 numbers (and added as such): their
// differences decide.
//
// A chunk takes such a CTA some 4.7 us, a chain of barriers, loads and products whose
// warps fill no unit; what counts is CTAs at work.  8191 tokens of 40 heads: 64 by 64
// 153 us (bytes: 25), 64 by 128 215, 128 by 64 221 (38); 1024 tokens of 8 heads of 64 19.
//
// A long sequence is cut into segments (by its length and the number of heads
// alone, so that a sequence's bits do not depend on the batch): a first kernel
// forms each segment's own state from zero, and the second starts each segment
// from the states and decays of those before it.
#include <type_traits>

#include "linear_plan.cuh"

namespace prism {
namespace {

using namespace lin;

// A CTA for each `width` columns of a (sequence, head).
template <int DK>
__global__ void __launch_bounds__(256) linear_few_kernel(const __grid_constant__ LinAttnArgs a, int width) {
  extern __shared__ __align__(128) uint8_t smem[];
  pdl_wait();
  const int slices = a.Dv / width, c0 = static_cast<int>(blockIdx.x % slices) * width;
  const int64_t s = blockIdx.x / slices;
  Span p;
  if (span_of(a, s, blockIdx.y == 0 && c0 == 0 && threadIdx.x == 0, p)) {
    if (p.n > kFewTokens) {   // only where it is malformed
      spoil(a, p, blockIdx.y, c0, width);
    } else {
      few_tokens<DK>(a, p, blockIdx.y, c0, width, reinterpret_cast<float*>(smem));
    }
  }
  pdl_trigger();
}

// ----------------------------------------------------------------- chunks ---
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Place of 16-byte piece `ch` of row `row` in a tile of rows of W values: the
// eight rows of a matrix touch all banks.
template <int W>
__device__ __forceinline__ uint32_t piece(int row, int ch) {
  return static_cast<uint32_t>(row * (W * 2) + ((ch ^ (row & 7)) << 4));
}

// Scores lie in blocks of 16 rows and 16 columns, those on and below the diagonal alone.
constexpr int kScoreBlocks = kChunk / 16 * (kChunk / 16 + 1) / 2;
__device__ __forceinline__ uint32_t score_place(int row, int ch) {
  const int m = row >> 4, r = row & 15;
  return static_cast<uint32_t>((m * (m + 1) / 2 + (ch >> 1)) * 512 + r * 32 + (((ch ^ (r >> 2)) & 1) << 4));
}

template <int DK, int DV>
struct Tile {
  static constexpr int kWarps = DV / 16, kThreads = kWarps * 32;
  static constexpr int kQ = kChunk * DK * 2, kV = kChunk * DV * 2, kP = kScoreBlocks * 512;
  static constexpr int kStage = 2 * kQ + kV;
  static constexpr int kBytes = 2 * kStage + 2 * kP;
  static constexpr int kLocalBytes = 2 * (kQ + kV);
};

// Segment `blockIdx.x % segs` of a (sequence, head).  kLocal: its state from
// zero, into the workspace.
template <int DK, int DV, bool kLocal>
__global__ void __launch_bounds__(Tile<DK, DV>::kThreads, 2)
    linear_chunk_kernel(const __grid_constant__ LinAttnArgs a, int max_segs) {
  using L = Tile<DK, DV>;
  constexpr int kWarps = L::kWarps, kThreads = L::kThreads, NT = DK / 8;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) float s_gh[2][kChunk], s_gl[2][kChunk];   // decays summed up to a token, in powers of two, in two parts
  __shared__ __align__(8) float s_eg[2][kChunk], s_w[2][kChunk], s_tot[2];   // those of G_i, G_C - G_i and G_C
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, lr = lane >> 2, lc = lane & 3;
  const int hv = blockIdx.y, hk = hv / a.G;
  const int64_t s = blockIdx.x / max_segs;
  const int seg = static_cast<int>(blockIdx.x % max_segs);
  Span p;
  const bool ok = span_of(a, s, !kLocal && seg == 0 && hv == 0 && tid == 0, p);
  if (!ok) return;
  if (p.bad || p.n <= kFewTokens) {
    if (kLocal || seg != 0) return;
    if (p.n > kFewTokens) {
      spoil(a, p, hv, 0, DV);
    } else {
      few_tokens<DK>(a, p, hv, 0, DV, reinterpret_cast<float*>(smem));
    }
    return;
  }
  const int64_t each = segment_chunks(p.n, a.cut);
  const int segs = static_cast<int>(segment_count(p.n, a.cut));
  if (seg >= segs || (kLocal && seg + 1 == segs)) return;   // nothing comes after the last one
  const int64_t t0 = seg * each * kChunk, t1 = min(p.n, t0 + each * kChunk);
  const int chunks = static_cast<int>((t1 - t0 + kChunk - 1) / kChunk);

  // the state, transposed: warp w has columns 16 w .. of it, lane (r, c) of tile t
  // columns r, r + 8 of those and rows 8 t + 2 c, + 1
  float st[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) st[t][0] = st[t][1] = st[t][2] = st[t][3] = 0.0f;
  constexpr int64_t kPart = DK * DV + 4;
  float* part = a.ws + (first_place(p.b, a.cut) * a.Hv + hv) * kPart;   // of the sequence's first segment
  const int64_t part_step = a.Hv * kPart;
  const int64_t at = (static_cast<int64_t>(2 * lc)) * DV + warp * 16 + lr;
  auto read_part = [&](const float* ps) {
    const float d = ps[DK * DV];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float4 x = *reinterpret_cast<const float4*>(ps + (t * kThreads + tid) * 4);
      st[t][0] = fmaf(d, st[t][0], x.x);
      st[t][1] = fmaf(d, st[t][1], x.y);
      st[t][2] = fmaf(d, st[t][2], x.z);
      st[t][3] = fmaf(d, st[t][3], x.w);
    }
  };
  auto write_part = [&](float* ps, float d) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
      *reinterpret_cast<float4*>(ps + (t * kThreads + tid) * 4) = make_float4(st[t][0], st[t][1], st[t][2], st[t][3]);
    if (tid == 0) ps[DK * DV] = d;
  };
  // The first place holds the state that the sequence starts from: with several
  // segments, the last may have written the state back before another begins.
  if (kLocal ? seg == 0 : segs == 1) {
    if (p.in >= 0) {
      const float* src = a.state + (p.in * a.Hv + hv) * (DK * DV) + at;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        st[t][0] = src[8 * t * DV];
        st[t][1] = src[(8 * t + 1) * DV];
        st[t][2] = src[8 * t * DV + 8];
        st[t][3] = src[(8 * t + 1) * DV + 8];
      }
    }
    if constexpr (kLocal) {
      write_part(part, 0.0f);
#pragma unroll
      for (int t = 0; t < NT; ++t) st[t][0] = st[t][1] = st[t][2] = st[t][3] = 0.0f;
    }
  } else if constexpr (!kLocal) {
    for (int i = 0; i <= seg; ++i) read_part(part + i * part_step);
  }

  const uint32_t base = smem_u32(smem);
  auto stage_k = [&](int c) { return base + (c & 1) * (kLocal ? L::kQ + L::kV : L::kStage); };
  auto stage_v = [&](int c) { return stage_k(c) + L::kQ; };
  auto stage_q = [&](int c) { return stage_v(c) + L::kV; };
  const uint32_t p_hi = base + 2 * L::kStage, p_lo = p_hi + L::kP;
  auto copy = [&](int c) {
    if (c < chunks) {
      const int64_t r0 = t0 + static_cast<int64_t>(c) * kChunk;
      auto rows = [&](auto width, uint32_t dst, const uint16_t* src, int64_t ld) {
        constexpr int W = decltype(width)::value;
#pragma unroll
        for (int i = tid; i < kChunk * W / 8; i += kThreads) {
          const int row = i / (W / 8), ch = i % (W / 8);
          const bool live = r0 + row < t1;
          cp_async_16(dst + piece<W>(row, ch), src + (live ? r0 + row : r0) * ld + ch * 8, live ? 16 : 0);
        }
      };
      rows(std::integral_constant<int, DK>(), stage_k(c), a.k + p.b * a.ldk_t + hk * a.ldk_h, a.ldk_t);
      rows(std::integral_constant<int, DV>(), stage_v(c), a.v + p.b * a.ldv_t + hv * a.ldv_h, a.ldv_t);
      if constexpr (!kLocal) rows(std::integral_constant<int, DK>(), stage_q(c), a.q + p.b * a.ldq_t + hk * a.ldq_h, a.ldq_t);
    }
    cp_async_commit();
  };
  // a chunk's decays: warp 0, two tokens a lane
  float dec[2];
  auto load_decay = [&](int c) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int64_t i = t0 + static_cast<int64_t>(c) * kChunk + 2 * lane + e;
      dec[e] = i < t1 ? decay_of(a, p.b + i, hv) : 0.0f;
    }
  };
  Sum log_total{0.0f, 0.0f};  // of the segment so far (warp 0)
  auto lay_decay = [&](int c) {
    const Decays d = sum_decays(dec);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * lane + e;
      s_gh[c & 1][i] = d.g[e].h;
      s_gl[c & 1][i] = d.g[e].l;
      s_eg[c & 1][i] = ex2(__fadd_rn(d.g[e].h, d.g[e].l));
      s_w[c & 1][i] = left_of(d, e);
    }
    if (lane == 0) s_tot[c & 1] = exp2f(__fadd_rn(d.total.h, d.total.l));
    log_total = join(log_total, d.total);
  };

  copy(0);
  if (warp == 0) {
    load_decay(0);
    lay_decay(0);
    load_decay(1);
  }
  for (int c = 0; c < chunks; ++c) {
    copy(c + 1);
    cp_async_wait<1>();
    __syncthreads();     // the chunk's rows and decays are there
    const uint32_t sk = stage_k(c), sv = stage_v(c), sq = stage_q(c);
    const int64_t r0 = t0 + static_cast<int64_t>(c) * kChunk;
    const int tiles = static_cast<int>(min(static_cast<int64_t>(kChunk), t1 - r0) + 15) >> 4;   // of 16 tokens that there are

    if constexpr (!kLocal) {
      // ---- scores of 16 rows and kCols columns a warp, decayed, into two bf16 parts
      constexpr int kCols = kChunk * kChunk / 16 / kWarps, kN = kCols / 8;
      const int m0 = kWarps == 8 ? (warp >> 1) * 16 : warp * 16, n0 = kWarps == 8 ? (warp & 1) * kCols : 0;
      float x[kN][4];
#pragma unroll
      for (int n = 0; n < kN; ++n) x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.0f;
      if (n0 <= m0 && m0 < 16 * tiles) {
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk) {
          uint32_t qa[4];
          ldmatrix_x4(sq + piece<DK>(m0 + (lane & 15), 2 * kk + (lane >> 4)), qa[0], qa[1], qa[2], qa[3]);
#pragma unroll
          for (int n = 0; n < kN; n += 2) {
            if (n0 + n * 8 > m0 + 15) continue;
            uint32_t kb[4];
            ldmatrix_x4(sk + piece<DK>(n0 + n * 8 + (lane & 7) + ((lane >> 4) << 3), 2 * kk + ((lane >> 3) & 1)), kb[0],
                        kb[1], kb[2], kb[3]);
            mma_bf16(x[n], qa, kb[0], kb[1]);
            mma_bf16(x[n + 1], qa, kb[2], kb[3]);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = m0 + lr + 8 * e;
        const float2 gi = make_float2(s_gh[c & 1][i], s_gl[c & 1][i]);
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          const int j = n0 + n * 8 + 2 * lc;
          const float2 gh = *reinterpret_cast<const float2*>(&s_gh[c & 1][j]), gl = *reinterpret_cast<const float2*>(&s_gl[c & 1][j]);
          float2 y = make_float2(j <= i ? x[n][2 * e] * ex2((gi.x - gh.x) + (gi.y - gl.x)) : 0.0f,
                                 j + 1 <= i ? x[n][2 * e + 1] * ex2((gi.x - gh.y) + (gi.y - gl.y)) : 0.0f);
          if (j > m0 + 15) continue;
          const uint32_t at_p = score_place(i, j >> 3) + (j & 7) * 2;
          const uint32_t hi = split_bf16(y), lo = pack_bf16(y.x, y.y);
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(p_hi + at_p), "r"(hi) : "memory");
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(p_lo + at_p), "r"(lo) : "memory");
        }
      }
      __syncthreads();
    }
    // next chunk's decays: their place was read before the barrier that began this chunk
    if (warp == 0 && c + 1 < chunks) {
      lay_decay(c + 1);
      load_decay(c + 2);
    }

    // the warp's 16 columns of V: k16 steps of 16 tokens
    uint32_t vf[kChunk / 16][4];
#pragma unroll
    for (int kk = 0; kk < kChunk / 16; ++kk)
      ldmatrix_x4_trans(sv + piece<DV>(kk * 16 + (lane & 7) + ((lane >> 4) << 3), 2 * warp + ((lane >> 3) & 1)), vf[kk]);

    if constexpr (!kLocal) {
      // ---- outputs: q S, decayed, and the scores times V
      float o[kChunk / 16][2][4];
#pragma unroll
      for (int m = 0; m < kChunk / 16; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n) o[m][n][0] = o[m][n][1] = o[m][n][2] = o[m][n][3] = 0.0f;
#pragma unroll
      for (int kk = 0; kk < DK / 16; ++kk) {
        uint32_t bh[2][2], bl[2][2];   // [column half][k half]
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float2 v = make_float2(st[2 * kk + k][2 * n], st[2 * kk + k][2 * n + 1]);
            bh[n][k] = split_bf16(v);
            bl[n][k] = pack_bf16(v.x, v.y);
          }
#pragma unroll
        for (int m = 0; m < kChunk / 16; ++m) {
          if (m >= tiles) break;
          uint32_t qa[4];
          ldmatrix_x4(sq + piece<DK>(m * 16 + (lane & 15), 2 * kk + (lane >> 4)), qa[0], qa[1], qa[2], qa[3]);
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            mma_bf16(o[m][n], qa, bh[n][0], bh[n][1]);
            mma_bf16(o[m][n], qa, bl[n][0], bl[n][1]);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < kChunk / 16; ++m) {
        if (m >= tiles) break;
        const float e0 = s_eg[c & 1][m * 16 + lr], e1 = s_eg[c & 1][m * 16 + lr + 8];
#pragma unroll
        for (int n = 0; n < 2; ++n) o[m][n][0] *= e0, o[m][n][1] *= e0, o[m][n][2] *= e1, o[m][n][3] *= e1;
#pragma unroll
        for (int kk = 0; kk <= m; ++kk) {
          uint32_t ph[4], pl[4];
          const uint32_t at_p = score_place(m * 16 + (lane & 15), 2 * kk + (lane >> 4));
          ldmatrix_x4(p_hi + at_p, ph[0], ph[1], ph[2], ph[3]);
          ldmatrix_x4(p_lo + at_p, pl[0], pl[1], pl[2], pl[3]);
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            mma_bf16(o[m][n], ph, vf[kk][n], vf[kk][2 + n]);
            mma_bf16(o[m][n], pl, vf[kk][n], vf[kk][2 + n]);
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int64_t i = r0 + m * 16 + lr + 8 * e;
          if (i >= t1) continue;
          uint16_t* dst = a.out + (p.b + i) * a.ldo_t + hv * a.ldo_h + warp * 16 + 2 * lc;
#pragma unroll
          for (int n = 0; n < 2; ++n)
            *reinterpret_cast<uint32_t*>(dst + 8 * n) = pack_bf16(o[m][n][2 * e] * a.scale, o[m][n][2 * e + 1] * a.scale);
        }
      }
    }

    // ---- the state after the chunk
    const float tot = s_tot[c & 1];
#pragma unroll
    for (int t = 0; t < NT; ++t) st[t][0] *= tot, st[t][1] *= tot, st[t][2] *= tot, st[t][3] *= tot;
#pragma unroll
    for (int kk = 0; kk < kChunk / 16; ++kk) {
      if (kk >= tiles) break;
      uint32_t va[3][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = kk * 16 + 2 * lc + 8 * (i >> 1);   // tokens of the operand's register
        float2 v = mul2(make_float2(bf16_lo(vf[kk][i]), bf16_hi(vf[kk][i])), *reinterpret_cast<const float2*>(&s_w[c & 1][j]));
        va[0][i] = split_bf16(v);
        va[1][i] = split_bf16(v);
        va[2][i] = pack_bf16(v.x, v.y);
      }
#pragma unroll
      for (int t = 0; t < NT; t += 2) {
        uint32_t kb[4];
        ldmatrix_x4_trans(sk + piece<DK>(kk * 16 + (lane & 15), t + (lane >> 4)), kb);
        // from zero, the small parts first, and then rounded to nearest: the tensor
        // cores' additions cut off, and the state would gather that
        float u[2][4] = {};
#pragma unroll
        for (int f = 2; f >= 0; --f) {
          mma_bf16(u[0], va[f], kb[0], kb[1]);
          mma_bf16(u[1], va[f], kb[2], kb[3]);
        }
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
          for (int e = 0; e < 4; ++e) st[t + f][e] += u[f][e];
      }
    }
    __syncthreads();     // the chunk's stage and scores are free
  }
  cp_async_wait<0>();

  if constexpr (kLocal) {
    write_part(part + (seg + 1) * part_step, exp2f(log_total.h + log_total.l));
  } else if (seg + 1 == segs && p.out >= 0) {
    float* dst = a.state + (p.out * a.Hv + hv) * (DK * DV) + at;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      dst[8 * t * DV] = st[t][0];
      dst[(8 * t + 1) * DV] = st[t][1];
      dst[8 * t * DV + 8] = st[t][2];
      dst[(8 * t + 1) * DV + 8] = st[t][3];
    }
  }
}

template <int DK, int DV>
cudaError_t launch_few(const LinAttnArgs& a, cudaStream_t stream) {
  // narrow slices where whole heads leave SMs empty
  const int width = a.S * a.Hv >= 2 * kSms ? DV : 32;
  const dim3 grid(static_cast<unsigned>(a.S * (DV / width)), a.Hv);
  return launch_kernel(linear_few_kernel<DK>, grid, dim3(kGroups * width / 4), few_smem(DK, width), stream, true, a, width);
}

template <int DK, int DV>
cudaError_t launch_shape(const LinAttnArgs& a, cudaStream_t stream) {
  if (a.max_len <= kFewTokens) return launch_few<DK, DV>(a, stream);
  if constexpr (DK == 128 && DV == 128) {
    return launch_linear_attention_tc(a, stream);
  } else {
    using L = Tile<DK, DV>;
    const int segs = static_cast<int>(most_segments(a.max_len, a.cut));
    const dim3 grid(static_cast<unsigned>(a.S * segs), a.Hv);
    cudaError_t e = cudaSuccess;
    if (segs > 1) {
      e = ensure_smem_attr(reinterpret_cast<const void*>(linear_chunk_kernel<DK, DV, true>), L::kLocalBytes);
      if (e == cudaSuccess)
        e = launch_kernel(linear_chunk_kernel<DK, DV, true>, grid, dim3(L::kThreads), L::kLocalBytes, stream, true, a, segs);
    }
    static_assert(few_smem(DK, DV) <= L::kBytes, "few tokens in the same memory");
    if (e == cudaSuccess) e = ensure_smem_attr(reinterpret_cast<const void*>(linear_chunk_kernel<DK, DV, false>), L::kBytes);
    if (e != cudaSuccess) return e;
    return launch_kernel(linear_chunk_kernel<DK, DV, false>, grid, dim3(L::kThreads), L::kBytes, stream, true, a, segs);
  }
}

}  // namespace

size_t linear_attention_workspace_bytes(int64_t T, int64_t max_len, int64_t Hv, int64_t Dk, int64_t Dv) {
  const Cut cut = cut_of(Hv, Dk == 128 && Dv == 128);
  if (most_segments(max_len, cut) <= 1) return 0;
  return static_cast<size_t>(first_place(T, cut) * Hv * (Dk * Dv + 4)) * 4;
}

cudaError_t launch_linear_attention(const LinAttnArgs& given, cudaStream_t stream) {
  LinAttnArgs a = given;
  a.cut = cut_of(a.Hv, a.Dk == 128 && a.Dv == 128);
  if (a.Dk == 64) return a.Dv == 64 ? launch_shape<64, 64>(a, stream) : launch_shape<64, 128>(a, stream);
  return a.Dv == 64 ? launch_shape<128, 64>(a, stream) : launch_shape<128, 128>(a, stream);
}

}  // namespace prism
