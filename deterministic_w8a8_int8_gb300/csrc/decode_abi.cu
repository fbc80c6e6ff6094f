// decode_abi.cu -- the extern "C" boundary of the decode-step operators:
// host-side argument checks (returned as prism_status before anything is
// enqueued) and dispatch to the launchers.  See include/prism.h.
#include "decode.cuh"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
constexpr int64_t kInt31 = (1LL << 31) - 1;
// Tokens of a sequence at most: the attention's 32-bit positions run up to some
// thousand past a text's end (pages that are looked up ahead).
constexpr int64_t kMaxTokens = (1LL << 31) - (1LL << 14);

// The cache's own arguments.  Fills c where they are sound.
int check_cache(const int8_t* k_codes, const int8_t* v_codes, const float* k_scale, const float* v_scale,
                const int32_t* page_table, int64_t ld_table, const int32_t* seq_lens, int64_t S, int64_t num_pages,
                int64_t max_pages, int64_t H, int64_t D, int64_t block, prism::KvPages& c) {
  if (num_pages <= 0 || max_pages <= 0 || H <= 0 || ld_table < max_pages) return PRISM_ERR_INVALID_ARG;
  if (k_codes == nullptr || v_codes == nullptr || k_scale == nullptr || v_scale == nullptr || page_table == nullptr ||
      seq_lens == nullptr)
    return PRISM_ERR_INVALID_ARG;
  int shift = 0;
  while ((1LL << shift) < block && shift < 8) ++shift;
  if ((1LL << shift) != block || block < 16 || block > 128) return PRISM_ERR_UNSUPPORTED;
  if (D != 64 && D != 128 && D != 256) return PRISM_ERR_UNSUPPORTED;
  if (S > (1 << 24) || H > 32767 || num_pages > kInt31 || max_pages > (kMaxTokens >> shift)) return PRISM_ERR_UNSUPPORTED;
  if (!aligned(k_codes, 16) || !aligned(v_codes, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4) ||
      !aligned(page_table, 4) || !aligned(seq_lens, 4))
    return PRISM_ERR_ALIGNMENT;
  c.k_codes = const_cast<int8_t*>(k_codes);
  c.v_codes = const_cast<int8_t*>(v_codes);
  c.k_scale = const_cast<float*>(k_scale);
  c.v_scale = const_cast<float*>(v_scale);
  c.table = page_table;
  c.ld_table = ld_table;
  c.lens = seq_lens;
  c.num_pages = num_pages;
  c.max_pages = max_pages;
  c.S = static_cast<int32_t>(S);
  c.H = static_cast<int32_t>(H);
  c.D = static_cast<int32_t>(D);
  c.block = static_cast<int32_t>(block);
  c.block_shift = shift;
  return PRISM_OK;
}

// A [T, H, D] bf16 operand: strides and alignment.
int check_rows(const void* p, int64_t ld_t, int64_t ld_h, int64_t T, int64_t H, int64_t D) {
  if (p == nullptr) return PRISM_ERR_INVALID_ARG;
  if ((T > 1 && ld_t < D) || (H > 1 && ld_h < D)) return PRISM_ERR_INVALID_ARG;
  if (ld_t % 8 != 0 || ld_h % 8 != 0 || !aligned(p, 16)) return PRISM_ERR_ALIGNMENT;
  return PRISM_OK;
}

}  // namespace

extern "C" {

int prism_kv_append(const void* k_bf16, int64_t ldk_t, int64_t ldk_h, const void* v_bf16, int64_t ldv_t,
                    int64_t ldv_h, int8_t* k_codes, int8_t* v_codes, float* k_scale, float* v_scale, void* k_open,
                    void* v_open, const int32_t* page_table, int64_t ld_table, const int32_t* seq_lens,
                    const int32_t* cu_new, int64_t S, int64_t T, int64_t max_new, int64_t num_pages,
                    int64_t max_pages, int64_t H_kv, int64_t D, int64_t block, int32_t* dev_error_word,
                    void* cuda_stream) {
  if (S < 0 || T < 0) return PRISM_ERR_INVALID_ARG;
  if (S == 0 || T == 0) return PRISM_OK;
  if (max_new < 1 || (cu_new == nullptr && T != S)) return PRISM_ERR_INVALID_ARG;
  if (T > kInt31) return PRISM_ERR_UNSUPPORTED;
  prism::KvAppendArgs a{};
  int st = check_cache(k_codes, v_codes, k_scale, v_scale, page_table, ld_table, seq_lens, S, num_pages, max_pages,
                       H_kv, D, block, a.c);
  if (st != PRISM_OK) return st;
  if ((st = check_rows(k_bf16, ldk_t, ldk_h, T, H_kv, D)) != PRISM_OK) return st;
  if ((st = check_rows(v_bf16, ldv_t, ldv_h, T, H_kv, D)) != PRISM_OK) return st;
  if (k_open == nullptr || v_open == nullptr) return PRISM_ERR_INVALID_ARG;
  if (!aligned(k_open, 16) || !aligned(v_open, 16) || !aligned(cu_new, 4) || !aligned(dev_error_word, 4))
    return PRISM_ERR_ALIGNMENT;
  a.k = static_cast<const uint16_t*>(k_bf16);
  a.ldk_t = ldk_t;
  a.ldk_h = ldk_h;
  a.v = static_cast<const uint16_t*>(v_bf16);
  a.ldv_t = ldv_t;
  a.ldv_h = ldv_h;
  a.k_open = static_cast<uint16_t*>(k_open);
  a.v_open = static_cast<uint16_t*>(v_open);
  a.cu_new = cu_new;
  a.T = T;
  a.max_new = std::min(max_new, T);
  a.err = reinterpret_cast<uint32_t*>(dev_error_word);
  return prism::record_cuda(prism::launch_kv_append(a, static_cast<cudaStream_t>(cuda_stream)));
}

size_t prism_kv_attention_workspace_bytes(int64_t S, int64_t T, int64_t max_q, int64_t max_pages, int64_t H_q,
                                          int64_t H_kv, int64_t D, int64_t block) {
  if (S <= 0 || T <= 0 || max_q <= 0 || max_pages <= 0 || H_q <= 0 || H_kv <= 0 || H_q % H_kv != 0) return 0;
  if ((D != 64 && D != 128 && D != 256) || (block != 16 && block != 32 && block != 64 && block != 128)) return 0;
  return prism::kv_attention_workspace_bytes(S, T, std::min(max_q, T), max_pages, H_q, H_kv, D, block);
}

int prism_kv_attention(const void* q_bf16, int64_t ldq_t, int64_t ldq_h, const int8_t* k_codes,
                       const int8_t* v_codes, const float* k_scale, const float* v_scale, const int32_t* page_table,
                       int64_t ld_table, const int32_t* seq_lens, const int32_t* cu_q, void* out_bf16, int64_t ldo_t,
                       int64_t ldo_h, float* lse, float sm_scale, int causal, int64_t window, int64_t S, int64_t T,
                       int64_t max_q, int64_t num_pages, int64_t max_pages, int64_t H_q, int64_t H_kv, int64_t D,
                       int64_t block, void* workspace, size_t workspace_bytes, int32_t* dev_error_word,
                       void* cuda_stream) {
  if (S < 0 || T < 0 || window < 0 || (causal != 0 && causal != 1)) return PRISM_ERR_INVALID_ARG;
  if (S == 0 || T == 0) return PRISM_OK;
  if (max_q < 1 || (cu_q == nullptr && T != S)) return PRISM_ERR_INVALID_ARG;
  if (window > 0 && !causal) return PRISM_ERR_INVALID_ARG;
  if (!(sm_scale > 0.0f) || sm_scale > 3e38f) return PRISM_ERR_INVALID_ARG;
  if (H_kv <= 0 || H_q <= 0 || H_q % H_kv != 0) return PRISM_ERR_INVALID_ARG;
  prism::KvAttentionArgs a{};
  int st = check_cache(k_codes, v_codes, k_scale, v_scale, page_table, ld_table, seq_lens, S, num_pages, max_pages,
                       H_kv, D, block, a.c);
  if (st != PRISM_OK) return st;
  if (H_q > (1 << 16) || T > kInt31 || T * H_q > kInt31) return PRISM_ERR_UNSUPPORTED;
  if ((st = check_rows(q_bf16, ldq_t, ldq_h, T, H_q, D)) != PRISM_OK) return st;
  if ((st = check_rows(out_bf16, ldo_t, ldo_h, T, H_q, D)) != PRISM_OK) return st;
  if (!aligned(lse, 4) || !aligned(cu_q, 4) || !aligned(dev_error_word, 4)) return PRISM_ERR_ALIGNMENT;
  max_q = std::min(max_q, T);
  const size_t need = prism::kv_attention_workspace_bytes(S, T, max_q, max_pages, H_q, H_kv, D, block);
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need) return PRISM_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return PRISM_ERR_ALIGNMENT;
  }
  a.q = static_cast<const uint16_t*>(q_bf16);
  a.ldq_t = ldq_t;
  a.ldq_h = ldq_h;
  a.out = static_cast<uint16_t*>(out_bf16);
  a.ldo_t = ldo_t;
  a.ldo_h = ldo_h;
  a.lse = lse;
  a.cu_q = cu_q;
  a.T = T;
  a.max_q = max_q;
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  a.causal = causal;
  a.window = window;
  a.Hq = static_cast<int32_t>(H_q);
  a.G = static_cast<int32_t>(H_q / H_kv);
  a.ws = workspace;
  a.err = reinterpret_cast<uint32_t*>(dev_error_word);
  return prism::record_cuda(prism::launch_kv_attention(a, static_cast<cudaStream_t>(cuda_stream)));
}

int prism_w4g_linear(const int8_t* q, int64_t ldq, const float* a_scale, const uint8_t* w4, int64_t ldw4,
                     const uint16_t* group_scale, int64_t lds, const uint16_t* group_offset, int64_t ldb,
                     const void* residual_bf16, int64_t ldr, void* out_bf16, int64_t ldo, int64_t M, int64_t N,
                     int64_t K, int64_t group, void* cuda_stream) {
  if (M < 0 || N < 0 || K <= 0 || group <= 0) return PRISM_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return PRISM_OK;
  if (q == nullptr || a_scale == nullptr || w4 == nullptr || group_scale == nullptr || out_bf16 == nullptr)
    return PRISM_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128) return PRISM_ERR_UNSUPPORTED;
  if (K % group != 0) return PRISM_ERR_INVALID_ARG;
  if (K > PRISM_MAX_K || N > kInt31 / 8 || M > 65535 * 64) return PRISM_ERR_UNSUPPORTED;
  if (ldq < K || ldw4 < K / 2 || lds < K / group || ldo < N || (group_offset != nullptr && ldb < K / group) ||
      (residual_bf16 != nullptr && ldr < N))
    return PRISM_ERR_INVALID_ARG;
  if (ldq % 16 != 0 || ldw4 % 16 != 0) return PRISM_ERR_ALIGNMENT;
  if (!aligned(q, 16) || !aligned(w4, 16) || !aligned(a_scale, 4) || !aligned(group_scale, 2) ||
      !aligned(group_offset, 2) || !aligned(residual_bf16, 2) || !aligned(out_bf16, 2))
    return PRISM_ERR_ALIGNMENT;
  prism::W4gArgs a{};
  a.q = q;
  a.ldq = ldq;
  a.a_scale = a_scale;
  a.w4 = w4;
  a.ldw4 = ldw4;
  a.scale = group_scale;
  a.lds = lds;
  a.offset = group_offset;
  a.ldb = ldb;
  a.residual = static_cast<const uint16_t*>(residual_bf16);
  a.ldr = ldr;
  a.out = static_cast<uint16_t*>(out_bf16);
  a.ldo = ldo;
  a.M = M;
  a.N = N;
  a.K = K;
  a.group = static_cast<int32_t>(group);
  return prism::record_cuda(prism::launch_w4g(a, static_cast<cudaStream_t>(cuda_stream)));
}

int prism_token_logprobs(const void* logits, int logits_f32, int64_t ldl, const int32_t* token_ids, int64_t ld_ids,
                         int64_t n_ids, int64_t R, int64_t V, int64_t top_k, float* logprobs, float* entropy,
                         int32_t* top_ids, float* top_logprobs, int32_t* dev_error_word, void* cuda_stream) {
  if (R < 0 || V <= 0 || n_ids < 0 || top_k < 0 || top_k > V || (logits_f32 != 0 && logits_f32 != 1))
    return PRISM_ERR_INVALID_ARG;
  if (R == 0) return PRISM_OK;
  if (logits == nullptr || ldl < V) return PRISM_ERR_INVALID_ARG;
  if (n_ids > 0 && (token_ids == nullptr || logprobs == nullptr || ld_ids < n_ids)) return PRISM_ERR_INVALID_ARG;
  if (top_k > 0 && (top_ids == nullptr || top_logprobs == nullptr)) return PRISM_ERR_INVALID_ARG;
  if (top_k > PRISM_MAX_TOP_K || V > kInt31 || R > kInt31 / 8 || n_ids > kInt31) return PRISM_ERR_UNSUPPORTED;
  if (!aligned(logits, logits_f32 ? 4 : 2) || !aligned(token_ids, 4) || !aligned(logprobs, 4) ||
      !aligned(entropy, 4) || !aligned(top_ids, 4) || !aligned(top_logprobs, 4) || !aligned(dev_error_word, 4))
    return PRISM_ERR_ALIGNMENT;
  prism::LogprobArgs a{};
  a.logits = logits;
  a.f32 = logits_f32;
  a.ldl = ldl;
  a.ids = token_ids;
  a.ld_ids = ld_ids;
  a.n_ids = static_cast<int32_t>(n_ids);
  a.R = R;
  a.V = V;
  a.top_k = static_cast<int32_t>(top_k);
  a.logprobs = logprobs;
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  a.err = reinterpret_cast<uint32_t*>(dev_error_word);
  return prism::record_cuda(prism::launch_token_logprobs(a, static_cast<cudaStream_t>(cuda_stream)));
}

}  // extern "C"
