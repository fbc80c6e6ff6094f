// decode.cuh -- arguments and launchers of the decode-step kernels: the paged
// int8 K/V cache's append and attention, the 4-bit group-scaled linear, and
// the token log probabilities.  Contracts in include/prism.h.
#pragma once

#include "common.cuh"

namespace prism {

// SMs that work is cut for, whatever the device has: the order of sums follows the
// cuts, so results are those of a call's sizes alone.
constexpr int kSms = 152;

// A paged cache as the kernels see it (dense [num_pages, H, block, D] codes).
struct KvPages {
  int8_t* k_codes;
  int8_t* v_codes;
  float* k_scale;
  float* v_scale;
  const int32_t* table;
  int64_t ld_table;
  const int32_t* lens;
  int64_t num_pages, max_pages;
  int32_t S, H, D, block, block_shift;
};

struct KvAppendArgs {
  KvPages c;
  const uint16_t* k;
  int64_t ldk_t, ldk_h;
  const uint16_t* v;
  int64_t ldv_t, ldv_h;
  uint16_t* k_open;
  uint16_t* v_open;
  const int32_t* cu_new;   // null: one row per sequence
  int64_t T, max_new;
  uint32_t* err;
};
cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t stream);

struct KvAttentionArgs {
  KvPages c;
  const uint16_t* q;
  int64_t ldq_t, ldq_h;
  uint16_t* out;
  int64_t ldo_t, ldo_h;
  float* lse;
  const int32_t* cu_q;     // null: one query per sequence
  int64_t T, max_q;
  float scale_log2;        // sm_scale * log2(e)
  int32_t causal;
  int64_t window;
  int32_t Hq, G;           // query heads, query heads per KV head
  void* ws;
  uint32_t* err;
};
size_t kv_attention_workspace_bytes(int64_t S, int64_t T, int64_t max_q, int64_t max_pages, int64_t Hq, int64_t Hkv,
                                    int64_t D, int64_t block);
cudaError_t launch_kv_attention(const KvAttentionArgs& a, cudaStream_t stream);
// Device status bits of its bounded waits, and their test mode (prism_debug_wait_expiry).
cudaError_t read_and_clear_kv_status(uint32_t* out);
cudaError_t set_kv_wait_expiry(unsigned long long limit_ns, int withhold);

struct W4gArgs {
  const int8_t* q;
  int64_t ldq;
  const float* a_scale;
  const uint8_t* w4;
  int64_t ldw4;
  const uint16_t* scale;
  int64_t lds;
  const uint16_t* offset;
  int64_t ldb;
  const uint16_t* residual;
  int64_t ldr;
  uint16_t* out;
  int64_t ldo;
  int64_t M, N, K;
  int32_t group;
};
cudaError_t launch_w4g(const W4gArgs& a, cudaStream_t stream);
// Device status bits of its bounded waits, and their test mode (prism_debug_wait_expiry).
cudaError_t read_and_clear_w4g_status(uint32_t* out);
cudaError_t set_w4g_wait_expiry(unsigned long long limit_ns, int withhold);

struct LogprobArgs {
  const void* logits;
  int32_t f32;
  int64_t ldl;
  const int32_t* ids;
  int64_t ld_ids;
  int32_t n_ids;
  int64_t R, V;
  int32_t top_k;
  float* logprobs;
  float* entropy;
  int32_t* top_ids;
  float* top_logprobs;
  uint32_t* err;
};
cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t stream);

// Two binary32 operations in one instruction, each rounded as by itself.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Sequence s's rows [b, e) of a packed [T, ...] input and its length; false
// (and the error bit) for offsets or a length outside their ranges.  The
// check needs nothing but the sequence's own entries.
struct SeqSpan {
  int32_t b, n;
  int64_t len;
};
__device__ __forceinline__ bool seq_span(const KvPages& c, const int32_t* cu, int64_t T, int s, bool len_after,
                                         SeqSpan& o) {
  const int32_t b = cu != nullptr ? cu[s] : s, e = cu != nullptr ? cu[s + 1] : s + 1;
  const int32_t len = c.lens[s];
  o.b = b;
  o.n = e - b;
  o.len = len;
  if (b < 0 || e < b || e > T || len < 0) return false;
  const int64_t last = len_after ? len : static_cast<int64_t>(len) + o.n;
  return last <= (c.max_pages << c.block_shift);
}

}  // namespace prism
