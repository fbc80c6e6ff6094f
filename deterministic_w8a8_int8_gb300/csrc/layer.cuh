// layer.cuh -- arguments and launchers of the operators between a layer's
// linears: norms and the gated activation down to codes, and linear attention.
// Contracts in include/prism.h.
#pragma once

#include "common.cuh"

namespace prism {

// A sum of binary32 numbers as the rounded sum and what is missing of it.
struct Sum {
  float h, l;
};
__device__ __forceinline__ Sum join(Sum a, Sum b) {
  const float s = __fadd_rn(a.h, b.h), t = __fsub_rn(s, a.h);
  const float e = __fadd_rn(__fsub_rn(a.h, __fsub_rn(s, t)), __fsub_rn(b.h, t));
  return Sum{s, __fadd_rn(e, __fadd_rn(a.l, b.l))};
}

struct RowCodes {          // where a row's values go (PRISM_FORM_*)
  int32_t form;
  void* q;
  int64_t ldq;
  float* a_scale;
};

struct NormArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* delta;   // null: none, and no h
  int64_t ldd;
  float alpha;
  const float* post;       // null: delta as it is
  const float* weight;
  float eps;
  float inv_n, inv_n_low;  // 1 / (values of a sum of squares), in two parts
  int64_t M, K;
  uint16_t* h;
  int64_t ldh;
  const uint16_t* gate;    // heads only; null: none
  int64_t ldg;
  const float* inv_s;      // heads only; null: ones
  int32_t D;               // heads only: channels of a head
  RowCodes o;
};
cudaError_t launch_norm_quant(const NormArgs& a, cudaStream_t stream);
cudaError_t launch_head_norm_quant(const NormArgs& a, cudaStream_t stream);

struct GluArgs {
  const uint16_t* x;       // [M, 2 F]
  int64_t ldx;
  const float* inv_s;
  int64_t M, F;
  RowCodes o;
};
cudaError_t launch_glu_quant(const GluArgs& a, cudaStream_t stream);

namespace lin {
// How long sequences are cut: `most` segments, of 2^shift tokens at least.
struct Cut {
  int64_t most;
  int32_t shift;
};
}  // namespace lin

struct LinAttnArgs {
  const uint16_t* q;
  int64_t ldq_t, ldq_h;
  const uint16_t* k;
  int64_t ldk_t, ldk_h;
  const uint16_t* v;
  int64_t ldv_t, ldv_h;
  const float* decay;
  int64_t ldd_t;           // 0: one for each head
  float* state;
  const int32_t* state_in;   // null: zeros
  const int32_t* state_out;  // null: not kept
  const int32_t* cu;         // null: one token each
  uint16_t* out;
  int64_t ldo_t, ldo_h;
  float scale;
  int64_t S, T, max_len, num_states;
  int32_t Hk, Hv, Dk, Dv, G;   // G: value heads of a key head
  lin::Cut cut;            // how sequences are cut (set by the launcher)
  int64_t places_each;     // workspace places of a sequence, or 0: by tokens (set by the launcher)
  float* ws;
  uint32_t* err;
};
size_t linear_attention_workspace_bytes(int64_t S, int64_t T, int64_t max_len, int64_t Hv, int64_t Dk, int64_t Dv);
cudaError_t launch_linear_attention(const LinAttnArgs& a, cudaStream_t stream);
// Device status bits of its bounded waits, and their test mode (prism_debug_wait_expiry).
cudaError_t read_and_clear_linear_status(uint32_t* out);
cudaError_t set_linear_wait_expiry(unsigned long long limit_ns, int withhold);

}  // namespace prism
