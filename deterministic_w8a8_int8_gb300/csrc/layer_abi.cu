// layer_abi.cu -- the extern "C" boundary of the operators between a layer's
// linears: host-side argument checks (returned as prism_status before anything
// is enqueued) and dispatch to the launchers.  See include/prism.h.
#include "layer.cuh"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
constexpr int64_t kInt31 = (1LL << 31) - 1;

// A [M, K] bf16 operand.
int check_matrix(const void* p, int64_t ld, int64_t K) {
  if (p == nullptr || ld < K) return PRISM_ERR_INVALID_ARG;
  return ld % 8 != 0 || !aligned(p, 16) ? PRISM_ERR_ALIGNMENT : PRISM_OK;
}

// Rows of K codes or values and their scales; fills o where they are sound.
int check_codes(int form, void* q, int64_t ldq, float* a_scale, int64_t K, prism::RowCodes& o) {
  if (form != PRISM_FORM_INT8 && form != PRISM_FORM_F16 && form != PRISM_FORM_BF16) return PRISM_ERR_INVALID_ARG;
  if (q == nullptr || ldq < K || (form != PRISM_FORM_BF16) != (a_scale != nullptr)) return PRISM_ERR_INVALID_ARG;
  if (K < 16 || K % 16 != 0 || K > PRISM_MAX_ROW) return PRISM_ERR_UNSUPPORTED;
  if (ldq % (form == PRISM_FORM_INT8 ? 16 : 8) != 0 || !aligned(q, 16) || !aligned(a_scale, 4)) return PRISM_ERR_ALIGNMENT;
  o = prism::RowCodes{form, q, ldq, a_scale};
  return PRISM_OK;
}

int check_eps(float eps) { return eps >= 1e-20f && eps <= 1.0f ? PRISM_OK : PRISM_ERR_INVALID_ARG; }

void set_mean(prism::NormArgs& a, int64_t n) {
  const double inv = 1.0 / static_cast<double>(n);
  a.inv_n = static_cast<float>(inv);
  a.inv_n_low = static_cast<float>(inv - static_cast<double>(a.inv_n));
}

// A [T, H, D] bf16 operand: strides and alignment.
int check_heads(const void* p, int64_t ld_t, int64_t ld_h, int64_t T, int64_t H, int64_t D) {
  if (p == nullptr) return PRISM_ERR_INVALID_ARG;
  if ((T > 1 && ld_t < D) || (H > 1 && ld_h < D)) return PRISM_ERR_INVALID_ARG;
  return ld_t % 8 != 0 || ld_h % 8 != 0 || !aligned(p, 16) ? PRISM_ERR_ALIGNMENT : PRISM_OK;
}

// Sizes of linear attention: S * H_v is searched for work within the kernels' bounded waits.
bool within(int64_t S, int64_t T, int64_t H_v) { return S <= (1 << 24) && T <= kInt31 && H_v <= 65535 && S * H_v <= (1 << 28); }

}  // namespace

extern "C" {

int prism_norm_quant(const void* x_bf16, int64_t ldx, const void* delta_bf16, int64_t ldd, float alpha,
                     const float* post_weight, const float* weight, float eps, int64_t M, int64_t K, void* h_bf16,
                     int64_t ldh, int form, void* q, int64_t ldq, float* a_scale, void* cuda_stream) {
  if (M < 0 || K <= 0) return PRISM_ERR_INVALID_ARG;
  if (M == 0) return PRISM_OK;
  prism::NormArgs a{};
  int st = check_codes(form, q, ldq, a_scale, K, a.o);
  if (st != PRISM_OK) return st;
  if ((st = check_matrix(x_bf16, ldx, K)) != PRISM_OK || (st = check_eps(eps)) != PRISM_OK) return st;
  if (weight == nullptr || (delta_bf16 == nullptr) != (h_bf16 == nullptr) ||
      (delta_bf16 == nullptr && post_weight != nullptr) || !(alpha > -3e38f && alpha < 3e38f))
    return PRISM_ERR_INVALID_ARG;
  if (!aligned(weight, 16) || !aligned(post_weight, 16)) return PRISM_ERR_ALIGNMENT;
  if (delta_bf16 != nullptr &&
      ((st = check_matrix(delta_bf16, ldd, K)) != PRISM_OK || (st = check_matrix(h_bf16, ldh, K)) != PRISM_OK))
    return st;
  if (h_bf16 != nullptr && ((h_bf16 == x_bf16 && ldh != ldx) || (h_bf16 == delta_bf16 && ldh != ldd)))
    return PRISM_ERR_INVALID_ARG;
  a.x = static_cast<const uint16_t*>(x_bf16);
  a.ldx = ldx;
  a.delta = static_cast<const uint16_t*>(delta_bf16);
  a.ldd = ldd;
  a.alpha = alpha;
  a.post = post_weight;
  a.weight = weight;
  a.eps = eps;
  set_mean(a, K);
  a.M = M;
  a.K = K;
  a.h = static_cast<uint16_t*>(h_bf16);
  a.ldh = ldh;
  return prism::record_cuda(prism::launch_norm_quant(a, static_cast<cudaStream_t>(cuda_stream)));
}

int prism_head_norm_quant(const void* x_bf16, int64_t ldx, const float* weight, const void* gate_bf16, int64_t ldg,
                          const float* inv_smooth, float eps, int64_t M, int64_t H, int64_t D, int form, void* q,
                          int64_t ldq, float* a_scale, void* cuda_stream) {
  if (M < 0 || H <= 0 || D <= 0) return PRISM_ERR_INVALID_ARG;
  if (M == 0) return PRISM_OK;
  if ((D != 64 && D != 128 && D != 256) || H > PRISM_MAX_ROW) return PRISM_ERR_UNSUPPORTED;
  prism::NormArgs a{};
  int st = check_codes(form, q, ldq, a_scale, H * D, a.o);
  if (st != PRISM_OK) return st;
  if ((st = check_matrix(x_bf16, ldx, H * D)) != PRISM_OK || (st = check_eps(eps)) != PRISM_OK) return st;
  if (weight == nullptr) return PRISM_ERR_INVALID_ARG;
  if (gate_bf16 != nullptr && (st = check_matrix(gate_bf16, ldg, H * D)) != PRISM_OK) return st;
  if (!aligned(weight, 16) || !aligned(inv_smooth, 16)) return PRISM_ERR_ALIGNMENT;
  a.x = static_cast<const uint16_t*>(x_bf16);
  a.ldx = ldx;
  a.weight = weight;
  a.eps = eps;
  set_mean(a, D);
  a.M = M;
  a.K = H * D;
  a.gate = static_cast<const uint16_t*>(gate_bf16);
  a.ldg = ldg;
  a.inv_s = inv_smooth;
  a.D = static_cast<int32_t>(D);
  return prism::record_cuda(prism::launch_head_norm_quant(a, static_cast<cudaStream_t>(cuda_stream)));
}

int prism_glu_quant(const void* gate_up_bf16, int64_t ldx, const float* inv_smooth, int64_t M, int64_t F, int form,
                    void* q, int64_t ldq, float* a_scale, void* cuda_stream) {
  if (M < 0 || F <= 0) return PRISM_ERR_INVALID_ARG;
  if (M == 0) return PRISM_OK;
  prism::GluArgs a{};
  int st = check_codes(form, q, ldq, a_scale, F, a.o);
  if (st != PRISM_OK) return st;
  if ((st = check_matrix(gate_up_bf16, ldx, 2 * F)) != PRISM_OK) return st;
  if (!aligned(inv_smooth, 16)) return PRISM_ERR_ALIGNMENT;
  a.x = static_cast<const uint16_t*>(gate_up_bf16);
  a.ldx = ldx;
  a.inv_s = inv_smooth;
  a.M = M;
  a.F = F;
  return prism::record_cuda(prism::launch_glu_quant(a, static_cast<cudaStream_t>(cuda_stream)));
}

size_t prism_linear_attention_workspace_bytes(int64_t S, int64_t T, int64_t max_len, int64_t H_v, int64_t D_k,
                                              int64_t D_v) {
  if (S <= 0 || T <= 0 || max_len <= 0 || H_v <= 0 || (D_k != 64 && D_k != 128) || (D_v != 64 && D_v != 128)) return 0;
  if (!within(S, T, H_v)) return 0;   // the call is refused
  return prism::linear_attention_workspace_bytes(S, T, std::min(max_len, T), H_v, D_k, D_v);
}

int prism_linear_attention(const void* q_bf16, int64_t ldq_t, int64_t ldq_h, const void* k_bf16, int64_t ldk_t,
                           int64_t ldk_h, const void* v_bf16, int64_t ldv_t, int64_t ldv_h, const float* log_decay,
                           int64_t ldd_t, float* state, const int32_t* state_in, const int32_t* state_out,
                           const int32_t* cu, void* out_bf16, int64_t ldo_t, int64_t ldo_h, float scale, int64_t S,
                           int64_t T, int64_t max_len, int64_t num_states, int64_t H_k, int64_t H_v, int64_t D_k,
                           int64_t D_v, void* workspace, size_t workspace_bytes, int32_t* dev_error_word,
                           void* cuda_stream) {
  if (S < 0 || T < 0) return PRISM_ERR_INVALID_ARG;
  if (S == 0) return PRISM_OK;
  if (max_len < 1 || num_states < 0 || (cu == nullptr && T != S)) return PRISM_ERR_INVALID_ARG;
  if (H_k <= 0 || H_v <= 0 || H_v % H_k != 0) return PRISM_ERR_INVALID_ARG;
  if (!(scale >= -0x1p64f && scale <= 0x1p64f)) return PRISM_ERR_INVALID_ARG;   // times 2^40 in chunks
  if ((D_k != 64 && D_k != 128) || (D_v != 64 && D_v != 128)) return PRISM_ERR_UNSUPPORTED;
  if (!within(S, T, H_v) || num_states > kInt31) return PRISM_ERR_UNSUPPORTED;
  if ((state_in != nullptr || state_out != nullptr) && (state == nullptr || num_states == 0)) return PRISM_ERR_INVALID_ARG;
  int st;
  if (T > 0) {   // no token: states are passed on alone
    if ((st = check_heads(q_bf16, ldq_t, ldq_h, T, H_k, D_k)) != PRISM_OK) return st;
    if ((st = check_heads(k_bf16, ldk_t, ldk_h, T, H_k, D_k)) != PRISM_OK) return st;
    if ((st = check_heads(v_bf16, ldv_t, ldv_h, T, H_v, D_v)) != PRISM_OK) return st;
    if ((st = check_heads(out_bf16, ldo_t, ldo_h, T, H_v, D_v)) != PRISM_OK) return st;
    if (log_decay == nullptr || (ldd_t != 0 && ldd_t < H_v)) return PRISM_ERR_INVALID_ARG;
  }
  if (!aligned(log_decay, 4) || !aligned(state, 16) || !aligned(state_in, 4) || !aligned(state_out, 4) ||
      !aligned(cu, 4) || !aligned(dev_error_word, 4))
    return PRISM_ERR_ALIGNMENT;
  max_len = std::min(max_len, std::max<int64_t>(T, 1));
  const size_t need = prism::linear_attention_workspace_bytes(S, T, max_len, H_v, D_k, D_v);
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need) return PRISM_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return PRISM_ERR_ALIGNMENT;
  }
  prism::LinAttnArgs a{};
  a.q = static_cast<const uint16_t*>(q_bf16);
  a.ldq_t = ldq_t;
  a.ldq_h = ldq_h;
  a.k = static_cast<const uint16_t*>(k_bf16);
  a.ldk_t = ldk_t;
  a.ldk_h = ldk_h;
  a.v = static_cast<const uint16_t*>(v_bf16);
  a.ldv_t = ldv_t;
  a.ldv_h = ldv_h;
  a.decay = log_decay;
  a.ldd_t = ldd_t;
  a.state = state;
  a.state_in = state_in;
  a.state_out = state_out;
  a.cu = cu;
  a.out = static_cast<uint16_t*>(out_bf16);
  a.ldo_t = ldo_t;
  a.ldo_h = ldo_h;
  a.scale = scale;
  a.S = S;
  a.T = T;
  a.max_len = max_len;
  a.num_states = num_states;
  a.Hk = static_cast<int32_t>(H_k);
  a.Hv = static_cast<int32_t>(H_v);
  a.Dk = static_cast<int32_t>(D_k);
  a.Dv = static_cast<int32_t>(D_v);
  a.G = static_cast<int32_t>(H_v / H_k);
  a.ws = static_cast<float*>(workspace);
  a.err = reinterpret_cast<uint32_t*>(dev_error_word);
  return prism::record_cuda(prism::launch_linear_attention(a, static_cast<cudaStream_t>(cuda_stream)));
}

}  // extern "C"
