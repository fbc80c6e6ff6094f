// linear_attention.cu -- linear attention with a decay for each head:
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale * q_t S_t
// with a state S [Dk, Dv] in binary32 for each (sequence, value head).
//
// Up to kFewTokens tokens of a sequence (decode steps, drafted tokens): the
// recurrence as it stands.  The state is read once into registers, every token
// updates it and reads it out, and it is written once: bytes, 8 Dk Dv a head,
// bound it (64 sequences of a token, 40 heads of 128 by 128: 54.8 us, 6.2 TB/s of
// states; one sequence 3.5 us, a launch and a state's way to the SM and back).
//
// More tokens go by in chunks of 64 (linear_attention_tc.cu).
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

template <int DK, int DV>
cudaError_t launch_few(const LinAttnArgs& a, cudaStream_t stream) {
  // narrow slices where whole heads leave SMs empty
  const int width = a.S * a.Hv >= 2 * kSms ? DV : 32;
  const dim3 grid(static_cast<unsigned>(a.S * (DV / width)), a.Hv);
  return launch_kernel(linear_few_kernel<DK>, grid, dim3(kGroups * width / 4), few_smem(DK, width), stream, true, a, width);
}

template <int DK, int DV>
cudaError_t launch_shape(const LinAttnArgs& a, cudaStream_t stream) {
  return a.max_len <= kFewTokens ? launch_few<DK, DV>(a, stream) : launch_linear_chunks<DK, DV>(a, stream);
}

}  // namespace

size_t linear_attention_workspace_bytes(int64_t S, int64_t T, int64_t max_len, int64_t Hv, int64_t Dk, int64_t Dv) {
  return static_cast<size_t>(places_of(S, T, max_len, cut_of(Hv)).total * Hv * (Dk * Dv + 4)) * 4;
}

cudaError_t launch_linear_attention(const LinAttnArgs& given, cudaStream_t stream) {
  LinAttnArgs a = given;
  a.cut = cut_of(a.Hv);
  a.places_each = places_of(a.S, a.T, a.max_len, a.cut).each;
  if (a.Dk == 64) return a.Dv == 64 ? launch_shape<64, 64>(a, stream) : launch_shape<64, 128>(a, stream);
  return a.Dv == 64 ? launch_shape<128, 64>(a, stream) : launch_shape<128, 128>(a, stream);
}

}  // namespace prism
