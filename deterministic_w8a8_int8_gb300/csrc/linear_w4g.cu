// linear_w4g.cu -- int8 activations times 4-bit weights with group scales.
#include <cuda_fp16.h>

#include "decode.cuh"

namespace prism {
namespace {

constexpr int kWarps = 4;

// One warp per (output channel, token); a lane takes every 32nd group, whose
// sums are exact integers, and adds them in binary32; then a fixed tree.
__global__ void __launch_bounds__(kWarps * 32) w4g_kernel(const __grid_constant__ W4gArgs a) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (n >= a.N) return;
  for (int64_t m = blockIdx.y; m < a.M; m += gridDim.y) {
    float y = 0.0f;
    for (int64_t g = lane; g < a.K / a.group; g += 32) {
      const uint8_t* w = a.w4 + n * a.ldw4 + g * (a.group / 2);
      const int8_t* q = a.q + m * a.ldq + g * a.group;
      int dot = 0, sum = 0;
      for (int i = 0; i < a.group / 2; ++i) {
        const int b = w[i];
        dot += q[2 * i] * (((b & 15) ^ 8) - 8) + q[2 * i + 1] * (((b >> 4) ^ 8) - 8);
        sum += q[2 * i] + q[2 * i + 1];
      }
      y = fmaf(static_cast<float>(dot), __half2float(__ushort_as_half(a.scale[n * a.lds + g])), y);
      if (a.offset != nullptr)
        y = fmaf(static_cast<float>(sum), __half2float(__ushort_as_half(a.offset[n * a.ldb + g])), y);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (lane == 0) {
      y = __fmul_rn(y, a.a_scale[m]);
      if (a.residual != nullptr) y = __fadd_rn(y, bf16_bits_to_float(a.residual[m * a.ldr + n]));
      a.out[m * a.ldo + n] = static_cast<uint16_t>(float_to_bf16_rne(y));
    }
  }
}

}  // namespace

cudaError_t launch_w4g(const W4gArgs& a, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((a.N + kWarps - 1) / kWarps), static_cast<unsigned>(std::min<int64_t>(a.M, 65535)));
  return launch_kernel(w4g_kernel, grid, dim3(kWarps * 32), 0, stream, true, a);
}

}  // namespace prism
