// bf16 rows times an NVFP4 weight matrix (one, or one a group): a warp an
// output column, lane l blocks of 16 features l, l + 32, ..
#include <cuda_runtime.h>

#include "launch.h"
#include "nvfp4.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) nvfp4_gemv_kernel(const GemvArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  if (col >= a.groups * a.N) return;
  const int64_t g = col / a.N, n = col - g * a.N;
  const int64_t k_tiles = (a.K / 16 + 3) / 4, scale_bytes = (a.N + 127) / 128 * k_tiles * 512;
  const uint8_t* codes = a.w_codes + col * (a.K / 2);
  const uint8_t* scales = a.w_scales + g * scale_bytes;
  const float gs = *a.gs_w;
  for (int64_t m = 0; m < a.M; ++m) {
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x) + m * a.x_sm + g * a.x_sg;
    float sum = 0.f;
    for (int64_t kb = lane; kb < a.K / 16; kb += 32) {
      float part = 0.f;
      for (int i = 0; i < 16; ++i) {
        const int code = codes[kb * 8 + i / 2] >> (4 * (i & 1)) & 15, e = code >> 1 & 3, frac = code & 1;
        const float mag = e > 0 ? (1.f + 0.5f * frac) * static_cast<float>(1 << (e - 1)) : 0.5f * frac;
        part = fmaf(code & 8 ? -mag : mag, __bfloat162float(x[kb * 16 + i]), part);
      }
      sum = fmaf(part, e4m3_to_f32(scales[sf_offset(n, kb, k_tiles)]), sum);
    }
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0)
      static_cast<__nv_bfloat16*>(a.out)[m * a.out_sm + g * a.out_sg + n] = __float2bfloat16_rn(sum * gs);
  }
}

}  // namespace

int launch_gemv(const GemvArgs& a, cudaStream_t stream, int /*num_sms*/) {
  const int64_t grid = (a.groups * a.N + kThreads / 32 - 1) / (kThreads / 32);
  if (grid > (int64_t(1) << 31) - 1) return MLA_ERR_INVALID_ARG;
  nvfp4_gemv_kernel<<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(a);
  return launch_status();
}

}  // namespace mla
