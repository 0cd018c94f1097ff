// The attention weight that a step's queries give to each key of the e4m3
// cache, summed over the heads: a CTA a block of 64 tokens, a warp a key.
#include <cuda_runtime.h>

#include "fp8_paged.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256, kBlock = MLA_FP8_BLOCK;

__global__ void __launch_bounds__(kThreads) fp8_key_weights_kernel(const Fp8WeightsArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t room = min(min(a.max_pages * a.page_size, a.row_len), static_cast<int64_t>(1) << 30);
  for (int b = blockIdx.y; b < a.batch; b += gridDim.y) {
    const int len = fp8_length(a.seq_lens[b], room, a.error_word, blockIdx.x == 0 && threadIdx.x == 0);
    for (int i = blockIdx.x; i * kBlock < len; i += gridDim.x) {
      const int64_t slot = fp8_block_slot(a.page_table + b * a.pt_stride, i, a.page_size, a.num_slots);
      const float scale = slot < 0 ? 0.f : a.scales[slot / kBlock];
      const bool good = scale >= kFp8ScaleMin && scale <= kFp8ScaleMax;
      if (!good && threadIdx.x == 0) flag_error(a.error_word, slot < 0 ? MLA_DEVERR_BOUNDS : MLA_DEVERR_SCALE);
      for (int t = i * kBlock + warp; t < min(len, (i + 1) * kBlock); t += kThreads / 32) {
        float sum = 0.f;
        if (good) {
          float key[18];
          for (int j = 0; j < 18; ++j) key[j] = e4m3_to_f32(a.cache[(slot + t % kBlock) * kFp8Key + 32 * j + lane]) * scale;
          for (int h = 0; h < a.num_heads; ++h) {
            const int64_t row = static_cast<int64_t>(b) * a.num_heads + h;
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + row * kFp8Key;
            float dot = 0.f;
            for (int j = 0; j < 18; ++j) dot = fmaf(__bfloat162float(q[32 * j + lane]), key[j], dot);
            for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
            sum += expf(dot * a.softmax_scale - a.lse[row]);
          }
        }
        if (lane == 0)
          a.out[b * a.out_stride + t] = (a.weights != nullptr ? a.weights[b * a.weights_stride + t] : 0.f) + sum;
      }
    }
  }
}

}  // namespace

int launch_fp8_key_weights(const Fp8WeightsArgs& a, cudaStream_t stream, int num_sms) {
  const dim3 grid(a.batch < 8 * num_sms ? 8 * num_sms / a.batch : 1, a.batch < 65535 ? a.batch : 65535);
  fp8_key_weights_kernel<<<grid, kThreads, 0, stream>>>(a);
  return launch_status();
}

}  // namespace mla
