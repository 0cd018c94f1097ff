// Absorbed MLA decode over the e4m3 latent cache (one scale per block of 64
// tokens).
#include <cuda_runtime.h>

#include "launch.h"
#include "nvfp4.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

constexpr int kKey = MLA_D_LATENT + MLA_D_ROPE;
constexpr int kBlock = MLA_FP8_BLOCK;
constexpr float kScaleMin = 8.673617379884035e-19f, kScaleMax = 1.152921504606847e18f;  // 2^-60, 2^60

// One CTA per (head, sequence): blocks of 64 keys, online softmax, fp32.
__global__ void __launch_bounds__(256) fp8_decode_kernel(const Fp8DecodeArgs p) {
  __shared__ float qs[kKey], ps[kBlock];
  __shared__ int64_t slot_s;
  __shared__ float scale_s;
  const int h = blockIdx.x, b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + (static_cast<int64_t>(b) * p.num_heads + h) * kKey;
  for (int i = threadIdx.x; i < kKey; i += 256) qs[i] = __bfloat162float(q[i]);
  int64_t len = p.seq_lens[b];
  const int64_t room = p.max_pages * p.page_size;
  if (len > room) {
    if (threadIdx.x == 0) flag_error(p.error_word, MLA_DEVERR_BOUNDS);
    len = room;
  }
  float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
  for (int64_t t0 = 0; t0 < len; t0 += kBlock) {
    __syncthreads();
    if (threadIdx.x == 0) {
      const int64_t page = p.page_table[b * p.pt_stride + t0 / p.page_size];
      const int64_t s = page * p.page_size + t0 % p.page_size;
      slot_s = (page < 0 || s + kBlock > p.num_slots) ? -1 : s;
      if (slot_s < 0) flag_error(p.error_word, MLA_DEVERR_BOUNDS);
      scale_s = slot_s >= 0 ? p.scales[s / kBlock] : 0.f;
      if (slot_s >= 0 && !(scale_s >= kScaleMin && scale_s <= kScaleMax)) {
        flag_error(p.error_word, MLA_DEVERR_SCALE);
        slot_s = -1;
      }
    }
    __syncthreads();
    if (slot_s < 0) continue;
    const int n = len - t0 < kBlock ? static_cast<int>(len - t0) : kBlock;
    const uint8_t* base = p.cache + slot_s * kKey;
    for (int k = warp; k < n; k += 8) {
      float s = 0.f;
      for (int i = lane; i < kKey; i += 32) s = fmaf(qs[i], e4m3_to_f32(base[static_cast<int64_t>(k) * kKey + i]), s);
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0) ps[k] = s * scale_s * p.softmax_scale;
    }
    __syncthreads();
    float mb = m;
    for (int k = 0; k < n; ++k) mb = fmaxf(mb, ps[k]);
    const float f = expf(m - mb);
    o0 *= f;
    o1 *= f;
    l *= f;
    m = mb;
    for (int k = 0; k < n; ++k) {
      const float e = expf(ps[k] - m);
      l += e;
      const uint32_t h2 =
          e4m3x2_to_f16x2_pair(*reinterpret_cast<const uint16_t*>(base + static_cast<int64_t>(k) * kKey + 2 * threadIdx.x));
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h2));
      o0 = fmaf(e * scale_s, v.x, o0);
      o1 = fmaf(e * scale_s, v.y, o1);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + (static_cast<int64_t>(b) * p.num_heads + h) * MLA_D_LATENT;
  reinterpret_cast<__nv_bfloat162*>(out)[threadIdx.x] = __floats2bfloat162_rn(o0 * inv, o1 * inv);
  if (p.lse != nullptr && threadIdx.x == 0)
    p.lse[static_cast<int64_t>(b) * p.num_heads + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t fp8_decode_workspace_bytes(int batch, int num_heads, int num_sms) {
  (void)batch; (void)num_heads; (void)num_sms;
  return 256;
}

int launch_fp8_decode(const Fp8DecodeArgs& a, cudaStream_t stream, int num_sms) {
  (void)num_sms;
  fp8_decode_kernel<<<dim3(a.num_heads, a.batch), 256, 0, stream>>>(a);
  return launch_status();
}

}  // namespace mla
