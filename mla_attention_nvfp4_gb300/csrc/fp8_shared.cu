// Absorbed MLA decode over the e4m3 cache for a batch whose sequences begin
// with the same tokens: a CTA a (sequence, head), 256 keys at a time.
#include <cuda_runtime.h>

#include "fp8_paged.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256, kBlock = MLA_FP8_BLOCK;

__global__ void __launch_bounds__(kThreads) fp8_shared_kernel(const Fp8DecodeArgs a, int64_t shared_len) {
  __shared__ float q[kFp8Key], p[kThreads], red[kThreads / 32];
  __shared__ int64_t from[kThreads];
  const int b = blockIdx.x / a.num_heads, tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  for (int j = tid; j < kFp8Key; j += kThreads)
    q[j] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[row * kFp8Key + j]);
  const int64_t room = min(a.max_pages * a.page_size, static_cast<int64_t>(1) << 30);
  const int len = fp8_length(a.seq_lens[b], room, a.error_word, tid == 0);
  float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
  int any = 0;
  __syncthreads();
  for (int base = 0; base < len; base += kThreads) {
    const int t = base + tid;
    float x = -INFINITY, scale = 0.f;
    from[tid] = -1;
    if (t < len) {
      const int owner = t < shared_len && len >= shared_len ? 0 : b;
      const int64_t slot = fp8_block_slot(a.page_table + owner * a.pt_stride, t / kBlock, a.page_size, a.num_slots);
      scale = slot < 0 ? 0.f : a.scales[slot / kBlock];
      if (scale >= kFp8ScaleMin && scale <= kFp8ScaleMax) {
        from[tid] = slot + t % kBlock;
        float dot = 0.f;
        for (int j = 0; j < kFp8Key; ++j) dot = fmaf(e4m3_to_f32(a.cache[from[tid] * kFp8Key + j]), q[j], dot);
        x = dot * scale * a.softmax_scale;
      } else {
        flag_error(a.error_word, slot < 0 ? MLA_DEVERR_BOUNDS : MLA_DEVERR_SCALE);
      }
    }
    float top = x;
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((tid & 31) == 0) red[tid >> 5] = top;
    __syncthreads();
    for (int i = 0; i < kThreads / 32; ++i) top = fmaxf(top, red[i]);
    const float now = fmaxf(m, top), by = now == -INFINITY ? 1.f : expf(m - now);
    const float e = from[tid] < 0 || x == -INFINITY ? 0.f : expf(x - now);
    any |= __syncthreads_or(from[tid] >= 0);
    p[tid] = e * scale;
    float sum = e;
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = sum;
    __syncthreads();
    l *= by, o0 *= by, o1 *= by, m = now;
    for (int i = 0; i < kThreads / 32; ++i) l += red[i];
    for (int i = 0; i < min(kThreads, len - base); ++i)
      if (from[i] >= 0) {
        const uint8_t* v = a.cache + from[i] * kFp8Key + 2 * tid;
        o0 = fmaf(p[i], e4m3_to_f32(v[0]), o0);
        o1 = fmaf(p[i], e4m3_to_f32(v[1]), o1);
      }
    __syncthreads();
  }
  if (any && l == 0.f) l = __uint_as_float(0x7FC00000u);  // all scores below fp32's range
  const float inv = l != 0.f ? 1.f / l : 0.f;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + row * MLA_D_LATENT + 2 * tid;
  out[0] = __float2bfloat16_rn(o0 * inv);
  out[1] = __float2bfloat16_rn(o1 * inv);
  if (a.lse != nullptr && tid == 0) a.lse[row] = l != 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t fp8_shared_workspace_bytes(int, int, int) { return 256; }

int launch_fp8_shared(const Fp8DecodeArgs& a, int64_t shared_len, cudaStream_t stream, int /*num_sms*/) {
  const int64_t rows = static_cast<int64_t>(a.batch) * a.num_heads;
  if (rows > (int64_t(1) << 31) - 1) return MLA_ERR_INVALID_ARG;
  fp8_shared_kernel<<<static_cast<unsigned>(rows), kThreads, 0, stream>>>(a, shared_len);
  return launch_status();
}

}  // namespace mla
