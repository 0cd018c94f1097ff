// Eviction from the e4m3 cache: of every sequence the most recent tokens and
// those of greatest weight, in order, moved to new pages.
//   choose: a CTA a sequence: the weight of rank n from four passes over its
//           bytes (counts of each byte's values among the weights that agree
//           above), then the indices in order;
//   move:   a CTA a new block of 64 tokens, whose scale follows the rule of
//           the append.
#include <cuda_runtime.h>

#include "fp8_paged.cuh"

namespace mla {
namespace {

constexpr int kBlock = MLA_FP8_BLOCK, kKey = kFp8Key;
constexpr int kChoose = 1024, kMove = 256;

// Weights as integers of the same order; NaN comes first, -0 is 0.
__device__ __forceinline__ uint32_t rank_key(float w) {
  if (isnan(w)) return 0;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kChoose) fp8_evict_choose_kernel(const Fp8EvictArgs a) {
  __shared__ int count[256], warp_sum[2][32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_left;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
    const float* w = a.weights + b * a.weights_stride;
    const int64_t room = min(min(a.max_pages * a.page_size, a.row_len), static_cast<int64_t>(1) << 30);
    const int len = fp8_length(a.seq_lens[b], room, a.error_word, tid == 0);
    const int n = fp8_length(min(len, a.keep), a.new_max_pages * a.page_size, a.error_word, tid == 0);
    const int old = len - min(len, min(a.recent, n));  // tokens that may go
    int left = n - (len - old);                        // of them stay
    // the smallest key that stays, and how many of those equal to it
    uint32_t prefix = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) count[tid] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
      for (int t = tid; t < old; t += kChoose) {
        const uint32_t k = rank_key(w[t]);
        if ((k & mask) == prefix) atomicAdd(&count[k >> shift & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int v = 255, l = left;
        while (v > 0 && count[v] < l) l -= count[v--];
        s_prefix = prefix | static_cast<uint32_t>(v) << shift;
        s_left = l;
      }
      __syncthreads();
      prefix = s_prefix;
      left = s_left;
    }
    // in order
    int done = 0, equal = 0;
    for (int base = 0; base < len; base += kChoose) {
      const int t = base + tid;
      const uint32_t k = t < old ? rank_key(w[t]) : 0;
      const bool tie = t < old && k == prefix, above = t < len && (t >= old || k > prefix);
      const uint32_t ties = __ballot_sync(0xffffffffu, tie);
      if (lane == 0) warp_sum[0][warp] = __popc(ties);
      __syncthreads();
      int before = equal;
      for (int i = 0; i < warp; ++i) before += warp_sum[0][i];
      for (int i = 0; i < 32; ++i) equal += warp_sum[0][i];
      const bool stays = above || (tie && before + __popc(ties & ((1u << lane) - 1)) < left);
      const uint32_t all = __ballot_sync(0xffffffffu, stays);
      if (lane == 0) warp_sum[1][warp] = __popc(all);
      __syncthreads();
      int at = done + __popc(all & ((1u << lane) - 1));
      for (int i = 0; i < warp; ++i) at += warp_sum[1][i];
      for (int i = 0; i < 32; ++i) done += warp_sum[1][i];
      if (stays && at < n) {
        a.kept[static_cast<int64_t>(b) * a.keep + at] = t;
        if (a.new_weights != nullptr) a.new_weights[b * a.new_weights_stride + at] = w[t];
      }
    }
    for (int i = n + tid; i < a.keep; i += kChoose) a.kept[static_cast<int64_t>(b) * a.keep + i] = -1;
    if (a.new_weights != nullptr)
      for (int64_t i = n + tid; i < a.new_row_len; i += kChoose) a.new_weights[b * a.new_weights_stride + i] = 0.f;
    if (tid == 0) a.new_lens[b] = n;
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kMove) fp8_evict_move_kernel(const Fp8EvictArgs a, int blocks) {
  const int b = blockIdx.x / blocks, i = blockIdx.x % blocks, tid = threadIdx.x;
  const int n = a.new_lens[b], rows = min(kBlock, n - i * kBlock);
  if (rows <= 0) return;
  __shared__ int64_t from[kBlock];
  __shared__ float scale[kBlock], most[kMove / 32];
  if (tid < rows) {
    const int t = a.kept[static_cast<int64_t>(b) * a.keep + i * kBlock + tid];
    const int64_t slot = fp8_block_slot(a.page_table + b * a.pt_stride, t / kBlock, a.page_size, a.num_slots);
    const float s = slot < 0 ? 0.f : a.scales[slot / kBlock];
    const bool good = s >= kFp8ScaleMin && s <= kFp8ScaleMax;
    if (!good) flag_error(a.error_word, slot < 0 ? MLA_DEVERR_BOUNDS : MLA_DEVERR_SCALE);
    from[tid] = good ? slot + t % kBlock : -1;
    scale[tid] = good ? s : 0.f;
  }
  __syncthreads();
  auto value = [&](int r, int j) { return from[r] < 0 ? 0.f : e4m3_to_f32(a.cache[from[r] * kKey + j]) * scale[r]; };
  float am = 0.f;
  for (int e = tid; e < rows * kKey; e += kMove) am = fmaxf(am, fabsf(value(e / kKey, e % kKey)));
  for (int o = 16; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
  if ((tid & 31) == 0) most[tid >> 5] = am;
  __syncthreads();
  for (int k = 0; k < kMove / 32; ++k) am = fmaxf(am, most[k]);
  const float s = fp8_block_scale(am);
  const int64_t to = fp8_block_slot(a.new_page_table + b * a.new_pt_stride, i, a.page_size, a.num_slots);
  if (to < 0) {
    if (tid == 0) flag_error(a.error_word, MLA_DEVERR_BOUNDS);
    return;
  }
  if (tid == 0) a.scales[to / kBlock] = s;
  for (int e = tid; e < rows * kKey; e += kMove)
    a.cache[to * kKey + e] = static_cast<uint8_t>(cvt_e4m3(value(e / kKey, e % kKey) * (1.f / s)));
}

}  // namespace

int launch_fp8_evict(const Fp8EvictArgs& a, cudaStream_t stream) {
  const int blocks = (a.keep + kBlock - 1) / kBlock;
  if (static_cast<int64_t>(a.batch) * blocks > (int64_t(1) << 31) - 1) return MLA_ERR_INVALID_ARG;
  fp8_evict_choose_kernel<<<a.batch, kChoose, 0, stream>>>(a);
  if (const int st = launch_status()) return st;
  fp8_evict_move_kernel<<<a.batch * blocks, kMove, 0, stream>>>(a, blocks);
  return launch_status();
}

}  // namespace mla
