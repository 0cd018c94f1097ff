// Eviction from the e4m3 cache: of every sequence the most recent tokens and
// those of greatest weight, in order, moved to new pages.
//
//   choose  a cluster a sequence, each CTA a part of its tokens, whose weights
//           wait in shared memory as integers of their order.  The weight of rank
//           n comes 11, 11 and 10 bits at a time: counts of their values among the
//           weights that agree above them, summed over the cluster by every CTA.
//           Then the tokens above it, and the first of those equal to it, find
//           their places from counts of the warps and CTAs before.  Bound by its
//           chain of loads and barriers: 5.8 us for 1000 tokens, 15 for 32
//           sequences to 32k.  (Rounds of 8 bits with a histogram a warp: 19; rounds of
//           11 with 8 copies of the histogram: 22, for clearing and adding them.)
//   move    a CTA a new block of 64 tokens, all its rows in registers while the
//           largest is found: 128k tokens in 24.7 us, 6.0 TB/s read and written.  Its
//           scale follows the append's rule.  (Amax and rounding on f16 pairs; with
//           integer bytes and fp32 29.7 us.  Persistent CTAs with warps that find the
//           next block's rows meanwhile: 34.)
#include <cuda_runtime.h>

#include "fp8_paged.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kBlock = MLA_FP8_BLOCK, kKey = kFp8Key;
constexpr int kChoose = 1024, kWarps = kChoose / 32;
constexpr int kHeld = 16384;          // weights in shared memory; the others of a longer part are read again
constexpr int kPart = 2048;           // tokens a CTA of a cluster takes at least, where there are so many
constexpr int kBins = 2048;
constexpr int kChooseBytes = kHeld * 4;
constexpr int kMove = 256, kUnits = kBlock * kKey / 16 / kMove;  // 16-byte units a thread

// Weights as integers of the same order; NaN comes first, -0 is 0.
__device__ __forceinline__ uint32_t rank_key(float w) {
  if (isnan(w)) return 0;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int2 cluster_load2(const int2* p, int rank) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(cluster_addr(smem_u32(p), rank)) : "memory");
  return v;
}

__global__ void __launch_bounds__(kChoose, 1) fp8_evict_choose_kernel(const Fp8EvictArgs a, int ctas) {
  extern __shared__ uint32_t held[];  // weights
  __shared__ alignas(16) int hist[2][kBins];  // of this CTA, in turn
  __shared__ int upper[kWarps], warp_counts[2][kWarps];
  __shared__ int2 counts;
  __shared__ uint32_t s_prefix;
  __shared__ int s_left;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / ctas, rank = blockIdx.x - b * ctas;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for the work ahead of this call
  const float* w = a.weights + b * a.weights_stride;
  const int64_t room = min(min(a.max_pages * a.page_size, a.row_len), static_cast<int64_t>(1) << 30);
  const bool first = rank == 0 && tid == 0;
  const int len = fp8_length(a.seq_lens[b], room, a.error_word, first);
  const int n = fp8_length(min(len, a.keep), a.new_max_pages * a.page_size, a.error_word, first);
  const int old = len - min(n, a.recent);  // tokens that may go (recent <= keep; a shorter new table keeps fewer)
  int left = n - (len - old);              // of them stay
  // this CTA's tokens, and its warps': consecutive ones, in 32s
  const int per = ((len + ctas - 1) / ctas + kChoose - 1) / kChoose * kChoose;
  const int t0 = min(rank * per, len), t1 = min(t0 + per, len), per_warp = per / kWarps;
  auto key_of = [&](int t) { return t - t0 < kHeld ? held[t - t0] : rank_key(w[t]); };
  for (int base = 0; base < min(t1 - t0, kHeld); base += 8 * kChoose) {  // (all loads of eight in flight)
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = base + j * kChoose + tid;
      v[j] = t0 + i < t1 && i < kHeld ? w[t0 + i] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = base + j * kChoose + tid;
      if (t0 + i < t1 && i < kHeld) held[i] = rank_key(v[j]);
    }
  }

  // the smallest key that stays, and how many of those equal to it
  uint32_t prefix = 0xFFFFFFFFu;  // (no weight's)
  if (left > 0) {
    prefix = 0;
#pragma unroll 1
    for (int round = 0; round < 3; ++round) {
      const int shift = round == 0 ? 21 : round == 1 ? 10 : 0, bins = round == 2 ? 1024 : kBins;
      const uint32_t mask = round == 0 ? 0u : round == 1 ? 0xFFE00000u : 0xFFFFFC00u;
      // thread i: bins 2 i and 2 i + 1
      int2* mine = reinterpret_cast<int2*>(hist[round & 1]) + tid;
      *mine = make_int2(0, 0);
      __syncthreads();
#pragma unroll 4
      for (int t = t0 + tid; t < min(t1, old); t += kChoose) {
        const uint32_t k = key_of(t);
        if ((k & mask) == prefix) atomicAdd(&hist[round & 1][k >> shift & (bins - 1)], 1);
      }
      int2 count;
      if (ctas > 1) {
        cluster_sync();
        int2 v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = c < ctas ? cluster_load2(mine, c) : make_int2(0, 0);
        count = make_int2(0, 0);
#pragma unroll
        for (int c = 0; c < 8; ++c) count.x += v[c].x, count.y += v[c].y;
      } else {
        __syncthreads();
        count = *mine;
      }
      // weights in larger bins: of the warp, and of the warps above
      int incl = count.x + count.y;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_down_sync(0xffffffffu, incl, o);
        if (lane + o < 32) incl += v;
      }
      if (lane == 0) upper[warp] = incl;
      __syncthreads();
      const int above = __reduce_add_sync(0xffffffffu, lane > warp ? upper[lane] : 0) + incl - count.x - count.y;
      const int more = above + count.y;  // for the lower of the two
      if (above < left && left <= more) {
        s_prefix = prefix | static_cast<uint32_t>(2 * tid + 1) << shift;
        s_left = left - above;
      } else if (more < left && left <= more + count.x) {
        s_prefix = prefix | static_cast<uint32_t>(2 * tid) << shift;
        s_left = left - more;
      }
      __syncthreads();
      prefix = s_prefix;
      left = s_left;
    }
  }

  // Places in order: what stays before this CTA, before this warp, and in it.
  const int w0 = min(t0 + warp * per_warp, t1), w1 = min(w0 + per_warp, t1);
  auto kind = [&](int t, bool& above, bool& tie) {  // of token t < w1
    const uint32_t k = t < min(w1, old) ? key_of(t) : 0;
    tie = t < min(w1, old) && k == prefix;
    above = t < w1 && (t >= old || k > prefix);
  };
  int n_above = 0, n_tie = 0;
#pragma unroll 4
  for (int t = w0; t < w1; t += 32) {
    bool above, tie;
    kind(t + lane, above, tie);
    n_above += __popc(__ballot_sync(0xffffffffu, above));
    n_tie += __popc(__ballot_sync(0xffffffffu, tie));
  }
  if (lane == 0) warp_counts[0][warp] = n_above, warp_counts[1][warp] = n_tie;
  __syncthreads();
  n_above = warp_counts[0][lane], n_tie = warp_counts[1][lane];
  int before_above = __reduce_add_sync(0xffffffffu, lane < warp ? n_above : 0);
  int before_tie = __reduce_add_sync(0xffffffffu, lane < warp ? n_tie : 0);
  if (ctas > 1) {
    n_above = __reduce_add_sync(0xffffffffu, n_above), n_tie = __reduce_add_sync(0xffffffffu, n_tie);
    if (tid == 0) counts = make_int2(n_above, n_tie);
    cluster_sync();
    const int2 other = lane < rank ? cluster_load2(&counts, lane) : make_int2(0, 0);
    before_above += __reduce_add_sync(0xffffffffu, other.x);
    before_tie += __reduce_add_sync(0xffffffffu, other.y);
    cluster_arrive();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the move's CTAs, which wait for this grid's end
  int32_t* kept = a.kept + static_cast<int64_t>(b) * a.keep;
  float* new_w = a.new_weights != nullptr ? a.new_weights + b * a.new_weights_stride : nullptr;
  for (int base = w0; base < w1; base += 128) {
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = new_w != nullptr && base + 32 * j + lane < w1 ? w[base + 32 * j + lane] : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = base + 32 * j + lane;
      bool above, tie;
      kind(t, above, tie);
      const uint32_t ties = __ballot_sync(0xffffffffu, tie), aboves = __ballot_sync(0xffffffffu, above), under = (1u << lane) - 1;
      const int ties_before = before_tie + __popc(ties & under);
      // (of the ties the first `left` stay)
      const int at = before_above + __popc(aboves & under) + min(left, ties_before);
      if ((above || (tie && ties_before < left)) && at < n) {
        kept[at] = t;
        if (new_w != nullptr) new_w[at] = v[j];
      }
      before_above += __popc(aboves);
      before_tie += __popc(ties);
    }
  }
  for (int64_t i = n + rank * kChoose + tid; i < a.keep; i += ctas * kChoose) kept[i] = -1;
  if (new_w != nullptr)
    for (int64_t i = n + rank * kChoose + tid; i < a.new_row_len; i += ctas * kChoose) new_w[i] = 0.f;
  if (first) a.new_lens[b] = n;
  if (ctas > 1) cluster_wait();  // (the others' shared memory is read until then)
}

// |codes| of two bytes; codes times a factor, rounded again.
__device__ __forceinline__ __half2 magnitudes(uint32_t two) {
  const uint32_t h2 = e4m3x2_to_f16x2_pair(two);
  return __habs2(*reinterpret_cast<const __half2*>(&h2));
}
__device__ __forceinline__ uint32_t scaled(uint32_t two, __half2 by) {
  const uint32_t h2 = e4m3x2_to_f16x2_pair(two);
  const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&h2), by);
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&p)));
  return r;
}

__global__ void __launch_bounds__(kMove, 4) fp8_evict_move_kernel(const Fp8EvictArgs a, int blocks) {
  const int b = blockIdx.x / blocks, i = blockIdx.x % blocks, tid = threadIdx.x;
  __shared__ int64_t from[kBlock];
  __shared__ float scale[kBlock], most[kMove / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for what was chosen
  // a chain of loads: token, page, its rows; the scales come with those
  const int at = i * kBlock + tid, t = tid < kBlock && at < a.keep ? a.kept[static_cast<int64_t>(b) * a.keep + at] : -1;
  int64_t slot = -1;
  if (t >= 0) {
    slot = fp8_block_slot(a.page_table + b * a.pt_stride, t / kBlock, a.page_size, a.num_slots);
    from[tid] = slot < 0 ? -1 : slot + t % kBlock;
  }
  const int rows = __syncthreads_count(t >= 0);
  if (rows == 0) return;
  uint4 v[kUnits];
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const int u = tid + j * kMove, r = u / (kKey / 16);
    v[j] = make_uint4(0, 0, 0, 0);
    if (r < rows && from[r] >= 0)
      v[j] = *reinterpret_cast<const uint4*>(a.cache + from[r] * kKey + u % (kKey / 16) * 16);
  }
  const int64_t to = fp8_block_slot(a.new_page_table + b * a.new_pt_stride, i, a.page_size, a.num_slots);
  if (t >= 0) {
    const float s = slot < 0 ? 0.f : a.scales[slot / kBlock];
    const bool good = s >= kFp8ScaleMin && s <= kFp8ScaleMax;
    if (!good) flag_error(a.error_word, slot < 0 ? MLA_DEVERR_BOUNDS : MLA_DEVERR_SCALE);
    scale[tid] = good ? s : 0.f;  // a key of zeros
  }
  __syncthreads();
  if (to < 0) {
    if (tid == 0) flag_error(a.error_word, MLA_DEVERR_BOUNDS);
    return;
  }
  float am = 0.f;
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const int r = (tid + j * kMove) / (kKey / 16);
    if (r < rows) {
      if (scale[r] == 0.f) v[j] = make_uint4(0, 0, 0, 0);
      const uint32_t q[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
      __half2 m = __float2half2_rn(0.f);  // (a NaN has no amax)
#pragma unroll
      for (int k = 0; k < 4; ++k) m = __hmax2(m, __hmax2(magnitudes(q[k]), magnitudes(q[k] >> 16)));
      am = fmaxf(am, fmaxf(__low2float(m), __high2float(m)) * scale[r]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
  if ((tid & 31) == 0) most[tid >> 5] = am;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kMove / 32; ++k) am = fmaxf(am, most[k]);
  const float s = fp8_block_scale(am), inv = 1.f / s;
  if (tid == 0) a.scales[to / kBlock] = s;
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const int u = tid + j * kMove, r = u / (kKey / 16);
    if (r >= rows) break;
    const float ratio = scale[r] * inv;
    if (ratio != 1.f && ratio != 0.f) {
      uint32_t* q = reinterpret_cast<uint32_t*>(&v[j]);
      if ((__float_as_uint(ratio) & 0x7FFFFFu) == 0 && ratio <= 32768.f) {
        // A power of two: products in f16, exact where e4m3 is not zero (codes have
        // 4 significant bits; below 2^-24 the factor is zero, and so are they).
        const __half2 by = __float2half2_rn(ratio);
#pragma unroll
        for (int k = 0; k < 4; ++k) q[k] = scaled(q[k], by) | scaled(q[k] >> 16, by) << 16;
      } else {
        // (a caller's own scale: the product is rounded to fp32 first)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t out = 0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t h2 = e4m3x2_to_f16x2_pair(q[k] >> (16 * h));
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
            out |= cvt_e4m3x2(f.x * ratio, f.y * ratio) << (16 * h);
          }
          q[k] = out;
        }
      }
    }
    *reinterpret_cast<uint4*>(a.cache + to * kKey + 16 * u) = v[j];
  }
}

}  // namespace

int launch_fp8_evict(const Fp8EvictArgs& a, cudaStream_t stream, int num_sms) {
  // new blocks a sequence, at most: of `keep` tokens, of those there can be, of the new pages
  const int64_t table = a.max_pages * a.page_size, row = a.row_len < table ? a.row_len : table;
  const int64_t room = a.new_max_pages * a.page_size < row ? a.new_max_pages * a.page_size : row;
  const int blocks = static_cast<int>(((a.keep < room ? a.keep : room) + kBlock - 1) / kBlock);
  if (static_cast<int64_t>(a.batch) * blocks > (int64_t(1) << 31) - 1) return MLA_ERR_INVALID_ARG;
  if (const int st = smem_limit_once(reinterpret_cast<const void*>(fp8_evict_choose_kernel), kChooseBytes, 36)) return st;
  // a cluster a sequence, as large as the SMs and its tokens allow (no more clusters than
  // run at once: 76 sequences of 1k to 32k cut to 1000 38.8 us, with four CTAs each 49.9;
  // 91 59.6 with one, 49.7 with two, but 91 of 1k to 8k 34.1 with one, 41.6 with two)
  int ctas = 1;
  while (ctas < 8 && a.batch * static_cast<int64_t>(ctas) * 2 <= num_sms && row > static_cast<int64_t>(ctas) * kPart) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.batch) * ctas);
  cfg.blockDim = dim3(kChoose);
  cfg.dynamicSmemBytes = kChooseBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // (griddepcontrol)
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  if (const int st = cuda_status(cudaLaunchKernelEx(&cfg, fp8_evict_choose_kernel, a, ctas))) return st;
  if (blocks == 0) return MLA_OK;  // (weights of no tokens)
  cfg.gridDim = dim3(static_cast<unsigned>(a.batch) * blocks);
  cfg.blockDim = dim3(kMove);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, fp8_evict_move_kernel, a, blocks));
}

}  // namespace mla
