// Query heads of the e4m3 decode as two e4m3 terms in shared memory.
#pragma once
#include <cuda_runtime.h>

#include "launch.h"
#include "nvfp4.cuh"
#include "sm100.cuh"

namespace mla {

constexpr float kGain = 16.f;  // queries' (and 32 heads' weights') second terms: at most 16 becomes 256
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kQueryFeatures = MLA_D_LATENT + MLA_D_ROPE;

__device__ __forceinline__ uint32_t cvt_e4m3x2_h2(uint32_t h2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
  return r;
}
__device__ __forceinline__ uint32_t h2_sub(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t h2_fma(uint32_t a, float s, uint32_t b) {
  const __half2 r =
      __hfma2(*reinterpret_cast<const __half2*>(&a), __float2half2_rn(s), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// kN heads first, first + step, .. of kH, by a warp: lane l holds features 8 l..
// and 256 + 8 l.. of each, and of one head's RoPE's (lanes 8 j.. the j-th's) 512 + 8
// (l % 8)...
template <int kN>
struct QueryHeads {
  uint4 v[kN][2], rope;

  // of q's rows (576 features a head), those below `heads`; the others are zeros
  __device__ __forceinline__ void load(const __nv_bfloat16* q, int lane, int first, int step, int heads) {
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int h = first + j * step;
      v[j][0] = v[j][1] = make_uint4(0, 0, 0, 0);
      if (h < heads) {
        const uint4* src = reinterpret_cast<const uint4*>(q) + static_cast<int64_t>(h) * (kQueryFeatures / 8);
        v[j][0] = src[lane];
        v[j][1] = src[lane + 32];
      }
    }
    const int h = first + (lane >> 3) * step;
    rope = make_uint4(0, 0, 0, 0);
    if (lane < 8 * kN && h < heads)
      rope = reinterpret_cast<const uint4*>(q)[static_cast<int64_t>(h) * (kQueryFeatures / 8) + 64 + (lane & 7)];
  }
};

// 8 features times inv as two terms, 8 bytes each.
__device__ __forceinline__ void query_split(const uint4& v, float inv, uint32_t at1, uint32_t at2) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  // in f16 pairs: 8 significant bits down to 2^-17, then steps of 2^-24
  uint32_t a[4], r[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float x0, x1;
    bf16x2_to_f32(w[j], x0, x1);
    const __half2 xh = __floats2half2_rn(x0 * inv, x1 * inv);
    const uint32_t xu = *reinterpret_cast<const uint32_t*>(&xh);
    a[j] = cvt_e4m3x2_h2(xu);
    r[j] = cvt_e4m3x2_h2(h2_fma(h2_sub(xu, e4m3x2_to_f16x2_pair(a[j])), kGain, 0));
  }
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at1), "r"(__byte_perm(a[0], a[1], 0x5410)),
               "r"(__byte_perm(a[2], a[3], 0x5410))
               : "memory");
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at2), "r"(__byte_perm(r[0], r[1], 0x5410)),
               "r"(__byte_perm(r[2], r[3], 0x5410))
               : "memory");
}

// q = 2^e (q1 + q2 / 16) of those heads, written at q0 as the product's operand:
// rows h (q1) and kH + h (q2) of four chunks of 128 features (128-byte swizzle),
// then of the RoPE (64-byte swizzle).  c[j]: log2(e) softmax_scale 2^e, or NaN for a
// head with an infinity or a NaN.
template <int kH, int kN>
__device__ __forceinline__ void query_terms(const QueryHeads<kN>& q, int lane, int first, int step, uint32_t q0,
                                            float softmax_scale, float (&c)[kN]) {
  constexpr uint32_t kChunk = 2 * kH * 128;
  auto words_max = [](const uint4& v) {  // of bf16 bits (sign dropped, they order like integers)
    return __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
  };
  const uint32_t rope_max = words_max(q.rope);
  float inv_rope = 0.f;
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    const int h = first + j * step;
    uint32_t m2 = __vmaxu2(words_max(q.v[j][0]), words_max(q.v[j][1]));
    if (lane >> 3 == j) m2 = __vmaxu2(m2, rope_max);
    m2 = __reduce_max_sync(0xffffffffu, max(m2 & 0xFFFF0000u, m2 << 16));
    // 2^e, the smallest with amax <= 448 * 2^e (448 = 1.75 * 2^8); a
    // head with an infinity or a NaN has NaN scores
    int ex = static_cast<int>(m2 >> 23) - 127 - 8 + ((m2 & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    ex = max(-126, min(120, ex));
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
    if (lane >> 3 == j) inv_rope = inv;
    c[j] = m2 >= 0x7F800000u ? __uint_as_float(0x7FC00000u)
                             : softmax_scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
    // row h (q1) and kH + h (q2) of a chunk; 16-byte units swizzled by the row
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int feature = 256 * k + 8 * lane;
      const uint32_t at = q0 + (feature >> 7) * kChunk + h * 128 + ((((feature & 127) >> 4) ^ (h & 7)) << 4) + (feature & 8);
      query_split(q.v[j][k], inv, at, at + kH * 128);
    }
  }
  if (lane < 8 * kN) {
    const int h = first + (lane >> 3) * step;
    const uint32_t at = q0 + 4 * kChunk + h * 64 + (((lane & 7) >> 1 ^ (h >> 1 & 3)) << 4) + (lane & 1) * 8;
    query_split(q.rope, inv_rope, at, at + kH * 64);
  }
}

}  // namespace mla
