// A query head of the e4m3 decode as two e4m3 terms in shared memory.
#pragma once
#include <cuda_runtime.h>

#include "nvfp4.cuh"
#include "sm100.cuh"

namespace mla {

constexpr float kGain = 16.f;  // queries' (and 32 heads' weights') second terms: at most 16 becomes 256
constexpr float kLog2e = 1.4426950408889634f;

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
// q = 2^e (q1 + q2 / 16), head h of kH, by a warp: lane l holds features 8 l..,
// and 256 + 8 l.., lanes 0..7 the RoPE's (512 + 8 l..).  Written at q0 as the
// product's operand: rows h (q1) and kH + h (q2) of four chunks of 128 features
// (128-byte swizzle), then of the RoPE (64-byte swizzle).  Returns log2(e)
// softmax_scale 2^e, or NaN for a head with an infinity or a NaN.
template <int kH>
__device__ __forceinline__ float query_terms(const uint4 (&v)[3], int lane, int h, uint32_t q0, float softmax_scale) {
  constexpr uint32_t kChunk = 2 * kH * 128;
  // amax from the bf16 bits (sign dropped, they order like integers)
  uint32_t m2 = 0;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) m2 = __vmaxu2(m2, w[j] & 0x7FFF7FFFu);
  }
  m2 = __reduce_max_sync(0xffffffffu, max(m2 & 0xFFFF0000u, m2 << 16));
  // 2^e, the smallest with amax <= 448 * 2^e (448 = 1.75 * 2^8); a
  // head with an infinity or a NaN has NaN scores
  int ex = static_cast<int>(m2 >> 23) - 127 - 8 + ((m2 & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  ex = max(-126, min(120, ex));
  const float inv = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
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
    const uint32_t w1[2] = {__byte_perm(a[0], a[1], 0x5410), __byte_perm(a[2], a[3], 0x5410)};
    const uint32_t w2[2] = {__byte_perm(r[0], r[1], 0x5410), __byte_perm(r[2], r[3], 0x5410)};
    // row h (q1) and kH + h (q2) of the chunk; 16-byte units swizzled by the row
    uint32_t a1, a2;
    if (k < 2) {
      const int feature = 256 * k + 8 * lane;
      const uint32_t base = q0 + (feature >> 7) * kChunk;
      const uint32_t unit = (feature & 127) >> 4, half = feature & 8;
      a1 = base + h * 128 + ((unit ^ (h & 7)) << 4) + half;
      a2 = a1 + kH * 128;
    } else {
      const uint32_t base = q0 + 4 * kChunk;
      const uint32_t unit = lane >> 1, half = (lane & 1) * 8;
      a1 = base + h * 64 + ((unit ^ ((h >> 1) & 3)) << 4) + half;
      a2 = a1 + kH * 64;
    }
    if (k < 2 || lane < 8) {
      asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(a1), "r"(w1[0]), "r"(w1[1]) : "memory");
      asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(a2), "r"(w2[0]), "r"(w2[1]) : "memory");
    }
  }
  return m2 >= 0x7F800000u ? __uint_as_float(0x7FC00000u)
                           : softmax_scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
}

}  // namespace mla
