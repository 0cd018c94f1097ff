// e4m3 GEMM with scales per block of 128, and the activations' quantiser.
#include <cuda_runtime.h>

#include "launch.h"
#include "nvfp4.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kGroup = MLA_FP8_GROUP;

// ---------------------------------------------------------------------------
// Quantiser: bf16 [M, K] -> e4m3 codes and one fp32 scale per 128 features.
// 16 lanes hold a group, 8 features each (one 16-byte load, one 8-byte
// store); four groups in flight per half-warp.
// ---------------------------------------------------------------------------
constexpr int kQuantThreads = 256;
constexpr int kQuantUnroll = 4;
constexpr int kQuantGroups = kQuantThreads / 16 * kQuantUnroll;  // groups per CTA

__global__ void __launch_bounds__(kQuantThreads) fp8_quantize_kernel(const __nv_bfloat16* __restrict__ x,
                                                                     int64_t x_stride, int64_t K, int n_groups,
                                                                     int row_groups, uint32_t magic, int shift,
                                                                     uint8_t* __restrict__ codes,
                                                                     float* __restrict__ scales) {
  const int sub = threadIdx.x & 15;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kQuantGroups + (threadIdx.x >> 4);
  uint4 v[kQuantUnroll];
  int64_t at[kQuantUnroll];  // offset of this thread's codes, or -1
#pragma unroll
  for (int i = 0; i < kQuantUnroll; ++i) {
    const int64_t g = first + i * (kQuantThreads / 16);
    v[i] = make_uint4(0, 0, 0, 0);
    at[i] = -1;
    if (g < n_groups) {
      const int64_t m = div_magic(static_cast<uint32_t>(g), magic, shift), j = g - m * row_groups;
      const int64_t k = j * kGroup + 8 * sub;
      if (k < K) {
        v[i] = *reinterpret_cast<const uint4*>(x + m * x_stride + k);
        at[i] = m * K + k;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kQuantUnroll; ++i) {
    const int64_t g = first + i * (kQuantThreads / 16);
    float f[8];
    bf16x2_to_f32(v[i].x, f[0], f[1]);
    bf16x2_to_f32(v[i].y, f[2], f[3]);
    bf16x2_to_f32(v[i].z, f[4], f[5]);
    bf16x2_to_f32(v[i].w, f[6], f[7]);
    float am = amax8(f);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
    // both quotients rounded to nearest: the scale by a division, the codes
    // by the correctly rounded reciprocal (div_rn)
    const float scale = fmaxf(__fdiv_rn(am, 448.f), 1.1754943508222875e-38f);
    const float inv = __frcp_rn(scale);
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float q[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        q[e] = isinf(scale) ? __fmul_rn(f[4 * k + e], inv) : div_rn(f[4 * k + e], scale, inv);
      w[k] = cvt_e4m3x2(q[0], q[1]) | (cvt_e4m3x2(q[2], q[3]) << 16);
    }
    if (at[i] >= 0) *reinterpret_cast<uint2*>(codes + at[i]) = make_uint2(w[0], w[1]);
    if (sub == 0 && g < n_groups) scales[g] = scale;
  }
}

// ---------------------------------------------------------------------------
// GEMM: 64 x 64 outputs per CTA, 4 x 4 per thread, fp32 on CUDA cores.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) fp8_gemm_kernel(const Fp8GemmArgs p) {
  __shared__ float sa[64][33], sw[64][33];
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * 64, n0 = static_cast<int64_t>(blockIdx.x) * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t kb_n = (p.K + kGroup - 1) / kGroup;
  float acc[4][4] = {};
  for (int64_t kb = 0; kb < kb_n; ++kb) {
    float part[4][4] = {};
    for (int64_t k0 = kb * kGroup; k0 < p.K && k0 < (kb + 1) * kGroup; k0 += 32) {
      __syncthreads();
      for (int i = threadIdx.x; i < 64 * 32; i += 256) {
        const int r = i >> 5, k = i & 31;
        sa[r][k] = (m0 + r < p.M && k0 + k < p.K) ? e4m3_to_f32(p.a[(m0 + r) * p.lda + k0 + k]) : 0.f;
        sw[r][k] = (n0 + r < p.N && k0 + k < p.K) ? e4m3_to_f32(p.w[(n0 + r) * p.ldw + k0 + k]) : 0.f;
      }
      __syncthreads();
      for (int k = 0; k < 32; ++k)
        for (int i = 0; i < 4; ++i)
          for (int j = 0; j < 4; ++j) part[i][j] = fmaf(sa[ty * 4 + i][k], sw[tx * 4 + j][k], part[i][j]);
    }
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
        if (m < p.M && n < p.N)
          acc[i][j] = fmaf(p.a_scales[m * kb_n + kb] * p.w_scales[n / kGroup * kb_n + kb], part[i][j], acc[i][j]);
      }
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m < p.M && n < p.N) static_cast<__nv_bfloat16*>(p.out)[m * p.ldc + n] = __float2bfloat16_rn(acc[i][j]);
    }
}

}  // namespace

int launch_fp8_quantize(const void* x, int64_t x_stride, int64_t M, int64_t K, uint8_t* codes, float* scales,
                        cudaStream_t stream, int num_sms) {
  (void)num_sms;
  const int row_groups = static_cast<int>((K + kGroup - 1) / kGroup);
  const int64_t groups = M * row_groups;  // < 2^31 (checked by the caller)
  uint32_t magic;
  int shift;
  magic_divisor(row_groups, &magic, &shift);
  const unsigned grid = static_cast<unsigned>((groups + kQuantGroups - 1) / kQuantGroups);
  fp8_quantize_kernel<<<grid, kQuantThreads, 0, stream>>>(static_cast<const __nv_bfloat16*>(x), x_stride, K,
                                                          static_cast<int>(groups), row_groups, magic, shift, codes,
                                                          scales);
  return launch_status();
}

int launch_fp8_gemm(const Fp8GemmArgs& a, cudaStream_t stream, int num_sms) {
  (void)num_sms;
  const dim3 grid(static_cast<unsigned>((a.N + 63) / 64), static_cast<unsigned>((a.M + 63) / 64));
  fp8_gemm_kernel<<<grid, 256, 0, stream>>>(a);
  return launch_status();
}

}  // namespace mla
