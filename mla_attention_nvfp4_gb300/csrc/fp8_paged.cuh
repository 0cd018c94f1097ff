// The e4m3 latent cache as its kernels find a sequence's keys in it.
#pragma once
#include <cuda_runtime.h>

#include "launch.h"
#include "nvfp4.cuh"

namespace mla {

constexpr int kFp8Key = MLA_D_LATENT + MLA_D_ROPE;
constexpr float kFp8ScaleMin = 8.673617379884035e-19f, kFp8ScaleMax = 1.152921504606847e18f;  // 2^-60, 2^60

// A block's scale: the smallest 2^e, -60 <= e <= 60, with amax <= 448 * 2^e (448 = 1.75 * 2^8):
// from amax's exponent and whether its fraction is above .75.
__device__ __forceinline__ float fp8_block_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < -60 ? -60 : e > 60 ? 60 : e;  // amax 0 and subnormal: -60; inf: 60
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// A sequence's length, at most what its page table and the caller's other
// rows hold (flagged where it is more).
__device__ __forceinline__ int fp8_length(int len, int64_t room, uint32_t* error_word, bool flag) {
  if (len <= 0) return 0;
  if (len <= room) return len;
  if (flag) flag_error(error_word, MLA_DEVERR_BOUNDS);
  return static_cast<int>(room);
}

// First slot of block i (64 tokens) of a sequence, or -1 where its page is
// out of the cache.
__device__ __forceinline__ int64_t fp8_block_slot(const int32_t* table, int64_t i, int page_size, int64_t num_slots) {
  const int64_t per = page_size / MLA_FP8_BLOCK, page = table[i / per];
  const int64_t slot = page * page_size + i % per * MLA_FP8_BLOCK;
  return page < 0 || slot + MLA_FP8_BLOCK > num_slots ? -1 : slot;
}

}  // namespace mla
