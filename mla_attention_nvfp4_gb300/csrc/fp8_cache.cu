// Append to the e4m3 latent cache: new tokens' latent and rotated RoPE key,
// one power-of-two scale per block of 64 tokens, and the rotation of the new
// queries' RoPE part by the same angles.  No tensor cores: 16-byte loads, one
// pass over the new rows, which wait in registers while their block's amax
// is found.
#include <cuda_runtime.h>

#include "launch.h"
#include "nvfp4.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBlock = MLA_FP8_BLOCK, kRows = kBlock / kWarps;  // rows of a block per warp
constexpr int kKey = MLA_D_LATENT + MLA_D_ROPE;
constexpr int kQPairs = 4 * kThreads / 8;  // (token, head) rows of 64 per query CTA
constexpr float kScaleMin = 8.673617379884035e-19f, kScaleMax = 1.152921504606847e18f;  // 2^-60, 2^60

// The smallest 2^e, -60 <= e <= 60, with amax <= 448 * 2^e (448 = 1.75 * 2^8):
// from amax's exponent and whether its fraction is above .75.
__device__ __forceinline__ float block_scale_pow2(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < -60 ? -60 : e > 60 ? 60 : e;  // amax 0 and subnormal: -60; inf: 60
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

__device__ __forceinline__ uint32_t bf16x2_pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// One pair turned by an angle: products and sums each rounded to float32, as
// the plain formula evaluates (no contraction), so that the rounding of the
// result to 8 or 16 bits sees the same value.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = a, y = b;
  a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  b = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
}

// Sequence b's new tokens: rows a.. of the batch, positions ctx .. ctx + n.
// False when its entries are out of range (flagged) or it has none.
struct Span {
  int64_t row, ctx, end;  // first row; first position; one past the last
};
__device__ __forceinline__ bool sequence_span(const Fp8AppendArgs& p, int b, Span& s, bool flag) {
  const int64_t a = p.cu_seqlens[b], e = p.cu_seqlens[b + 1], ctx = p.context_lens[b];
  uint32_t bits = 0;
  int64_t n = e - a;
  bool ok = true;
  if (a < 0 || e > p.num_tokens || n < 0 || ctx < 0) {
    bits = MLA_DEVERR_BOUNDS;
    ok = false;
  } else {
    if (n > p.max_new) {
      bits = MLA_DEVERR_BOUNDS;
      n = p.max_new;
    }
    int64_t end = ctx + n;
    const int64_t room = p.max_pages * p.page_size;
    const int64_t most = room < p.max_position ? room : p.max_position;
    if (end > most) {
      bits = MLA_DEVERR_BOUNDS;
      end = most;
    }
    s = Span{a, ctx, end};
    ok = end > ctx;
  }
  if (bits != 0 && flag) flag_error(p.error_word, bits);
  return ok;
}

// The work of sequence b is cut into key parts (one block of 64 tokens each)
// and query parts (kQPairs rows of 64 each); a grid of num_seqs * (n_kv + n_q)
// CTAs covers the longest sequence, and CTAs past a sequence's end return.
template <bool kInterleaved>
__global__ void __launch_bounds__(kThreads) fp8_append_kernel(const Fp8AppendArgs p, int n_kv, int n_q) {
  const int per = n_kv + n_q;
  const int b = blockIdx.x / per, part = blockIdx.x % per;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Span sp;
  if (!sequence_span(p, b, sp, part == 0 && tid == 0)) return;

  if (part >= n_kv) {
    // ------------------------------------------------------------- queries
    // (token, head) rows; 8 threads a row.  Interleaved: thread c holds
    // features [8c, 8c + 8), four pairs; otherwise threads 0..3 hold
    // features [8c, 8c + 8) and their partners 32 further on.
    const int64_t total = (sp.end - sp.ctx) * p.num_heads;
    const int64_t first = static_cast<int64_t>(part - n_kv) * kQPairs;
    constexpr int kPer = kInterleaved ? 8 : 4;  // threads a row
    constexpr int kIter = kQPairs * kPer / kThreads;
    const int c = tid % kPer;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q_pe);
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.q_out);
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int64_t pair = first + i * (kThreads / kPer) + tid / kPer;
      if (pair >= total) break;
      const int64_t t = pair / p.num_heads;
      const int h = static_cast<int>(pair - t * p.num_heads);
      const float* cs = p.cos_sin + (sp.ctx + t) * 64;
      const __nv_bfloat16* src = q + (sp.row + t) * p.q_st + h * p.q_sh + 8 * c;
      __nv_bfloat16* dst = o + (sp.row + t) * p.qo_st + h * p.qo_sh + 8 * c;
      if constexpr (kInterleaved) {
        uint4 v = *reinterpret_cast<const uint4*>(src);
        const float4 cc = *reinterpret_cast<const float4*>(cs + 4 * c);
        const float4 ss = *reinterpret_cast<const float4*>(cs + 32 + 4 * c);
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
        const float cw[4] = {cc.x, cc.y, cc.z, cc.w}, sw[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float x, y;
          bf16x2_to_f32(w[k], x, y);
          turn(x, y, cw[k], sw[k]);
          w[k] = bf16x2_pack(x, y);
        }
        *reinterpret_cast<uint4*>(dst) = v;
      } else {
        uint4 v = *reinterpret_cast<const uint4*>(src), u = *reinterpret_cast<const uint4*>(src + 32);
        uint32_t *vw = reinterpret_cast<uint32_t*>(&v), *uw = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 cc = *reinterpret_cast<const float2*>(cs + 8 * c + 2 * k);
          const float2 ss = *reinterpret_cast<const float2*>(cs + 32 + 8 * c + 2 * k);
          float x0, x1, y0, y1;
          bf16x2_to_f32(vw[k], x0, x1);
          bf16x2_to_f32(uw[k], y0, y1);
          turn(x0, y0, cc.x, ss.x);
          turn(x1, y1, cc.y, ss.y);
          vw[k] = bf16x2_pack(x0, x1);
          uw[k] = bf16x2_pack(y0, y1);
        }
        *reinterpret_cast<uint4*>(dst) = v;
        *reinterpret_cast<uint4*>(dst + 32) = u;
      }
    }
    return;
  }

  // ------------------------------------------------------------------ keys
  const int64_t pos0 = (sp.ctx / kBlock + part) * kBlock;  // position of the block's first token
  if (pos0 >= sp.end) return;
  const int lo = sp.ctx > pos0 ? static_cast<int>(sp.ctx - pos0) : 0;  // the block's rows written here
  const int hi = sp.end < pos0 + kBlock ? static_cast<int>(sp.end - pos0) : kBlock;
  const int64_t page = p.page_table[b * p.pt_stride + pos0 / p.page_size];
  const int64_t slot0 = page * p.page_size + pos0 % p.page_size;
  if (page < 0 || slot0 + kBlock > p.num_slots) {
    if (tid == 0) flag_error(p.error_word, MLA_DEVERR_BOUNDS);
    return;
  }
  float* scale_ptr = p.scales + slot0 / kBlock;
  const float was = lo > 0 ? *scale_ptr : 0.f;

  // This warp's rows, all loads first: lane l holds latent features
  // [16 l, 16 l + 16) and pair l of the RoPE key.
  uint4 va[kRows], vb[kRows];
  float r0[kRows], r1[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = warp + i * kWarps;
    va[i] = vb[i] = make_uint4(0, 0, 0, 0);
    r0[i] = r1[i] = 0.f;
    if (r >= lo && r < hi) {
      const int64_t row = sp.row + (pos0 + r - sp.ctx);
      const uint4* src =
          reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.kv_c) + row * p.kv_stride + 16 * lane);
      va[i] = src[0];
      vb[i] = src[1];
      const __nv_bfloat16* pe = static_cast<const __nv_bfloat16*>(p.k_pe) + row * p.pe_stride;
      if constexpr (kInterleaved) {
        bf16x2_to_f32(*reinterpret_cast<const uint32_t*>(pe + 2 * lane), r0[i], r1[i]);
      } else {
        r0[i] = __bfloat162float(pe[lane]);
        r1[i] = __bfloat162float(pe[lane + 32]);
      }
      const float* cs = p.cos_sin + (pos0 + r) * 64;
      turn(r0[i], r1[i], cs[lane], cs[lane + 32]);
    }
  }
  float am = 0.f;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const uint32_t w[8] = {va[i].x, va[i].y, va[i].z, va[i].w, vb[i].x, vb[i].y, vb[i].z, vb[i].w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float x, y;
      bf16x2_to_f32(w[k], x, y);
      am = fmaxf(am, fmaxf(fabsf(x), fabsf(y)));
    }
    am = fmaxf(am, fmaxf(fabsf(r0[i]), fabsf(r1[i])));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
  __shared__ float red[kWarps];
  if (lane == 0) red[warp] = am;
  __syncthreads();  // also: every thread has read the earlier scale
#pragma unroll
  for (int i = 0; i < kWarps; ++i) am = fmaxf(am, red[i]);

  const float need = block_scale_pow2(am);
  const bool keep = lo > 0 && was >= kScaleMin && was <= kScaleMax;
  if (lo > 0 && !keep && tid == 0) flag_error(p.error_word, MLA_DEVERR_SCALE);
  const float scale = keep ? fmaxf(was, need) : need;
  uint8_t* rec0 = p.cache + slot0 * kKey;
  if (keep && scale != was) {
    // the block's scale grows: its earlier tokens' codes in the new scale
    const float ratio = was / scale;
    for (int i = tid; i < lo * (kKey / 16); i += kThreads) {
      uint4* ptr = reinterpret_cast<uint4*>(rec0) + i;
      uint4 v = *ptr;
      uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t out = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t h2 = e4m3x2_to_f16x2_pair(w[k] >> (16 * j));
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
          out |= cvt_e4m3x2(f.x * ratio, f.y * ratio) << (16 * j);
        }
        w[k] = out;
      }
      *ptr = v;
    }
  }
  if (tid == 0) *scale_ptr = scale;
  const float inv = 1.f / scale;  // exact: a power of two (or the caller's larger scale, rounded)
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = warp + i * kWarps;
    if (r < lo || r >= hi) continue;
    const uint32_t w[8] = {va[i].x, va[i].y, va[i].z, va[i].w, vb[i].x, vb[i].y, vb[i].z, vb[i].w};
    uint32_t out[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float a, c, d, e;
      bf16x2_to_f32(w[2 * k], a, c);
      bf16x2_to_f32(w[2 * k + 1], d, e);
      out[k] = cvt_e4m3x2(a * inv, c * inv) | (cvt_e4m3x2(d * inv, e * inv) << 16);
    }
    uint8_t* rec = rec0 + static_cast<int64_t>(r) * kKey;
    *reinterpret_cast<uint4*>(rec + 16 * lane) = make_uint4(out[0], out[1], out[2], out[3]);
    const uint32_t rope = cvt_e4m3x2(r0[i] * inv, r1[i] * inv);
    if constexpr (kInterleaved) {
      *reinterpret_cast<uint16_t*>(rec + MLA_D_LATENT + 2 * lane) = static_cast<uint16_t>(rope);
    } else {
      rec[MLA_D_LATENT + lane] = static_cast<uint8_t>(rope);
      rec[MLA_D_LATENT + 32 + lane] = static_cast<uint8_t>(rope >> 8);
    }
  }
}

}  // namespace

int launch_fp8_append(const Fp8AppendArgs& a, cudaStream_t stream) {
  // n consecutive tokens touch at most (n + 62) / 64 + 1 blocks
  const int64_t n = a.max_new < a.num_tokens ? a.max_new : a.num_tokens;
  const int64_t n_kv = (n + kBlock - 2) / kBlock + 1;
  const int64_t n_q = (n * a.num_heads + kQPairs - 1) / kQPairs;
  const int64_t grid = a.num_seqs * (n_kv + n_q);
  if (grid > (int64_t(1) << 31) - 1) return MLA_ERR_INVALID_ARG;
  Fp8AppendArgs p = a;
  p.max_new = static_cast<int>(n);
  if (a.interleaved)
    fp8_append_kernel<true><<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(p, static_cast<int>(n_kv),
                                                                                  static_cast<int>(n_q));
  else
    fp8_append_kernel<false><<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(p, static_cast<int>(n_kv),
                                                                                   static_cast<int>(n_q));
  return launch_status();
}

}  // namespace mla
