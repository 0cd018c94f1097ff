// Append to the e4m3 latent cache: new tokens' latent and rotated RoPE key,
// one power-of-two scale per block of 64 tokens, and the rotation of the new
// queries' RoPE part by the same angles.  No tensor cores; HBM-bound.  A
// block's new rows wait in shared memory (bulk copies, a row each) while
// their amax is found, so that few registers and many bytes are in flight.
// 8 x 4096 tokens with 16 query heads: 26.5 us, 4.9 TB/s (59 us with the rows in
// registers); 64 sequences of one token, 128 heads: 3.3 us, a launch and one
// chain of loads (lengths, page, scale and codes, store).
#include <cuda_runtime.h>

#include "fp8.cuh"
#include "fp8_paged.cuh"
#include "launch.h"
#include "nvfp4.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBlock = MLA_FP8_BLOCK, kRows = kBlock / kWarps;  // rows of a block per warp
constexpr int kKey = MLA_D_LATENT + MLA_D_ROPE;
constexpr int kQPairs = kThreads;  // (token, head) rows of 64 per query CTA
constexpr int kPeBytes = MLA_D_ROPE * 2, kKvBytes = MLA_D_LATENT * 2;
constexpr int kSmemBytes = kBlock * (kKvBytes + kPeBytes);  // 72 KB: three CTAs an SM
constexpr float kScaleMin = kFp8ScaleMin, kScaleMax = kFp8ScaleMax;

// One pair turned by an angle: products and sums each rounded to float32, as
// the plain formula evaluates (no contraction), so that the rounding of the
// result to 8 or 16 bits sees the same value.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = a, y = b;
  a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  b = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
}

// Sequence b's new tokens: rows a.. of the batch, its tokens ctx .. ctx + n,
// whose angles are those of rows `ahead` further on.  False when its entries
// are out of range (flagged) or it has none.
struct Span {
  int64_t row, ctx, end, ahead;  // first row; first token; one past the last; position less token
};
__device__ __forceinline__ bool sequence_span(const Fp8AppendArgs& p, int b, Span& s, bool flag) {
  const int64_t a = p.cu_seqlens[b], e = p.cu_seqlens[b + 1], ctx = p.context_lens[b];
  const int64_t position = p.positions != nullptr ? p.positions[b] : ctx;
  uint32_t bits = 0;
  int64_t n = e - a;
  bool ok = true;
  if (a < 0 || e > p.num_tokens || n < 0 || ctx < 0 || position < 0) {
    bits = MLA_DEVERR_BOUNDS;
    ok = false;
  } else {
    if (n > p.max_new) {
      bits = MLA_DEVERR_BOUNDS;
      n = p.max_new;
    }
    int64_t end = ctx + n;
    const int64_t room = p.max_pages * p.page_size, angles = p.max_position - (position - ctx);
    const int64_t most = room < angles ? room : angles;
    if (end > most) {
      bits = MLA_DEVERR_BOUNDS;
      end = most;
    }
    s = Span{a, ctx, end, position - ctx};
    ok = end > ctx;
  }
  if (bits != 0 && flag) flag_error(p.error_word, bits);
  return ok;
}

// The work of sequence b is cut into key parts (one block of 64 tokens each)
// and query parts (kQPairs rows of 64 each); a grid of num_seqs * (n_kv + n_q)
// CTAs covers the longest sequence, and CTAs past a sequence's end return.
template <bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 3) fp8_append_kernel(const Fp8AppendArgs p, int n_kv, int n_q) {
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
    // all loads first (q_out may be q_pe: every thread writes what it read)
    constexpr int kVec = kInterleaved ? 1 : 2;  // 16-byte units a row and thread
    uint4 v[kIter][kVec];
    int row_of[kIter];  // token of the sequence, or -1
    int head_of[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int64_t pair = first + i * (kThreads / kPer) + tid / kPer;
      row_of[i] = -1;
      head_of[i] = 0;
      if (pair < total) {
        row_of[i] = static_cast<int>(pair / p.num_heads);
        head_of[i] = static_cast<int>(pair - static_cast<int64_t>(row_of[i]) * p.num_heads);
        const __nv_bfloat16* src = q + (sp.row + row_of[i]) * p.q_st + head_of[i] * p.q_sh + 8 * c;
        v[i][0] = *reinterpret_cast<const uint4*>(src);
        if constexpr (!kInterleaved) v[i][1] = *reinterpret_cast<const uint4*>(src + 32);
      }
    }
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      if (row_of[i] < 0) break;
      const float* cs = p.cos_sin + (sp.ctx + sp.ahead + row_of[i]) * 64;
      __nv_bfloat16* dst = o + (sp.row + row_of[i]) * p.qo_st + head_of[i] * p.qo_sh + 8 * c;
      uint32_t* w = reinterpret_cast<uint32_t*>(&v[i][0]);
      if constexpr (kInterleaved) {
        const float4 cc = *reinterpret_cast<const float4*>(cs + 4 * c);
        const float4 ss = *reinterpret_cast<const float4*>(cs + 32 + 4 * c);
        const float cw[4] = {cc.x, cc.y, cc.z, cc.w}, sw[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float x, y;
          bf16x2_to_f32(w[k], x, y);
          turn(x, y, cw[k], sw[k]);
          w[k] = bf16x2_pack(x, y);
        }
        *reinterpret_cast<uint4*>(dst) = v[i][0];
      } else {
        uint32_t* u = reinterpret_cast<uint32_t*>(&v[i][kVec - 1]);
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          const float4 cc = *reinterpret_cast<const float4*>(cs + 8 * c + 2 * k);
          const float4 ss = *reinterpret_cast<const float4*>(cs + 32 + 8 * c + 2 * k);
          const float cw[4] = {cc.x, cc.y, cc.z, cc.w}, sw[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float x0, x1, y0, y1;
            bf16x2_to_f32(w[k + j], x0, x1);
            bf16x2_to_f32(u[k + j], y0, y1);
            turn(x0, y0, cw[2 * j], sw[2 * j]);
            turn(x1, y1, cw[2 * j + 1], sw[2 * j + 1]);
            w[k + j] = bf16x2_pack(x0, x1);
            u[k + j] = bf16x2_pack(y0, y1);
          }
        }
        *reinterpret_cast<uint4*>(dst) = v[i][0];
        *reinterpret_cast<uint4*>(dst + 32) = v[i][kVec - 1];
      }
    }
    return;
  }

  // ------------------------------------------------------------------ keys
  const int64_t pos0 = (sp.ctx / kBlock + part) * kBlock;  // the block's first token
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

  extern __shared__ __align__(128) uint8_t smem[];  // latent rows, then RoPE rows
  __shared__ uint64_t bar;
  if (tid == 0) {
    mbar_init(&bar, 1);
    fence_mbar_init();
    mbar_expect_tx(&bar, (hi - lo) * (kKvBytes + kPeBytes));
  }
  __syncthreads();
  if (tid >= lo && tid < hi) {
    const int64_t row = sp.row + (pos0 + tid - sp.ctx);
    bulk_load(smem_u32(smem) + tid * kKvBytes, static_cast<const __nv_bfloat16*>(p.kv_c) + row * p.kv_stride, kKvBytes,
              &bar);
    bulk_load(smem_u32(smem) + kBlock * kKvBytes + tid * kPeBytes,
              static_cast<const __nv_bfloat16*>(p.k_pe) + row * p.pe_stride, kPeBytes, &bar);
  }
  // Rows warp, warp + 8, ..: lane l holds latent features [8 l, 8 l + 8) and
  // [256 + 8 l, ..), and pair l of the RoPE key, whose angles come meanwhile.
  float cosine[kRows], sine[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = warp + i * kWarps;
    cosine[i] = sine[i] = 0.f;
    if (r >= lo && r < hi) {
      const float* cs = p.cos_sin + (pos0 + sp.ahead + r) * 64;
      cosine[i] = cs[lane];
      sine[i] = cs[lane + 32];
    }
  }
  if (!mbar_wait_cta(&bar, 0, p.error_word)) {
    if (tid == 0) drain_copies(&bar, 1, 1);
    return;  // nothing is written
  }
  auto latent = [&](int r, int half) { return *reinterpret_cast<const uint4*>(smem + r * kKvBytes + 512 * half + 16 * lane); };
  auto rope = [&](int r, int i, float& a, float& b) {  // the rotated pair
    const uint8_t* pe = smem + kBlock * kKvBytes + r * kPeBytes;
    if constexpr (kInterleaved) {
      bf16x2_to_f32(reinterpret_cast<const uint32_t*>(pe)[lane], a, b);
    } else {
      a = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(pe)[lane]);
      b = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(pe)[lane + 32]);
    }
    turn(a, b, cosine[i], sine[i]);
  };
  float am = 0.f;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = warp + i * kWarps;
    if (r < lo || r >= hi) continue;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint4 v = latent(r, half);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float x, y;
        bf16x2_to_f32(w[k], x, y);
        am = fmaxf(am, fmaxf(fabsf(x), fabsf(y)));
      }
    }
    float x, y;
    rope(r, i, x, y);
    am = fmaxf(am, fmaxf(fabsf(x), fabsf(y)));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
  __shared__ float red[kWarps];
  if (lane == 0) red[warp] = am;
  __syncthreads();  // also: every thread has read the earlier scale
#pragma unroll
  for (int i = 0; i < kWarps; ++i) am = fmaxf(am, red[i]);

  const float need = fp8_block_scale(am);
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
    uint8_t* rec = rec0 + static_cast<int64_t>(r) * kKey;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint4 v = latent(r, half);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t out[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float a, b2, c, d;
        bf16x2_to_f32(w[2 * k], a, b2);
        bf16x2_to_f32(w[2 * k + 1], c, d);
        out[k] = cvt_e4m3x2(a * inv, b2 * inv) | (cvt_e4m3x2(c * inv, d * inv) << 16);
      }
      *reinterpret_cast<uint2*>(rec + 256 * half + 8 * lane) = make_uint2(out[0], out[1]);
    }
    float x, y;
    rope(r, i, x, y);
    const uint32_t two = cvt_e4m3x2(x * inv, y * inv);
    if constexpr (kInterleaved) {
      *reinterpret_cast<uint16_t*>(rec + MLA_D_LATENT + 2 * lane) = static_cast<uint16_t>(two);
    } else {
      rec[MLA_D_LATENT + lane] = static_cast<uint8_t>(two);
      rec[MLA_D_LATENT + 32 + lane] = static_cast<uint8_t>(two >> 8);
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
  auto* kern = a.interleaved ? fp8_append_kernel<true> : fp8_append_kernel<false>;
  if (const int st = smem_limit_once(reinterpret_cast<const void*>(kern), kSmemBytes, a.interleaved ? 21 : 22)) return st;
  kern<<<static_cast<unsigned>(grid), kThreads, kSmemBytes, stream>>>(p, static_cast<int>(n_kv), static_cast<int>(n_q));
  return launch_status();
}

}  // namespace mla
