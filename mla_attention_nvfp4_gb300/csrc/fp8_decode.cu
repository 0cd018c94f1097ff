// Absorbed MLA decode over the e4m3 latent cache (one scale per block of 64
// tokens) on tcgen05.
//
// The cached bytes are the tensor cores' operands as they lie: tiles of 128
// keys x 576 features arrive by TMA and serve both products, the keys as
// 128-row operand of S^T = K Q^T (K-major) and the values as 128-row operand
// of O^T = V^T P^T (read feature-major, one 128-feature chunk at a time).
// Queries and probabilities are the other operand: 32 heads a CTA, so that a
// call with few heads pays for few, and a key is a TMEM lane, so that masking
// a key masks a thread.
//
// Two e4m3 terms, side by side as columns of that operand, carry 8 bits:
//   q = 2^e (q1 + q2) with q1 = e4m3(q 2^-e), q2 = e4m3(q 2^-e - q1): a bf16
//       query exactly (its 8 bits split 4 + 4), down to 2^-17 of the head's
//       largest feature, below which it is held to an absolute 2^-19 of it;
//   p = p1 + p2 / 16 likewise, at most 2^-8 off relative (what bf16 would be).
//       The largest p lies between 2^kReset and 2^kTop, so that the absolute
//       floor, one step 2^-9 of the second term, lies 2^17 or more below it.
//       There the second term is rounded with an offset that runs evenly
//       through a step over 32 neighbouring keys: a long tail of equal, tiny
//       weights, which rounding to nearest would push to one side, keeps its
//       sum.
//
// Scales: with s the block's scale, x = log2(e) softmax_scale s q.k8,
// l = sum 2^(x - m) and O = sum (s 2^(x - m)) k8; m is a per-head reference
// that follows the maximum of x + log2 s lazily: it is raised, and O and l
// rescaled, only when a weight would exceed 2^kTop.
//
// One CTA per SM, persistent over a contiguous range of the batch's tiles
// (every range the same size, cut anywhere in a sequence); cut sequences are
// merged by LSE in a second kernel, in range order.
//   warp 0       TMA producer: 128-feature chunks of latent in a ring, RoPE apart;
//   warp 1       issues the score products, up to two tiles ahead;
//   warp 14      issues the value products (issuers of their own, so that
//                neither's waits leave the tensor cores without work);
//   warps 2..9   softmax (thread = key; warps 2..5 heads 0..15, 6..9 the rest);
//   warps 10..13 the next piece's queries to two terms, the last one's output.
#include <cuda.h>
#include <cuda_runtime.h>

#include "fp8.cuh"
#include "launch.h"
#include "nvfp4.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kKey = MLA_D_LATENT + MLA_D_ROPE;
constexpr int kBlock = MLA_FP8_BLOCK;
constexpr int kTile = 128;  // keys
constexpr int kH = 32, kMine = 16;  // heads per CTA; per softmax thread
constexpr int kSoftmax = 256, kHelper = 128, kThreads = 96 + kSoftmax + kHelper;
constexpr float kScaleMin = 8.673617379884035e-19f, kScaleMax = 1.152921504606847e18f;  // 2^-60, 2^60
constexpr float kTop = 8.5f;    // weights stay at or below 2^8.5 = 362 (e4m3: 448)
constexpr float kReset = 4.0f;  // a raised reference puts the tile's largest weight at 2^4
constexpr float kGain = 16.f;   // of the second term: the first's rounding error, at most 16, becomes 256
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;

// Shared memory: latent chunks (128 keys x 128 features, four a tile), RoPE
// tiles, two pieces' queries (rows q1 0..31, q2 32..63; four chunks of 128
// features and the RoPE), weights (row = key: p1 | p2), the rest.
constexpr int kSlots = 8, kRopes = 2;
constexpr uint32_t kChunkBytes = kTile * 128, kRopeBytes = kTile * 64;
constexpr uint32_t kQChunk = 2 * kH * 128, kQBytes = 2 * kH * kKey;
constexpr uint32_t kOffRope = kSlots * kChunkBytes, kOffQ = kOffRope + kRopes * kRopeBytes;
constexpr uint32_t kOffP = kOffQ + 2 * kQBytes, kOffMisc = kOffP + kTile * 2 * kH;
constexpr uint32_t kColS = 256;  // TMEM: O^T in columns 0..255 (64 per chunk: p1 | p2), then two S^T of 64 (q1 | q2)

struct Misc {
  uint64_t full[kSlots], empty[kSlots], rfull[kRopes], rempty[kRopes];
  uint64_t s_full[2], s_free[2], p_ready, pv_done, q_ready[2], sums_ready, o_free;
  alignas(16) float c[2][kH], m[kH], move[kH], factor[kH], inv[kH];
  float part[4][kH];
  int64_t scan[kThreads / 32], t0, t1, off0;
  int b0;
  uint32_t raised;  // heads whose reference moves, a bit each
  uint32_t tmem;
  volatile int abort;
};
constexpr uint32_t kSmemBytes = kOffMisc + static_cast<uint32_t>(sizeof(Misc));
static_assert(kSmemBytes <= 232448, "shared memory budget");

struct Params {
  Fp8DecodeArgs a;
  uint32_t page_magic;  // division by page_size / 64
  int page_shift;
  int ranges, groups;  // ranges of tiles; head groups (grid = ranges * groups)
  bool split;
  int64_t* offsets;  // [batch + 1] first tile of each sequence, then tiles per range
  float* part_lse;   // log2 units, [range][group][2][kH]
  float* part_o;     // the same rows of 512
};

__device__ __forceinline__ int clipped_len(const Fp8DecodeArgs& a, int b) {
  const int64_t room = a.max_pages * a.page_size;
  const int n = a.seq_lens[b];
  return n <= 0 ? 0 : n <= room ? n : static_cast<int>(room);
}
__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

// Block i (64 tokens) of sequence b: its page table entry, and its first slot
// given that entry, or -1 (page out of range).
__device__ __forceinline__ int block_page(const Params& p, int b, int i) {
  return p.a.page_table[b * p.a.pt_stride + div_magic(i, p.page_magic, p.page_shift)];
}
__device__ __forceinline__ int block_slot(const Params& p, int page, int i) {
  const int in = i - static_cast<int>(div_magic(i, p.page_magic, p.page_shift)) * (p.a.page_size / kBlock);
  const int64_t slot = static_cast<int64_t>(page) * p.a.page_size + static_cast<int64_t>(in) * kBlock;
  return page < 0 || slot + kBlock > p.a.num_slots ? -1 : static_cast<int>(slot);
}

// Calls f(b, len, first tile, last tile + 1, tiles of b, part) for every
// piece of this CTA's work; part: 0 for the piece its range begins with.
template <class F>
__device__ __forceinline__ void for_each_piece(const Params& p, const Misc& ms, int range, F f) {
  // one loop (and one copy of f's code) for both forms: a range of tiles, or
  // whole sequences range, range + ranges, ...
  const bool split = p.split;
  int64_t t = split ? ms.t0 : 0, off = split ? ms.off0 : 0;
  const int64_t t0 = t, t1 = split ? ms.t1 : 0;
  for (int b = split ? ms.b0 : range; split ? t < t1 : b < p.a.batch; b += split ? 1 : p.ranges) {
    const int len = clipped_len(p.a, b), n = tiles_of(len);
    const int s = split ? static_cast<int>(t - off) : 0;
    const int e = split && t1 - off < n ? static_cast<int>(t1 - off) : n;
    if (n > 0 || !split) f(b, len, s, e, n, t == t0 ? 0 : 1);
    if (split) {
      if (n > 0) t = off + e;
      off += n;
    }
  }
}

// mbar_wait with the loop kept out of line: one try where it is used.
__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, uint32_t* err, volatile int* abort) {
  return mbar_wait(bar, parity, err, abort);
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, uint32_t* err, volatile int* abort) {
  return mbar_test(bar, parity) || wait_long(bar, parity, err, abort);
}

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
__device__ __forceinline__ void softmax_bar() { asm volatile("bar.sync 1, %0;" ::"n"(kSoftmax) : "memory"); }
__device__ __forceinline__ bool softmax_any(bool v) {
  int r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\tsetp.ne.s32 a, %1, 0;\n\tbarrier.cta.red.or.pred b, 2, %2, a;\n\t"
      "selp.s32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"(static_cast<int>(v)), "n"(kSoftmax)
      : "memory");
  return r != 0;
}

// The plan: this CTA's range of the batch's tiles, and its first sequence.
__device__ __forceinline__ void make_plan(const Params& p, Misc& ms, int range, bool publish) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, B = p.a.batch;
  const int per_thread = (B + kThreads - 1) / kThreads;
  const int first = tid * per_thread, last = min(first + per_thread, B);
  int64_t sum = 0;
  for (int b = first; b < last; ++b) sum += tiles_of(clipped_len(p.a, b));
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) ms.scan[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += ms.scan[w];
    total += ms.scan[w];
  }
  const int64_t per = (total + p.ranges - 1) / p.ranges;
  const int64_t t0 = range * per, t1 = t0 + per < total ? t0 + per : total;
  int64_t off = before + incl - sum;
  if (tid == 0) {
    ms.t0 = t0;
    ms.t1 = t1;
  }
  for (int b = first; b < last; ++b) {
    const int n = tiles_of(clipped_len(p.a, b));
    if (publish) p.offsets[b] = off;
    if (t0 >= off && t0 < off + n) {
      ms.b0 = b;
      ms.off0 = off;
    }
    off += n;
  }
  if (publish && tid == 0) {
    p.offsets[B] = total;
    p.offsets[B + 1] = per;
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    fp8_decode_kernel(const __grid_constant__ CUtensorMap tm_lat, const __grid_constant__ CUtensorMap tm_rope,
                      const Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc& ms = *reinterpret_cast<Misc*>(smem + kOffMisc);
  const uint32_t s0 = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int range = blockIdx.x / p.groups, group = blockIdx.x % p.groups;
  uint32_t* err = p.a.error_word;

  if (threadIdx.x == 0) {
    ms.abort = 0;
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&ms.full[i], 1);
      mbar_init(&ms.empty[i], 1);
    }
    for (int i = 0; i < kRopes; ++i) {
      mbar_init(&ms.rfull[i], 1);
      mbar_init(&ms.rempty[i], 1);
    }
    mbar_init(&ms.s_full[0], 1);
    mbar_init(&ms.s_full[1], 1);
    mbar_init(&ms.s_free[0], kSoftmax / 32);
    mbar_init(&ms.s_free[1], kSoftmax / 32);
    mbar_init(&ms.p_ready, kSoftmax / 32);
    mbar_init(&ms.pv_done, 1);
    mbar_init(&ms.q_ready[0], kHelper / 32);
    mbar_init(&ms.q_ready[1], kHelper / 32);
    mbar_init(&ms.sums_ready, kSoftmax / 32);
    mbar_init(&ms.o_free, kHelper / 32);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ms.tmem, 512);
    tmem_relinquish();
  }
  if (p.split) make_plan(p, ms, range, blockIdx.x == 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms.tmem;
  auto slot_addr = [&](int i) { return s0 + i * kChunkBytes; };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tmap(&tm_lat);
      prefetch_tmap(&tm_rope);
    }
    int n = 0;
    bool ok = true;
    for_each_piece(p, ms, range, [&](int b, int len, int s, int e, int, int) {
      const int n_blocks = (len + kBlock - 1) / kBlock;
      int y = 0;  // lane i: row of block (first block of the batch of 32) + i; past the cache where there is none
      for (int t = s; t < e && ok; ++t, ++n) {
        const int at = (2 * (t - s)) & 31;
        if (at == 0) {
          const int i = 2 * t + lane;
          const int slot = i < n_blocks && i < 2 * e ? block_slot(p, block_page(p, b, i), i) : -1;
          y = static_cast<int>(slot < 0 ? p.a.num_slots : slot);
        }
        const int y0 = __shfl_sync(0xffffffffu, y, at), y1 = __shfl_sync(0xffffffffu, y, at + 1);
        if (lane == 0) {
#pragma unroll
          for (int d = 0; d < 4 && ok; ++d) {
            const int k = 4 * n + d, i = k % kSlots;
            ok = wait(&ms.empty[i], ((k / kSlots) & 1) ^ 1, err, &ms.abort);
            if (!ok) break;
            mbar_expect_tx(&ms.full[i], kChunkBytes);
            tma_load_bytes(slot_addr(i), &tm_lat, 128 * d, y0, &ms.full[i]);
            tma_load_bytes(slot_addr(i) + kChunkBytes / 2, &tm_lat, 128 * d, y1, &ms.full[i]);
          }
          if (ok) {
            const int i = n % kRopes;
            ok = wait(&ms.rempty[i], ((n / kRopes) & 1) ^ 1, err, &ms.abort);
            if (ok) {
              const uint32_t dst = s0 + kOffRope + i * kRopeBytes;
              mbar_expect_tx(&ms.rfull[i], kRopeBytes);
              tma_load_bytes(dst, &tm_rope, MLA_D_LATENT, y0, &ms.rfull[i]);
              tma_load_bytes(dst + kRopeBytes / 2, &tm_rope, MLA_D_LATENT, y1, &ms.rfull[i]);
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0) != 0;
      }
    });
  } else if (warp == 1) {
    // -------------------------------------------------------- score products
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3(128, 2 * kH, false, false);
      bool ok = true;
      auto ready = [&](uint64_t* bar, int parity) {
        ok = ok && wait(bar, parity, err, &ms.abort);
        return ok;
      };
      int n = 0, piece = 0;
      for_each_piece(p, ms, range, [&](int, int, int s, int e, int, int) {
        if (s >= e || !ready(&ms.q_ready[piece & 1], (piece >> 1) & 1)) return;
        const uint32_t q = s0 + kOffQ + (piece & 1) * kQBytes;
        for (int t = s; t < e; ++t, ++n) {
          const uint32_t d = tmem + kColS + (n & 1) * 2 * kH;
          if (!ready(&ms.s_free[n & 1], ((n >> 1) & 1) ^ 1)) return;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int k = 4 * n + c, i = k % kSlots;
            if (!ready(&ms.full[i], (k / kSlots) & 1)) return;
            tc_fence_after();
            const uint64_t da = smem_desc_sw128(slot_addr(i), 0, 1024), db = smem_desc_sw128(q + c * kQChunk, 0, 1024);
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_e4m3(d, da + 2 * j, db + 2 * j, idesc, (c > 0 || j > 0) ? 1u : 0u);
          }
          const int i = n % kRopes;
          if (!ready(&ms.rfull[i], (n / kRopes) & 1)) return;
          tc_fence_after();
          const uint64_t da = smem_desc_sw64(s0 + kOffRope + i * kRopeBytes, 512);
          const uint64_t db = smem_desc_sw64(q + 4 * kQChunk, 512);
#pragma unroll
          for (int j = 0; j < 2; ++j) mma_e4m3(d, da + 2 * j, db + 2 * j, idesc, 1u);
          mma_commit(&ms.rempty[i]);
          mma_commit(&ms.s_full[n & 1]);
        }
        ++piece;
      });
    }
  } else if (warp == 14) {
    // -------------------------------------------------------- value products
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3(128, 2 * kH, true, true);
      bool ok = true;
      int n = 0, piece = 0;
      for_each_piece(p, ms, range, [&](int, int, int s, int e, int, int) {
        if (s >= e) return;
        for (int t = s; t < e; ++t, ++n) {
          ok = ok && wait(&ms.p_ready, n & 1, err, &ms.abort);
          // the previous piece's output has been read
          if (t == s && piece > 0) ok = ok && wait(&ms.o_free, (piece - 1) & 1, err, &ms.abort);
          if (!ok) return;
          tc_fence_after();
          const uint64_t db = smem_desc_sw64(s0 + kOffP, 512);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int i = (4 * n + c) % kSlots;
            // V^T: 128 features of the chunk as rows, 32 keys (4096 bytes) a
            // step.  The scores of this tile are done (P came of them), so
            // the chunk is free after these.
            const uint64_t da = smem_desc_sw128(slot_addr(i), 0, 1024);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_e4m3(tmem + 64 * c, da + 256 * j, db + 128 * j, idesc, (t > s || j > 0) ? 1u : 0u);
            mma_commit(&ms.empty[i]);
          }
          mma_commit(&ms.pv_done);
        }
        ++piece;
      });
    }
  } else if (warp < 10) {
    // ------------------------------------------------------------- softmax
    // A wait that gives up leaves these warps running through their loops
    // (they meet at named barriers); the error word tells.
    const int quad = warp & 3, tid = threadIdx.x - 64, wg = tid >> 7;
    const int hb = wg * kMine;         // this thread's first head
    const int key = quad * 32 + lane;  // of the tile: a TMEM lane
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const int h0 = group * kH, heads = min(kH, p.a.num_heads - h0);
    // offset of the second term's rounding: (j + 1/2) / 32 - 1/2 of a step
    // 2^-9, j the lane's bits reversed
    const float off = ((__brev(lane) >> 27) + 0.5f) * (1.f / 32) - 0.5f;
    const __half2 dither_h = __float2half2_rn(off * 0.001953125f);
    const uint32_t dither = *reinterpret_cast<const uint32_t*>(&dither_h);
    int n = 0, piece = 0;
    for_each_piece(p, ms, range, [&](int b, int len, int s, int e, int tiles, int part) {
      float* lse = p.a.lse != nullptr ? p.a.lse + static_cast<int64_t>(b) * p.a.num_heads + h0 : nullptr;
      if (s >= e) {  // no keys
        uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.a.out) +
                                              (static_cast<int64_t>(b) * p.a.num_heads + h0) * MLA_D_LATENT);
        for (int i = tid; i < heads * (MLA_D_LATENT / 8); i += kSoftmax) out[i] = make_uint4(0, 0, 0, 0);
        if (lse != nullptr && tid < heads) lse[tid] = -INFINITY;
        return;
      }
      if (s == 0 && tid == 0 && group == 0 && p.a.seq_lens[b] > len) flag_error(err, MLA_DEVERR_BOUNDS);

      // Page table entries two tiles ahead, block scales one, each loaded an
      // iteration before it is used.
      const int n_blocks = (len + kBlock - 1) / kBlock;
      auto page_at = [&](int t) {
        const int i = 2 * t + (quad >> 1);
        return t < e && i < n_blocks ? block_page(p, b, i) : 0;
      };
      auto slot_at = [&](int t, int page) {  // -2: no such block; -1: its page is out of range
        const int i = 2 * t + (quad >> 1);
        return t < e && i < n_blocks ? block_slot(p, page, i) : -2;
      };
      int slot_n = slot_at(s, page_at(s)), page_n = page_at(s + 1);
      float scale_n = slot_n >= 0 ? p.a.scales[slot_n / kBlock] : 0.f;

      if (tid < kH) ms.m[tid] = 0.f;
      wait(&ms.q_ready[piece & 1], (piece >> 1) & 1, err, &ms.abort);  // c is there
      softmax_bar();                                 // and m
      const float* cs = ms.c[piece & 1] + hb;
      const float* mr = ms.m + hb;
      float l[kMine];
#pragma unroll
      for (int h = 0; h < kMine; ++h) l[h] = 0.f;
      bool set = false;  // the references follow some key
      for (int t = s; t < e; ++t, ++n) {
        const int slot = slot_n;
        const bool sb_ok = slot >= 0 && scale_n >= kScaleMin && scale_n <= kScaleMax;
        const float sb = sb_ok ? scale_n : 1.f, lsb = log2f(sb);
        if (lane == 0 && (quad & 1) == 0 && wg == 0 && slot != -2 && !sb_ok)
          flag_error(err, slot < 0 ? MLA_DEVERR_BOUNDS : MLA_DEVERR_SCALE);
        const bool valid = sb_ok && t * kTile + key < len;

        wait(&ms.s_full[n & 1], (n >> 1) & 1, err, &ms.abort);
        tc_fence_after();
        float x[kMine], top = -INFINITY;
        {
          const uint32_t src = lanes + kColS + (n & 1) * 2 * kH + hb;
          uint32_t v[16], u[16];
          tmem_ld16(src, v);
          tmem_ld16(src + kH, u);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ms.s_free[n & 1]);
#pragma unroll
          for (int h = 0; h < kMine; h += 4) {
            const float4 cc = *reinterpret_cast<const float4*>(cs + h), mm = *reinterpret_cast<const float4*>(mr + h);
            const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, mv[4] = {mm.x, mm.y, mm.z, mm.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float sum = __uint_as_float(v[h + j]) + __uint_as_float(u[h + j]);
              x[h + j] = valid ? fmaf(sum * sb, cv[j], -mv[j]) : -INFINITY;
              top = fmaxf(top, x[h + j]);
            }
          }
        }
        if (softmax_any(top + lsb > kTop || (!set && valid))) {
          // Raise the references of the heads that need it: each head's
          // maximum over the warp's keys by exchanging halves (lane i ends
          // with head hb + i / 2), then over the warps.
          float v[kMine];
#pragma unroll
          for (int h = 0; h < kMine; ++h) v[h] = x[h] + lsb;
#pragma unroll
          for (int o = 16; o > 1; o >>= 1) {
            const bool up = (lane & o) != 0;
#pragma unroll
            for (int h = 0; h < kMine / 2; ++h) {
              if (h < o / 2) {
                const float give = up ? v[h] : v[h + o / 2], keep = up ? v[h + o / 2] : v[h];
                v[h] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, o));
              }
            }
          }
          v[0] = fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
          ms.part[quad][hb + lane / 2] = v[0];
          softmax_bar();
          if (tid < kH) {
            const float mx = fmaxf(fmaxf(ms.part[0][tid], ms.part[1][tid]), fmaxf(ms.part[2][tid], ms.part[3][tid]));
            const bool raise = isfinite(mx) && (!set || mx > kTop);
            const float by = raise ? mx - kReset : 0.f;
            ms.move[tid] = by;
            ms.factor[tid] = !set ? 0.f : ex2_approx(-by);
            ms.m[tid] += by;
            const uint32_t raised = __ballot_sync(0xffffffffu, raise);
            if (lane == 0) ms.raised = raised;
          }
          softmax_bar();
#pragma unroll
          for (int h = 0; h < kMine; h += 4) {
            const float4 mv = *reinterpret_cast<const float4*>(&ms.move[hb + h]);
            const float4 fv = *reinterpret_cast<const float4*>(&ms.factor[hb + h]);
            x[h] -= mv.x, x[h + 1] -= mv.y, x[h + 2] -= mv.z, x[h + 3] -= mv.w;
            l[h] *= fv.x, l[h + 1] *= fv.y, l[h + 2] *= fv.z, l[h + 3] *= fv.w;
          }
          if (t > s) {
            // O holds earlier tiles: once their products are done, the
            // columns of 16 heads at a time, two value chunks per warp
            wait(&ms.pv_done, (n - 1) & 1, err, &ms.abort);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 64; c += 16) {
              const int g = c & (kH - 1);
              if (((ms.raised >> g) & 0xFFFFu) == 0) continue;
              const uint32_t at = lanes + 128 * wg + c;
              uint32_t a[16], u[16];
              tmem_ld16(at, a);
              tmem_ld16(at + 64, u);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                const float4 f4 = *reinterpret_cast<const float4*>(&ms.factor[g + i]);
                const float fv[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  a[i + j] = __float_as_uint(__uint_as_float(a[i + j]) * fv[j]);
                  u[i + j] = __float_as_uint(__uint_as_float(u[i + j]) * fv[j]);
                }
              }
              tmem_st16(at, a);
              tmem_st16(at + 64, u);
            }
            tmem_st_wait();
          }
          set = true;
        }
        slot_n = slot_at(t + 1, page_n);
        scale_n = slot_n >= 0 ? p.a.scales[slot_n / kBlock] : 0.f;
        page_n = page_at(t + 2);
        // weights and their two terms; words of four heads
        uint32_t w1[kMine / 4], w2[kMine / 4];
#pragma unroll
        for (int h = 0; h < kMine; h += 4) {
          uint32_t a[2], r[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float e0 = ex2_approx(x[h + 2 * j]), e1 = ex2_approx(x[h + 2 * j + 1]);
            l[h + 2 * j] += e0;
            l[h + 2 * j + 1] += e1;
            const __half2 ph = __floats2half2_rn(e0 * sb, e1 * sb);
            const uint32_t pu = *reinterpret_cast<const uint32_t*>(&ph);
            a[j] = cvt_e4m3x2_h2(pu);
            r[j] = cvt_e4m3x2_h2(h2_fma(h2_sub(pu, e4m3x2_to_f16x2_pair(a[j])), kGain, dither));
          }
          w1[h / 4] = a[0] | (a[1] << 16);
          w2[h / 4] = r[0] | (r[1] << 16);
        }
        // the previous tile's products have read P
        if (n > 0) wait(&ms.pv_done, (n - 1) & 1, err, &ms.abort);
        {
          // row = key, 64 bytes p1 | p2, 16-byte units swizzled by the row
          const uint32_t row = s0 + kOffP + key * 64, sw = (key >> 1) & 3;
          sts128(row + ((wg ^ sw) << 4), make_uint4(w1[0], w1[1], w1[2], w1[3]));
          sts128(row + (((wg + 2) ^ sw) << 4), make_uint4(w2[0], w2[1], w2[2], w2[3]));
        }
        // a row that is no key of the sequence may hold any bytes (NaN too):
        // as values they are zeros
        if (!valid && slot >= 0) {
#pragma unroll 1
          for (int c = 2 * wg; c < 2 * wg + 2; ++c) {
            const uint32_t row = slot_addr((4 * n + c) % kSlots) + key * 128;
#pragma unroll
            for (int i = 0; i < 8; ++i) sts128(row + 16 * i, make_uint4(0, 0, 0, 0));
          }
        }
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.p_ready);
      }

      // Sums over the keys: halves exchanged as above, then across the warps.
#pragma unroll
      for (int o = 16; o > 1; o >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int h = 0; h < kMine / 2; ++h) {
          if (h < o / 2) {
            const float give = up ? l[h] : l[h + o / 2], keep = up ? l[h + o / 2] : l[h];
            l[h] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
        }
      }
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], 1);
      ms.part[quad][hb + lane / 2] = l[0];
      softmax_bar();
      // the previous piece's output warps have read inv
      if (piece > 0) wait(&ms.o_free, (piece - 1) & 1, err, &ms.abort);
      if (tid < kH) {
        const float sum = (ms.part[0][tid] + ms.part[1][tid]) + (ms.part[2][tid] + ms.part[3][tid]);
        ms.inv[tid] = sum != 0.f ? 1.f / sum : 0.f;  // NaN stays NaN
        const float l2 = sum != 0.f ? ms.m[tid] + log2f(sum) : -INFINITY;
        if (e - s < tiles)
          p.part_lse[((static_cast<int64_t>(range) * p.groups + group) * 2 + part) * kH + tid] = l2;
        else if (lse != nullptr && tid < heads)
          lse[tid] = l2 * kLn2;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.sums_ready);
      softmax_bar();  // part and m are free for the next piece
      ++piece;
    });
  } else {
    // ----------------------------------------------------- queries, output
    const int quad = warp & 3;
    const int row = quad * 32 + lane;  // of a value chunk: a TMEM lane
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const int h0 = group * kH, heads = min(kH, p.a.num_heads - h0);
    int n_last = -1;  // last tile of the pieces so far
    // A piece's queries are laid out while the piece before it runs, its
    // output written while the piece after it starts.
    struct { int b, part, whole, n; } done = {-1, 0, 0, 0};
    int piece = 0, written = 0;
    auto output = [&]() {
      // sums first: then the last tile's products are the next phase of pv_done
      wait(&ms.sums_ready, written & 1, err, &ms.abort);
      wait(&ms.pv_done, done.n & 1, err, &ms.abort);
      tc_fence_after();
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.a.out) +
                           (static_cast<int64_t>(done.b) * p.a.num_heads + h0) * MLA_D_LATENT;
      float* part_o = p.part_o + ((static_cast<int64_t>(range) * p.groups + group) * 2 + done.part) * kH * MLA_D_LATENT;
      // thread = feature; neighbouring threads swap halves of two heads so
      // that each stores two features of one
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        const int d = 128 * c + row;
        uint32_t v[32], u[32];
        tmem_ld32(lanes + 64 * c, v);
        tmem_ld32(lanes + 64 * c + 32, u);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 iv4 = *reinterpret_cast<const float4*>(&ms.inv[i]);
          const float iv[4] = {iv4.x, iv4.y, iv4.z, iv4.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            v[i + j] = __float_as_uint(fmaf(__uint_as_float(u[i + j]), 1.f / kGain, __uint_as_float(v[i + j])) * iv[j]);
        }
        if (c == 3) {  // O and inv are free
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ms.o_free);
        }
        if (done.whole) {
          const int odd = lane & 1;
          uint32_t* dst = reinterpret_cast<uint32_t*>(out + odd * MLA_D_LATENT + (d - odd));
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float mine = __uint_as_float(odd ? v[i + 1] : v[i]);
            const float got = __shfl_xor_sync(0xffffffffu, __uint_as_float(odd ? v[i] : v[i + 1]), 1);
            const __nv_bfloat162 o = odd ? __floats2bfloat162_rn(got, mine) : __floats2bfloat162_rn(mine, got);
            if (i + odd < heads) dst[i * (MLA_D_LATENT / 2)] = *reinterpret_cast<const uint32_t*>(&o);
          }
        } else {
          float* dst = part_o + d;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i < heads) dst[i * MLA_D_LATENT] = __uint_as_float(v[i]);
        }
      }
      ++written;
    };
    for_each_piece(p, ms, range, [&](int b, int, int s, int e, int tiles, int part) {
      if (s >= e) return;
      // Queries: a warp takes every fourth head; lane l features 8 l.., and
      // 256 + 8 l.., lanes 0..7 the RoPE's; two heads' loads in flight.
      // Their buffer's last reader, the piece before the last, is written.
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.a.q) +
                               (static_cast<int64_t>(b) * p.a.num_heads + h0) * kKey;
      const uint32_t dst = s0 + kOffQ + (piece & 1) * kQBytes;
      auto load_head = [&](int h, uint4(&v)[3]) {
        v[0] = v[1] = v[2] = make_uint4(0, 0, 0, 0);
        if (h < heads) {
          const uint4* src = reinterpret_cast<const uint4*>(q + static_cast<int64_t>(h) * kKey);
          v[0] = src[lane];
          v[1] = src[lane + 32];
          if (lane < 8) v[2] = src[lane + 64];
        }
      };
      uint4 v_next[3], v_after[3];
      load_head(quad, v_next);
      load_head(quad + 4, v_after);
#pragma unroll 1
      for (int h = quad; h < kH; h += 4) {
        uint4 v[3];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          v[k] = v_next[k];
          v_next[k] = v_after[k];
        }
        load_head(h + 8, v_after);
        // amax from the bf16 bits (sign dropped, they order like integers)
        uint32_t m2 = 0;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            m2 = max(m2, w[j] & 0x7FFF0000u);
            m2 = max(m2, (w[j] << 16) & 0x7FFF0000u);
          }
        }
        m2 = __reduce_max_sync(0xffffffffu, m2);
        // 2^e, the smallest with amax <= 448 * 2^e (448 = 1.75 * 2^8)
        int ex = static_cast<int>(m2 >> 23) - 127 - 8 + ((m2 & 0x7FFFFFu) > 0x600000u ? 1 : 0);
        ex = max(-60, min(60, ex));
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
        if (lane == 0)
          ms.c[piece & 1][h] = p.a.softmax_scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
          uint32_t w1[2], w2[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float x0, x1, x2, x3;
            bf16x2_to_f32(w[2 * j], x0, x1);
            bf16x2_to_f32(w[2 * j + 1], x2, x3);
            x0 *= inv, x1 *= inv, x2 *= inv, x3 *= inv;
            const uint32_t a = cvt_e4m3x2(x0, x1), c = cvt_e4m3x2(x2, x3);
            const uint32_t ha = e4m3x2_to_f16x2_pair(a), hc = e4m3x2_to_f16x2_pair(c);
            const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&ha));
            const float2 fc = __half22float2(*reinterpret_cast<const __half2*>(&hc));
            w1[j] = a | (c << 16);
            w2[j] = cvt_e4m3x2(x0 - fa.x, x1 - fa.y) | (cvt_e4m3x2(x2 - fc.x, x3 - fc.y) << 16);
          }
          // row h (q1) and kH + h (q2) of the chunk; 16-byte units swizzled by the row
          uint32_t a1, a2;
          if (k < 2) {
            const int feature = 256 * k + 8 * lane;
            const uint32_t base = dst + (feature >> 7) * kQChunk;
            const uint32_t unit = (feature & 127) >> 4, half = feature & 8;
            a1 = base + h * 128 + ((unit ^ (h & 7)) << 4) + half;
            a2 = a1 + kH * 128;
          } else {
            const uint32_t base = dst + 4 * kQChunk;
            const uint32_t unit = lane >> 1, half = (lane & 1) * 8;
            a1 = base + h * 64 + ((unit ^ ((h >> 1) & 3)) << 4) + half;
            a2 = a1 + kH * 64;
          }
          if (k < 2 || lane < 8) {
            asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(a1), "r"(w1[0]), "r"(w1[1]) : "memory");
            asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(a2), "r"(w2[0]), "r"(w2[1]) : "memory");
          }
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.q_ready[piece & 1]);
      ++piece;
      if (done.b >= 0) output();
      n_last += e - s;
      done = {b, part, e - s == tiles, n_last};
    });
    if (done.b >= 0) output();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// Merge of the pieces of cut sequences, in range order, by LSE; sequences
// without keys get their zeros here.  CTA = (sequence, head), thread = four
// features.
__global__ void __launch_bounds__(128) fp8_decode_merge_kernel(const Params p) {
  const int b = blockIdx.x / p.a.num_heads, h = blockIdx.x % p.a.num_heads, tid = threadIdx.x;
  const int64_t off = p.offsets[b], end = p.offsets[b + 1], per = p.offsets[p.a.batch + 1];
  const int64_t row = static_cast<int64_t>(b) * p.a.num_heads + h;
  uint2* out = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.a.out) + row * MLA_D_LATENT) + tid;
  if (off == end) {
    *out = make_uint2(0, 0);
    if (p.a.lse != nullptr && tid == 0) p.a.lse[row] = -INFINITY;
    return;
  }
  const int64_t r0 = off / per, r1 = (end - 1) / per;
  if (r0 == r1) return;  // one piece: written already
  const int g = h / kH;
  auto piece = [&](int64_t r) {  // its row of partial results
    const int part = r == r0 && r * per < off ? 1 : 0;
    return ((r * p.groups + g) * 2 + part) * kH + h % kH;
  };
  float m = -INFINITY;
  for (int64_t r = r0; r <= r1; ++r) m = fmaxf(m, p.part_lse[piece(r)]);
  const float ref = m == -INFINITY ? 0.f : m;
  float sum = 0.f, o[4] = {};
  for (int64_t r = r0; r <= r1; ++r) {
    const int64_t i = piece(r);
    const float w = ex2_approx(p.part_lse[i] - ref);
    sum += w;
    const float4 v = reinterpret_cast<const float4*>(p.part_o + i * MLA_D_LATENT)[tid];
    o[0] = fmaf(w, v.x, o[0]);
    o[1] = fmaf(w, v.y, o[1]);
    o[2] = fmaf(w, v.z, o[2]);
    o[3] = fmaf(w, v.w, o[3]);
  }
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(o[0] * inv, o[1] * inv);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(o[2] * inv, o[3] * inv);
  *out = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  if (p.a.lse != nullptr && tid == 0) p.a.lse[row] = sum != 0.f ? (ref + log2f(sum)) * kLn2 : -INFINITY;
}

struct Layout {
  int ranges, groups;
  size_t lse, o, total;
};
Layout layout(int batch, int num_heads, int num_sms) {
  Layout l;
  l.groups = (num_heads + kH - 1) / kH;
  l.ranges = num_sms / l.groups > 1 ? num_sms / l.groups : 1;
  const size_t rows = static_cast<size_t>(l.ranges) * l.groups * 2 * kH;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  l.lse = up((static_cast<size_t>(batch) + 2) * sizeof(int64_t));
  l.o = up(l.lse + rows * sizeof(float));
  l.total = l.o + rows * MLA_D_LATENT * sizeof(float);
  return l;
}

}  // namespace

size_t fp8_decode_workspace_bytes(int batch, int num_heads, int num_sms) {
  return layout(batch, num_heads, num_sms).total;
}

int launch_fp8_decode(const Fp8DecodeArgs& a, cudaStream_t stream, int num_sms) {
  const Layout l = layout(a.batch, a.num_heads, num_sms);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  uint32_t magic;
  int shift;
  magic_divisor(a.page_size / kBlock, &magic, &shift);
  Params p{a, magic, shift, l.ranges, l.groups, ws != nullptr, reinterpret_cast<int64_t*>(ws), reinterpret_cast<float*>(ws + l.lse),
           reinterpret_cast<float*>(ws + l.o)};
  if (static_cast<int64_t>(a.batch) * a.num_heads > (int64_t(1) << 31) - 1) return MLA_ERR_INVALID_ARG;
  CUtensorMap lat, rope;
  if (!encode_byte_map(&lat, a.cache, kKey, a.num_slots, kKey, 128, kBlock, false) ||
      !encode_byte_map(&rope, a.cache, kKey, a.num_slots, kKey, 64, kBlock, true)) {
    set_last_error("cuTensorMapEncodeTiled failed for the cache");
    return MLA_ERR_LAUNCH;
  }
  if (const int st = smem_limit_once(reinterpret_cast<const void*>(fp8_decode_kernel), static_cast<int>(kSmemBytes), 19))
    return st;
  fp8_decode_kernel<<<static_cast<unsigned>(p.ranges) * p.groups, kThreads, kSmemBytes, stream>>>(lat, rope, p);
  if (const int st = launch_status()) return st;
  if (!p.split) return MLA_OK;
  fp8_decode_merge_kernel<<<static_cast<unsigned>(a.num_heads) * a.batch, 128, 0, stream>>>(p);
  return launch_status();
}

}  // namespace mla
