// The attention weight that a decode step's queries give to each key of the
// e4m3 cache, summed over the heads:
//   out[b, t] = weights[b, t] + sum_h 2^(log2(e) (softmax_scale q_bh . key_t - lse_bh)).
//
// The decode's score product alone, on tcgen05: tiles of 128 keys x 576
// features arrive by TMA as they lie and are the 128-row operand, the queries'
// two e4m3 terms (fp8_query.cuh) the other, so that a key is a TMEM lane and
// the sum over the heads stays in its thread.  HBM-bound: all heads meet a tile
// while it is there, and no result of one tile is needed by another.  Up to 128
// heads are one CTA's, whose queries then leave room for one tile in flight, not
// two; more heads take a launch each 128.
// Times: 32 sequences of 1k to 32k, 16 heads 32.2 us (5.7 TB/s); 64 x 4096, 64 heads
// 29.8, 128 heads 43.7 (3.7 TB/s: the one tile in flight, chunk by chunk behind its
// products, and the pieces' starts); 1 x 1000, 16 heads 4.7, a chain of latencies.
//
// One CTA per SM, persistent over an equal part of the batch's tiles (and of
// its pieces' starts, a sequence's queries being converted anew):
//   warp 0      TMA producer; 128-feature chunks and the RoPE's in turn;
//   warp 1      issues the products, a tile ahead;
//   warps 2..   queries to two terms; then a tile each four of them, in turn:
//               thread = key.
#include <cuda.h>
#include <cuda_runtime.h>

#include "fp8.cuh"
#include "fp8_paged.cuh"
#include "fp8_query.cuh"
#include "launch.h"
#include "nvfp4.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kKey = kFp8Key, kBlock = MLA_FP8_BLOCK, kTile = 128;
// Groups of four warps that take a tile each in turn: two keep up with the
// tiles; with 64 heads and more the queries want four.
template <int kH>
constexpr int kGroups = kH >= 64 ? 4 : 2;
template <int kH>
constexpr int kThreads = 64 + 128 * kGroups<kH>;
constexpr uint32_t kChunkBytes = kTile * 128, kRopeBytes = kTile * 64, kTileBytes = 4 * kChunkBytes + kRopeBytes;
constexpr int kStart = 2;  // a piece's start, in tiles
constexpr int kInfo = 4;   // tiles whose scales are kept

template <int kH>
struct Cfg {
  static constexpr int tiles = kH == 128 ? 1 : 2;  // in shared memory
  static constexpr int slots = 5 * tiles;          // chunks of them
  static constexpr uint32_t off_rope = 4 * tiles * kChunkBytes, off_q = tiles * kTileBytes;
  static constexpr uint32_t off_misc = off_q + 2 * kH * kKey;
  static constexpr uint32_t columns = 4 * kH;  // of TMEM: two tiles' scores of 2 kH
};

template <int kH>
struct Misc {
  uint64_t full[Cfg<kH>::slots], empty[Cfg<kH>::slots], info_full[kInfo];
  // A tile's scores are there: a barrier a group of sum warps, of whose tiles it waits
  // for every one (of two by the scores' place, four groups would each miss every
  // other phase, and could take a tile's for that four tiles before).
  uint64_t s_full[kGroups<kH>], s_free[2], q_ready, q_free, retired;
  alignas(16) float2 head[2][kH];  // of a piece, in turn: factor of its scores, log2(e) lse
  float scale[kInfo][2];           // of a tile's two blocks; 0: none of the sequence's
  int64_t scan[kThreads<kH> / 32], t0, t1, off0;
  int b0, len0;  // the part's first sequence, its keys
  uint32_t tmem;
  int copies;
  volatile int abort;
};

template <int kH>
constexpr uint32_t smem_bytes() {
  return Cfg<kH>::off_misc + static_cast<uint32_t>(sizeof(Misc<kH>));
}
static_assert(smem_bytes<128>() <= 232448 && smem_bytes<64>() <= 232448, "shared memory budget");

struct Params {
  Fp8WeightsArgs a;
  uint32_t page_magic;  // division by page_size / 64
  int page_shift;
  int h0;  // first head of this launch
};

__device__ __forceinline__ int64_t room_of(const Fp8WeightsArgs& a) {
  const int64_t table = a.max_pages * a.page_size, most = (int64_t{1} << 31) - 2 * kTile;
  const int64_t room = table < a.row_len ? table : a.row_len;
  return room < most ? room : most;
}
__device__ __forceinline__ int length_of(const Params& p, int b) {
  return fp8_length(p.a.seq_lens[b], room_of(p.a), nullptr, false);
}
__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }
__device__ __forceinline__ int cost_of(int len) { return len > 0 ? tiles_of(len) + kStart : 0; }

// The pieces of a CTA's part, one after another: tiles [s, e) of sequence b
// (len keys).  A part is one of the sequences' costs, of which the first kStart
// of a sequence are its start and the rest its tiles.
struct Pieces {
  int b = 0, len = 0, s = 0, e = 0;

  template <class M>
  __device__ __forceinline__ Pieces(const Params& p, const M& ms)
      : next_(ms.b0), t_(ms.t0), t1_(ms.t1), off_(ms.off0), next_len_(ms.len0) {}
  __device__ __forceinline__ bool next(const Params& p) {
    while (t_ < t1_ && next_ < p.a.batch) {
      b = next_;
      len = next_len_;
      const int64_t first = off_ + kStart, end = off_ + cost_of(len), hi = t1_ < end ? t1_ : end;
      s = t_ > first ? static_cast<int>(t_ - first) : 0;
      e = hi > first ? static_cast<int>(hi - first) : 0;
      t_ = hi;
      if (hi == end) {
        off_ = end;
        ++next_;
        next_len_ = load(p);  // ahead of its use
      }
      if (s < e) return true;
    }
    return false;
  }

 private:
  __device__ __forceinline__ int load(const Params& p) const { return next_ < p.a.batch ? length_of(p, next_) : 0; }
  int next_;
  int64_t t_;
  const int64_t t1_;
  int64_t off_;
  int next_len_;
};

// This CTA's part of the sequences' costs, and its first sequence.
template <int kThreads, class M>
__device__ __forceinline__ void make_plan(const Params& p, M& ms) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, B = p.a.batch;
  const int per_thread = (B + kThreads - 1) / kThreads;
  const int first = min(tid * per_thread, B), last = min(first + per_thread, B);
  int64_t sum = 0;
#pragma unroll 1
  for (int b = first; b < last; ++b) {
    sum += cost_of(length_of(p, b));
    if (blockIdx.x == 0 && p.a.seq_lens[b] > room_of(p.a)) flag_error(p.a.error_word, MLA_DEVERR_BOUNDS);
  }
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) ms.scan[warp] = incl;
  __syncthreads();
  int64_t total = 0, off = incl - sum;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) off += ms.scan[i];
    total += ms.scan[i];
  }
  const int64_t per = (total + gridDim.x - 1) / gridDim.x, t0 = blockIdx.x * per;
  if (tid == 0) {
    ms.t0 = t0;
    ms.t1 = t0 + per < total ? t0 + per : total;
  }
#pragma unroll 1
  for (int b = first; b < last; ++b) {
    const int len = length_of(p, b), n = cost_of(len);
    if (t0 >= off && t0 < off + n) {
      ms.b0 = b;
      ms.len0 = len;
      ms.off0 = off;
    }
    off += n;
  }
}

template <int kH>
__global__ void __launch_bounds__(kThreads<kH>, 1)
    fp8_key_weights_kernel(const __grid_constant__ CUtensorMap tm_lat, const __grid_constant__ CUtensorMap tm_rope,
                           const __grid_constant__ Params p) {
  using C = Cfg<kH>;
  constexpr int kQueryWarps = 4 * kGroups<kH>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc<kH>& ms = *reinterpret_cast<Misc<kH>*>(smem + C::off_misc);
  const uint32_t s0 = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = min(kH, p.a.num_heads - p.h0);
  uint32_t* err = p.a.error_word;

  if (threadIdx.x == 0) {
    ms.abort = 0;
    ms.b0 = p.a.batch;  // a part without tiles
    ms.off0 = 0;
    for (int i = 0; i < C::slots; ++i) {
      mbar_init(&ms.full[i], 1);
      mbar_init(&ms.empty[i], 1);
    }
    for (int i = 0; i < kInfo; ++i) mbar_init(&ms.info_full[i], 1);
    for (int i = 0; i < kGroups<kH>; ++i) mbar_init(&ms.s_full[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&ms.s_free[i], 4);
    mbar_init(&ms.q_ready, kQueryWarps);
    mbar_init(&ms.q_free, 1);
    mbar_init(&ms.retired, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ms.tmem, C::columns);
    tmem_relinquish();
  }
  // The next call's CTAs may take the place of those that end; nothing is read
  // before the work ahead of this call is done.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();  // (b0 is set before the plan)
  make_plan<kThreads<kH>>(p, ms);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms.tmem;
  // chunk c of tile n (4: the RoPE)
  auto slot_addr = [&](int n, int c) {
    return c < 4 ? s0 + (n % C::tiles * 4 + c) * kChunkBytes : s0 + C::off_rope + n % C::tiles * kRopeBytes;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tmap(&tm_lat);
      prefetch_tmap(&tm_rope);
    }
    int n = 0, copies = 0;  // tiles; of them with this lane's chunk asked for
    bool ok = true;
    const int per_page = p.a.page_size / kBlock;
    for (Pieces it(p, ms); ok && it.next(p);) {
      const int s = it.s, e = it.e, n_blocks = min((it.len + kBlock - 1) / kBlock, 2 * e);
      const int32_t* table = p.a.page_table + it.b * p.a.pt_stride;
      // 32 blocks (16 tiles) at a time, one a lane: the block's first slot
      // (past the cache where there is none, so that it reads as zeros) and its
      // scale.  The next 32 page table entries are loaded ahead.
      auto page_of = [&](int i) { return i < n_blocks ? table[div_magic(i, p.page_magic, p.page_shift)] : -1; };
      int page = page_of(2 * s + lane), y = 0;
      float scale = 0.f;
#pragma unroll 1
      for (int t = s; t < e && ok; ++t, ++n) {
        const int at = (2 * (t - s)) & 31;
        if (at == 0) {
          const int i = 2 * t + lane, in = i - static_cast<int>(div_magic(i, p.page_magic, p.page_shift)) * per_page;
          const int64_t slot = static_cast<int64_t>(page) * p.a.page_size + static_cast<int64_t>(in) * kBlock;
          const bool there = page >= 0 && slot + kBlock <= p.a.num_slots;
          page = page_of(i + 32);
          y = static_cast<int>(there ? slot : p.a.num_slots);
          scale = there ? p.a.scales[slot / kBlock] : 0.f;
        }
        const int y0 = __shfl_sync(0xffffffffu, y, at), y1 = __shfl_sync(0xffffffffu, y, at + 1);
        if (lane < 5) {  // a chunk a lane
          const int c = lane, i = n % C::tiles * 5 + c;
          ok = mbar_wait(&ms.empty[i], ((n / C::tiles) & 1) ^ 1, err, &ms.abort);
          if (ok) {
            const uint32_t bytes = c < 4 ? kChunkBytes : kRopeBytes, dst = slot_addr(n, c);
            const CUtensorMap* map = c < 4 ? &tm_lat : &tm_rope;
            mbar_expect_tx(&ms.full[i], bytes);
            tma_load_bytes(dst, map, 128 * c, y0, &ms.full[i]);
            tma_load_bytes(dst + bytes / 2, map, 128 * c, y1, &ms.full[i]);
            ++copies;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        // the scales (waited for after the copies); the place of tile n - 4,
        // whose sums are done: this tile's chunks took those of a later one
        if (at == 0) {
          const bool block = 2 * t + lane < n_blocks, good = scale >= kFp8ScaleMin && scale <= kFp8ScaleMax;
          if (block && !good && p.h0 == 0) flag_error(err, y == p.a.num_slots ? MLA_DEVERR_BOUNDS : MLA_DEVERR_SCALE);
          if (!good) scale = 0.f;
        }
        const float sc0 = __shfl_sync(0xffffffffu, scale, at), sc1 = __shfl_sync(0xffffffffu, scale, at + 1);
        if (lane == 0 && ok) {
          ms.scale[n % kInfo][0] = sc0;
          ms.scale[n % kInfo][1] = sc1;
          mbar_arrive(&ms.info_full[n % kInfo]);
        }
        ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0) != 0;
      }
    }
    // (chunk c of tile n is copy 5 n + c; of the last tile some lanes may have given up)
    copies = __reduce_max_sync(0xffffffffu, copies);
    if (lane == 0) ms.copies = 5 * copies;
  } else if (warp == 1) {
    // ------------------------------------------------------------- products
    // The loop is short: all chunks in one copy, descriptors by additions, and
    // what a wait says told to the warp once a tile (products of chunks that never
    // came are never read; with a vote a chunk the issue took a microsecond a tile).
    constexpr uint32_t idesc = idesc_e4m3(128, 2 * kH, false, false);
    const uint64_t dq = smem_desc_sw128(s0 + C::off_q, 0, 1024), dk = smem_desc_sw128(s0, 0, 1024);
    const uint64_t dq_rope = smem_desc_sw64(s0 + C::off_q + 4 * 2 * kH * 128, 512), dk_rope = smem_desc_sw64(s0 + C::off_rope, 512);
    auto ready = [&](uint64_t* bar, int parity) { return mbar_test(bar, parity) || mbar_wait(bar, parity, err, &ms.abort); };
    bool ok = true;
    int n = 0, piece = 0;
    for (Pieces it(p, ms); ok && it.next(p); ++piece) {
      ok = __all_sync(0xffffffffu, ready(&ms.q_ready, piece & 1));
      tc_fence_after();
#pragma unroll 1
      for (int t = it.s; ok && t < it.e; ++t, ++n) {
        const int half = uniform(n & 1), place = C::tiles == 2 ? half : 0;  // of its scores, its chunks
        const uint32_t d = tmem + half * 2 * kH;
        ok = ready(&ms.s_free[half], ((n >> 1) & 1) ^ 1);
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 5; ++c) {
          ok &= ready(&ms.full[5 * place + c], (n / C::tiles) & 1);
          __syncwarp();
          if (elect_one()) {
            if (c < 4) {
              const uint64_t da = dk + (4 * place + c) * (kChunkBytes >> 4), db = dq + c * (2 * kH * 128 >> 4);
#pragma unroll
              for (int j = 0; j < 4; ++j) mma_e4m3(d, da + 2 * j, db + 2 * j, idesc, (c > 0 || j > 0) ? 1u : 0u);
            } else {
              const uint64_t da = dk_rope + place * (kRopeBytes >> 4);
#pragma unroll
              for (int j = 0; j < 2; ++j) mma_e4m3(d, da + 2 * j, dq_rope + 2 * j, idesc, 1u);
            }
            mma_commit(&ms.empty[5 * place + c]);
            if (c == 4) {
              mma_commit(&ms.s_full[n % kGroups<kH>]);
              if (t + 1 == it.e) mma_commit(&ms.q_free);
            }
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
    }
    retire_products(&ms.retired, err);
  } else {
    // ------------------------------------------------------- queries, sums
    // A wait that gives up leaves these warps running through their loops; the
    // error word tells.
    const int quad = warp & 3, group = (warp - 2) >> 2, key = quad * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    int n = 0, piece = 0;
    for (Pieces it(p, ms); it.next(p); ++piece) {
      const int b = it.b, len = it.len;
      const int64_t row0 = static_cast<int64_t>(b) * p.a.num_heads + p.h0;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.a.q) + row0 * kKey;
      float2* head = ms.head[piece & 1];
      constexpr int kMine = kH / kQueryWarps;
      constexpr int kN = kMine > 4 ? 2 : kMine;  // heads at a time (of 128 two, the next two's loads in flight)
      QueryHeads<kN> mine;
      mine.load(q, lane, warp - 2, kQueryWarps, heads);
      const float lse = lane < kMine && warp - 2 + lane * kQueryWarps < heads
                            ? p.a.lse[row0 + warp - 2 + lane * kQueryWarps] * kLog2e
                            : INFINITY;  // (no head: its weights are 2^-inf)
      if (piece > 0) mbar_wait(&ms.q_free, (piece - 1) & 1, err, &ms.abort);
#pragma unroll 1
      for (int j0 = 0; j0 < kMine; j0 += kN) {
        const int h0 = warp - 2 + j0 * kQueryWarps;
        const QueryHeads<kN> now = mine;
        if (kMine > kN) mine.load(q, lane, h0 + kN * kQueryWarps, kQueryWarps, heads);
        float c[kN];
        query_terms<kH>(now, lane, h0, kQueryWarps, s0 + C::off_q, p.a.softmax_scale, c);
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          const int h = h0 + j * kQueryWarps;
          if (lane == j0 + j) head[h] = make_float2(h < heads ? c[j] : 0.f, lse);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.q_ready);
      mbar_wait(&ms.q_ready, piece & 1, err, &ms.abort);  // (all heads' factors)

#pragma unroll 1
      for (int t = it.s; t < it.e; ++t, ++n) {
        if (n % kGroups<kH> != group) continue;
        const int at = t * kTile + key;
        float before = 0.f;
        if (p.a.weights != nullptr && at < len) before = p.a.weights[b * p.a.weights_stride + at];
        mbar_wait(&ms.info_full[n % kInfo], (n / kInfo) & 1, err, &ms.abort);
        const float scale = ms.scale[n % kInfo][quad >> 1];
        mbar_wait(&ms.s_full[group], (n / kGroups<kH>) & 1, err, &ms.abort);
        tc_fence_after();
        const uint32_t src = lanes + (n & 1) * 2 * kH;
        float sum[4] = {};
#pragma unroll
        for (int g = 0; g < kH; g += 16) {
          uint32_t v[16], u[16];
          tmem_ld16(src + g, v);
          tmem_ld16(src + kH + g, u);
          tmem_ld_wait();
          if (g + 16 == kH) {  // the scores' place is free
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.s_free[n & 1]);
          }
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float4 f = *reinterpret_cast<const float4*>(&head[g + i]);
            const float x0 = fmaf(__uint_as_float(u[i]), 1.f / kGain, __uint_as_float(v[i])) * scale;
            const float x1 = fmaf(__uint_as_float(u[i + 1]), 1.f / kGain, __uint_as_float(v[i + 1])) * scale;
            sum[i & 3] += ex2_approx(fmaf(x0, f.x, -f.y));
            sum[(i + 1) & 3] += ex2_approx(fmaf(x1, f.z, -f.w));
          }
        }
        const float all = (sum[0] + sum[1]) + (sum[2] + sum[3]);
        if (at < len) p.a.out[b * p.a.out_stride + at] = before + (scale > 0.f ? all : 0.f);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::columns);
  if (warp == 0 && lane == 0 && ms.abort) drain_copies(ms.full, C::slots, ms.copies);
}

template <int kH>
int launch(const Params& p, const CUtensorMap& lat, const CUtensorMap& rope, int slot, int ctas, cudaStream_t stream) {
  constexpr int bytes = static_cast<int>(smem_bytes<kH>());
  const auto kern = fp8_key_weights_kernel<kH>;
  if (const int st = smem_limit_once(reinterpret_cast<const void*>(kern), bytes, slot)) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads<kH>);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // (griddepcontrol)
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, kern, lat, rope, p));
}

}  // namespace

int launch_fp8_key_weights(const Fp8WeightsArgs& a, cudaStream_t stream, int num_sms) {
  Params p{a, 0, 0, 0};
  magic_divisor(a.page_size / kBlock, &p.page_magic, &p.page_shift);
  CUtensorMap lat, rope;
  if (!encode_byte_map(&lat, a.cache, kKey, a.num_slots, kKey, 128, kBlock, false) ||
      !encode_byte_map(&rope, a.cache, kKey, a.num_slots, kKey, 64, kBlock, true)) {
    set_last_error("cuTensorMapEncodeTiled failed for the cache");
    return MLA_ERR_LAUNCH;
  }
  for (; p.h0 < a.num_heads; p.h0 += 128) {
    const int heads = a.num_heads - p.h0;
    const int st = heads <= 16   ? launch<16>(p, lat, rope, 32, num_sms, stream)
                   : heads <= 32 ? launch<32>(p, lat, rope, 33, num_sms, stream)
                   : heads <= 64 ? launch<64>(p, lat, rope, 34, num_sms, stream)
                                 : launch<128>(p, lat, rope, 35, num_sms, stream);
    if (st != MLA_OK) return st;
    // the next heads are added to these
    p.a.weights = a.out;
    p.a.weights_stride = a.out_stride;
  }
  return MLA_OK;
}

}  // namespace mla
