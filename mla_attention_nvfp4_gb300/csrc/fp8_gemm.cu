// e4m3 GEMM with scales per block of 128, and the activations' quantiser.
#include <cuda.h>
#include <cuda_runtime.h>

#include "encode_tiled.h"
#include "fp8.cuh"
#include "launch.h"
#include "nvfp4.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kGroup = MLA_FP8_GROUP;

// ---------------------------------------------------------------------------
// Quantiser: bf16 [M, K] -> e4m3 codes and one fp32 scale per 128 features.
// 8 lanes hold a group, 16 features each (two 16-byte loads, one 16-byte
// store; 8 features where K asks for it); two groups in flight per 8 lanes.
// HBM-bound, but only with few instructions an element: maxima on bf16
// pairs, quotients on pairs of floats.  8192 x 16384: 64.5 us (6.3 TB/s; 75 with
// one element at a time); 64 x 7168: 2.1 us.
// x / scale is rounded to nearest by Markstein's method: with y = 1 / scale
// rounded to nearest and q0 = x y, the remainder x - q0 scale is exact in one
// fused multiply-add (tiny groups are scaled up for that), and q0 + y remainder
// is the quotient, rounded once.
// ---------------------------------------------------------------------------
constexpr int kQuantThreads = 256;
constexpr int kQuantUnroll = 2;
constexpr int kQuantGroups = kQuantThreads / 8 * kQuantUnroll;  // groups per CTA

__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t times_2_64(uint32_t a) {
  const __nv_bfloat162 r =
      __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), __float2bfloat162_rn(18446744073709551616.f));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__global__ void __launch_bounds__(kQuantThreads) fp8_quantize_kernel(const __nv_bfloat16* __restrict__ x,
                                                                     int64_t x_stride, int64_t K, int n_groups,
                                                                     int row_groups, uint32_t magic, int shift,
                                                                     uint8_t* __restrict__ codes,
                                                                     float* __restrict__ scales) {
  const int sub = threadIdx.x & 7;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kQuantGroups + (threadIdx.x >> 3);
  uint4 v[kQuantUnroll][2];
  int64_t at[kQuantUnroll];  // offset of this thread's codes
  int have[kQuantUnroll];    // 8-feature halves it holds
#pragma unroll
  for (int i = 0; i < kQuantUnroll; ++i) {
    const int64_t g = first + i * (kQuantThreads / 8);
    v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
    at[i] = 0;
    have[i] = 0;
    if (g < n_groups) {
      const int64_t m = div_magic(static_cast<uint32_t>(g), magic, shift), j = g - m * row_groups;
      const int64_t k = j * kGroup + 16 * sub;
      const uint4* src = reinterpret_cast<const uint4*>(x + m * x_stride + k);
      have[i] = k + 16 <= K ? 2 : k + 8 <= K ? 1 : 0;
      if (have[i] > 0) v[i][0] = src[0];
      if (have[i] > 1) v[i][1] = src[1];
      at[i] = m * K + k;
    }
  }
#pragma unroll
  for (int i = 0; i < kQuantUnroll; ++i) {
    const int64_t g = first + i * (kQuantThreads / 8);
    uint32_t w[8] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w, v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
    uint32_t m2 = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m2 = max_abs2(m2, w[k] & 0x7FFF7FFFu);  // NaN gives the other operand
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m2 = max_abs2(m2, __shfl_xor_sync(0xffffffffu, m2, o));
    float lo, hi;
    bf16x2_to_f32(m2, lo, hi);
    float am = fmaxf(lo, hi), least = 1.1754943508222875e-38f, down = 1.f;
    if (__builtin_expect(am < 2.42861286636753e-17f, 0)) {  // 448 * 2^-64
      // A tiny group times 2^64, exactly, with the same quotients: the exact
      // remainder reaches 2^-46 below a numerator, and fp32 ends at 2^-149.
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = times_2_64(w[k]);
      am *= 18446744073709551616.f;
      least *= 18446744073709551616.f;
      down = 5.421010862427522e-20f;
    }
    // both quotients rounded to nearest, from correctly rounded reciprocals
    // (div_rn); 1 / 448 rounded is a constant
    const float den = isinf(am) ? am : fmaxf(div_rn(am, 448.f, 0.0022321429569274187f), least);
    const float scale = den * down;
    const float inv = __frcp_rn(den);
    const uint64_t ninv2 = pack2(-inv, -inv), den2 = pack2(den, den);
    uint32_t out[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t code = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float a, b;
        bf16x2_to_f32(w[2 * k + j], a, b);
        // everything with 1 / -scale, the quotient's sign turned at the end: a
        // remainder of zero then leaves -0 as it is
        const uint64_t num = pack2(a, b);
        const uint64_t q0 = mul2(num, ninv2);
        uint64_t r = num;
        fma2(r, q0, den2);  // the exact remainder
        uint64_t q = q0;
        fma2(q, r, ninv2);
        unpack2(isinf(den) ? q0 : q, a, b);
        code |= cvt_e4m3x2(-a, -b) << (16 * j);
      }
      out[k] = code;
    }
    if (have[i] == 2 && (K & 15) == 0) {
      *reinterpret_cast<uint4*>(codes + at[i]) = make_uint4(out[0], out[1], out[2], out[3]);
    } else {
      if (have[i] > 0) *reinterpret_cast<uint2*>(codes + at[i]) = make_uint2(out[0], out[1]);
      if (have[i] > 1) *reinterpret_cast<uint2*>(codes + at[i] + 8) = make_uint2(out[2], out[3]);
    }
    if (sub == 0 && g < n_groups) scales[g] = scale;
  }
}

// ---------------------------------------------------------------------------
// GEMM.  The scales vary along K, so the tensor cores' accumulator holds one
// block of 128 features at a time and the epilogue warps add it, scaled, to
// fp32 sums in registers, while the next block's products fill the other
// accumulator.
//
// Large: 128 x 256 outputs per tile, persistent CTAs.
//   warp 0        TMA producer: A and W tiles of one K block, 128-byte swizzle,
//                 kStages in flight;
//   warps 1, 2    MMA issuers, one an accumulator: four products of K = 32 per
//                 block;
//   warps 4..11   sums: warps 4..7 columns 0..127, warps 8..11 columns 128..255
//                 (each half has one weight scale per block), thread = row;
//                 they take the registers the first warpgroup gives up
//                 (128 sums, 32 columns being added and 32 being loaded each).
// 4096 x 7168 x 16384: 363 to 384 us from run to run, as power allows, 2500 to
// 2650 TFLOP/s (457 us with one issuer and each load waited for before its sums;
// the pairs below compare two forms at one time).  A K block takes 520 cycles of products
// by themselves, and 920 here, where 48 KB are copied into shared memory as 48
// are read from it: 512 rows take 59 us with the sums and without them.  A CTA
// pair's 256 x 256 tile halves the weights' part of that and takes as long (60
// us; its products alone 45), for then the sums bound it: 128 multiply-adds a
// thread and block beside the scales' loads and waits of 100 to 140 cycles.
// Sixteen sum warps of 64 columns: 413 us, not 360; sums on pairs (f32x2) and
// accumulators freed before two thirds of the sums: the same; the next
// accumulator asked for ahead: 389, not 360; row scales staged in shared memory: 73, not
// 59, for 512 rows.
// ---------------------------------------------------------------------------
constexpr int kBM = 128, kBN = 256;
constexpr int kStages = 4;
constexpr int kThreads = 384;
constexpr int kRegsIssue = 40, kRegsSum = 232;  // of 168 x 3 warpgroups at launch
constexpr uint32_t kABytes = kBM * kGroup, kWBytes = kBN * kGroup;
constexpr uint32_t kStageBytes = kABytes + kWBytes;
constexpr uint32_t kRowBytes = 32 * 128;  // a sum warp's rows on their way out
constexpr uint32_t kSmAlloc = kStages * kStageBytes + 1024, kSmAllocRows = kSmAlloc + 8 * kRowBytes;
constexpr int kRaster = 8;  // row tiles that share the weights passing through L2
static_assert(kSmAllocRows + 512 <= 232448, "shared memory budget");

struct Params {
  const float* a_scales;
  const float* w_scales;
  int64_t M, N, ldc;
  int kb;  // blocks of 128 features
  __nv_bfloat16* c;
  int tiles_m, tiles_n;
  uint32_t* error_word;
};

// Tile t: groups of kRaster row tiles, inside a group column by column.
__device__ __forceinline__ void tile_of(int t, int tiles_m, int tiles_n, int& mt, int& nt) {
  const int group = t / (kRaster * tiles_n);
  const int rows = min(kRaster, tiles_m - group * kRaster);
  const int in = t - group * kRaster * tiles_n;
  mt = group * kRaster + in % rows;
  nt = in / rows;
}

struct alignas(8) Barriers {
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], retired[2];
};

// kSectors: the output's rows begin at multiples of 32 bytes.  (Both endings
// in one kernel: 4096 x 7168 x 16384 386 us, not 357.)
template <bool kSectors>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Barriers bars;
  __shared__ uint32_t tmem_base_s;
  __shared__ volatile int abort_s;
  __shared__ int issued_s;  // K blocks whose copies were
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t s0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int n_tiles = p.tiles_m * p.tiles_n;
  uint32_t* err = p.error_word;

  if (threadIdx.x == 0) {
    abort_s = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.acc_full[i], 1);
      mbar_init(&bars.acc_empty[i], 8);
      mbar_init(&bars.retired[i], 1);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_s, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_s;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == 0 && lane == 0) {
      prefetch_tmap(&tm_a);
      prefetch_tmap(&tm_w);
      int it = 0;
      for (int t = blockIdx.x; t < n_tiles && !abort_s; t += gridDim.x) {
        int mt, nt;
        tile_of(t, p.tiles_m, p.tiles_n, mt, nt);
        for (int kb = 0; kb < p.kb; ++kb, ++it) {
          const int s = it % kStages;
          if (!mbar_wait(&bars.empty[s], ((it / kStages) & 1) ^ 1, err, &abort_s)) break;
          mbar_expect_tx(&bars.full[s], kStageBytes);
          tma_load_bytes(s0 + s * kStageBytes, &tm_a, kb * kGroup, mt * kBM, &bars.full[s]);
          tma_load_bytes(s0 + s * kStageBytes + kABytes, &tm_w, kb * kGroup, nt * kBN, &bars.full[s]);
        }
      }
      issued_s = it;
    } else if (warp == 1 || warp == 2) {
      // An issuer for each accumulator, every other K block: one alone takes
      // longer to get from one block's products to the next one's (its waits
      // and commits, about 900 cycles) than these run (520).
      constexpr uint32_t idesc = idesc_e4m3(kBM, kBN, false, false);
      const int buf = uniform(warp - 1);
      const uint32_t d = uniform(tmem + buf * kBN);
      const int mine = n_tiles > static_cast<int>(blockIdx.x) ? (n_tiles - 1 - blockIdx.x) / gridDim.x + 1 : 0;
      const int64_t blocks = static_cast<int64_t>(mine) * p.kb;
      for (int64_t i = buf; i < blocks; i += 2) {
        const uint32_t it = static_cast<uint32_t>(i);
        const int s = uniform(it % kStages);
        const uint64_t da = smem_desc_sw128(s0 + s * kStageBytes, 0, 1024);
        const uint64_t db = smem_desc_sw128(s0 + s * kStageBytes + kABytes, 0, 1024);
        // (a stage is always the same issuer's, so its phases come in turn)
        static_assert(kStages % 2 == 0, "stages alternate between the issuers");
        if (!__all_sync(0xffffffffu, mbar_wait(&bars.full[s], (it / kStages) & 1, err, &abort_s) &&
                                         mbar_wait(&bars.acc_empty[buf], ((it >> 1) & 1) ^ 1, err, &abort_s)))
          break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < 4; ++j)  // 32 bytes a step along the swizzled row
            mma_e4m3(d, da + 2 * j, db + 2 * j, idesc, j > 0 ? 1u : 0u);
          mma_commit(&bars.acc_full[buf]);
          mma_commit(&bars.empty[s]);
        }
        __syncwarp();
      }
      retire_products(&bars.retired[buf], err);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSum));
    const int quad = warp & 3, half = (warp - 4) >> 2;  // TMEM lane quarter; column half
    const int r = quad * 32 + lane;
    const uint32_t src = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * 128;
    int it = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < n_tiles; t += gridDim.x) {
      int mt, nt;
      tile_of(t, p.tiles_m, p.tiles_n, mt, nt);
      const int64_t row = static_cast<int64_t>(mt) * kBM + r, col0 = static_cast<int64_t>(nt) * kBN + half * 128;
      const bool live = row < p.M && col0 < p.N;
      const float* as = p.a_scales + (live ? row : 0) * p.kb;
      const float* ws = p.w_scales + (live ? col0 / kGroup : 0) * p.kb;
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.f;
      // scales two blocks ahead of their use (multiplied only there)
      const int last = p.kb - 1;
      float a0 = as[0], w0 = ws[0], a1 = as[min(1, last)], w1 = ws[min(1, last)];
      // 32 columns at a time, the next ones' load under the current ones' sums
      // (the next block's too)
      uint32_t v[32], u[32];
      auto add = [&](const uint32_t(&x)[32], int c, float sc) {
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[32 * c + i] = fmaf(__uint_as_float(x[i]), sc, acc[32 * c + i]);
      };
      auto filled = [&](int at) {
        const bool in = mbar_wait(&bars.acc_full[at & 1], (at >> 1) & 1, err, &abort_s);
        tc_fence_after();
        return __all_sync(0xffffffffu, in) != 0;  // (a wait may give up in some lanes only)
      };
      ok = filled(it);
      if (ok) {
        tmem_ld32(src + (it & 1) * kBN, v);
        tmem_ld_wait(v);
      }
      for (int kb = 0; ok && kb < p.kb; ++kb, ++it) {
        const uint32_t at = src + (it & 1) * kBN;
        const float a2 = as[min(kb + 2, last)], w2 = ws[min(kb + 2, last)];
        const float sc = a0 * w0;
        tmem_ld32(at + 32, u);
        add(v, 0, sc);
        tmem_ld_wait(u);
        tmem_ld32(at + 64, v);
        add(u, 1, sc);
        tmem_ld_wait(v);
        tmem_ld32(at + 96, u);
        add(v, 2, sc);
        tmem_ld_wait(u);
        tc_fence_before();  // the accumulator may be filled again
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.acc_empty[it & 1]);
        const bool more = kb < last;
        if (more) {
          ok = filled(it + 1);
          if (ok) tmem_ld32(src + ((it + 1) & 1) * kBN, v);
        }
        add(u, 3, sc);
        if (more) tmem_ld_wait(v);
        a0 = a1;
        w0 = w1;
        a1 = a2;
        w1 = w2;
      }
      if (!ok || col0 >= p.N) continue;
      const int n = p.N - col0 < 128 ? static_cast<int>(p.N - col0) : 128;
      if constexpr (kSectors) {
        // whole sectors, 32 bytes a store
        __nv_bfloat16* dst = p.c + row * p.ldc + col0;
        if (row < p.M) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float* f = acc + 16 * i;
            if (16 * i + 16 <= n) {
              uint32_t w[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) w[j] = bf16x2_pack(f[2 * j], f[2 * j + 1]);
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 16 * i), "r"(w[0]),
                           "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                           : "memory");
            } else {
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (16 * i + j < n) dst[16 * i + j] = __float2bfloat16_rn(f[j]);
            }
          }
        }
      } else {
        // Rows at any address: 64 columns at a time through shared memory
        // (16-byte units swizzled by the row), so that a warp writes
        // neighbouring columns of one row (4096 x 7160 x 512: one thread's
        // row by itself, 187 us).
        const uint32_t stage = s0 + kStages * kStageBytes + (warp - 4) * kRowBytes;
        const int rows = static_cast<int>(min(int64_t{32}, p.M - (row - lane)));
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          __syncwarp();  // the part before has been read
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float* f = acc + 64 * part + 8 * i;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * 128 + ((i ^ (lane & 7)) << 4)),
                         "r"(bf16x2_pack(f[0], f[1])), "r"(bf16x2_pack(f[2], f[3])), "r"(bf16x2_pack(f[4], f[5])),
                         "r"(bf16x2_pack(f[6], f[7]))
                         : "memory");
          }
          __syncwarp();
          const int c = 64 * part + 2 * lane;
          uint16_t* dst = reinterpret_cast<uint16_t*>(p.c) + (row - lane) * p.ldc + col0 + c;
          for (int r = 0; r < rows; ++r, dst += p.ldc) {
            uint32_t w;
            asm volatile("ld.shared.b32 %0, [%1];"
                         : "=r"(w)
                         : "r"(stage + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4)
                         : "memory");
            if (c + 1 < n && (reinterpret_cast<uintptr_t>(dst) & 3u) == 0) {
              *reinterpret_cast<uint32_t*>(dst) = w;
            } else {
              if (c < n) dst[0] = static_cast<uint16_t>(w);
              if (c + 1 < n) dst[1] = static_cast<uint16_t>(w >> 16);
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
  if (warp == 0 && lane == 0 && abort_s) drain_copies(bars.full, kStages, issued_s);
}

// ---------------------------------------------------------------------------
// Few rows: the weights are the tensor cores' 128-row operand and kT tokens
// the other one (N = kT), so that few tokens cost few products and the
// weights stream through; the K blocks of a tile are split over a cluster's
// CTAs, whose fp32 sums are added through distributed shared memory in rank
// order.
//   warp 0 producer, warp 1 and the last one MMA issuers, between them four
//   warps of sums per 64 tokens: thread = weight row.
// N 7168, K 16384: 16 rows 23 us, 64 rows 25.8 (4.6 TB/s), 128 rows 36;
// 1 x 576 x 7168: 5.3 us, of which the launch takes half.
// ---------------------------------------------------------------------------
constexpr int kMaxSplits = 8;   // portable cluster size
constexpr int kScaleBlocks = 16;  // K blocks whose scales are staged at a time

template <int kT>
struct Small {
  static constexpr int halves = kT == 128 ? 2 : 1, tokens = kT / halves;  // groups of sum warps, tokens of each
  static constexpr int sum_threads = 128 * halves, threads = 96 + sum_threads;
  static constexpr int resident = kT <= 32 ? 3 : kT == 64 ? 2 : 1;  // CTAs an SM holds
  static constexpr int stages = kT == 16 ? 4 : kT == 32 ? 3 : kT == 64 ? 4 : 6;
  static constexpr uint32_t w_bytes = 128 * kGroup, t_bytes = kT * kGroup, stage_bytes = w_bytes + t_bytes;
  static constexpr uint32_t sum_bytes = kT * 128 * 4;
  static constexpr uint32_t pipe = stages * stage_bytes;
  static constexpr uint32_t alloc = (pipe > sum_bytes ? pipe : sum_bytes) + 1024;
  static constexpr uint32_t cols = 2 * kT;
};

__device__ __forceinline__ float4 ld_cluster(uint32_t addr, uint32_t rank) {
  uint32_t remote;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(remote)
               : "memory");
  return v;
}

// grid (splits, weight tiles, token tiles), cluster (splits, 1, 1)
template <int kT>
__global__ void __launch_bounds__(Small<kT>::threads, Small<kT>::resident)
    fp8_gemm_small_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                          const Params p) {
  using S = Small<kT>;
  constexpr int kTok = S::tokens;
  extern __shared__ uint8_t smem_raw[];
  __shared__ struct alignas(8) {
    uint64_t full[S::stages], empty[S::stages], acc_full[2], acc_empty[2], retired[2];
  } bars;
  __shared__ alignas(16) float scale_s[kScaleBlocks][kT];
  __shared__ uint32_t tmem_base_s;
  __shared__ volatile int abort_s;
  __shared__ int issued_s;  // K blocks whose copies were
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t s0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int splits = gridDim.x, rank = blockIdx.x;
  const int n0 = blockIdx.y * 128, m0 = blockIdx.z * kT;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.kb) * rank / splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.kb) * (rank + 1) / splits);
  uint32_t* err = p.error_word;

  if (threadIdx.x == 0) {
    abort_s = 0;
    for (int s = 0; s < S::stages; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.acc_full[i], 1);
      mbar_init(&bars.acc_empty[i], 4 * S::halves);
      mbar_init(&bars.retired[i], 1);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_s, S::cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_s;

  const int half = (warp - 2) >> 2;  // of the sum warps
  uint64_t acc[kTok / 2];
#pragma unroll
  for (int i = 0; i < kTok / 2; ++i) acc[i] = 0;
  if (warp == 0) {
    if (lane == 0) {
      prefetch_tmap(&tm_a);
      prefetch_tmap(&tm_w);
      int it = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % S::stages;
        if (!mbar_wait(&bars.empty[s], ((it / S::stages) & 1) ^ 1, err, &abort_s)) break;
        mbar_expect_tx(&bars.full[s], S::stage_bytes);
        tma_load_bytes(s0 + s * S::stage_bytes, &tm_w, kb * kGroup, n0, &bars.full[s]);
        tma_load_bytes(s0 + s * S::stage_bytes + S::w_bytes, &tm_a, kb * kGroup, m0, &bars.full[s]);
      }
      issued_s = it;
    }
  } else if (warp == 1 || warp == S::threads / 32 - 1) {
    // an issuer for each accumulator, as above
    constexpr uint32_t idesc = idesc_e4m3(128, kT, false, false);
    const int buf = uniform(warp == 1 ? 0 : 1);
    const uint32_t d = uniform(tmem + buf * kT);
    for (int it = buf; it < kb1 - kb0; it += 2) {
      const int s = uniform(it % S::stages);
      const uint64_t da = smem_desc_sw128(s0 + s * S::stage_bytes, 0, 1024);
      const uint64_t db = smem_desc_sw128(s0 + s * S::stage_bytes + S::w_bytes, 0, 1024);
      // The accumulator first: that block it - 2 is summed says that every
      // earlier block is in, so that the stage's phase is this block's or the
      // one before (an odd number of stages gives a stage to both issuers in
      // turn, and a wait tells phases apart by their parity alone).
      if (!__all_sync(0xffffffffu, mbar_wait(&bars.acc_empty[buf], ((it >> 1) & 1) ^ 1, err, &abort_s) &&
                                       mbar_wait(&bars.full[s], (it / S::stages) & 1, err, &abort_s)))
        break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_e4m3(d, da + 2 * j, db + 2 * j, idesc, j > 0 ? 1u : 0u);
        mma_commit(&bars.acc_full[buf]);
        mma_commit(&bars.empty[s]);
      }
      __syncwarp();
    }
    retire_products(&bars.retired[buf], err);
  } else {
    constexpr int kSumThreads = S::sum_threads;
    const int quad = warp & 3, tid = threadIdx.x - 64;
    const uint32_t src = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * kTok;
    const float* ws = p.w_scales + static_cast<int64_t>(blockIdx.y) * p.kb;
    // scales of the next kScaleBlocks blocks: token by token along K
    constexpr int kPer = kScaleBlocks * kT / kSumThreads;
    float next[kPer];
    auto fetch = [&](int kb_at) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int idx = i * kSumThreads + tid, kb = kb_at + idx % kScaleBlocks;
        const int64_t m = m0 + idx / kScaleBlocks;
        next[i] = (kb < kb1 && m < p.M) ? p.a_scales[m * p.kb + kb] * ws[kb] : 0.f;
      }
    };
    fetch(kb0);
    for (int kb = kb0, it = 0; kb < kb1; ++kb, ++it) {
      const int j = it % kScaleBlocks, buf = it & 1;
      if (j == 0) {
        asm volatile("bar.sync 1, %0;" ::"n"(kSumThreads) : "memory");  // the previous blocks' scales have been read
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int idx = i * kSumThreads + tid;
          scale_s[idx % kScaleBlocks][idx / kScaleBlocks] = next[i];
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kSumThreads) : "memory");
        if (kb + kScaleBlocks < kb1) fetch(kb + kScaleBlocks);
      }
      // a wait that gives up still takes part in the barriers above
      mbar_wait(&bars.acc_full[buf], (it >> 1) & 1, err, &abort_s);
      tc_fence_after();
      constexpr int kW = kTok < 32 ? kTok : 32;
#pragma unroll
      for (int c = 0; c < kTok / kW; ++c) {
        uint32_t v[kW];
        if constexpr (kW == 32)
          tmem_ld32(src + buf * kT + kW * c, v);
        else
          tmem_ld16(src + buf * kT + kW * c, v);
        tmem_ld_wait();
        if (c == kTok / kW - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.acc_empty[buf]);
        }
#pragma unroll
        for (int i = 0; i < kW / 4; ++i) {
          const float4 sc = *reinterpret_cast<const float4*>(&scale_s[j][half * kTok + kW * c + 4 * i]);
          fma2(acc[kW / 2 * c + 2 * i], pack2(v[4 * i], v[4 * i + 1]), pack2(sc.x, sc.y));
          fma2(acc[kW / 2 * c + 2 * i + 1], pack2(v[4 * i + 2], v[4 * i + 3]), pack2(sc.z, sc.w));
        }
      }
    }
  }

  // Results: thread = weight row (output column), tokens one after another:
  // a warp writes 32 neighbouring columns of one output row.
  const int r = (warp & 3) * 32 + lane;
  const int64_t n = static_cast<int64_t>(n0) + r;
  const bool sums = warp >= 2 && threadIdx.x < 64 + S::sum_threads;
  if (splits == 1) {
    if (sums && n < p.N) {
#pragma unroll
      for (int i = 0; i < kTok / 2; ++i) {
        float lo, hi;
        unpack2(acc[i], lo, hi);
        const int64_t m = m0 + half * kTok + 2 * i;
        if (m < p.M) p.c[m * p.ldc + n] = __float2bfloat16_rn(lo);
        if (m + 1 < p.M) p.c[(m + 1) * p.ldc + n] = __float2bfloat16_rn(hi);
      }
    }
  } else {
    // every product has read its operands (each sum waited for them), so the
    // stages' memory holds the sums [token][row]
    __syncthreads();
    if (sums) {
      const uint32_t at = s0 + (half * kTok * 128 + r) * 4;
#pragma unroll
      for (int i = 0; i < kTok / 2; ++i) {
        float lo, hi;
        unpack2(acc[i], lo, hi);
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + 1024 * i), "f"(lo) : "memory");
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + 1024 * i + 512), "f"(hi) : "memory");
      }
    }
    cluster_sync();
    const int live = static_cast<int>(p.M - m0 < kT ? p.M - m0 : kT);
    // four neighbouring columns of a row at a time
    for (int e = rank * S::threads + threadIdx.x; e < live * 32; e += splits * S::threads) {
      float4 v[kMaxSplits];
#pragma unroll
      for (int c = 0; c < kMaxSplits; ++c)
        if (c < splits) v[c] = ld_cluster(s0 + e * 16, c);
      float f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < kMaxSplits; ++c)
        if (c < splits) {
          f[0] += v[c].x;
          f[1] += v[c].y;
          f[2] += v[c].z;
          f[3] += v[c].w;
        }
      const int64_t col = static_cast<int64_t>(n0) + 4 * (e & 31);
      __nv_bfloat16* dst = p.c + (static_cast<int64_t>(m0) + (e >> 5)) * p.ldc + col;
      if (col + 4 <= p.N && (reinterpret_cast<uintptr_t>(dst) & 7u) == 0) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(bf16x2_pack(f[0], f[1]), bf16x2_pack(f[2], f[3]));
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (col + i < p.N) dst[i] = __float2bfloat16_rn(f[i]);
      }
    }
    cluster_sync();  // no CTA leaves while another reads its sums
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, S::cols);
  if (warp == 0 && lane == 0 && abort_s) drain_copies(bars.full, S::stages, issued_s);
}

template <int kT>
int launch_small(const CUtensorMap& tm_a, const CUtensorMap& tm_w, const Params& p, int splits, int slot,
                 cudaStream_t stream) {
  const void* kern = reinterpret_cast<const void*>(fp8_gemm_small_kernel<kT>);
  if (const int st = smem_limit_once(kern, static_cast<int>(Small<kT>::alloc), slot)) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(splits, p.tiles_n, p.tiles_m);
  cfg.blockDim = dim3(Small<kT>::threads);
  cfg.dynamicSmemBytes = Small<kT>::alloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = splits;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, fp8_gemm_small_kernel<kT>, tm_a, tm_w, p));
}

}  // namespace

int launch_fp8_quantize(const void* x, int64_t x_stride, int64_t M, int64_t K, uint8_t* codes, float* scales,
                        cudaStream_t stream) {
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

bool encode_byte_map(CUtensorMap* map, const void* base, int64_t width, int64_t rows, int64_t stride, uint32_t box_x,
                     uint32_t box_rows, bool swizzle64) {
  const EncodeTiledFn fn = encode_tiled_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride)};
  const cuuint32_t box[2] = {box_x, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int launch_fp8_gemm(const Fp8GemmArgs& a, cudaStream_t stream, int num_sms) {
  const int kb = static_cast<int>((a.K + kGroup - 1) / kGroup);
  const int64_t tm = (a.M + kBM - 1) / kBM, tn = (a.N + kBN - 1) / kBN;
  const int kt = a.M <= 16 ? 16 : a.M <= 32 ? 32 : a.M <= 64 ? 64 : 128;  // tokens of the streaming form's tile
  const int64_t sn = (a.N + 127) / 128, sm = (a.M + kt - 1) / kt;

  // Which form, and into how many parts K is cut, by an estimate in K blocks
  // of one streaming CTA's time (0.5 us), however many share its SM, until
  // together they take what HBM gives (kPerBlock blocks of 128 weights x 128
  // in the time of one); a wave of CTAs costs kOverhead blocks more, and a
  // large tile's block 7/8 of one.  Clusters do not fill every place an SM
  // offers: nine tenths count.  Measured, N 7168, K 16384: 64 rows, 34 us with
  // 2 parts, 25 with 4 (one wave each), 30 with 8 (two waves); 16 rows, 24 with
  // 4, 28 with 8; 128 rows, 36 us streaming, 58 as large tiles; 256 rows, 66
  // and 58; 512 rows, 127 and 59.  Over 77 shapes of 65 to 2048 rows the form
  // chosen was within 7 % of the faster one.
  constexpr int kOverhead = 6, kPerBlock = 200;
  const int64_t places = static_cast<int64_t>(num_sms) * (kt <= 32 ? 3 : kt == 64 ? 2 : 1) * 9 / 10;
  int splits = 1;
  int64_t best = INT64_MAX;
  for (int s = 1; s <= kMaxSplits && s <= kb; ++s) {
    const int64_t waves = (sn * sm * s + places - 1) / places;
    int64_t cost = waves * ((kb + s - 1) / s);
    if (cost < sn * sm * kb / kPerBlock) cost = sn * sm * kb / kPerBlock;
    cost += waves * kOverhead;
    if (cost < best) {
      best = cost;
      splits = s;
    }
  }
  // More tiles than a grid's second and third dimensions hold are large ones.
  const int64_t waves = (tm * tn + num_sms - 1) / num_sms;
  const bool large = sn > 65535 || sm > 65535 || (a.M > 64 && waves * kb * 7 / 8 + kOverhead < best);
  CUtensorMap tm_a, tm_w;
  if (!encode_byte_map(&tm_a, a.a, a.K, a.M, a.lda, kGroup, static_cast<uint32_t>(large ? kBM : kt), false) ||
      !encode_byte_map(&tm_w, a.w, a.K, a.N, a.ldw, kGroup, large ? kBN : 128, false)) {
    set_last_error("cuTensorMapEncodeTiled failed for the GEMM operands");
    return MLA_ERR_LAUNCH;
  }
  Params p{a.a_scales, a.w_scales, a.M, a.N, a.ldc, kb, static_cast<__nv_bfloat16*>(a.out), 0, 0, a.error_word};
  if (large) {
    if (tm * tn > int64_t(1) << 30) return MLA_ERR_INVALID_ARG;  // (a tile's index and a grid more fit an int)
    p.tiles_m = static_cast<int>(tm);
    p.tiles_n = static_cast<int>(tn);
    const int grid = static_cast<int>(tm * tn < num_sms ? tm * tn : num_sms);
    const bool sectors = ((reinterpret_cast<uintptr_t>(a.out) | static_cast<uintptr_t>(a.ldc * 2)) & 31u) == 0;
    const auto kern = sectors ? fp8_gemm_kernel<true> : fp8_gemm_kernel<false>;
    const uint32_t smem = sectors ? kSmAlloc : kSmAllocRows;
    if (const int st =
            smem_limit_once(reinterpret_cast<const void*>(kern), static_cast<int>(smem), sectors ? 14 : 23))
      return st;
    kern<<<grid, kThreads, smem, stream>>>(tm_a, tm_w, p);
    return launch_status();
  }
  p.tiles_m = static_cast<int>(sm);
  p.tiles_n = static_cast<int>(sn);
  switch (kt) {
    case 16: return launch_small<16>(tm_a, tm_w, p, splits, 15, stream);
    case 32: return launch_small<32>(tm_a, tm_w, p, splits, 16, stream);
    case 64: return launch_small<64>(tm_a, tm_w, p, splits, 17, stream);
    default: return launch_small<128>(tm_a, tm_w, p, splits, 18, stream);
  }
}

}  // namespace mla
