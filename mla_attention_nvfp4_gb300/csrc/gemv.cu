// bf16 rows times an NVFP4 weight matrix (one, or one a group):
//   out[m, g, n] = gs sum_k x[m, g, k] code[g, n, k] scale[g, n, k / 16].
//
// Every weight is 9/16 of a byte, read once for up to 16 rows: HBM would bound it
// (9.9 us for 7168 x 16384).  What does is the latency of the weights' conversion: of
// some 290 instructions a warp for 16 rows x 256 features 160 are the codes' conversion
// and the scales' products, in chains that four warps a scheduler do not hide (one row
// of x issues in 42 % of the cycles, 16 rows in 38 %; at full issue one row's would
// take 7 us), beside a start of 2.7 us and the clusters' sum of 2.4.  The sums run on
// mma.sync m16n8k16 (f16 operands, fp32 sums): weights are its 16 rows, x its 8 columns.
// (tcgen05 wants its operands in shared memory: f16 weights would be written there and
// read again.)
//   weights  code * scale has 6 significant bits between 2^-10 and 2688: exact in
//            f16.  A thread of a quad holds a quarter of a step's features of a row,
//            whole blocks of 16.  Which feature of an instruction they are is free,
//            as long as x agrees: its rows lie in shared memory in the order of the
//            fragments.
//   x        bf16 in f16, after a power of two a row and 256 features that brings
//            the largest to 2^14 or more: exact down to 2^-31 of it (f16's steps
//            are 2^-24), within 2^-39 of it below.  Infinities and NaN are kept.
// The 8 warps of a CTA take 16 or 32 rows each, or share rows and split the
// features of a stage; a cluster of up to 10 CTAs splits K, and its CTAs each add
// up and write a part of the rows: no workspace, and sums in a fixed order.
// Weights come by TMA into a ring (a box of lines of 128 or 64 bytes, and the
// scales as they lie), x is read ahead of them (asked for behind 25 MB of weights
// it came 5 us later).
// Times, calls overlapping in a graph: 1 x 7168 x 16384 17.9 us (3.7 TB/s), 16 rows
// 27.6, 1 x 576 x 7168 4.2, 4 rows of 128 matrices of 512 x 128 3.5, of 128 x 512 5.5,
// 16 x 1024 x 7168 8.6.  What was tried beside that: weights
// from global memory to registers (23.3 us), three CTAs an SM (clusters of 8 then
// fill the SMs one and a half times: 31 us), 16 warps a CTA (16 rows: 31.8 us).
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "fp8.cuh"
#include "launch.h"
#include "nvfp4.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxStages = 8;  // of weights in shared memory
constexpr int kCtas = 2;       // an SM
constexpr uint32_t kShare = (222 / kCtas) * 1024;  // of an SM's shared memory for each of them
constexpr uint32_t kLimit = 224 * 1024;            // of 227 KB, where a stage is large
constexpr int kMaxSplits = 10;                     // (above 8: not portable, asked for)

constexpr int kXBlock = 256;                       // features of a row of x that share a power of two
constexpr int kMinStages = 3;

// kGroups: of 16 rows a warp, for which it reads x once.
template <int kGroups>
struct Cfg {
  static constexpr int rows = 16 * kGroups * kWarps;  // of a row tile
  static constexpr int step = 256 / kGroups;          // features a warp takes at a time: a quarter a thread of a quad
  static constexpr uint32_t line = step / 2, code_bytes = rows * line, sf_bytes = step / 64 * 512;
  static constexpr int log = kGroups == 2 ? 5 : 4;    // of a warp's rows
  // a stage's bytes, with 2^row_log warps that have rows of their own
  static constexpr uint32_t stage(int row_log) {
    return code_bytes + (kWarps >> row_log) * ((1 << (log + row_log)) > 128 ? 2u : 1u) * sf_bytes;
  }
  // x's, a chunk: a row of a block for each warp at least, in whole stages
  __host__ __device__ static constexpr int chunk(int pad, int subs) {
    const int a = kXBlock / step / subs, b = kXBlock / step * kWarps / (pad * subs);
    return a > b ? (a > 1 ? a : 1) : (b > 1 ? b : 1);
  }
};

struct Params {
  GemvArgs a;
  int row_log;    // 2^row_log warps with rows of their own; the others take further steps of a stage
  int splits;     // CTAs a cluster
  int tiles;      // of C::rows rows, a group
  int sf_tiles;   // of 128 rows, a group
  int row_stages;  // of a whole row
  int stages;      // in shared memory
  int64_t k_tiles, scale_bytes;
};

// 8 codes to f16 pairs, in order.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
// kPad: rows of x a CTA takes, at most.  kSplit: clusters split K (a kernel without
// their code ends sooner: 4 x 128 heads x 512 x 128 3.5 us, not 3.8).
template <int kPad, int kGroups, bool kSplit>
__global__ void __launch_bounds__(kThreads, kCtas)
    nvfp4_gemv_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ Params p) {
  using C = Cfg<kGroups>;
  const int splits = kSplit ? p.splits : 1;
  constexpr int kTiles = kPad > 8 ? 2 : 1;  // groups of 8 columns of the products
  constexpr int kStep = C::step, kXStep = kPad * kStep * 2;  // bytes of x a step
  extern __shared__ __align__(1024) uint8_t smem[];  // stages of weights, two chunks of x; then the CTA's sums
  __shared__ float factor[2][kWarps][kPad];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages];
  __shared__ volatile int abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane >> 2, t = lane & 3;
  const int row_warps = 1 << p.row_log, subs = kWarps >> p.row_log, cta_rows = 1 << (C::log + p.row_log);
  uint32_t id = blockIdx.x / splits;
  const int split = blockIdx.x - id * splits;
  const int sub = id & (subs - 1);
  id >>= 3 - p.row_log;
  const int64_t g = id / p.tiles;
  const int tile = id - static_cast<uint32_t>(g) * p.tiles;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kPad;
  const int rows = static_cast<int>(p.a.M - m0 < kPad ? p.a.M - m0 : kPad);
  const int row_warp = warp & (row_warps - 1), k_warp = warp >> p.row_log;
  const int first = p.row_stages * split / splits, count = p.row_stages * (split + 1) / splits - first;  // count >= 1
  const int sf_tiles = cta_rows > 128 ? 2 : 1;  // this CTA's rows are of
  const uint32_t stage_bytes = C::code_bytes + sf_tiles * subs * C::sf_bytes;
  const uint32_t base = smem_u32(smem), x_base = base + p.stages * stage_bytes;

  // Weights: lines of 128 bytes, step by step the CTA's rows, their 16-byte
  // pieces swizzled by the row (rows past the matrix: zeros, or the next group's);
  // then the steps' scales as they lie.
  const int64_t n0 = static_cast<int64_t>(tile) * C::rows + sub * cta_rows;
  const int sf_there = static_cast<int>(min(p.sf_tiles - n0 / 128, static_cast<int64_t>(sf_tiles)));
  const uint8_t* scales = p.a.w_scales + g * p.scale_bytes + n0 / 128 * p.k_tiles * 512;
  int issued = 0;
  auto load = [&](int i) {  // by one thread
    const int slot = i % p.stages, step = (first + i) * subs;
    const uint32_t dst = base + slot * stage_bytes;
    const int64_t left = p.k_tiles - static_cast<int64_t>(step) * (kStep / 64);  // tiles of 4 blocks
    const int tiles = left < kStep / 64 * subs ? static_cast<int>(left) : kStep / 64 * subs;
    mbar_expect_tx(&full[slot], C::code_bytes + max(sf_there, 0) * tiles * 512);
    for (int k = 0; k < subs; ++k)
      tma_load_bytes(dst + k * (cta_rows * C::line), &map, (step + k) * C::line, static_cast<int>(g * p.a.N + n0), &full[slot]);
    for (int k = 0; k < sf_there; ++k)
      bulk_load(dst + C::code_bytes + k * subs * C::sf_bytes, scales + (k * p.k_tiles + static_cast<int64_t>(step) * (kStep / 64)) * 512,
                tiles * 512, &full[slot]);
    issued = i + 1;
  };
  if (tid == 0) {
    abort = 0;
    prefetch_tmap(&map);
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    fence_mbar_init();
  }
  // The next call's CTAs may take the place of those that end; nothing is read
  // before the work ahead of this call is done (and by no load that takes memory
  // for constant: it was not when these CTAs began).
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // x, a chunk of stages at a time: a warp takes rows of blocks of 256 features (a
  // chunk has one for each warp at least), 8 features a lane.  A unit of 8 is piece
  // u % kPieces of the quad's thread u / kPieces, of the step u / (4 kPieces).
  constexpr int kPieces = kStep / 32;
  const int chunk = C::chunk(kPad, subs), chunk_steps = chunk * subs;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.a.x) + m0 * p.a.x_sm + g * p.a.x_sg;
  const int unit = kPieces == 8 ? (lane & 3) * 8 + (lane >> 2) : (lane & 16) + (lane & 3) * 4 + (lane >> 2 & 3);
  auto read_x = [&](int i, int pair) {  // i: the chunk's first stage
    const int r = pair % kPad, k = (first + i) * subs * kStep + pair / kPad * kXBlock + 8 * unit;
    return i < count && r < rows && k < p.a.K ? *reinterpret_cast<const uint4*>(x + r * p.a.x_sm + k) : make_uint4(0, 0, 0, 0);
  };
  auto stage_x = [&](int buffer, int pair, uint4 v) {
    uint32_t* q = reinterpret_cast<uint32_t*>(&v);
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) most = __vmaxu2(most, q[j] & 0x7FFF7FFFu);
    most = __reduce_max_sync(0xffffffffu, max(most & 0xFFFFu, most >> 16));
    if (most >= 0x7F80u) {  // an infinity or a NaN: the largest of the others
      most = 0;
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = q[j] & 0x7FFFu, hi = q[j] >> 16 & 0x7FFFu;
        most = max(most, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
      }
      most = __reduce_max_sync(0xffffffffu, most);
    }
    // 2^e <= largest < 2^(e + 1); times 2^(14 - e).  (Below 2^-112 the factor
    // stays at 2^126, where f16's steps are below all of bf16's.)
    const int e = max(static_cast<int>(most >> 7) - 127, -112);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
    const int r = pair % kPad, s = pair / kPad;
    if (lane == 0) factor[buffer][s][r] = __uint_as_float(static_cast<uint32_t>(127 + e - 14) << 23);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float lo, hi;
      bf16x2_to_f32(q[j], lo, hi);
      const __half2 h = __floats2half2_rn(lo * up, hi * up);
      q[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    const int piece = unit % kPieces, thread = unit / kPieces & 3, step = s * (kXBlock / kStep) + unit / (4 * kPieces);
    sts128(x_base + (buffer * chunk_steps + step) * kXStep + 16 * (piece * (4 * kPad) + 4 * r + thread), v);
  };
  constexpr int kAhead = kPad > 8 ? 2 : 1;  // rows of x a warp has in registers ahead,
  constexpr int kDepth = 3;                 // of so many chunks
  const int pairs_x = kPad * chunk_steps * kStep / kXBlock;
  uint4 next[kDepth][kAhead];
  auto read_ahead = [&](uint4 (&v)[kAhead], int i) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) v[j] = read_x(i, warp + kWarps * j);
  };
  auto stage_all = [&](int i, int buffer) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) stage_x(buffer, warp + kWarps * j, next[0][j]);
#pragma unroll 1
    for (int pair = warp + kWarps * kAhead; pair < pairs_x; pair += kWarps) stage_x(buffer, pair, read_x(i, pair));
#pragma unroll
    for (int d = 0; d + 1 < kDepth; ++d)
#pragma unroll
      for (int j = 0; j < kAhead; ++j) next[d][j] = next[d + 1][j];
  };
  // (before the weights are asked for, behind which it would wait)
#pragma unroll
  for (int d = 0; d < kDepth; ++d) read_ahead(next[d], d * chunk);
  if (tid == 0) {
    for (int i = 0; i < p.stages && i < count; ++i) load(i);
  }
  stage_all(0, 0);

  float total[kGroups][kTiles][4] = {};
  // where this thread's weights, scales and x lie in a stage
  const int r0 = row_warp * (16 * kGroups) + quad, line0 = k_warp * cta_rows + r0, in_tile = (sub * cta_rows + r0) & 127;
  const uint32_t code_at = base + line0 * C::line + (kGroups == 1 ? (2 * t) ^ (line0 & 7) : t ^ (line0 >> 1 & 3)) * 16;
  // (a warp's rows are some of 32 whose scales are 16 bytes apart)
  const uint32_t scale_at = base + C::code_bytes + ((r0 >> 7) * subs + k_warp) * C::sf_bytes +
                            (kGroups == 1 ? t * 512 : (t >> 1) * 512 + (t & 1) * 2) + (in_tile & 31) * 16 + (in_tile >> 5) * 4;
  uint32_t x_at[kTiles];
#pragma unroll
  for (int c = 0; c < kTiles; ++c)  // (columns past the rows are whatever they are, and not written)
    x_at[c] = x_base + k_warp * kXStep + 16 * (4 * min(8 * c + quad, kPad - 1) + t);
  const int blocks = static_cast<int>(p.a.K / 16);  // of a row
  int slot = 0, phase = 0, buffer = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < count; i0 += chunk, buffer ^= 1) {
    __syncthreads();  // the chunk's x is there, and the one before has been read
    read_ahead(next[kDepth - 1], i0 + kDepth * chunk);
#pragma unroll 1
    for (int i = i0; i < min(i0 + chunk, count); ++i) {
      // (A wait that gives up, which the error word tells, leaves the warps
      // running through their loops; the sums are then whatever they are.)
      wait(&full[slot], phase, p.a.error_word, &abort);
      const uint32_t at = slot * stage_bytes, in_chunk = (buffer * chunk + i - i0) * subs;
      const uint32_t x_in = in_chunk * kXStep;
      uint32_t sf[2 * kGroups];  // of rows r0, r0 + 8, ..: four or two blocks' of a thread
#pragma unroll
      for (int r = 0; r < 2 * kGroups; ++r) sf[r] = kGroups == 1 ? lds32(scale_at + at + 128 * r) : lds16(scale_at + at + 128 * r);
      constexpr int kBlocks = kStep / 64;
      const int block = ((first + i) * subs + k_warp) * (kStep / 16) + kBlocks * t;
      if (block + kBlocks > blocks) {  // the last blocks of a row may be two of four, or none (the padding may hold NaN)
        const uint32_t mask = blocks - block == 2 ? 0xFFFFu : 0u;
#pragma unroll
        for (int r = 0; r < 2 * kGroups; ++r) sf[r] &= mask;
      }
      float acc[kGroups][kTiles][4] = {};
#pragma unroll
      for (int b2 = 0; b2 < kStep / 128; ++b2) {  // two blocks of 16
        uint4 v[2 * kGroups];
        uint32_t sc[2 * kGroups];  // f16 pairs of their scales
#pragma unroll
        for (int r = 0; r < 2 * kGroups; ++r) {
          v[r] = lds128((code_at ^ (b2 << 4)) + at + r * (8 * C::line));
          sc[r] = e4m3x2_to_f16x2_pair(sf[r] >> (16 * b2));
        }
#pragma unroll
        for (int b1 = 0; b1 < 2; ++b1) {
          uint4 u[kTiles][2];
#pragma unroll
          for (int c = 0; c < kTiles; ++c)
#pragma unroll
            for (int half = 0; half < 2; ++half)
              u[c][half] = lds128(x_at[c] + x_in + (4 * b2 + 2 * b1 + half) * (64 * kPad));
#pragma unroll
          for (int gr = 0; gr < kGroups; ++gr) {
            uint32_t a[2][8];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint4 w = v[2 * gr + r];
              const uint32_t s2 = __byte_perm(sc[2 * gr + r], 0, b1 ? 0x3232 : 0x1010);
              uint32_t h[4];
              codes_to_f16(b1 ? w.z : w.x, h);
#pragma unroll
              for (int j = 0; j < 4; ++j) a[r][j] = h2_mul(h[j], s2);
              codes_to_f16(b1 ? w.w : w.y, h);
#pragma unroll
              for (int j = 0; j < 4; ++j) a[r][4 + j] = h2_mul(h[j], s2);
            }
#pragma unroll
            for (int c = 0; c < kTiles; ++c)
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                mma_f16(acc[gr][c], a[0][4 * half], a[1][4 * half], a[0][4 * half + 1], a[1][4 * half + 1], u[c][half].x,
                        u[c][half].y);
                mma_f16(acc[gr][c], a[0][4 * half + 2], a[1][4 * half + 2], a[0][4 * half + 3], a[1][4 * half + 3],
                        u[c][half].z, u[c][half].w);
              }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);
#pragma unroll
      for (int c = 0; c < kTiles; ++c)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float f = factor[buffer][((i - i0) * subs + k_warp) * kStep / kXBlock][min(8 * c + 2 * t + j, kPad - 1)];
#pragma unroll
          for (int gr = 0; gr < kGroups; ++gr) {
            total[gr][c][j] = fmaf(acc[gr][c][j], f, total[gr][c][j]);
            total[gr][c][j + 2] = fmaf(acc[gr][c][j + 2], f, total[gr][c][j + 2]);
          }
        }
      // the stage before is free once all warps have read it
      if (tid == 0 && i > 0 && i - 1 + p.stages < count) {
        const int before = i - 1;
        wait(&empty[before % p.stages], (before / p.stages) & 1, p.a.error_word, &abort);
        load(before + p.stages);
      }
      if (++slot == p.stages) slot = 0, phase ^= 1;
    }
    if (i0 + chunk < count) stage_all(i0 + chunk, buffer ^ 1);
  }
  if (tid == 0 && abort) drain_copies(full, p.stages, issued);
  __syncthreads();

  // [k warp][column][row of the CTA], over the warps' features, then over the
  // cluster's, each CTA a part of the (column, row) pairs
  float* sums = reinterpret_cast<float*>(smem);
  const int pairs = rows * cta_rows;
#pragma unroll
  for (int c = 0; c < kTiles; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = 8 * c + 2 * t + (j & 1);
      if (col < rows) {
#pragma unroll
        for (int gr = 0; gr < kGroups; ++gr)
          sums[k_warp * pairs + col * cta_rows + r0 + 16 * gr + 8 * (j >> 1)] = total[gr][c][j];
      }
    }
  __syncthreads();
  if (subs > 1 && splits > 1) {
    for (int e = tid; e < pairs; e += kThreads) {
      float v = sums[e];
      for (int k = 1; k < subs; ++k) v += sums[k * pairs + e];
      sums[e] = v;
    }
  }
  if (splits > 1) cluster_sync();
  const float gs = *p.a.gs_w;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.a.out) + m0 * p.a.out_sm + g * p.a.out_sg + n0;
  for (int e = split * kThreads + tid; e < pairs; e += splits * kThreads) {
    const int col = e >> (C::log + p.row_log), r = e & (cta_rows - 1);
    float v = 0.f;
    if (splits > 1) {
      for (int k = 0; k < splits; ++k) v += cluster_load(base + 4 * e, k);
    } else {
      for (int k = 0; k < subs; ++k) v += sums[k * pairs + e];
    }
    if (n0 + r < p.a.N) out[col * p.a.out_sm + r] = __float2bfloat16_rn(v * gs);
  }
  if (splits > 1) cluster_sync();  // (the others' shared memory is read until here)
}

// A CTA's shared memory with 2^row_log warps that have rows of their own: two chunks
// of x, and as many stages of weights as its share of an SM holds (or three, where
// that is more than its share: one CTA an SM).
struct Form {
  int stages;
  uint32_t bytes;
};
template <int kPad, int kGroups>
constexpr Form form_of(int row_log) {
  using C = Cfg<kGroups>;
  const int subs = kWarps >> row_log;
  const uint32_t x = 2u * C::chunk(kPad, subs) * subs * kPad * C::step * 2, stage = C::stage(row_log);
  int stages = x + kMinStages * stage >= kShare ? kMinStages : static_cast<int>((kShare - x) / stage);
  if (stages > kMaxStages) stages = kMaxStages;
  return Form{stages, x + stages * stage};
}

// Clusters of a size and a form that the current device holds at once, asked for once.
template <int kPad, int kGroups>
int resident_clusters(int splits, int row_log, int dev, int num_sms) {
  static std::atomic<int> known[64][4][kMaxSplits + 1];
  const uint32_t bytes = form_of<kPad, kGroups>(row_log).bytes;
  const int most = num_sms * (bytes <= kShare ? kCtas : 1) / splits;
  if (dev >= 64) return splits > 8 ? -1 : most;
  int n = known[dev][row_log][splits].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaError_t st;
    if (splits == 1) {
      st = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, nvfp4_gemv_kernel<kPad, kGroups, false>, kThreads, bytes);
      n *= num_sms;
    } else {
      const auto kern = nvfp4_gemv_kernel<kPad, kGroups, true>;
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = splits;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(static_cast<unsigned>(splits * num_sms));
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = bytes;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      st = splits > 8 ? cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) : cudaSuccess;
      if (st == cudaSuccess) st = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
    }
    if (st != cudaSuccess || n < 1) {
      (void)cudaGetLastError();
      n = splits > 8 ? -1 : most;  // -1: none
    }
    known[dev][row_log][splits].store(n, std::memory_order_relaxed);
  }
  return n;
}

template <int kPad, int kGroups>
int launch(Params p, int slot, int num_sms, cudaStream_t stream) {
  using C = Cfg<kGroups>;
  static_assert(kMinStages * C::code_bytes >= C::rows * kPad * sizeof(float), "the sums fit in the stages of weights");
  const auto split_kern = nvfp4_gemv_kernel<kPad, kGroups, true>, whole_kern = nvfp4_gemv_kernel<kPad, kGroups, false>;
  if (const int st = smem_limit_once(reinterpret_cast<const void*>(split_kern), static_cast<int>(kLimit), slot)) return st;
  if (const int st = smem_limit_once(reinterpret_cast<const void*>(whole_kern), static_cast<int>(kLimit), slot + 9)) return st;

  p.tiles = static_cast<int>((p.a.N + C::rows - 1) / C::rows);

  int dev = 0;
  if (const int st = cuda_status(cudaGetDevice(&dev))) return st;
  // Rows a CTA, and K's parts (a cluster of up to 10; a step a warp at least): the
  // shortest time, as waves of the clusters that the SMs hold at once, each of a
  // CTA's stages and of a start and an end that take about as long as four.
  const int64_t steps = (p.a.K + C::step - 1) / C::step, m_tiles = (p.a.M + kPad - 1) / kPad, units = p.a.groups * p.tiles;
  int64_t best_time = INT64_MAX, ctas = 0;
  for (int log = 3; log >= 0; --log) {
    const int subs = kWarps >> log;
    if (form_of<kPad, kGroups>(log).bytes > kLimit) break;
    const int64_t stages = (steps + subs - 1) / subs;
    for (int s = 1; s <= kMaxSplits && s <= stages; ++s) {
      const int64_t held = resident_clusters<kPad, kGroups>(s, log, dev, num_sms), clusters = units * subs * m_tiles;
      if (held < 1) continue;
      const int64_t time = (clusters + held - 1) / held * ((stages + s - 1) / s + 4);
      if (time < best_time) best_time = time, ctas = units * subs * s, p.row_log = log, p.splits = s;
    }
  }
  if (ctas > (int64_t(1) << 31) - 1 || m_tiles > 65535) return MLA_ERR_INVALID_ARG;
  const int subs = kWarps >> p.row_log;
  const Form form = form_of<kPad, kGroups>(p.row_log);
  p.row_stages = static_cast<int>((steps + subs - 1) / subs);
  p.stages = form.stages;

  CUtensorMap map;
  if (!encode_byte_map(&map, p.a.w_codes, p.a.K / 2, p.a.groups * p.a.N, p.a.K / 2, C::line, 1 << (C::log + p.row_log), kGroups == 2)) {
    set_last_error("cuTensorMapEncodeTiled failed for the weights");
    return MLA_ERR_LAUNCH;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(m_tiles));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = form.bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // (griddepcontrol)
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.splits > 1 ? 2 : 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, p.splits > 1 ? split_kern : whole_kern, map, p));
}

}  // namespace

int launch_gemv(const GemvArgs& a, cudaStream_t stream, int num_sms) {
  Params p = {};
  p.a = a;
  p.sf_tiles = static_cast<int>((a.N + 127) / 128);
  p.k_tiles = (a.K / 16 + 3) / 4;
  p.scale_bytes = p.sf_tiles * p.k_tiles * 512;
  // Two groups of 16 rows a warp, in steps of half the features, where x is much
  // (more than 8 rows: 16 x 7168 x 16384 27.6 us, with one 28.5) or a row of weights
  // short (4 x 128 heads x 512 x 128 3.5 us, with one 5.9; x 512 6.8, with one 7.9).
  // One otherwise: 1 x 7168 x 16384 17.9 us, with two 20.4; 1 x 576 x 7168 4.0, with two
  // 4.4.  (Near the border the matrices' number counts too: 4 x 128 heads x 512 x 1024
  // 12.5 us, with two 11.7; 4 x 16 heads x 512 x 512 4.2, with one 3.8; x 256 3.8, with
  // one 2.7.)
  const bool two = a.K <= 512;
  constexpr int kSlot = 37;  // 9 and 9 more
  if (a.M <= 1) return two ? launch<1, 2>(p, kSlot, num_sms, stream) : launch<1, 1>(p, kSlot + 1, num_sms, stream);
  if (a.M <= 2) return two ? launch<2, 2>(p, kSlot + 2, num_sms, stream) : launch<2, 1>(p, kSlot + 3, num_sms, stream);
  if (a.M <= 4) return two ? launch<4, 2>(p, kSlot + 4, num_sms, stream) : launch<4, 1>(p, kSlot + 5, num_sms, stream);
  if (a.M <= 8) return two ? launch<8, 2>(p, kSlot + 6, num_sms, stream) : launch<8, 1>(p, kSlot + 7, num_sms, stream);
  return launch<16, 2>(p, kSlot + 8, num_sms, stream);
}

}  // namespace mla
