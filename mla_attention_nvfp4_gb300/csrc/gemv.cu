// bf16 rows times an NVFP4 weight matrix (one, or one a group):
//   out[m, g, n] = gs sum_k x[m, g, k] code[g, n, k] scale[g, n, k / 16].
//
// HBM-bound: every weight is 9/16 of a byte, read once for up to 16 rows.  The
// sums run on mma.sync m16n8k16 (f16 operands, fp32 sums): weights are its 16
// rows, x its 8 columns, and what an instruction could do beyond the bytes' rate
// counts for nothing here.  (tcgen05 would want the weights unpacked in shared
// memory first; here they go from global memory to registers, are converted
// there and multiplied.)
//   weights  code * scale has 6 significant bits between 2^-10 and 2688: exact in
//            f16.  A thread holds 64 weights of two rows (32 bytes each) a step of
//            256 features: four whole blocks of 16, whose scales are one word.
//            Which feature of an instruction they are is free, as long as x
//            agrees: its rows lie in shared memory in the order of the fragments.
//   x        bf16 in f16, after a power of two a row and 2048 features that brings
//            the largest to 2^14 or more: exact down to 2^-31 of it (f16's steps
//            are 2^-24), within 2^-39 of it below.  Infinities and NaN are kept.
//   rows     a warp's 16 are 4 consecutive ones of each 32 of a 128-row tile: so
//            their scales are 64 consecutive bytes of the swizzled layout.
// The 8 warps of a CTA take kRows rows of 16 and split the features of a step
// range over the rest; a cluster of up to 8 CTAs splits K, and its CTAs each add
// up and write a part of the rows: no workspace, and sums in a fixed order.
#include <cuda_runtime.h>

#include "launch.h"
#include "nvfp4.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kStep = 256;      // features a step: 64 a thread of a quad
constexpr int kChunk = 8;       // steps whose x is in shared memory at a time
#ifndef D1
#define D1 2
#define D2 2
#define B1 2
#define B2 2
#endif
template <int kTiles>
constexpr int kDepthOf = kTiles == 1 ? D1 : D2;  // steps of weights in flight
template <int kTiles>
constexpr int kCtas = kTiles == 1 ? B1 : B2;     // an SM

struct Params {
  GemvArgs a;
  int row_warps;   // warps with rows of their own: 16 row_warps rows a CTA
  int splits;      // CTAs a cluster
  int tiles;       // of 128 rows, a group
  int steps;       // of a whole row
  int64_t k_tiles, scale_bytes;
};

struct Weights {  // a step's of one thread: two rows
  uint4 code[2][2];
  uint32_t scale[2];
};

template <bool kWide>
__device__ __forceinline__ void load_row(const uint8_t* p, int bytes, uint4 (&v)[2]) {
  if constexpr (kWide) {
    if (bytes > 0)
      asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x), "=r"(v[1].y), "=r"(v[1].z),
                     "=r"(v[1].w)
                   : "l"(p));
    else
      v[0] = v[1] = make_uint4(0, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      v[i] = bytes > 16 * i ? __ldg(reinterpret_cast<const uint4*>(p) + i) : make_uint4(0, 0, 0, 0);
  }
}

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
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr, int rank) {
  float v;
  asm volatile(
      "{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
      : "=f"(v)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

// kTiles: groups of 8 rows of x.
template <int kTiles, bool kWide>
__global__ void __launch_bounds__(kThreads, kCtas<kTiles>) nvfp4_gemv_kernel(const Params p) {
  constexpr int kCols = 8 * kTiles, kDepth = kDepthOf<kTiles>;
  extern __shared__ __align__(16) uint8_t smem[];  // a chunk's x; then the CTA's sums
  __shared__ uint32_t row_max[kCols][kWarps];
  __shared__ float factor[kCols];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane >> 2, t = lane & 3;
  const int split = blockIdx.x % p.splits, subs = kWarps / p.row_warps;
  int64_t id = blockIdx.x / p.splits;
  const int sub = static_cast<int>(id % subs);
  id /= subs;
  const int tile = static_cast<int>(id % p.tiles);
  const int64_t g = id / p.tiles;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kCols;
  const int rows = static_cast<int>(p.a.M - m0 < kCols ? p.a.M - m0 : kCols);
  const int row_warp = warp % p.row_warps, k_warp = warp / p.row_warps;
  const int first = static_cast<int>(static_cast<int64_t>(p.steps) * split / p.splits);
  const int last = static_cast<int>(static_cast<int64_t>(p.steps) * (split + 1) / p.splits);

  // this thread's two rows of the tile, and where its bytes of step 0 are
  const int in_tile = 4 * (sub * p.row_warps + row_warp) + (quad & 3) + 32 * (quad >> 2);
  const int64_t n = static_cast<int64_t>(tile) * 128 + in_tile;
  const int64_t row_bytes = p.a.K / 2;
  const uint8_t* codes = p.a.w_codes + (g * p.a.N + n) * row_bytes + 32 * t;
  const uint8_t* scales = p.a.w_scales + g * p.scale_bytes + (tile * p.k_tiles + t) * 512 + (in_tile & 31) * 16 + (in_tile >> 5) * 4;
  const bool have[2] = {n < p.a.N, n + 64 < p.a.N};
  auto load = [&](Weights& w, int s) {
    const int64_t left = row_bytes - static_cast<int64_t>(s) * (kStep / 2) - 32 * t;
    const int bytes = left >= 32 ? 32 : left > 0 ? static_cast<int>(left) : 0;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int b = have[r] ? bytes : 0;
      load_row<kWide>(codes + 64 * r * row_bytes + static_cast<int64_t>(s) * (kStep / 2), b, w.code[r]);
      w.scale[r] = 0;
      if (b > 0) w.scale[r] = __ldg(reinterpret_cast<const uint32_t*>(scales + 8 * r + static_cast<int64_t>(s) * 2048));
      if (!kWide && b == 16) w.scale[r] &= 0xFFFFu;  // two of the four blocks
    }
  };
  const int mine = first + k_warp < last ? (last - first - k_warp + subs - 1) / subs : 0;  // steps of this warp
  Weights w[kDepth];
#pragma unroll
  for (int d = 0; d < kDepth; ++d)
    if (d < mine) load(w[d], first + k_warp + subs * d);

  float total[kTiles][4] = {};
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.a.x) + m0 * p.a.x_sm + g * p.a.x_sg;
  // threads of one row of x while it is staged: 32 to 256
  const int per_row = rows > 4 ? 32 : rows > 2 ? 64 : rows > 1 ? 128 : 256;
  int i = 0;  // this warp's steps
#pragma unroll 1
  for (int chunk = first; chunk < last; chunk += kChunk) {
    // ------------------------------------------------- x into shared memory
    const int steps = min(kChunk, last - chunk);
    const int64_t k0 = static_cast<int64_t>(chunk) * kStep;
    const int units = steps * (kStep / 8);                                                        // of 8 features
    const int there = static_cast<int>(min(static_cast<int64_t>(units), (p.a.K - k0) / 8));       // not past the row's end
    if (chunk > first) __syncthreads();  // the last chunk's x has been read
    for (int r = tid / per_row; r < rows; r += kThreads / per_row) {
      const uint4* src = reinterpret_cast<const uint4*>(x + r * p.a.x_sm + k0);
      uint32_t most = 0;
#pragma unroll 4
      for (int u = tid % per_row; u < there; u += per_row) {
        const uint4 v = __ldg(src + u);
        const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) most = __vmaxu2(most, q[j] & 0x7FFF7FFFu);
      }
      most = max(most & 0xFFFFu, most >> 16);
      most = __reduce_max_sync(0xffffffffu, most);
      if (most >= 0x7F80u) {  // an infinity or a NaN: the largest of the others
        most = 0;
        for (int u = tid % per_row; u < there; u += per_row) {
          const uint4 v = __ldg(src + u);
          const uint32_t q[4] = {v.x, v.y, v.z, v.w};
          for (int j = 0; j < 4; ++j) {
            const uint32_t lo = q[j] & 0x7FFFu, hi = q[j] >> 16 & 0x7FFFu;
            most = max(most, lo < 0x7F80u ? lo : 0u);
            most = max(most, hi < 0x7F80u ? hi : 0u);
          }
        }
        most = __reduce_max_sync(0xffffffffu, most);
      }
      if (lane == 0) row_max[r][tid % per_row / 32] = most;
    }
    __syncthreads();
    for (int r = tid / per_row; r < rows; r += kThreads / per_row) {
      uint32_t most = 0;
      for (int k = 0; k < per_row / 32; ++k) most = max(most, row_max[r][k]);
      // 2^e <= largest < 2^(e + 1); times 2^(14 - e).  (Below 2^-112 the factor
      // stays at 2^126, where f16's steps are below all of bf16's.)
      const int e = max(static_cast<int>(most >> 7) - 127, -112);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
      if (tid % per_row == 0) factor[r] = __uint_as_float(static_cast<uint32_t>(127 + e - 14) << 23);
      const uint4* src = reinterpret_cast<const uint4*>(x + r * p.a.x_sm + k0);
#pragma unroll 4
      for (int u = tid % per_row; u < units; u += per_row) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (u < there) v = __ldg(src + u);
        uint32_t* q = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float lo, hi;
          bf16x2_to_f32(q[j], lo, hi);
          const __half2 h = __floats2half2_rn(lo * up, hi * up);
          q[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        // unit u of a step is piece u % 8 of the quad's thread u / 8
        const int s = u >> 5, piece = u & 7, thread = u >> 3 & 3;
        reinterpret_cast<uint4*>(smem)[(s * 8 + piece) * (4 * rows) + 4 * r + thread] = v;
      }
    }
    __syncthreads();
    // ------------------------------------------------------------- products
    float acc[kTiles][4] = {};
    const int end = min(mine, (chunk - first + steps - k_warp + subs - 1) / subs);
#pragma unroll 1
    while (i < end) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        if (i % kDepth == d && i < end) {
          const int s = first + k_warp + subs * i;
          const uint4* xs = reinterpret_cast<const uint4*>(smem) + (s - chunk) * 8 * (4 * rows) + lane;
          uint32_t sc[2][2];  // f16 pairs of two blocks' scales
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            sc[r][0] = e4m3x2_to_f16x2_pair(w[d].scale[r]);
            sc[r][1] = e4m3x2_to_f16x2_pair(w[d].scale[r] >> 16);
          }
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            uint32_t a[2][8];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint4 v = w[d].code[r][b >> 1];
              const uint32_t lo = b & 1 ? v.z : v.x, hi = b & 1 ? v.w : v.y;
              const uint32_t s2 = __byte_perm(sc[r][b >> 1], 0, b & 1 ? 0x3232 : 0x1010);
              uint32_t h[4];
              codes_to_f16(lo, h);
#pragma unroll
              for (int j = 0; j < 4; ++j) a[r][j] = h2_mul(h[j], s2);
              codes_to_f16(hi, h);
#pragma unroll
              for (int j = 0; j < 4; ++j) a[r][4 + j] = h2_mul(h[j], s2);
            }
#pragma unroll
            for (int c = 0; c < kTiles; ++c) {
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (8 * c + quad < rows) v = xs[(2 * b + half) * (4 * rows) + 32 * c];
                mma_f16(acc[c], a[0][4 * half], a[1][4 * half], a[0][4 * half + 1], a[1][4 * half + 1], v.x, v.y);
                mma_f16(acc[c], a[0][4 * half + 2], a[1][4 * half + 2], a[0][4 * half + 3], a[1][4 * half + 3], v.z, v.w);
              }
            }
          }
          if (i + kDepth < mine) load(w[d], s + subs * kDepth);
          ++i;
        }
      }
    }
#pragma unroll
    for (int c = 0; c < kTiles; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = 8 * c + 2 * t + (j & 1);
        if (col < rows) total[c][j] = fmaf(acc[c][j], factor[col], total[c][j]);
      }
  }

  // ----------------------------------------------------------------- sums
  // [k warp][column][row of the CTA], over the warps' features, then over the
  // cluster's, each CTA a part of the (column, row) pairs
  __syncthreads();
  float* sums = reinterpret_cast<float*>(smem);
  const int cta_rows = 16 * p.row_warps, pairs = rows * cta_rows;
#pragma unroll
  for (int c = 0; c < kTiles; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = 8 * c + 2 * t + (j & 1);
      if (col < rows) sums[k_warp * pairs + col * cta_rows + row_warp * 16 + quad + 8 * (j >> 1)] = total[c][j];
    }
  __syncthreads();
  if (subs > 1 && p.splits > 1) {
    for (int e = tid; e < pairs; e += kThreads) {
      float v = sums[e];
      for (int k = 1; k < subs; ++k) v += sums[k * pairs + e];
      sums[e] = v;
    }
  }
  if (p.splits > 1) cluster_sync();
  const float gs = *p.a.gs_w;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.a.out) + m0 * p.a.out_sm + g * p.a.out_sg;
  const uint32_t base = smem_u32(sums);
  for (int e = split * kThreads + tid; e < pairs; e += p.splits * kThreads) {
    const int col = e / cta_rows, r = e - col * cta_rows;
    float v = 0.f;
    if (p.splits > 1) {
      for (int k = 0; k < p.splits; ++k) v += ld_cluster(base + 4 * e, k);
    } else {
      for (int k = 0; k < subs; ++k) v += sums[k * pairs + e];
    }
    // row r of the CTA: warp r / 16, its row r % 16 as above
    const int q = r & 15;
    const int64_t at = static_cast<int64_t>(tile) * 128 + 4 * (sub * p.row_warps + (r >> 4)) + (q & 3) + 32 * (q >> 2);
    if (at < p.a.N) out[col * p.a.out_sm + at] = __float2bfloat16_rn(v * gs);
  }
  if (p.splits > 1) cluster_sync();  // (the others' shared memory is read until here)
}

template <int kTiles, bool kWide>
int launch(const Params& p, int64_t ctas, int64_t m_tiles, int slot, cudaStream_t stream) {
  const auto kern = nvfp4_gemv_kernel<kTiles, kWide>;
  const int rows = static_cast<int>(p.a.M < 8 * kTiles ? p.a.M : 8 * kTiles);
  const int steps = (p.steps + p.splits - 1) / p.splits;
  const int x_bytes = (steps < kChunk ? steps : kChunk) * kStep * 2 * rows, sum_bytes = kWarps * 16 * rows * 4;
  constexpr int kMost = kChunk * kStep * 2 * 8 * kTiles;
  static_assert(kMost >= kWarps * 16 * 8 * kTiles * 4, "a chunk's x is the larger part");
  if (const int st = smem_limit_once(reinterpret_cast<const void*>(kern), kMost, slot)) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(m_tiles));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = x_bytes > sum_bytes ? x_bytes : sum_bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.splits;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.splits > 1 ? 1 : 0;
  return cuda_status(cudaLaunchKernelEx(&cfg, kern, p));
}

}  // namespace

int launch_gemv(const GemvArgs& a, cudaStream_t stream, int num_sms) {
  Params p;
  p.a = a;
  p.tiles = static_cast<int>((a.N + 127) / 128);
  p.steps = static_cast<int>((a.K + kStep - 1) / kStep);
  p.k_tiles = (a.K / 16 + 3) / 4;
  p.scale_bytes = p.tiles * p.k_tiles * 512;
  // All the rows of a tile a CTA (x is staged once a CTA) and K split over up to
  // 8 CTAs, so that whole waves of CTAs fill the SMs; fewer rows where that leaves
  // SMs without work.  A warp has a step of features at least.
  const int tiles = a.M <= 8 ? 1 : 2;
  const int64_t m_tiles = (a.M + 8 * tiles - 1) / (8 * tiles);
  const int64_t slots = static_cast<int64_t>(num_sms) * (tiles == 1 ? kCtas<1> : kCtas<2>);
  const int64_t units = a.groups * p.tiles * m_tiles;
  double best_share = 0;
  int64_t best = 0;
  for (int rw = kWarps; rw >= 1; rw /= 2) {
    const int subs = kWarps / rw;
    for (int s = 1; s <= 8 && (s == 1 || s * subs <= p.steps); ++s) {
      const int64_t ctas = units * subs * s, waves = (ctas + slots - 1) / slots;
      const double share = static_cast<double>(ctas) / static_cast<double>(waves * slots);
      if (share > best_share * 1.05) best_share = share, best = ctas / m_tiles, p.row_warps = rw, p.splits = s;
    }
    if (best_share > 0.7) break;
  }
  if (best > (int64_t(1) << 31) - 1 || m_tiles > 65535) return MLA_ERR_INVALID_ARG;
  const bool wide = a.K % 64 == 0 && (reinterpret_cast<uintptr_t>(a.w_codes) & 31u) == 0;
  if (tiles == 1)
    return wide ? launch<1, true>(p, best, m_tiles, 26, stream) : launch<1, false>(p, best, m_tiles, 27, stream);
  return wide ? launch<2, true>(p, best, m_tiles, 28, stream) : launch<2, false>(p, best, m_tiles, 29, stream);
}

}  // namespace mla
