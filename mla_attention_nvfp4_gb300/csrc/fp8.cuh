// Pieces the e4m3 kernels share: byte tensor maps and their copies, the
// 8-bit tcgen05 product, wide TMEM loads.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sm100.cuh"

namespace mla {

// A row-major byte matrix [rows, width] with `stride` bytes between rows as a
// tensor map; box_x x box_rows bytes a copy, swizzled by 128 or 64 bytes;
// bytes past the matrix read as zero.
bool encode_byte_map(CUtensorMap* map, const void* base, int64_t width, int64_t rows, int64_t stride, uint32_t box_x,
                     uint32_t box_rows, bool swizzle64);

namespace sm100 {

__device__ __forceinline__ void tma_load_bytes(uint32_t dst, const void* tmap, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      ::"r"(dst), "l"(tmap), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

// Shared-memory descriptor of a 64-byte-swizzled operand (mode 4): atoms of 8
// rows x 64 bytes, `sbo` bytes from one group of 8 rows to the next.
__device__ __forceinline__ uint64_t smem_desc_sw64(uint32_t saddr, uint32_t sbo) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32 |
         static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(4) << 61;
}

// D[tmem] (+)= A[smem] * B[smem]^T with e4m3 operands (K = 32), fp32 sums.
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Waits for the warp's loads; v, which one of them wrote, is not read before.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}

// What a CTA has in flight when it ends, after a wait that gave up too, would
// touch memory that is no longer its own.  So an issuer waits for its products
// (below), which have waited for their copies; and, where a role gave up, one
// thread waits, with a limit, at the CTA's end for the last copies into each
// ring of stages (full: their barriers; issued: all that were).
__device__ __noinline__ inline void drain_copies(uint64_t* full, uint32_t stages, uint32_t issued) {
  for (uint32_t i = issued > stages ? issued - stages : 0; i < issued; ++i)
    for (int n = 0; n < 4096 && !mbar_test(&full[i % stages], (i / stages) & 1); ++n) {
    }
}

// One lane of a converged warp, the same one each time (a commit follows the
// products of its own thread).  Loops that issue products are run by the whole
// warp, their descriptors made of values that the compiler knows to be the
// warp's (uniform), and only the issue itself is one lane's: the operands are
// uniform registers, and values of a one-lane branch are moved there one by
// one (e4m3 decode, 64 x 4096 keys, 128 heads: 94 us so, 88 in this way).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
template <typename T>
__device__ __forceinline__ T uniform(T v) {
  return __shfl_sync(0xffffffffu, v, 0);
}

// An issuer (a whole warp) waits for its products, before it leaves; retired: a
// barrier of its own, of one arrival.
__device__ __forceinline__ void retire_products(uint64_t* retired, uint32_t* error_word) {
  __syncwarp();
  if (elect_one()) mma_commit(retired);
  __syncwarp();
  mbar_wait(retired, 0, error_word, nullptr);
}

// Instruction descriptor of kind::f8f6f4, e4m3 operands (format 0), fp32
// accumulator: the fields of idesc_f32acc.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool a_mn, bool b_mn) {
  return idesc_f32acc(M, N, 0u, a_mn, b_mn);
}

// 32 lanes x 32 bits, 32 consecutive columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// One column: lane = this thread's.
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, float& v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=f"(v) : "r"(taddr));
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, float v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "f"(v) : "memory");
}

// acc (two floats) += v (two floats) * s (two floats), each a fused
// multiply-add rounded to nearest.
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t v, uint64_t s) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(s));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

}  // namespace sm100
}  // namespace mla
