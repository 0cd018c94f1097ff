// Absorbed MLA decode over the e4m3 latent cache (one scale per block of 64
// tokens) on tcgen05.
//
// The cached bytes are the tensor cores' operands as they lie: tiles of 128
// keys x 576 features arrive by TMA and serve both products, the keys as
// 128-row operand of S^T = K Q^T (K-major) and the values as 128-row operand
// of O^T = V^T P^T (read feature-major, one 128-feature chunk at a time).
// Queries and probabilities are the other operand, kH heads a CTA (32 or 64),
// so that a call with few heads pays for few, and a key is a TMEM lane, so
// that masking a key masks a thread.
//
// Two 8-bit terms carry 8 significant bits:
//   q = 2^e (q1 + q2 / 16) with q1 = e4m3(q 2^-e), q2 = e4m3(16 (q 2^-e - q1)):
//       a bf16 query exactly (its 8 bits split 4 + 4), down to 2^-13 of the
//       head's largest feature: there q 2^-e is 2^-6, from where on q1's rest
//       is a multiple of 2^-13 and 16 times it one of e4m3's smallest step,
//       2^-9.  Features below that are held to half a step, 2^-21 of the
//       largest.  (16 times the rest, at most 256, still fits; without the
//       factor both limits lie 2^4 higher.)  The terms are 2 kH columns of one
//       product, added as S^T is read.
//   p = p1 + p2 with p1 = e4m3(p), at most 2^-8 off relative (what bf16 would
//       be; f16, to which p is rounded before, adds 2^-12).  The largest p lies
//       between 2^kReset and 2^kTop; p2 has a step of 2^-13 or more, 2^17 or
//       more below it:
//         32 heads: p2 = e4m3(16 (p - p1)), both terms in one product, with
//           accumulators of their own;
//         64 heads: one accumulator (TMEM holds no more), two products, and
//           p2 = e5m2 of p - p1 in steps of 2^-13 (e5m2's own steps are
//           smaller below 2^-11, and change from one power of two to the next).
//       Before either rounding comes an offset that runs evenly through such a
//       step over 32 neighbouring keys: a long tail of equal, tiny weights,
//       which rounding to nearest would push to one side, keeps its sum.  The
//       offsets stay below half a step: a weight of zero is zero.
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
//   warps 2..9   queries to two terms, softmax (thread = key; warps 2..5 the
//                first half of the heads, 6..9 the second);
//   warps 10..13 rescale O where references were raised, while the softmax
//                goes on; a piece's output, while the next one starts.
// The code of each role is kept short (rolled loops, one copy): unrolled
// further, the warps waited for instructions more than for anything else.
// Times (merge included; pairs below compare two forms at one time): 64 x 4096
// keys, 128 heads 88.9 us, 64 heads 65, 16 heads 46; 128 sequences of 1k to
// 32k, 16 heads 135 us (5.2 TB/s), 128 heads 324 (1020 TFLOP/s); 1 x 65536, 128
// heads 37.5; 1 x 100, 16 heads 9.9 (12.3 with the merge), launches and one chain
// of latencies.  With 64 heads a CTA, shared memory bounds a tile: the
// operands of its products (18 x 8 KB and 32 x 6 KB), the copies in (72 KB) and
// P take 3300 cycles at 128 bytes a cycle, of about 4400.  CTAs of 32 heads
// read every key twice as often (64 x 4096, 128 heads: 131 us).  What was
// tried beside that: the next tile into L2 ahead (no faster), the merge put in
// place before the decode ends (1 x 65536: 58 us, not 50), two value chunks'
// scores issued at once (90 us, not 88), references found by votes instead of
// exchanges (111 us, not 94).
//
// A batch with a shared prefix (kShared) is the same work on lists of keys: the
// prefix, once for every kH rows (sequence, head) of the batch, whatever
// sequences they are of, and each sequence's own keys.  All pieces leave partial
// results, and a row's merge takes those of the prefix and its own.  64 x (16384 +
// 1..2048) keys, 16 heads 59.0 us (the decode 119, 110 where its tables name the same
// pages: a tile of keys serves 64 rows, not 16); 32 x (32768 + 1000), 128 heads 251
// (1199 TFLOP/s; the decode 273, and 253 of the same pages: its rows were full, only
// HBM is spared); 4 x (2048 + 64), 16 heads 14.8, latencies of start, one tile and
// merge (the decode 15.9); 16 x (12800 + 100), 16 heads 28.4 (37.2), 128 x (4096 + 64),
// one head 25.0 (65.1), where the starts are most of it.
#include <cuda.h>
#include <cuda_runtime.h>

#include "fp8.cuh"
#include "fp8_query.cuh"
#include "launch.h"
#include "nvfp4.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kKey = MLA_D_LATENT + MLA_D_ROPE;
constexpr int kBlock = MLA_FP8_BLOCK;
constexpr int kTile = 128;  // keys
constexpr int kSoftmax = 256, kOutput = 128, kThreads = 96 + kSoftmax + kOutput;
constexpr float kScaleMin = 8.673617379884035e-19f, kScaleMax = 1.152921504606847e18f;  // 2^-60, 2^60
constexpr float kTop = 8.5f;    // weights stay at or below 2^8.5 = 362 (e4m3: 448)
constexpr float kReset = 4.0f;  // a raised reference puts the tile's largest weight at 2^4
constexpr float kBelow = -3.402823466e38f;  // a piece's LSE where all its scores are below fp32's range
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kPiece = 3, kMerge = 2;  // what a piece's start and a merge cost, in tiles
// The merge gives a row of results 2 kSub warps, not 2, from kManyPieces ranges
// a sequence on.  1 x 65536 keys, 128 heads: 37.5 us in all (49.2 with 2 warps
// a row; kSub 4: 38.3, 16: 37.5); 2 x 32768: 41.3 (48.6); 4 x 16384, at 19
// ranges a sequence: 42.7 (41.1).
constexpr int kSub = 8, kManyPieces = 24;
constexpr uint32_t kChunkBytes = kTile * 128, kRopeBytes = kTile * 64;
constexpr uint32_t kColS = 256;  // TMEM: O^T in columns 0..255 (64 per value chunk), then two S^T of 2 kH (q1 | q2)

// Shared memory: a ring of latent chunks (128 keys x 128 features, four a
// tile), RoPE tiles, queries (rows q1, then q2; four chunks of 128 features
// and the RoPE), weights (rows of 64 bytes, one per key: p1 | p2, or p1 and
// p2 apart), the rest.
template <int kH>
struct Cfg {
  static_assert(kH == 32 || kH == 64, "heads per CTA");
  static constexpr int mine = kH / 2;  // heads per softmax thread
  static constexpr int slots = kH == 64 ? 8 : 10, ropes = kH == 64 ? 1 : 2, info = 4;
  static constexpr int terms = kH / 32;  // value products per chunk
  static constexpr uint32_t q_chunk = 2 * kH * 128;
  static constexpr uint32_t off_rope = slots * kChunkBytes, off_q = off_rope + ropes * kRopeBytes;
  static constexpr uint32_t off_p = off_q + 2 * kH * kKey, off_misc = off_p + kTile * 64 * terms;
};

template <int kH>
struct Misc {
  using C = Cfg<kH>;
  uint64_t full[C::slots], empty[C::slots], rfull[C::ropes], rempty[C::ropes], info_full[C::info];
  uint64_t s_full[2], s_free[2], p_ready, pv_done, q_ready, sums_ready, o_free, moved[2], rescaled[2], retired[2];
  alignas(16) float c[kH], m[kH];
  alignas(16) float move[2][kH];  // what a tile raises the references by, in turn
  alignas(16) float inv[kH];      // a piece's references, then 1 / its sums
  alignas(16) float sums[4][kH];
  int top[kH];            // a hit head's maximum, as an integer that orders like it
  uint32_t raised[2][2];  // heads (of either half) whose part of O is to be rescaled
  uint32_t hits[2], moves[2];  // heads (of either half) that may have to be raised; that are
  float scale[C::info][2];  // of a tile's two blocks; 0: the block is no part of the sequence
  int64_t t0, t1, off0;
  int b0, longest;  // first sequence's keys (shared: of the first list's sequences)
  uint32_t tmem;
  int chunks, ropes;  // copies issued
  volatile int abort;
};

template <int kH>
constexpr uint32_t smem_bytes() {
  return Cfg<kH>::off_misc + static_cast<uint32_t>(sizeof(Misc<kH>));
}
static_assert(smem_bytes<64>() <= 232448 && smem_bytes<32>() <= 232448, "shared memory budget");

// A batch with a shared prefix (groups is 1, cuts one entry a list): lists of
// keys with up to kH query rows each, one after another.  First the prefix, once
// for every kH of the batch's rows (sequence, head); then the keys that are each
// sequence's own, once for every kH of its heads.  A list in a range has its
// partial results at list + range: pieces follow each other in both.
struct SharedPlan {
  int64_t len;                 // of the prefix
  int prefix, lists, groups;   // lists of the prefix, of all; per sequence
  int own_rows;                // rows of an own list's partial results
  int64_t own;                 // the first of those rows
};

struct Params {
  Fp8DecodeArgs a;
  uint32_t page_magic;  // division by page_size / 64
  int page_shift;
  int ranges, groups;  // ranges of tiles; head groups (grid = ranges * groups)
  bool split;
  int2* cuts;      // [batch]: a sequence's first range, and its pieces | (1 << 30 where the first is part 1)
  float* part_lse;   // log2 units, [range][group][2][kH]
  float* part_o;     // the same rows of 512
  SharedPlan sh;
};

__device__ __forceinline__ int clipped_len(const Fp8DecodeArgs& a, int b) {
  const int64_t table = a.max_pages * a.page_size, most = (int64_t{1} << 31) - 2 * kTile;  // (lengths are rounded up)
  const int64_t room = table < most ? table : most;
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

// The pieces of a CTA's work, one after another: tiles [s, e) of sequence b
// (len keys, n tiles, from block `block` of its page table), query rows row ..
// row + rows of the batch's.  Cut form: the pieces of a range of tiles; part is
// 0 for the one the range begins with, else 1.  Whole form: sequences range,
// range + ranges, ..., those without keys too.
template <int kH, bool kShared>
struct Pieces {
  int b = 0, len = 0, s = 0, e = 0, n = 0, part = 0;
  const int rows;
  static constexpr int block = 0;
  __device__ __forceinline__ int64_t row(const Params& p) const { return static_cast<int64_t>(b) * p.a.num_heads + h0_; }
  __device__ __forceinline__ int64_t part_row(const Params& p, int range) const {
    return ((static_cast<int64_t>(range) * p.groups + h0_ / kH) * 2 + part) * kH;
  }

  template <class M>
  __device__ __forceinline__ Pieces(const Params& p, const M& ms, int range)
      : rows(min(kH, p.a.num_heads - static_cast<int>(blockIdx.x % p.groups) * kH)), h0_(blockIdx.x % p.groups * kH), split_(p.split), step_(p.split ? 1 : p.ranges), next_(p.split ? ms.b0 : range), t_(p.split ? ms.t0 : 0),
        t0_(t_), t1_(p.split ? ms.t1 : 0), off_(p.split ? ms.off0 : 0) {
    next_len_ = p.split ? ms.longest : load(p);
  }
  __device__ __forceinline__ bool next(const Params& p) {
    do {
      if (split_ ? t_ >= t1_ : next_ >= p.a.batch) return false;
      b = next_;
      len = next_len_;
      n = tiles_of(len);
      next_ += step_;
      next_len_ = load(p);  // ahead of its use
      s = split_ ? static_cast<int>(t_ - off_) : 0;
      e = split_ && t1_ - off_ < n ? static_cast<int>(t1_ - off_) : n;
      part = t_ == t0_ ? 0 : 1;
      if (split_) {
        if (n > 0) t_ = off_ + e;
        off_ += n;
      }
    } while (split_ && n == 0);
    return true;
  }

 private:
  __device__ __forceinline__ int load(const Params& p) const { return next_ < p.a.batch ? clipped_len(p.a, next_) : 0; }
  const int h0_;
  const bool split_;
  const int step_;
  int next_, next_len_;
  int64_t t_;
  const int64_t t0_, t1_;
  int64_t off_;
};

// The keys and rows of a list.
struct KeyList {
  int b, rows;  // page table row
  int64_t row;
  int first, last;  // prefix: the sequences of its rows
};
template <int kH>
__device__ __forceinline__ KeyList key_list(const Params& p, int v) {
  const uint32_t H = p.a.num_heads;  // (rows are at most 2^30)
  KeyList k;
  if (v < p.sh.prefix) {
    const uint32_t row = static_cast<uint32_t>(v) * kH;
    k.row = row;
    k.rows = min(static_cast<uint32_t>(p.a.batch) * H - row, static_cast<uint32_t>(kH));
    k.b = 0;
    k.first = static_cast<int>(row / H);
    k.last = static_cast<int>((row + k.rows - 1) / H);
  } else {
    const uint32_t u = v - p.sh.prefix, groups = p.sh.groups;
    k.b = k.first = k.last = static_cast<int>(u / groups);
    const int g = static_cast<int>(u - k.b * groups);
    k.row = k.b * H + g * kH;
    k.rows = min(kH, p.a.num_heads - g * kH);
  }
  return k;
}
// Its keys, given the longest of its sequences' lengths (an own list's only one).
__device__ __forceinline__ int list_keys(const Params& p, int v, int longest) {
  const int shared = static_cast<int>(p.sh.len);
  if (v < p.sh.prefix) return longest >= shared ? shared : 0;
  return longest >= shared ? longest - shared : longest;
}
// What a list takes, in tiles: its start, where it has any.  (64 rows: 32 x
// (32768 + 1000) keys, 128 heads, 256 us; with 3 tiles a start, 4, 6: 297, 274,
// 256: the CTAs of the many short lists were the last to end.)
template <int kH>
constexpr int kStart = kH == 64 ? 5 : 3;
template <int kH>
__device__ __forceinline__ int list_cost(int tiles) {
  return tiles > 0 ? tiles + kStart<kH> : 0;
}

// The same for lists: a range is one of their costs, of which the first kStart
// of a list are its start and the rest its tiles.
template <int kH>
struct Pieces<kH, true> {
  int b = 0, len = 0, s = 0, e = 0, n = 0, rows = 0, block = 0, list = 0;
  __device__ __forceinline__ int64_t row(const Params&) const { return row_; }
  __device__ __forceinline__ int64_t part_row(const Params& p, int range) const {
    const int64_t prefix = p.sh.prefix;
    return list < prefix ? (static_cast<int64_t>(list) + range) * kH
                         : p.sh.own + (list - prefix + range) * static_cast<int64_t>(p.sh.own_rows);
  }
  template <class M>
  __device__ __forceinline__ Pieces(const Params& p, const M& ms, int)
      : next_(ms.b0), t_(ms.t0), t1_(ms.t1), off_(ms.off0), lane_(threadIdx.x & 31) {
    longest_ = ms.longest;  // (the plan has it)
  }
  // (called by whole warps)
  __device__ __forceinline__ bool next(const Params& p) {
    while (t_ < t1_ && next_ < p.sh.lists) {
      const int v = next_;
      const int longest = __reduce_max_sync(0xffffffffu, longest_);
      len = list_keys(p, v, longest);
      n = tiles_of(len);
      const int64_t first = off_ + kStart<kH>, end = off_ + list_cost<kH>(n), hi = t1_ < end ? t1_ : end;
      s = t_ > first ? static_cast<int>(t_ - first) : 0;
      e = hi > first ? static_cast<int>(hi - first) : 0;
      t_ = hi;
      if (hi == end) {
        off_ = end;
        ++next_;
        longest_ = load(p);  // ahead of its use
      }
      if (s < e) {
        const KeyList k = key_list<kH>(p, v);
        list = v;
        b = k.b;
        rows = k.rows;
        row_ = k.row;
        block = v >= p.sh.prefix && longest >= p.sh.len ? static_cast<int>(p.sh.len / kBlock) : 0;
        return true;
      }
    }
    return false;
  }

 private:
  __device__ __forceinline__ int load(const Params& p) const {
    int most = 0;
    if (next_ < p.sh.lists) {
      const KeyList k = key_list<kH>(p, next_);
      for (int i = k.first + lane_; i <= k.last; i += 32) most = max(most, clipped_len(p.a, i));
    }
    return most;
  }
  int64_t row_ = 0;
  int next_, longest_;
  int64_t t_;
  const int64_t t1_;
  int64_t off_;
  const int lane_;
};

__device__ __forceinline__ uint32_t cvt_e5m2x2_h2(uint32_t h2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
  return r;
}
// Rounded to multiples of 2^-13 where below 2^-4: the steps of f16 numbers in
// [2^-3, 2^-2).  (Larger ones lose what is far below their step in e5m2.)
__device__ __forceinline__ uint32_t h2_steps(uint32_t a) {
  const __half2 mid = __float2half2_rn(0.1875f);
  const __half2 r = __hsub2(__hadd2(*reinterpret_cast<const __half2*>(&a), mid), mid);
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Floats as integers of the same order, for an integer maximum.
__device__ __forceinline__ int ordered(float v) {
  const int i = __float_as_int(v);
  return i >= 0 ? i : i ^ 0x7FFFFFFF;
}
__device__ __forceinline__ float from_ordered(int i) { return __int_as_float(i >= 0 ? i : i ^ 0x7FFFFFFF); }

// Barriers of one half of the softmax warps (128 threads): kH / 2 heads,
// whose references and sums are that half's alone.
__device__ __forceinline__ void half_bar(int wg) { asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory"); }
__device__ __forceinline__ bool half_any(int wg, bool v) {
  int r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\tsetp.ne.s32 a, %1, 0;\n\tbarrier.cta.red.or.pred b, %2, 128, a;\n\t"
      "selp.s32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"(static_cast<int>(v)), "r"(3 + wg)
      : "memory");
  return r != 0;
}

// The plan: this CTA's range of the batch's tiles, and its first sequence; or
// of the lists' costs, and its first list.  scan: two words of shared memory a
// warp.
template <int kH, bool kShared, class M>
__device__ __forceinline__ void make_plan(const Params& p, M& ms, int64_t* scan, int range, bool publish) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, B = kShared ? p.sh.lists : p.a.batch;
  int longest = 0;  // of the sequence, or the list's sequences
  auto cost_of = [&](int b) {
    if constexpr (kShared) {
      const KeyList k = key_list<kH>(p, b);
      longest = 0;
#pragma unroll 1
      for (int i = k.first; i <= k.last; ++i) longest = max(longest, clipped_len(p.a, i));
      return list_cost<kH>(tiles_of(list_keys(p, b, longest)));
    } else {
      longest = clipped_len(p.a, b);
      return tiles_of(longest);
    }
  };
  const int per_thread = (B + kThreads - 1) / kThreads;
  const int first = tid * per_thread, last = min(first + per_thread, B);
  int64_t sum = 0;
  int most = 0;
#pragma unroll 1
  for (int b = first; b < last; ++b) {
    const int n = cost_of(b);
    sum += n;
    most = max(most, n);
  }
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 31) {
    scan[2 * warp] = incl;
    scan[2 * warp + 1] = most;
  }
  __syncthreads();
  int64_t all = lane < kThreads / 32 ? scan[2 * lane] : 0;
  most = __reduce_max_sync(0xffffffffu, lane < kThreads / 32 ? static_cast<int>(scan[2 * lane + 1]) : 0);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, all, o);
    if (lane >= o) all += v;
  }
  const int64_t total = __shfl_sync(0xffffffffu, all, 31);
  const int64_t before = warp > 0 ? __shfl_sync(0xffffffffu, all, max(warp - 1, 0)) : 0;
  // (64-bit division only where it is needed)
  auto divide = [](int64_t a, int64_t b) {
    return (a | b) >> 31 ? a / b : static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
  };
  const int64_t per = divide(total + p.ranges - 1, p.ranges);
  // A CTA each for whole sequences, where that takes no longer than equal
  // ranges: those begin two pieces (of one sequence's end and the next one's
  // start; one, if they are of a tile or the batch of a sequence), and the cut
  // ones are merged.
  // (A list's cost has its start; a range begins one more, that of a cut list.)
  const bool uncut =
      B <= p.ranges && (kShared ? most <= per + kStart<kH>
                                : most + kPiece <= per + (per > 1 && B > 1 ? 2 : 1) * kPiece + kMerge);
  const int64_t t0 = uncut ? 0 : range * per;
  int64_t off = before + incl - sum;
  if constexpr (kShared) {
    if (tid == 0) {
      ms.t0 = t0;
      ms.t1 = uncut ? 0 : t0 + per < total ? t0 + per : total;
    }
    __syncthreads();  // (an uncut list's thread writes them again)
#pragma unroll 1
    for (int b = first; b < last; ++b) {
      const int n = cost_of(b);
      if (publish) {
        const int r0 = n > 0 ? static_cast<int>(divide(off + kStart<kH>, per)) : 0, r1 = n > 0 ? static_cast<int>(divide(off + n - 1, per)) : -1;
        p.cuts[b] = uncut ? make_int2(b, n > 0 ? 1 : 0) : make_int2(r0, r1 - r0 + 1);
        // (by its first list, which may have no keys)
        const KeyList k = key_list<kH>(p, b);
        if (b >= p.sh.prefix && (b - p.sh.prefix) % p.sh.groups == 0 && p.a.seq_lens[k.b] > clipped_len(p.a, k.b))
          flag_error(p.a.error_word, MLA_DEVERR_BOUNDS);
      }
      if (uncut ? b == range : t0 >= off && t0 < off + n) {
        ms.b0 = b;
        ms.off0 = off;
        ms.longest = longest;
        if (uncut) {
          ms.t0 = off;
          ms.t1 = off + n;
        }
      }
      off += n;
    }
    return;
  }
  if (tid == 0) {
    ms.t0 = t0;
    ms.t1 = t0 + per < total ? t0 + per : total;
    if (uncut) {
      ms.b0 = range;
      ms.longest = range < B ? clipped_len(p.a, range) : 0;
      ms.t1 = tiles_of(ms.longest);
    }
  }
#pragma unroll 1
  for (int b = first; b < last; ++b) {
    const int n = cost_of(b);
    if (publish) {
      const int r0 = n > 0 ? static_cast<int>(divide(off, per)) : 0, r1 = n > 0 ? static_cast<int>(divide(off + n - 1, per)) : -1;
      p.cuts[b] = uncut ? make_int2(b, n > 0 ? 1 : 0) : make_int2(r0, (r1 - r0 + 1) | (r0 * per < off ? 1 << 30 : 0));
    }
    if (!uncut && t0 >= off && t0 < off + n) {
      ms.b0 = b;
      ms.off0 = off;
      ms.longest = longest;
    }
    off += n;
  }
}

template <int kH, bool kShared>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_decode_kernel(const __grid_constant__ CUtensorMap tm_lat, const __grid_constant__ CUtensorMap tm_rope,
                      const Params p) {
  using C = Cfg<kH>;
  using Work = Pieces<kH, kShared>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc<kH>& ms = *reinterpret_cast<Misc<kH>*>(smem + C::off_misc);
  const uint32_t s0 = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int range = blockIdx.x / p.groups, group = blockIdx.x % p.groups;
  uint32_t* err = p.a.error_word;

  if (threadIdx.x == 0) {
    ms.abort = 0;
    ms.hits[0] = ms.hits[1] = 0;
    ms.b0 = 0;  // a range without tiles has no first sequence
    ms.off0 = 0;
#pragma unroll 1
    for (int i = 0; i < C::slots; ++i) {
      mbar_init(&ms.full[i], 1);
      mbar_init(&ms.empty[i], 1);
    }
    for (int i = 0; i < C::ropes; ++i) {
      mbar_init(&ms.rfull[i], 1);
      mbar_init(&ms.rempty[i], 1);
    }
#pragma unroll 1
    for (int i = 0; i < C::info; ++i) mbar_init(&ms.info_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms.s_full[i], 1);
      mbar_init(&ms.s_free[i], kSoftmax / 32);
    }
    mbar_init(&ms.p_ready, kSoftmax / 32);
    mbar_init(&ms.pv_done, 1);
    mbar_init(&ms.q_ready, kSoftmax / 32);
    mbar_init(&ms.sums_ready, kSoftmax / 32);
    mbar_init(&ms.o_free, kOutput / 32);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms.moved[i], kSoftmax / 32);
      mbar_init(&ms.rescaled[i], kOutput / 32);
      mbar_init(&ms.retired[i], 1);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ms.tmem, 512);
    tmem_relinquish();
  }
  if constexpr (kShared) asm volatile("griddepcontrol.wait;" ::: "memory");  // for the work ahead of this call
  if (p.split) make_plan<kH, kShared>(p, ms, reinterpret_cast<int64_t*>(&ms.sums[0][0]), range, blockIdx.x == 0);
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
    int n = 0, chunks = 0, ropes = 0;  // tiles; copies issued
    bool ok = true;
    for (Work it(p, ms, range); it.next(p);) {
      const int b = it.b, len = it.len, s = it.s, e = it.e;
      // 32 blocks (16 tiles) at a time, one a lane: the block's first slot
      // (past the cache where there is none, so that it reads as zeros) and
      // its scale.  The next 32 page table entries are loaded ahead.
      if (!kShared && s == 0 && group == 0 && lane == 0 && p.a.seq_lens[b] > len) flag_error(err, MLA_DEVERR_BOUNDS);
      const int n_blocks = min((len + kBlock - 1) / kBlock, 2 * e);
      auto page_of = [&](int i) { return i < n_blocks ? block_page(p, b, i + it.block) : -1; };
      int page = page_of(2 * s + lane), y = 0;
      float scale = 0.f;
#pragma unroll 1
      for (int t = s; t < e && ok; ++t, ++n) {
        const int at = (2 * (t - s)) & 31;
        if (at == 0) {
          const int i = 2 * t + lane;
          const int slot = i < n_blocks ? block_slot(p, page, i + it.block) : -1;
          page = page_of(i + 32);
          y = static_cast<int>(slot < 0 ? p.a.num_slots : slot);
          scale = slot < 0 ? 0.f : p.a.scales[slot / kBlock];
        }
        const int y0 = __shfl_sync(0xffffffffu, y, at), y1 = __shfl_sync(0xffffffffu, y, at + 1);
        if (lane == 0) {
#pragma unroll 1
          for (int d = 0; d < 4 && ok; ++d) {
            const int k = 4 * n + d, i = k % C::slots;
            ok = wait(&ms.empty[i], ((k / C::slots) & 1) ^ 1, err, &ms.abort);
            if (!ok) break;
            mbar_expect_tx(&ms.full[i], kChunkBytes);
            tma_load_bytes(slot_addr(i), &tm_lat, 128 * d, y0, &ms.full[i]);
            tma_load_bytes(slot_addr(i) + kChunkBytes / 2, &tm_lat, 128 * d, y1, &ms.full[i]);
            chunks = k + 1;
          }
          if (ok) {
            const int i = n % C::ropes;
            ok = wait(&ms.rempty[i], ((n / C::ropes) & 1) ^ 1, err, &ms.abort);
            if (ok) {
              const uint32_t dst = s0 + C::off_rope + i * kRopeBytes;
              mbar_expect_tx(&ms.rfull[i], kRopeBytes);
              tma_load_bytes(dst, &tm_rope, MLA_D_LATENT, y0, &ms.rfull[i]);
              tma_load_bytes(dst + kRopeBytes / 2, &tm_rope, MLA_D_LATENT, y1, &ms.rfull[i]);
              ropes = n + 1;
            }
          }
        }
        // the blocks' scales (waited for after the copies); tile n - 4, whose
        // place they take, is done: this tile's chunks took those of tile n - 3
        // or a later one
        if (at == 0) {
          const bool block = 2 * t + lane < n_blocks, good = scale >= kScaleMin && scale <= kScaleMax;
          if (block && !good) flag_error(err, y == p.a.num_slots ? MLA_DEVERR_BOUNDS : MLA_DEVERR_SCALE);
          if (!good) scale = 0.f;
        }
        const float sc0 = __shfl_sync(0xffffffffu, scale, at), sc1 = __shfl_sync(0xffffffffu, scale, at + 1);
        if (lane == 0 && ok) {
          ms.scale[n % C::info][0] = sc0;
          ms.scale[n % C::info][1] = sc1;
          mbar_arrive(&ms.info_full[n % C::info]);
        }
        ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0) != 0;
      }
    }
    if (lane == 0) {
      ms.chunks = chunks;
      ms.ropes = ropes;
    }
  } else if (warp == 1) {
    // -------------------------------------------------------- score products
    constexpr uint32_t idesc = idesc_e4m3(128, 2 * kH, false, false);
    const uint64_t dq = smem_desc_sw128(s0 + C::off_q, 0, 1024);
    const uint64_t dq_rope = smem_desc_sw64(s0 + C::off_q + 4 * C::q_chunk, 512);
    bool ok = true;
    auto ready = [&](uint64_t* bar, int parity) {
      ok = __all_sync(0xffffffffu, ok && wait(bar, parity, err, &ms.abort));
      return ok;
    };
    int n = 0, piece = 0;
    for (Work it(p, ms, range); ok && it.next(p);) {
      const int s = it.s, e = it.e;
      if (s >= e) continue;
      if (!ready(&ms.q_ready, piece & 1)) break;
#pragma unroll 1
      for (int t = s; t < e; ++t, ++n) {
        const uint32_t d = uniform(tmem + kColS + (n & 1) * 2 * kH);
        if (!ready(&ms.s_free[n & 1], ((n >> 1) & 1) ^ 1)) break;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          const int k = 4 * n + c, i = uniform(k % C::slots);
          if (!ready(&ms.full[i], (k / C::slots) & 1)) break;
          tc_fence_after();
          const uint64_t da = smem_desc_sw128(slot_addr(i), 0, 1024), db = dq + uniform(c) * (C::q_chunk >> 4);
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_e4m3(d, da + 2 * j, db + 2 * j, idesc, (c > 0 || j > 0) ? 1u : 0u);
          }
          __syncwarp();
        }
        const int i = uniform(n % C::ropes);
        if (!ready(&ms.rfull[i], (n / C::ropes) & 1)) break;
        tc_fence_after();
        const uint64_t da = smem_desc_sw64(s0 + C::off_rope + i * kRopeBytes, 512);
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < 2; ++j) mma_e4m3(d, da + 2 * j, dq_rope + 2 * j, idesc, 1u);
          mma_commit(&ms.rempty[i]);
          mma_commit(&ms.s_full[n & 1]);
        }
        __syncwarp();
      }
      ++piece;
    }
    retire_products(&ms.retired[0], err);
  } else if (warp == 14) {
    // -------------------------------------------------------- value products
    const uint64_t dp = smem_desc_sw64(s0 + C::off_p, 512);
    bool ok = true;
    auto ready = [&](uint64_t* bar, int parity) {
      ok = __all_sync(0xffffffffu, ok && wait(bar, parity, err, &ms.abort));
    };
    int n = 0, piece = 0, k = 0;  // tiles, pieces, tiles that are no piece's first
    for (Work it(p, ms, range); ok && it.next(p);) {
      const int s = it.s, e = it.e;
      if (s >= e) continue;
#pragma unroll 1
      for (int t = s; t < e; ++t, ++n) {
        ready(&ms.p_ready, n & 1);
        // O as it is to be added to: the previous piece's read, this one's
        // rescaled
        if (t > s) {
          ready(&ms.rescaled[k & 1], (k >> 1) & 1);
          ++k;
        } else if (piece > 0) {
          ready(&ms.o_free, (piece - 1) & 1);
        }
        if (!ok) break;
        tc_fence_after();
        // 64 heads: two chunks at a time (64x4096, 128 heads: 86.8 us, 88.0
        // one by one; 32 heads are faster one by one, 135.5 us, not 136.4 for
        // 128 sequences to 32k of 16 heads)
        constexpr int kStep = C::terms;
#pragma unroll 1
        for (int c = 0; c < 4; c += kStep) {
          const int i = uniform((4 * n + c) % C::slots);
          static_assert(C::slots % kStep == 0, "neighbouring chunks in neighbouring slots");
          // V^T: 128 features of the chunk as rows, 32 keys (4096 bytes) a
          // step.  The scores of this tile are done (P came of them), so
          // the chunk is free after these.
          const uint64_t da = smem_desc_sw128(slot_addr(i), 0, 1024);
          const uint32_t d = uniform(tmem + 64 * c);
          if (elect_one()) {
#pragma unroll
            for (int x = 0; x < kStep; ++x) {
#pragma unroll
              for (int term = 0; term < C::terms; ++term) {
                // e4m3 x e4m3, or e4m3 x e5m2 (format 1) for the second term
                const uint32_t idesc = idesc_e4m3(128, 64, true, true) | (term == 1 ? 1u << 10 : 0u);
                const uint64_t db = dp + term * (kTile * 64 >> 4);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  mma_e4m3(d + 64 * x, da + x * (kChunkBytes >> 4) + 256 * j, db + 128 * j, idesc,
                           (t > s || term > 0 || j > 0) ? 1u : 0u);
              }
              mma_commit(&ms.empty[i + x]);
            }
            if (c + kStep == 4) mma_commit(&ms.pv_done);
          }
          __syncwarp();
        }
      }
      ++piece;
    }
    retire_products(&ms.retired[1], err);
  } else if (warp < 10) {
    // ---------------------------------------------------- queries, softmax
    // A wait that gives up leaves these warps running through their loops
    // (they meet at named barriers); the error word tells.
    constexpr int kMine = C::mine;
    const int quad = warp & 3, wg = (warp - 2) >> 2, tid = (threadIdx.x - 64) & 127;
    const int hb = wg * kMine;         // this thread's first head
    const int key = quad * 32 + lane;  // of the tile: a TMEM lane
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    // offset of the second term's rounding: (j + 1/2) / 32 - 1/2, j the
    // lane's bits reversed, of a step 2^-13 (32 heads: 2^-9, after the gain)
    const float off = ((__brev(lane) >> 27) + 0.5f) * (1.f / 32) - 0.5f;
    const __half2 dither_h = __float2half2_rn(off * (kH == 32 ? kGain : 1.f) * 0.0001220703125f);
    const uint32_t dither = *reinterpret_cast<const uint32_t*>(&dither_h);
    int n = 0, piece = 0, k = 0;
    for (Work it(p, ms, range); it.next(p);) {
      const int len = it.len, s = it.s, e = it.e, heads = it.rows;
      const int64_t row = it.row(p);
      if (!kShared && s >= e) {  // no keys
        uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.a.out) + row * MLA_D_LATENT);
        for (int i = threadIdx.x - 64; i < heads * (MLA_D_LATENT / 8); i += kSoftmax) out[i] = make_uint4(0, 0, 0, 0);
        if (p.a.lse != nullptr)
          for (int i = threadIdx.x - 64; i < heads; i += kSoftmax) p.a.lse[row + i] = -INFINITY;
        continue;
      }
      // Queries (the previous piece's last scores, which this half has read,
      // were the last to use them): a warp takes every fourth head of its
      // half, four at a time (of 64 heads two, the next two's loads in flight: 32 x
      // (32768 + 1000) shared keys, 128 heads 254 us, with four 255; 128 sequences to
      // 32k of 16 heads 135, with two 139).
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.a.q) + row * kKey;
      const int limit = min(heads, hb + kMine);
      constexpr int kN = kH == 64 ? 2 : 4;
      QueryHeads<kN> next;
      next.load(q, lane, hb + quad, 4, limit);
#pragma unroll 1
      for (int h = hb + quad; h < hb + kMine; h += 4 * kN) {
        const QueryHeads<kN> now = next;
        if (kMine > 4 * kN) next.load(q, lane, h + 4 * kN, 4, limit);
        float c[kN];
        query_terms<kH>(now, lane, h, 4, s0 + C::off_q, p.a.softmax_scale, c);
#pragma unroll
        for (int j = 0; j < kN; ++j)
          if (lane == j) ms.c[h + 4 * j] = c[j];
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.q_ready);
      const float* cs = ms.c + hb;
      float* mr = ms.m + hb;  // the references
      if (tid < kMine) {
        mr[tid] = 0.f;
        ms.top[hb + tid] = ordered(-INFINITY);
      }
      half_bar(wg);

      float l[kMine];
#pragma unroll
      for (int h = 0; h < kMine; ++h) l[h] = 0.f;
      bool seen = false;  // there was a key
      uint32_t unset = static_cast<uint32_t>((uint64_t{1} << kMine) - 1);  // heads whose reference follows no key yet
#pragma unroll 1
      for (int t = s; t < e; ++t, ++n) {
        wait(&ms.info_full[n % C::info], (n / C::info) & 1, err, &ms.abort);
        const float scale = ms.scale[n % C::info][quad >> 1];
        const float sb = scale > 0.f ? scale : 1.f, lsb = log2f(sb);
        const bool valid = scale > 0.f && t * kTile + key < len;
        const bool full = __all_sync(0xffffffffu, valid);

        wait(&ms.s_full[n & 1], (n >> 1) & 1, err, &ms.abort);
        tc_fence_after();
        const uint32_t src = lanes + kColS + (n & 1) * 2 * kH + hb;
        float x[kMine], top = -INFINITY;
#pragma unroll
        for (int g = 0; g < kMine; g += 16) {
          uint32_t v[16], u[16];
          tmem_ld16(src + g, v);
          tmem_ld16(src + kH + g, u);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const int h = g + i;
            const float4 cc = *reinterpret_cast<const float4*>(cs + h), mm = *reinterpret_cast<const float4*>(mr + h);
            const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, mv[4] = {mm.x, mm.y, mm.z, mm.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              x[h + j] =
                  fmaf(fmaf(__uint_as_float(u[i + j]), 1.f / kGain, __uint_as_float(v[i + j])) * sb, cv[j], -mv[j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.s_free[n & 1]);
        if (!full) {
#pragma unroll
          for (int h = 0; h < kMine; ++h) x[h] = valid ? x[h] : -INFINITY;
        }
#pragma unroll
        for (int h = 0; h < kMine; ++h) top = fmaxf(top, x[h]);
        // Raise the references of the heads that need it.
        const bool any = __any_sync(0xffffffffu, top + lsb > kTop || (unset != 0 && valid));
        if (any) {
          // A head's maximum: halves exchanged until lane i holds head
          // i * kMine / 32 of the warp's keys, then over the warps.
          float f[kMine / 2];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const bool up = (lane & o) != 0;
            const int half = kMine * o / 32;
            if (half == 0) f[0] = fmaxf(f[0], __shfl_xor_sync(0xffffffffu, f[0], o));
#pragma unroll
            for (int h = 0; h < kMine / 2; ++h) {
              if (h < half) {
                const float lo = o == 16 ? x[h] : f[h], hi = o == 16 ? x[h + half] : f[(h + half) % (kMine / 2)];
                f[h] = fmaxf(up ? hi : lo, __shfl_xor_sync(0xffffffffu, up ? lo : hi, o));
              }
            }
          }
          const int h = lane * kMine / 32;
          if ((unset >> h & 1) != 0 || f[0] + lsb > kTop) {
            atomicMax(&ms.top[hb + h], ordered(f[0] + lsb));
            atomicOr(&ms.hits[wg], 1u << h);
          }
        }
        if (half_any(wg, any)) {
          if (tid < 32) {
            const bool hit = (ms.hits[wg] >> lane & 1) != 0;
            const float mx = hit ? from_ordered(ms.top[hb + lane]) : 0.f;
            const bool raise = hit && isfinite(mx) && ((unset >> lane & 1) != 0 || mx > kTop);
            const float by = raise ? mx - kReset : 0.f;
            if (lane < kMine) ms.move[k & 1][hb + lane] = by;
            if (raise) mr[lane] += by;
            if (hit) ms.top[hb + lane] = ordered(-INFINITY);
            const uint32_t raised = __ballot_sync(0xffffffffu, raise);
            if (lane == 0) {
              ms.hits[wg] = 0;
              ms.moves[wg] = raised;
              // without earlier weights O is zero (or yet to be written)
              ms.raised[k & 1][wg] = raised & ~unset;
            }
          }
          half_bar(wg);
          const uint32_t moves = ms.moves[wg];
#pragma unroll
          for (int h = 0; h < kMine; h += 4) {
            if (moves >> h & 15) {
              const float4 mv = *reinterpret_cast<const float4*>(&ms.move[k & 1][hb + h]);
              const float by[4] = {mv.x, mv.y, mv.z, mv.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                x[h + j] -= by[j];
                if ((unset >> (h + j) & 1) == 0) l[h + j] *= ex2_approx(-by[j]);  // (else 0, or NaN)
              }
            }
          }
          seen = true;
          unset &= ~moves;
        } else if (tid == 0) {
          ms.raised[k & 1][wg] = 0;
        }
        if (t > s) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&ms.moved[k & 1]);
          ++k;
        }
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
            const uint32_t rest = h2_sub(pu, e4m3x2_to_f16x2_pair(a[j]));
            r[j] = kH == 32 ? cvt_e4m3x2_h2(h2_fma(rest, kGain, dither)) : cvt_e5m2x2_h2(h2_steps(h2_fma(rest, 1.f, dither)));
          }
          w1[h / 4] = a[0] | (a[1] << 16);
          w2[h / 4] = r[0] | (r[1] << 16);
        }
        // the previous tile's products have read P
        if (n > 0) wait(&ms.pv_done, (n - 1) & 1, err, &ms.abort);
        {
          // row = key, 64 bytes: heads of one term, or p1 | p2; 16-byte units
          // swizzled by the row
          const uint32_t row = s0 + C::off_p + key * 64, sw = (key >> 1) & 3;
          if constexpr (kH == 64) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint32_t at = row + (((2 * wg + c) ^ sw) << 4);
              sts128(at, make_uint4(w1[4 * c], w1[4 * c + 1], w1[4 * c + 2], w1[4 * c + 3]));
              sts128(at + kTile * 64, make_uint4(w2[4 * c], w2[4 * c + 1], w2[4 * c + 2], w2[4 * c + 3]));
            }
          } else {
            sts128(row + ((wg ^ sw) << 4), make_uint4(w1[0], w1[1], w1[2], w1[3]));
            sts128(row + (((wg + 2) ^ sw) << 4), make_uint4(w2[0], w2[1], w2[2], w2[3]));
          }
        }
        // a row that is no key of the sequence may hold any bytes (NaN too):
        // as values they are zeros
        if (!valid) {
#pragma unroll 1
          for (int c = 2 * wg; c < 2 * wg + 2; ++c) {
            const uint32_t row = slot_addr((4 * n + c) % C::slots) + key * 128;
#pragma unroll
            for (int i = 0; i < 8; ++i) sts128(row + 16 * ((i + lane) & 7), make_uint4(0, 0, 0, 0));  // all banks
          }
        }
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.p_ready);
      }

      // The weights' sums over this warp's keys, exchanged as above, for the
      // output warps (done with the previous piece's).
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const bool up = (lane & o) != 0;
        const int half = kMine * o / 32;
        if (half == 0) l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
#pragma unroll
        for (int h = 0; h < kMine / 2; ++h) {
          if (h < half) {
            const float give = up ? l[h] : l[h + half], keep = up ? l[h + half] : l[h];
            l[h] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
        }
      }
      if (piece > 0) wait(&ms.o_free, (piece - 1) & 1, err, &ms.abort);
      ms.sums[quad][hb + lane * kMine / 32] = l[0];
      if (tid < kMine) ms.inv[hb + tid] = seen ? mr[tid] : -INFINITY;  // -inf: no keys
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.sums_ready);
      half_bar(wg);  // c is free for the next piece
      ++piece;
    }
  } else {
    // --------------------------------------------------------------- output
    const int quad = warp & 3, tid = (threadIdx.x - 64) & 127;
    const int row = quad * 32 + lane;  // of a value chunk: a TMEM lane
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    int piece = 0, n_last = -1, k = 0;  // the piece's last tile; tiles that are no piece's first
    for (Work it(p, ms, range); it.next(p);) {
      if (it.s >= it.e) continue;
      const int heads = it.rows;
      const bool whole = !kShared && it.e - it.s == it.n;
      const int64_t out_row = it.row(p), part_row = it.part_row(p, range);
      n_last += it.e - it.s;
      // the next sequence's or list's queries, into L2 meanwhile
      int64_t next_row = out_row + p.a.num_heads;
      int next_rows = it.b + 1 < p.a.batch ? heads : 0;
      if constexpr (kShared) {
        next_rows = 0;
        if (it.list + 1 < p.sh.lists) {
          const KeyList k = key_list<kH>(p, it.list + 1);
          next_row = k.row;
          next_rows = k.rows;
        }
      }
      if (next_rows > 0) {
        const char* q = static_cast<const char*>(p.a.q) + next_row * (kKey * 2);
        for (int i = tid; i < next_rows * (kKey * 2 / 128); i += kOutput)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(q + 128 * i));
      }
      // Rescaling: a head's columns of the value chunks (kH 32: of both terms)
      // times 2^-move, once the tile before is in.
#pragma unroll 1
      for (int n = n_last - (it.e - it.s) + 1; n < n_last; ++n, ++k) {
        wait(&ms.moved[k & 1], (k >> 1) & 1, err, &ms.abort);
        uint64_t raised = ms.raised[k & 1][0] | static_cast<uint64_t>(ms.raised[k & 1][1]) << (kH / 2);
        if (raised != 0) {
          wait(&ms.pv_done, n & 1, err, &ms.abort);
          tc_fence_after();
#pragma unroll 1
          for (; raised != 0; raised &= raised - 1) {
            const int h = __ffsll(static_cast<long long>(raised)) - 1;
            const float f = ex2_approx(-ms.move[k & 1][h]);
            constexpr int kCols = 256 / kH;
            float o[kCols];
#pragma unroll
            for (int i = 0; i < kCols; ++i) tmem_ld1(lanes + kH * i + h, o[i]);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < kCols; ++i) tmem_st1(lanes + kH * i + h, o[i] * f);
          }
          tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.rescaled[k & 1]);
      }
      // sums first: then the last tile's products are the next phase of pv_done
      wait(&ms.sums_ready, piece & 1, err, &ms.abort);
      if (tid < kH) {
        const float m = ms.inv[tid];
        float sum = (ms.sums[0][tid] + ms.sums[1][tid]) + (ms.sums[2][tid] + ms.sums[3][tid]);
        // a score above fp32's range, or all of a sequence's below it (of a
        // piece's: kBelow, and the merge decides)
        const bool below = sum == 0.f && m != -INFINITY;
        if (isinf(sum) || (below && whole)) sum = __uint_as_float(0x7FC00000u);
        ms.inv[tid] = sum != 0.f ? 1.f / sum : 0.f;  // NaN stays NaN
        const float l2 = sum != 0.f ? m + log2f(sum) : below ? kBelow : -INFINITY;
        if (!whole) {
          if (!kShared || tid < heads) p.part_lse[part_row + tid] = l2;
        } else if (p.a.lse != nullptr && tid < heads)
          p.a.lse[out_row + tid] = l2 * kLn2;
      }
      asm volatile("bar.sync 5, %0;" ::"n"(kOutput) : "memory");
      wait(&ms.pv_done, n_last & 1, err, &ms.abort);
      tc_fence_after();
      // thread = feature; neighbouring threads swap halves of two heads so
      // that each stores two features of one
#pragma unroll 1
      for (int i = 0; i < 4 * C::terms; ++i) {
        const int c = i / C::terms, g = 32 * (i % C::terms);  // value chunk, first head
        const int d = 128 * c + row;
        uint32_t v[32];
        tmem_ld32(lanes + 64 * c + g, v);
        if constexpr (kH == 32) {  // p1's and p2's products
          uint32_t u[32];
          tmem_ld32(lanes + 64 * c + 32, u);
          tmem_ld_wait();
#pragma unroll
          for (int h = 0; h < 32; ++h)
            v[h] = __float_as_uint(fmaf(__uint_as_float(u[h]), 1.f / kGain, __uint_as_float(v[h])));
        } else {
          tmem_ld_wait();
        }
#pragma unroll
        for (int h = 0; h < 32; h += 4) {
          const float4 iv = *reinterpret_cast<const float4*>(&ms.inv[g + h]);
          v[h] = __float_as_uint(__uint_as_float(v[h]) * iv.x);
          v[h + 1] = __float_as_uint(__uint_as_float(v[h + 1]) * iv.y);
          v[h + 2] = __float_as_uint(__uint_as_float(v[h + 2]) * iv.z);
          v[h + 3] = __float_as_uint(__uint_as_float(v[h + 3]) * iv.w);
        }
        if (i == 4 * C::terms - 1) {  // O and inv are free
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ms.o_free);
        }
        if (whole) {
          const int odd = lane & 1;
          uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.a.out) +
                                                      (out_row + g + odd) * MLA_D_LATENT + (d - odd));
#pragma unroll
          for (int h = 0; h < 32; h += 2) {
            const float mine = __uint_as_float(odd ? v[h + 1] : v[h]);
            const float got = __shfl_xor_sync(0xffffffffu, __uint_as_float(odd ? v[h] : v[h + 1]), 1);
            const __nv_bfloat162 o = odd ? __floats2bfloat162_rn(got, mine) : __floats2bfloat162_rn(mine, got);
            if (g + h + odd < heads) dst[h * (MLA_D_LATENT / 2)] = *reinterpret_cast<const uint32_t*>(&o);
          }
        } else {
          float* dst = p.part_o + (part_row + g) * MLA_D_LATENT + d;
#pragma unroll
          for (int h = 0; h < 32; ++h)
            if (g + h < heads) dst[h * MLA_D_LATENT] = __uint_as_float(v[h]);
        }
      }
      ++piece;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
  if (warp == 0 && lane == 0 && ms.abort) {
    drain_copies(ms.full, C::slots, ms.chunks);
    drain_copies(ms.rfull, C::ropes, ms.ropes);
  }
}

// Merge of the pieces of cut sequences, in range order, by LSE (of a prefix
// before those of a sequence's own keys); sequences without keys get their
// zeros here.  kSub warps = half the features of one (sequence, head), 8 a
// lane; each takes every kSub-th piece.
template <int kSub>
constexpr int merge_threads = kSub > 1 ? 64 * kSub : 256;
template <int kH, int kSub, bool kShared>
__global__ void __launch_bounds__(merge_threads<kSub>) fp8_decode_merge_kernel(const Params p) {
  if constexpr (kShared) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the next call's, which wait)
  const int lane = threadIdx.x & 31;
  const int64_t id = (static_cast<int64_t>(blockIdx.x) * merge_threads<kSub> + threadIdx.x) / (32 * kSub);
  const int sub = kSub > 1 ? (threadIdx.x >> 5) % kSub : 0;
  const int64_t row = id >> 1;
  if (row >= static_cast<int64_t>(p.a.batch) * p.a.num_heads) return;
  const int b = static_cast<int>(row / p.a.num_heads), h = static_cast<int>(row - static_cast<int64_t>(b) * p.a.num_heads);
  const int half = static_cast<int>(id & 1);
  // its pieces, and the row of partial results of each
  int n, n0 = 0, first = 0;
  int64_t row0, own0 = 0;
  if constexpr (kShared) {
    const int own = p.sh.prefix + b * p.sh.groups + h / kH, list = static_cast<int>(row / kH);
    const int2 mine = p.cuts[own];
    const bool shares = p.sh.prefix > 0 && clipped_len(p.a, b) >= p.sh.len;
    const int2 pre = shares ? p.cuts[list] : make_int2(0, 0);
    n0 = pre.y;
    n = n0 + mine.y;
    row0 = (static_cast<int64_t>(list) + pre.x) * kH + row % kH;
    own0 = p.sh.own + (own - p.sh.prefix + mine.x - static_cast<int64_t>(n0)) * p.sh.own_rows + h % kH;
  } else {
    const int2 cut = p.cuts[b];
    n = cut.y & ~(1 << 30), first = cut.y >> 30;  // pieces; part of the first
    if (n == 1) return;                           // written already
    row0 = cut.x * static_cast<int64_t>(p.groups) * 2 * kH + (h / kH) * 2 * kH + h % kH;
  }
  auto part_of = [&](int i) {
    if constexpr (kShared)
      return i < n0 ? row0 + static_cast<int64_t>(i) * kH : own0 + static_cast<int64_t>(i) * p.sh.own_rows;
    else
      return row0 + i * (static_cast<int64_t>(p.groups) * 2 * kH) + (i == 0 ? first * kH : 0);
  };
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.a.out) + row * MLA_D_LATENT + 256 * half + 4 * lane;
  // lane i: LSE of piece i, i + 32, ...
  auto lse_of = [&](int i) { return i < n ? p.part_lse[part_of(i)] : -INFINITY; };
  float m = -INFINITY;
  for (int i = lane; i < n; i += 32) m = fmaxf(m, lse_of(i));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float ref = m == -INFINITY ? 0.f : m;
  float sum = 0.f, acc[8] = {};
  for (int base = 0; base < n; base += 32) {
    const float w_mine = ex2_approx(lse_of(base + lane) - ref);
    const int count = min(32, n - base);
#pragma unroll 4
    for (int j = sub; j < count; j += kSub) {
      const float w = __shfl_sync(0xffffffffu, w_mine, j);
      const int i = base + j;
      const float4* o = reinterpret_cast<const float4*>(p.part_o + part_of(i) * MLA_D_LATENT + 256 * half + 4 * lane);
      const float4 u = o[0], v = o[32];
      sum += w;
      acc[0] = fmaf(w, u.x, acc[0]), acc[1] = fmaf(w, u.y, acc[1]);
      acc[2] = fmaf(w, u.z, acc[2]), acc[3] = fmaf(w, u.w, acc[3]);
      acc[4] = fmaf(w, v.x, acc[4]), acc[5] = fmaf(w, v.y, acc[5]);
      acc[6] = fmaf(w, v.z, acc[6]), acc[7] = fmaf(w, v.w, acc[7]);
    }
  }
  if (kSub > 1) {  // (one row a CTA: its warps left above together or are all here)
    __shared__ float part[2 * kSub][9][32];
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int k = 0; k < 8; ++k) part[warp][k][lane] = acc[k];
    part[warp][8][lane] = sum;
    __syncthreads();
    if (sub != 0) return;
    for (int s = 1; s < kSub; ++s) {
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] += part[warp + s][k][lane];
      sum += part[warp + s][8][lane];
    }
  }
  if (m == kBelow) sum = __uint_as_float(0x7FC00000u);
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[4 * k] * inv, acc[4 * k + 1] * inv);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(acc[4 * k + 2] * inv, acc[4 * k + 3] * inv);
    *reinterpret_cast<uint2*>(out + 128 * k) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
  if (p.a.lse != nullptr && half == 0 && lane == 0) p.a.lse[row] = sum != 0.f ? (ref + log2f(sum)) * kLn2 : -INFINITY;
}

int heads_per_cta(int num_heads) { return num_heads <= 32 ? 32 : 64; }

struct Layout {
  int ranges, groups;
  size_t lse, o, total;
};
Layout layout(int batch, int num_heads, int num_sms) {
  const int kh = heads_per_cta(num_heads);
  Layout l;
  l.groups = (num_heads + kh - 1) / kh;
  l.ranges = num_sms / l.groups > 1 ? num_sms / l.groups : 1;
  const size_t rows = static_cast<size_t>(l.ranges) * l.groups * 2 * kh;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  l.lse = up(static_cast<size_t>(batch) * sizeof(int2));
  l.o = up(l.lse + rows * sizeof(float));
  l.total = l.o + rows * MLA_D_LATENT * sizeof(float);
  return l;
}

template <int kH, bool kShared>
int launch(const Params& p, const CUtensorMap& lat, const CUtensorMap& rope, int slot, cudaStream_t stream) {
  constexpr int bytes = static_cast<int>(smem_bytes<kH>());
  const auto kern = fp8_decode_kernel<kH, kShared>;
  if (const int st = smem_limit_once(reinterpret_cast<const void*>(kern), bytes, slot)) return st;
  if constexpr (kShared) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.ranges));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // (griddepcontrol)
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (const int st = cuda_status(cudaLaunchKernelEx(&cfg, kern, lat, rope, p))) return st;
  } else {
    kern<<<static_cast<unsigned>(p.ranges) * p.groups, kThreads, bytes, stream>>>(lat, rope, p);
    if (const int st = launch_status()) return st;
  }
  if (!p.split) return MLA_OK;
  // A CTA a row where the rows are cut into many pieces.
  const int64_t rows = static_cast<int64_t>(p.a.num_heads) * p.a.batch;
  if (p.ranges / kManyPieces >= (kShared ? p.sh.prefix : p.a.batch))
    fp8_decode_merge_kernel<kH, kSub, kShared><<<static_cast<unsigned>(rows), merge_threads<kSub>, 0, stream>>>(p);
  else
    fp8_decode_merge_kernel<kH, 1, kShared><<<static_cast<unsigned>((rows + 3) / 4), 256, 0, stream>>>(p);
  return launch_status();
}

int cache_maps(const Fp8DecodeArgs& a, CUtensorMap* lat, CUtensorMap* rope) {
  if (encode_byte_map(lat, a.cache, kKey, a.num_slots, kKey, 128, kBlock, false) &&
      encode_byte_map(rope, a.cache, kKey, a.num_slots, kKey, 64, kBlock, true))
    return MLA_OK;
  set_last_error("cuTensorMapEncodeTiled failed for the cache");
  return MLA_ERR_LAUNCH;
}

// Shared prefix: the batch's rows decide on the heads a CTA.
struct SharedLayout {
  int kh;
  SharedPlan plan;
  size_t lse, o, total;
};
SharedLayout shared_layout(int kh, int batch, int num_heads, int num_sms, int64_t shared_len) {
  SharedLayout l;
  const int64_t rows = static_cast<int64_t>(batch) * num_heads;
  l.kh = kh;
  constexpr int64_t kNever = (int64_t(1) << 31) - kBlock;  // (longer than a sequence can be)
  l.plan.len = shared_len < kNever ? shared_len : kNever;
  l.plan.prefix = static_cast<int>((rows + l.kh - 1) / l.kh);
  l.plan.groups = (num_heads + l.kh - 1) / l.kh;
  l.plan.lists = l.plan.prefix + batch * l.plan.groups;
  l.plan.own_rows = num_heads < l.kh ? num_heads : l.kh;
  l.plan.own = (static_cast<int64_t>(l.plan.prefix) + num_sms) * l.kh;
  const size_t all = l.plan.own + (static_cast<int64_t>(batch) * l.plan.groups + num_sms) * l.plan.own_rows;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  l.lse = up(static_cast<size_t>(l.plan.lists) * sizeof(int2));
  l.o = up(l.lse + all * sizeof(float));
  l.total = l.o + all * MLA_D_LATENT * sizeof(float);
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
  // Where the page table holds too few keys for a sequence to be cut (as
  // make_plan decides, with one tile or more a range), plan and merge are left
  // out: 1 x 100 keys, 16 heads, 9.9 us, not 12.3.  (The table's width decides,
  // since lengths are on the device: a wider one costs the 12.3, however few keys
  // it is used for.)
  const bool split =
      ws != nullptr && (a.batch > l.ranges || a.max_pages * a.page_size > (1 + kMerge) * kTile);
  Params p{a, magic, shift, l.ranges, l.groups, split, reinterpret_cast<int2*>(ws), reinterpret_cast<float*>(ws + l.lse),
           reinterpret_cast<float*>(ws + l.o), SharedPlan{}};
  if (static_cast<int64_t>(a.batch) * a.num_heads > (int64_t(1) << 31) - 1) return MLA_ERR_INVALID_ARG;
  CUtensorMap lat, rope;
  if (const int st = cache_maps(a, &lat, &rope)) return st;
  return heads_per_cta(a.num_heads) == 64 ? launch<64, false>(p, lat, rope, 19, stream)
                                          : launch<32, false>(p, lat, rope, 20, stream);
}

size_t fp8_shared_workspace_bytes(int batch, int num_heads, int num_sms) {
  const size_t a = shared_layout(32, batch, num_heads, num_sms, 0).total;
  const size_t b = shared_layout(64, batch, num_heads, num_sms, 0).total;
  return a > b ? a : b;
}

int launch_fp8_shared(const Fp8DecodeArgs& a, int64_t shared_len, cudaStream_t stream, int num_sms) {
  // 64 rows a CTA, where the keys are read half as often and a tile of 64 rows
  // takes little longer than one of 32; 32 where no CTA would have two tiles of
  // the prefix, and its start counts (but not for heads that fill 64 rows: their
  // own keys may be many).  4 x (2048 + 64) keys of 16 heads 14.8 us with 32 rows, 17.9
  // with 64; 64 x (4096 + 64) 31.8 and 34.9, x (8192 + 64) 42.8 and 41.8, x (32768 + 64)
  // 113 and 85.  (Long prefixes of few rows would do better with 32 up to about 100
  // tiles a list: 4 x (32768 + 64) 23.1 and 27.9.)
  const int64_t rows = static_cast<int64_t>(a.batch) * a.num_heads;
  const bool few = a.num_heads <= 32 && (rows + 31) / 32 * ((shared_len + kTile - 1) / kTile) <= num_sms;
  const SharedLayout l = shared_layout(few ? 32 : 64, a.batch, a.num_heads, num_sms, shared_len);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  uint32_t magic;
  int shift;
  magic_divisor(a.page_size / kBlock, &magic, &shift);
  const Params p{a, magic, shift, num_sms, 1, true, reinterpret_cast<int2*>(ws), reinterpret_cast<float*>(ws + l.lse),
                 reinterpret_cast<float*>(ws + l.o), l.plan};
  CUtensorMap lat, rope;
  if (const int st = cache_maps(a, &lat, &rope)) return st;
  return l.kh == 64 ? launch<64, true>(p, lat, rope, 24, stream) : launch<32, true>(p, lat, rope, 25, stream);
}

}  // namespace mla
