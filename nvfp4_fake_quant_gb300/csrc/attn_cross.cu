// Attention of many query rows over the paged NVFP4 cache, every row of a sequence seeing all
// of the sequence's cached keys:
//   S_j = scale q~ . K~_j,  o = sum_j exp(S_j - lse) V~_j,  lse = ln sum exp S_j
// The rows of a (sequence, KV head) are its tokens times the query heads that share the KV
// head.  Two callers: cross attention (the keys: an encoder's states), and single tokens
// behind a shared prefix (a "sequence": the batch entries that share it; the keys: the
// prefix, read once for all of them).
//
// Work split.  Tiles (256 rows x one page of 128 keys) of all (sequence, KV head, row tile)
// lie one after another on one line, cut into equal runs, one CTA each, whatever the lengths.
// A segment (one sequence, KV head and row tile) inside a run is written by it; one that
// crosses runs leaves (m, l, sum p V~) per run in the workspace, joined in run order by a
// second kernel: results do not vary from run to run.
//
// One CTA, twenty warps:
//   producer   K codes by tensor-map loads with the swizzle the MMA reads, the record's rest
//              by bulk copies, into a ring of stages, with a description of each tile
//   4 decode   V's codes times scales, exactly, to f16 rows in shared memory (scales run
//              along D, so codes cannot be the FP4 operand of a product over keys), once for
//              both streams; the first of them brings K's scales into the scale operand's order
//   4 query    q~ of the segments, up to two ahead (of the first with the help of the softmax and
//              decode warps); rows without keys
//   2 x S      S = Q~ K~^T as block-scaled FP4 tcgen05 MMAs on the codes.  A unit is 128 rows x
//              64 keys; the units of two streams (two halves of the rows; of 128 rows or fewer
//              two halves of the keys, joined where the segment ends) go in turn through three
//              buffers of 64 columns, so that S of the next unit is there when a stream's
//              softmax has ended
//   PV         O += P V~ as f16 MMAs, P from tensor memory (over the S it came from)
//   2 x 4      softmax, one thread a row, a warpgroup for each stream.  The maximum that p
//              refers to is raised only where a score exceeds it by 8 (log2); the row's thread
//              then rescales O itself
// p is rounded to f16, its sum taken before the rounding; all sums are fp32.  p is 2^7 where the
// score is the reference maximum, so at most 2^15: f16 has no more room above, and 2^32 below the
// best key a p is still seen (from 1 on, keys 2^25 below a dominant one vanished from O, not from
// the sum).
//
// Measured, in a replayed graph: 32760 tokens x 12 heads over 512 keys 113.5 us (0.91 PFLOP/s, 46%
// of the bf16 rate; plain 9203 us), four latents of up to 6272 tokens 101.5 us, nine short pieces
// 23.6 us; 32 sequences x 64 heads behind 131072 shared keys 131 us with the join and the sequences' own
// keys (1.05 PFLOP/s; one read of the prefix takes 22 us).  A tile takes 3400 to 3800 cycles, of
// which its MMAs need 1280 and its exponentials 1024: the bound is the chain of waits between the
// roles (150 to 300 cycles each beside four other warps of the scheduler), and in short segments q~
// and the rows on their way out (4000 cycles a segment).  Slower were: P beside S with S a unit
// ahead for each stream (146 us where this is 130), the same with two warps for P V~ at 80
// registers (147), one warp for S and two for P V~ (140), 128-key units, sixteen softmax warps.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "nvq_internal.h"
#include "nvq_kv.cuh"
#include "nvq_ptx.cuh"
#include "nvq_quant.cuh"

namespace nvq {

namespace {

constexpr int kRows = 128;     // query rows of a unit
constexpr int kPair = 256;     // and of a tile
constexpr int kKeys = 64;      // keys of a unit
constexpr int kThreads = 640;
constexpr int kDecodeWarp = 8, kQWarp = 12, kProducerWarp = 16, kSWarp = 17, kPvWarp = 19;
constexpr int kSegs = 8;       // descriptions of segments: the query warps are two ahead of S, the
                               // softmax of an end may be one behind it
constexpr float kUp = 7.f;     // p is 2^kUp at the reference maximum
// tensor memory columns: S of unit u at 64 (u % 3), O of the two streams, the scales of q~ (two
// buffers of both streams) and of K (of each stream two: a copy never overwrites what an MMA in
// flight may read, see the S warps).  Heads of 64 leave columns 320 to 447 unused.
constexpr uint32_t kO = 192, kSfQ = 448, kSfK = 480;

enum : int { kStart = 1, kEnd = 2, kAbsent = 4, kBoth = 8 };
enum : int { kValid = 127, kUnitStart = 128, kUnitEnd = 256, kUnitLast = 512 };

struct Tile {
  int flags, valid;  // kBoth: over 128 rows; keys of the page that hold tokens
  int rows, seg;     // of the segment; segments before it in the run
};

template <int D>
struct Cfg {
  static constexpr int kStages = D == 128 ? 3 : 8;
  static constexpr uint32_t kRec = record_bytes(D);
  static constexpr uint32_t kV = kRows * D * 2;          // a page's V~ in f16
  static constexpr uint32_t kQ = kRows * D / 2;          // codes of q~
  static constexpr uint32_t kQSc = D / 64 * 512;         // and scales
  static constexpr uint32_t kVAt = kStages * kRec;       // [2]
  static constexpr uint32_t kQAt = kVAt + 2 * kV;        // [2][2 halves]
  static constexpr uint32_t kQScAt = kQAt + 4 * kQ;      // [2][2]
  static constexpr uint32_t kOutAt = kQScAt + 4 * kQSc;  // rows of o on their way out: of each
  static constexpr uint32_t kOut = 32 * D * 2;           // warp 32 of 2 D bytes
  static constexpr uint32_t kMlAt = kOutAt + kPair / 32 * kOut;  // float2 [2][128]: streams' (m, l)
  static constexpr uint32_t kDescAt = kMlAt + 2 * kRows * 8;
  static constexpr uint32_t kSegAt = kDescAt + kStages * 16;   // Segment [kSegs]
  static constexpr uint32_t kUnitAt = kSegAt + kSegs * 48;       // int [2 streams][3 (4)]
  static constexpr uint32_t kBarAt = kUnitAt + 32;
  static constexpr int kBars = 3 * kStages + 4 * 2 + 4 * 3 + 2 * 2 + 3 + 8 + kSegs + 1;
  // heads of 64: padded so that no CTA of the few-rows linear lies beside one
  static constexpr uint32_t kUsed = kBarAt + kBars * 8 + 1024;
  static constexpr uint32_t kSmem = kUsed > 152 * 1024 ? kUsed : 152 * 1024;
  static_assert(kRec % 1024 == 0 && kQ % 1024 == 0 && kOutAt % 1024 == 0, "swizzle atoms");
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(apart_from_linear_small(kSmem), "tensor memory");
};

// A segment that begins in a run and goes on in later ones: the line's last tile of it (below 0:
// there is none) and the number of tiles of the line.
struct Split {
  int64_t end, all;
  int slot, rows, row0, tok0, hk, pad;
};

// A segment as the query warps hand it to the others.
struct Segment {
  int row0, rows;  // its first row among the rows of its (sequence, KV head), and their number
  int tok0, hk;    // first token of the sequence; KV head
  int slot;        // where the segment's part goes (-1: it is whole)
  int s, i, i_end, len;  // its pages in the run, of a sequence of len keys
  int pad[3];
};

struct CrossArgs {
  const uint16_t* q;
  int64_t ld_q;
  int T;
  const uint8_t* pool;
  int64_t num_pages;
  const int32_t* table;
  int64_t ld_table;
  int max_pages;
  const int32_t* lens;
  const int32_t* cu;
  int per_seq;  // tokens of each sequence where cu is null
  int B, H, Hkv, G;
  int tiles;  // whole warps' rows of o go by the tensor map: G divides 32
  Scales scale;
  __nv_bfloat16* o;  // or, where null, o32 with the logarithms (base 2) in lse
  float* o32;
  float* lse;
  Split* split;  // [runs]
  float* parts;  // [2 runs][part_rows] (m, l), then [part_rows][D]
  int part_rows, runs;
  uint64_t runs_magic;  // 2^64 / runs, rounded up
  int* err;
};

__host__ __device__ constexpr int64_t part_floats(int rows, int D) {
  return static_cast<int64_t>(rows) * (D + 2);
}

struct Extent {
  int tok0, toks, len, row_tiles, key_tiles;
};

// Where a run begins: tile i of (sequence s, KV head hk, row tile rt), the sequence's first tile
// at seg0 of the line.
struct Start {
  int64_t seg0;
  Extent e;
  int s, hk, rt, i;
};

// What is wrong with a sequence: something to report; offsets that decrease, so that sequences
// would have rows in common; rows without keys (of the scan alone).
enum : int { kReport = 1, kFalls = 2, kEmpty = 4 };

__device__ __forceinline__ Extent extent(const CrossArgs& a, int s, int* wrong) {
  Extent e;
  if (a.cu == nullptr) {
    e.tok0 = s * a.per_seq;
    e.toks = a.per_seq;
    *wrong = 0;
  } else {
    const int lo = a.cu[s], hi = a.cu[s + 1];
    e.tok0 = min(max(lo, 0), a.T);
    const int end = min(max(hi, 0), a.T);
    e.toks = max(end - e.tok0, 0);
    *wrong = (lo != e.tok0 || hi != end ? kReport : 0) | (end < e.tok0 ? kReport | kFalls : 0);
  }
  const int cap = a.max_pages * kPage, n = a.lens[s];
  if (n > cap) *wrong |= kReport;
  e.len = max(0, min(n, cap));
  e.row_tiles = (e.toks * a.G + kPair - 1) / kPair;
  e.key_tiles = e.row_tiles > 0 ? (e.len + kPage - 1) / kPage : 0;
  return e;
}

// The segments of a run, one after another: sequence s (its first tile at seg0 of the line),
// KV head hk, row tile rt, of it the tiles i .. i_end - 1.
struct Walk {
  Extent e;
  int64_t seg0, first;
  int s, hk, rt, i, i_end, left;  // left: tiles of the run from this segment on
  __device__ __forceinline__ Walk(const Start& st, int n_tiles)
      : e(st.e), seg0(st.seg0), s(st.s), hk(st.hk), rt(st.rt), i(st.i), left(n_tiles) {
    cut();
  }
  __device__ __forceinline__ void cut() {
    first = seg0 + (static_cast<int64_t>(hk) * e.row_tiles + rt) * e.key_tiles;
    i_end = min(e.key_tiles, i + left);
  }
  __device__ __forceinline__ bool next(const CrossArgs& a) {
    left -= i_end - i;
    if (left == 0) return false;
    i = 0;
    if (++rt == e.row_tiles) {
      rt = 0;
      if (++hk == a.Hkv) {
        hk = 0;
        seg0 += static_cast<int64_t>(e.row_tiles) * e.key_tiles * a.Hkv;
        int wrong;
#pragma unroll 1
        do {
          e = extent(a, ++s, &wrong);
        } while (e.key_tiles == 0);
      }
    }
    cut();
    return true;
  }
  __device__ __forceinline__ int row0() const { return rt * kPair; }
  __device__ __forceinline__ int rows(const CrossArgs& a) const {
    return min(kPair, e.toks * a.G - row0());
  }
};

// The value of lane 0, which the compiler then keeps where tcgen05 instructions take it from.
template <class T>
__device__ __forceinline__ T uniform(T v) {
  return __shfl_sync(0xFFFFFFFFu, v, 0);
}

// mbar_wait_warp in few instructions.  Twenty warps of six roles run their own code at once, and
// what does not fit the instruction caches costs more than all arithmetic (with the waits of
// nvq_ptx.cuh inline, loops unrolled and masks in the softmax's chunks the kernel was 113 KB, three
// warps of eleven waited for instructions and a tile took 3350 cycles).  A wait gives up after two
// seconds, or when another thread has.  (With a suspend-time hint of a
// microsecond on the try_wait a warp now and then slept all of it: not faster.)
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, uint32_t abort) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b32 t0, t, v;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE;\n\t"
      "mov.u32 t0, %%globaltimer_lo;\n\t"
      "AGAIN:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE;\n\t"
      "mov.u32 t, %%globaltimer_lo;\n\t"
      "sub.u32 t, t, t0;\n\t"
      "setp.gt.u32 q, t, 2000000000;\n\t"
      "@q st.volatile.shared.u32 [%3], 1;\n\t"
      "ld.volatile.shared.u32 v, [%3];\n\t"
      "setp.eq.u32 q, v, 0;\n\t"
      "@q bra AGAIN;\n\t"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(abort)
      : "memory");
  return __all_sync(0xFFFFFFFFu, ok != 0);
}

// The same for a wait that lasts as long as a segment, which may have any number of tiles: it gives
// up only where no tile has begun (`begun` has not changed) for two seconds.
__device__ __forceinline__ bool wait_segment(uint64_t* bar, uint32_t parity, volatile int* abort,
                                             const volatile int* begun) {
  int seen = *begun;
  uint64_t t0 = globaltimer_ns();
  bool ok;
#pragma unroll 1
  while (!(ok = mbar_try_wait(bar, parity)) && *abort == 0) {
    const int now = *begun;
    const uint64_t t = globaltimer_ns();
    if (now != seen) {
      seen = now;
      t0 = t;
    } else if (t - t0 > NVQ_WAIT_LIMIT_NS) {
      *abort = 1;
    }
  }
  return __all_sync(0xFFFFFFFFu, ok);
}

// q~ of a segment by N threads, thread t taking block t % (D/16) of every kStep-th row: codes into
// the swizzled rows of the A operand, scales into the 512-byte blocks of the scale operand, of the
// two halves one after another.  Rows beyond the segment's: zeros.  kAhead rows' values are on
// their way (four spill beside the rest: 32760 rows x 12 heads 133 us; two 123 us, one 144 us; two
// with the rows brought to L2 before, 120 us).
template <int D, int N>
struct QueryTile {
  static constexpr int kBlocks = D / 16, kStep = N / kBlocks;
  static constexpr int kAhead = N == 128 ? 2 : 4;
  uint4 lo[kAhead], hi[kAhead];
  const uint16_t* base;              // block t % kBlocks of the segment's first query head
  int tok, g, rows, step_t, step_g;  // the next row's token and query head; a step's

  __device__ __forceinline__ void begin(const CrossArgs& a, const Segment& sg, int t) {
    rows = sg.rows;
    base = a.q + sg.tok0 * a.ld_q + static_cast<int64_t>(sg.hk * a.G) * D + t % kBlocks * 16;
    const int row = sg.row0 + t / kBlocks;
    tok = row / a.G;
    g = row - tok * a.G;
    step_t = kStep / a.G;
    step_g = kStep - step_t * a.G;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) load(a, t / kBlocks + u * kStep, lo[u], hi[u]);
  }
  __device__ __forceinline__ void load(const CrossArgs& a, int n, uint4& lo, uint4& hi) {
    lo = hi = make_uint4(0, 0, 0, 0);
    if (n < rows) {
      const uint16_t* src = base + tok * a.ld_q + g * D;
      lo = ld16(src);
      hi = ld16(src + 8);
    }
    tok += step_t;
    if ((g += step_g) >= a.G) {
      g -= a.G;
      ++tok;
    }
  }
  __device__ __forceinline__ void quantize(const CrossArgs& a, uint8_t* codes, uint8_t* scales,
                                           int t) {
    const int end = rows > kRows ? kPair : kRows;
    if constexpr (kAhead * kStep >= kPair) {  // all loads are on their way
#pragma unroll 1
      for (int n = t / kBlocks; n < end; n += kStep) {
        row(lo[0], hi[0], codes, scales, n, t % kBlocks);
#pragma unroll
        for (int u = 0; u + 1 < kAhead; ++u) {
          lo[u] = lo[u + 1];
          hi[u] = hi[u + 1];
        }
      }
    } else {
#pragma unroll 1
      for (int n0 = t / kBlocks; n0 < end; n0 += kAhead * kStep) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int n = n0 + u * kStep;
          const uint4 x = lo[u], y = hi[u];
          load(a, n + kAhead * kStep, lo[u], hi[u]);
          row(x, y, codes, scales, n, t % kBlocks);
        }
      }
    }
  }
  // block j of row n
  static __device__ __forceinline__ void row(const uint4& x, const uint4& y, uint8_t* codes,
                                             uint8_t* scales, int n, int j) {
    const uint32_t v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    const Codes16 r = codes16_unit(v);
    const int swz = D == 128 ? (n >> 1) & 3 : (n >> 2) & 1;  // 64- and 32-byte swizzles
    // the halves' codes and scales lie one behind the other
    *reinterpret_cast<uint2*>(codes + n * (D / 2) + (((j >> 1) ^ swz) << 4) + (j & 1) * 8) =
        make_uint2(r.codes[0], r.codes[1]);
    scales[(n >> 7) * (D / 64 * 512) + (j >> 2) * 512 + (n & 31) * 16 + (n >> 5 & 3) * 4 +
           (j & 3)] = static_cast<uint8_t>(r.sbyte);
  }
};

// V~ of a page as f16 rows of 64 elements (128 bytes, swizzled; elements 64.. in a second block)
// by four warps, 32 keys each.  A lane takes 32 elements (16 bytes of codes, two scales) of a
// key; lanes of consecutive pieces read consecutive bytes.  In heads of 128 the lanes of a row's
// second half take their words in another order, so that no two of eight lanes write the same
// banks.  Keys behind the last token become zeros: their bytes may be anything.
template <int D>
__device__ __forceinline__ void decode_v(const uint8_t* rec, uint8_t* dst, int valid, int warp,
                                         int lane) {
  constexpr int kPieces = D / 32, kKeys = 32 / kPieces;
  const int piece = lane % kPieces, flip = piece >> 1;
#pragma unroll 1
  for (int i = 0; i < kPieces; ++i) {
    const int key = 32 * warp + i * kKeys + lane / kPieces;
    const uint4 c =
        *reinterpret_cast<const uint4*>(rec + v_codes_at(D) + key * (D / 2) + piece * 16);
    uint32_t sc =
        *reinterpret_cast<const uint16_t*>(rec + v_scales_at(D) + key * (D / 16) + piece * 2);
    if (key >= valid) sc = 0;
    const uint32_t s2 = e4m3x2_to_f16x2(sc);
    const uint32_t sa = __byte_perm(s2, 0, 0x1010), sb = __byte_perm(s2, 0, 0x3232);
    const uint32_t w[4] = {flip ? c.z : c.x, flip ? c.w : c.y, flip ? c.x : c.z, flip ? c.y : c.w};
    const uint32_t s[2] = {flip ? sb : sa, flip ? sa : sb};
    uint8_t* row = dst + (piece >> 1) * (kRows * 128) + key * 128;
    const int chunk = ((piece & 1) * 4 + 2 * flip) ^ (key & 7);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      uint32_t h[4];
      e2m1x8_to_f16x2(w[x], h);
      *reinterpret_cast<uint4*>(row + ((chunk ^ x) << 4)) =
          make_uint4(hmul2(h[0], s[x >> 1]), hmul2(h[1], s[x >> 1]), hmul2(h[2], s[x >> 1]),
                     hmul2(h[3], s[x >> 1]));
    }
  }
}

// Four kind::f16 UMMAs (K = 16 each) into the accumulator d: A in tensor memory at a + 8 k, B
// through b0 advanced by 2048 k bytes; commits to c0 and, unless it is 0, to c1.
__device__ __forceinline__ void umma_f16_ts4_w(uint32_t d, uint32_t a, uint64_t b0, uint32_t idesc,
                                               uint32_t acc, uint32_t c0, uint32_t c1) {
  asm volatile(
      "{\n\t.reg .pred p, e, t, q;\n\t.reg .b32 lo, hi, a1, a2, a3;\n\t"
      ".reg .b64 b1, b2, b3;\n\t"
      "setp.ne.b32 p, %2, 0;\n\t"
      "setp.eq.u32 t, 0, 0;\n\t"
      "mov.b64 {lo, hi}, %4;\n\t"
      "add.u32 lo, lo, 128;\n\tmov.b64 b1, {lo, hi};\n\t"
      "add.u32 lo, lo, 128;\n\tmov.b64 b2, {lo, hi};\n\t"
      "add.u32 lo, lo, 128;\n\tmov.b64 b3, {lo, hi};\n\t"
      "add.u32 a1, %3, 8;\n\tadd.u32 a2, %3, 16;\n\tadd.u32 a3, %3, 24;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.and.u32 q, %6, 0, e;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%3], %4, %1, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %1, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %1, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %1, t;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%6];\n\t}"
      ::"r"(d), "r"(idesc), "r"(acc), "r"(a), "l"(b0), "r"(c0), "r"(c1)
      : "memory");
}

// What is written as a row's lse: the natural logarithm (-inf of a row with a NaN, as for single
// tokens), or base 2 beside an output in fp32 (there NaN, so that who folds it in sees it).
// The fast logarithm may be off by 2^-22 of its value, 2^-18 for 131072 keys, a part of what the
// sums of S are off by (with log2f 32760 rows x 12 heads x 512 keys took 113.7 us, not 112.5).
__device__ __forceinline__ float row_lse(const CrossArgs& a, float m, float l) {
  if (l == 0.f) return -INFINITY;
  const float v = m + __log2f(l);
  if (a.o == nullptr) return v;
  return l > 0.f ? v * kLn2 : -INFINITY;
}

// 32 lanes x 8 columns (32x32b shape).
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
               "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(const uint32_t* v) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(v[0]), __uint_as_float(v[1]));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// p = 2^(s scale + neg_m) of 32 scores, their sums added to l, p as f16 pairs.
__device__ __forceinline__ void exponentials(const uint32_t (&s)[32], uint64_t scale2,
                                             uint64_t neg_m, uint64_t& l2, uint32_t (&p)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float p0, p1;
    up2(fma2(pk2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), scale2, neg_m), p0, p1);
    p0 = ex2_f32(p0);
    p1 = ex2_f32(p1);
    l2 = add2(l2, pk2(p0, p1));
    p[i] = pack_f16x2_rn(p0, p1);
  }
}

// A token without visible keys: o = 0 (in fp32 left as it is), lse = -inf.
template <int D>
__device__ __forceinline__ void empty_token(const CrossArgs& a, int tok, int lane) {
  const int64_t row0 = static_cast<int64_t>(tok) * a.H;
  if (a.o != nullptr)
#pragma unroll 1
    for (int x = lane; x < a.H * (D / 8); x += 32)
      reinterpret_cast<uint4*>(a.o + row0 * D)[x] = make_uint4(0, 0, 0, 0);
  if (a.lse != nullptr)
#pragma unroll 1
    for (int x = lane; x < a.H; x += 32) a.lse[row0 + x] = -INFINITY;
}

// Tells the other warps of a segment of the run [u0, u1), and the join of one that begins in it
// and goes on behind it.
__device__ __forceinline__ void describe(const CrossArgs& a, const Walk& w, int run, int64_t u0,
                                         int64_t u1, int64_t all, Segment& to,
                                         uint64_t* described) {
  const bool begins = w.first >= u0, ends = w.first + w.e.key_tiles <= u1;
  // a part that begins with the run goes to the run's slot 0, one inside it to slot 1
  const int slot = begins && ends ? -1 : 2 * run + (w.first > u0 ? 1 : 0);
  to = {w.row0(), w.rows(a), w.e.tok0, w.hk, slot, w.s, w.i, w.i_end, w.e.len, {0, 0, 0}};
  mbar_arrive(described);
  if (begins && !ends)
    a.split[run] = {w.first + w.e.key_tiles - 1, all, slot, w.rows(a), w.row0(), w.e.tok0, w.hk, 0};
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    cross_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap to,
                 const CrossArgs a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int64_t warp_sum[kThreads / 32];
  __shared__ alignas(8) unsigned char walk_bytes[sizeof(Walk)];  // of the query warps' first thread
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word, begun;  // begun: the tile that the producer is at
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023u) &
                                             ~static_cast<uintptr_t>(1023u));
  Tile* desc = reinterpret_cast<Tile*>(smem + C::kDescAt);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarAt);
  uint64_t* empty = full + C::kStages;   // S and the PV and decode warps done with it
  uint64_t* k_ready = empty + C::kStages;  // K's scales in order
  uint64_t* v_full = k_ready + C::kStages;  // [2], four decode warps
  uint64_t* v_empty = v_full + 2;         // [2]
  uint64_t* q_full = v_empty + 2;         // [2], four query warps
  uint64_t* q_empty = q_full + 2;         // [2]
  uint64_t* s_full = q_empty + 2;         // [2 streams][3], by the units of the stream
  uint64_t* p_full = s_full + 6;          // [3] by the unit's buffer, four softmax warps
  uint64_t* pv_done = p_full + 3;         // [3]
  uint64_t* o_full = pv_done + 3;         // [2 streams]: a segment's last PV is done
  uint64_t* o_read = o_full + 2;          // [2 streams], eight: two by each of its softmax warps,
                                          // or one by each of both streams'
  uint64_t* drain = o_read + 2;           // [3]
  uint64_t* merge = drain + 3;            // [2 streams][4]: by 32 rows, the stream's keys are done
  uint64_t* described = merge + 8;        // [kSegs]
  uint64_t* q_first = described + kSegs;  // the other warps that quantize the run's first segment
  Segment* segs = reinterpret_cast<Segment*>(smem + C::kSegAt);
  int* units = reinterpret_cast<int*>(smem + C::kUnitAt);  // by s_full: keys with tokens, flags
  float2* ml = reinterpret_cast<float2*>(smem + C::kMlAt);
  const uint32_t abort = smem_u32(&abort_word);
  const auto walk = [&]() -> Walk& { return *reinterpret_cast<Walk*>(walk_bytes); };
  pdl_trigger();

  if (threadIdx.x == 32 * kProducerWarp) {  // (the first warps look at sequences meanwhile)
    abort_word = begun = 0;
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 2 + 1 + 4);
      mbar_init(&k_ready[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&v_full[i], 4);
      mbar_init(&v_empty[i], 1);
      mbar_init(&q_full[i], 4);
      mbar_init(&q_empty[i], 2);
      mbar_init(&o_full[i], 1);
      mbar_init(&o_read[i], 8);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&s_full[i], 2);  // the MMAs, and what the S warp tells of the unit
      mbar_init(&s_full[3 + i], 2);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
      mbar_init(&drain[i], 1);
    }
    for (int i = 0; i < 8; ++i) mbar_init(&merge[i], 1);
    for (int i = 0; i < kSegs; ++i) mbar_init(&described[i], 1);
    mbar_init(q_first, kQWarp);
    fence_mbar_init();
  }
  if (warp == kPvWarp) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
    tma_prefetch_desc(&tk);
  }
  pdl_wait();  // before this nothing that another kernel may have written is read
  // ---- the run of this CTA: a scan over the sequences
  const int per = (a.B + kThreads - 1) / kThreads;
  const int s_lo = min(a.B, static_cast<int>(threadIdx.x) * per), s_hi = min(a.B, s_lo + per);
  int64_t mine = 0;
  int any = 0;
  Extent e{};
#pragma unroll 1
  for (int s = s_lo; s < s_hi; ++s) {
    int wrong;
    e = extent(a, s, &wrong);
    any |= wrong | (e.toks > 0 && e.key_tiles == 0 ? kEmpty : 0);
    mine += static_cast<int64_t>(e.row_tiles) * e.key_tiles * a.Hkv;
  }
  if ((any & kReport) && blockIdx.x == 0) atomicMax(a.err, kErrTable);
  int64_t scan = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, scan, off);
    if (lane >= off) scan += v;
  }
  if (lane == 31) warp_sum[warp] = scan;
  // sequences with rows in common would write them in any order: then nobody has rows
  const bool falls = __syncthreads_or(any & kFalls);
  int64_t all = 0;
  const int busy = ((a.B + per - 1) / per + 31) / 32;  // warps that have sequences
#pragma unroll 1
  for (int w = 0; w < busy; ++w) {
    if (w < warp) scan += warp_sum[w];
    all += warp_sum[w];
  }
  const int64_t before = scan - mine;  // tiles before this thread's sequences
  if (falls) all = mine = 0;
  const int run = blockIdx.x;
  const Runs line(all, a.runs, a.runs_magic);
  const int64_t u0 = line.begin(run), u1 = line.begin(run + 1);
  if (mine > 0 && before <= u0 && u0 < before + mine) {
    int64_t at = before;
    int s = s_lo;
    if (per > 1) {
#pragma unroll 1
      for (;; ++s) {
        int wrong;
        e = extent(a, s, &wrong);
        const int64_t n = static_cast<int64_t>(e.row_tiles) * e.key_tiles * a.Hkv;
        if (u0 < at + n) break;
        at += n;
      }
    }
    // the run's first segment of the sequence, and the first of its tiles
    int hk, rt, i;
    const int64_t x = u0 - at;
    if (x < (int64_t{1} << 31)) {
      const uint32_t y = static_cast<uint32_t>(x), nth = y / static_cast<uint32_t>(e.key_tiles);
      i = static_cast<int>(y - nth * e.key_tiles);
      hk = static_cast<int>(nth / static_cast<uint32_t>(e.row_tiles));
      rt = static_cast<int>(nth - hk * e.row_tiles);
    } else {
      const int64_t nth = x / e.key_tiles;
      i = static_cast<int>(x - nth * e.key_tiles);
      hk = static_cast<int>(nth / e.row_tiles);
      rt = static_cast<int>(nth - static_cast<int64_t>(hk) * e.row_tiles);
    }
    // the run's first segment, described before anyone looks
    const Start st{at, e, s, hk, rt, i};
    const Walk w(st, static_cast<int>(u1 - u0));
    walk() = w;
    a.split[run].end = -1;
    describe(a, w, run, u0, u1, all, segs[0], &described[0]);
  }
  if (u0 == u1 && threadIdx.x == 0) a.split[run].end = -1;
  tc_fence_before();
  const bool empties = __syncthreads_or(any & kEmpty) && !falls;
  tc_fence_after();
  const uint32_t tmem = uniform(tmem_slot);
  const int n_tiles = uniform(static_cast<int>(u1 - u0));

  // ---- the run's first segment: nothing can begin before its q~, which took the query warps alone
  // 9000 cycles, so all that would wait for it help (64 tokens behind a shared prefix 55 -> 53 us)
  if (warp < kProducerWarp && n_tiles > 0) {
    QueryTile<D, 32 * kProducerWarp> q;
    q.begin(a, segs[0], threadIdx.x);
    q.quantize(a, smem + C::kQAt, smem + C::kQScAt, threadIdx.x);
    fence_proxy_async_smem();
    mbar_arrive_warp(warp < kQWarp ? q_first : &q_full[0]);
  }

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    bool ok = true;
    int n = 0;
    Ring ring;
#pragma unroll 1
    for (int seg = 0; n < n_tiles && ok; ++seg) {
      if (!(ok = wait(&described[seg % kSegs], (seg / kSegs) & 1, abort))) break;
      const Segment& sg = segs[seg % kSegs];
      const int hk = sg.hk, len = sg.len, i0 = sg.i, i_end = sg.i_end;
      const int32_t* table = a.table + sg.s * a.ld_table;
      Tile td{0, 0, sg.rows, seg};
      int pages = 0;  // this lane's page number: of tile i0 + 32 k + lane
#pragma unroll 1
      for (int i = i0; i < i_end; ++i, ++n, ring.next(C::kStages)) {
        if (((i - i0) & 31) == 0) pages = i + lane < i_end ? table[i + lane] : -1;
        const int page = __shfl_sync(0xFFFFFFFFu, pages, (i - i0) & 31);
        const bool there = page >= 0 && page < a.num_pages;
        td.flags = (i == i0 ? kStart : 0) | (i == i_end - 1 ? kEnd : 0) | (there ? 0 : kAbsent) |
                   (td.rows > kRows ? kBoth : 0);
        td.valid = there ? min(kPage, len - i * kPage) : 0;
        if (!there && lane == 0) atomicMax(a.err, kErrTable);
        const int st = ring.s;
        if (!(ok = wait(&empty[st], ring.phase ^ 1, abort))) break;
        if (lane == 0) {
          desc[st] = td;
          begun = n;
        }
        __syncwarp();
        uint8_t* dst = smem + st * C::kRec;
        if (there) {
          const int rec = page * a.Hkv + hk;
          mbar_arrive_expect_tx_w(&full[st], C::kRec);
          tma_load_4d_w(dst, &tk, 0, 0, rec, 0, &full[st]);
          bulk_load_w(dst + v_codes_at(D),
                      a.pool + static_cast<int64_t>(rec) * record_bytes(D) + v_codes_at(D),
                      C::kRec - v_codes_at(D), &full[st]);
        } else {
          mbar_arrive_expect_tx_w(&full[st], 0);
        }
      }
    }
    if (!ok) {  // let the copies already issued land before the block leaves
#pragma unroll 1
      for (int m = max(0, n - C::kStages); m < n; ++m)
        mbar_wait_warp(&full[m % C::kStages], (m / C::kStages) & 1, nullptr, 10000000ull);
    }
  } else if (warp == kSWarp || warp == kSWarp + 1) {
    // ------------------------------------------------------------ S = Q~ K~^T of a stream's units
    constexpr uint32_t idesc = idesc_mxf4nvf4(kRows, kKeys);
    constexpr uint32_t lay = D == 128 ? 4u : 6u, sbo = 4 * D;  // swizzle, bytes of 8 rows
    const int stream = warp - kSWarp;
    const uint64_t q_d0 = sdesc(smem_u32(smem + C::kQAt), 16, sbo, lay);
    const uint64_t k_d0 = sdesc(smem_u32(smem), 16, sbo, lay);
    Ring ring, unit;  // the buffer of the stream's next unit, every other one
    if (stream == 1) unit.next(3);
    int word = 0;     // units of the stream so far, modulo 3
    bool ok = true;
#pragma unroll 1
    for (int n = 0; n < n_tiles && ok; ++n, ring.next(C::kStages)) {
      const int st = ring.s;
      if (!wait(&k_ready[st], ring.phase, abort)) break;
      const int flags = uniform(desc[st].flags), seg = uniform(desc[st].seg);
      const int valid = desc[st].valid;
      const int qb = seg & 1, both = flags & kBoth ? 1 : 0;
      const int half = both ? stream : 0;  // of the rows
      if ((flags & kStart) && !wait(&q_full[qb], (seg >> 1) & 1, abort)) break;
      if (n == 0 && !wait(q_first, 0, abort)) break;
      const uint32_t sfq = tmem + kSfQ + 16 * qb + 8 * stream;
      const uint32_t sfk = tmem + kSfK + 16 * stream + 8 * (n & 1);
      const uint64_t qd = q_d0 + static_cast<uint64_t>((2 * qb + half) * (C::kQ >> 4));
      const uint64_t qds[2] = {qd, qd + 2};
#pragma unroll 1
      for (int j = 0; j <= both; ++j) {
        const int key = both ? j : stream;
        const bool last = j == both;
        const uint64_t kd =
            k_d0 + static_cast<uint64_t>(st * (C::kRec >> 4) + key * (kKeys * D / 2 >> 4));
        const uint64_t kds[2] = {kd, kd + 2};
        uint64_t* const ready = &s_full[3 * stream + word];
        if (lane == 0)  // (the PV of the stream's unit three before is done: the word is free)
          units[4 * stream + word] =
              max(0, min(kKeys, valid - kKeys * key)) |
              ((flags & kStart) && j == 0 ? kUnitStart : 0) |
              (last ? ((flags & kEnd) ? kUnitEnd : 0) | (n == n_tiles - 1 ? kUnitLast : 0) : 0);
        word = word == 2 ? 0 : word + 1;
        // the buffer is free when the PV of the unit three before has read the P over it
        if (!(ok = wait(&pv_done[unit.s], unit.phase ^ 1, abort))) break;
        tc_fence_after();
        if (j == 0) {
          // The copies go to columns whose last readers have completed: the stream's MMAs of tile
          // n - 2 (the PVs waited for lie behind them), and of q's of segment seg - 2, which the
          // query warps waited for.
          if (flags & kStart) {
#pragma unroll
            for (int k = 0; k < D / 64; ++k)
              tmem_cp_32x128_x4_w(sfq + 4 * k,
                                  smem_u32(smem + C::kQScAt + (2 * qb + half) * C::kQSc) + 512 * k);
          }
          if (!(flags & kAbsent)) {
#pragma unroll
            for (int k = 0; k < D / 64; ++k)
              tmem_cp_32x128_x4_w(sfk + 4 * k,
                                  smem_u32(smem + st * C::kRec + k_scales_at(D)) + 512 * k);
          }
        }
        if (!(flags & kAbsent)) {
          umma_fp4_group_w<D / 64>(tmem + 64 * unit.s, qds, kds, idesc, sfq, sfk + 2 * key,
                                   bar_u32(ready), last ? bar_u32(&empty[st]) : 0u);
        } else {
          umma_commit_w(ready);
          if (last) umma_commit_w(&empty[st]);
        }
        mbar_arrive_warp(ready);
        unit.next(3);
        unit.next(3);
      }
      if (flags & kEnd) umma_commit_w(&q_empty[qb]);
    }
    umma_commit_w(&drain[stream]);  // the MMAs in flight end before the block
    mbar_wait_warp(&drain[stream], 0, nullptr, 10000000ull);
  } else if (warp == kPvWarp) {
    // ------------------------------------------------------------ O += P V~
    constexpr uint32_t idesc = idesc_f16(kRows, D, 0, 0, 1);
    const uint64_t v_d0 = sdesc_sw128(smem_u32(smem + C::kVAt), kRows * 128, 1024);
    Ring ring, unit;
    bool ok = true;
#pragma unroll 1
    for (int n = 0; n < n_tiles && ok; ++n, ring.next(C::kStages)) {
      const int b = n & 1;
      if (!wait(&full[ring.s], ring.phase, abort)) break;
      const int flags = uniform(desc[ring.s].flags), seg = uniform(desc[ring.s].seg);
      mbar_arrive_warp(&empty[ring.s]);
      const int halves = flags & kBoth ? 2 : 1;
      if (!wait(&v_full[b], (n >> 1) & 1, abort)) break;
#pragma unroll 1
      for (int u = 0; u < 2 * halves; ++u, unit.next(3)) {
        const int stream = u & 1, key = halves == 2 ? u >> 1 : u;
        const bool first = (flags & kStart) && u < 2;
        // O of the stream's segment before has been read
        if (first && seg > 0 && !(ok = wait(&o_read[stream], (seg - 1) & 1, abort))) break;
        if (!(ok = wait(&p_full[unit.s], unit.phase, abort))) break;
        tc_fence_after();
        umma_f16_ts4_w(tmem + kO + D * stream, tmem + 64 * unit.s,
                       v_d0 + static_cast<uint64_t>(b) * (C::kV >> 4) + 512 * key, idesc,
                       first ? 0u : 1u, bar_u32(&pv_done[unit.s]),
                       u == 2 * halves - 1 ? bar_u32(&v_empty[b]) : 0u);
        if ((flags & kEnd) && u >= 2 * halves - 2) umma_commit_w(&o_full[stream]);
      }
    }
    umma_commit_w(&drain[2]);
    mbar_wait_warp(&drain[2], 0, nullptr, 10000000ull);
  } else if (warp >= kDecodeWarp && warp < kQWarp) {
    // ------------------------------------------------------------ V~
    Ring ring;
#pragma unroll 1
    for (int n = 0; n < n_tiles; ++n, ring.next(C::kStages)) {
      const int st = ring.s, b = n & 1;
      if (!wait(&full[st], ring.phase, abort)) break;
      if (warp == kDecodeWarp) {
        if (!(desc[st].flags & kAbsent)) {
          arrange_scales<D>(smem + st * C::kRec + k_scales_at(D), lane);
          fence_proxy_async_smem();
        }
        mbar_arrive_warp(&k_ready[st]);
      }
      if (!wait(&v_empty[b], ((n >> 1) & 1) ^ 1, abort)) break;
      decode_v<D>(smem + st * C::kRec, smem + C::kVAt + b * C::kV, desc[st].valid,
                  warp - kDecodeWarp, lane);
      fence_proxy_async_smem();
      mbar_arrive_warp(&v_full[b]);
      mbar_arrive_warp(&empty[st]);
    }
  } else if (warp < kDecodeWarp) {
    // ------------------------------------------------------------ softmax
    const int stream = warp >> 2, quarter = warp & 3;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t o_at = lanes + kO + D * stream;
    const uint64_t scale2 = pk2(a.scale.fused, a.scale.fused);
    float m = -INFINITY;  // reference maximum (log2 units)
    uint64_t l2 = pk2(0.f, 0.f);
    uint32_t u = stream;           // its units are every other one
    uint32_t ends = 0, joins = 0;  // segments, and those whose keys were shared, so far
    int rows = 0;                  // of the segment
    int what = n_tiles > 0 ? 0 : kUnitLast;  // the S warp's word
    // s_full is the stream's own: a barrier of both would be phases ahead or behind of one of them,
    // whose parity would tell it of an older phase's end
    Ring mine_full;
#pragma unroll 1
    for (; !(what & kUnitLast); u += 2, mine_full.next(3)) {
      const uint32_t buf = u % 3;
      if (!wait(&s_full[3 * stream + mine_full.s], mine_full.phase, abort)) break;
      tc_fence_after();
      what = units[4 * stream + mine_full.s];
      if (what & kUnitStart) {
        m = -INFINITY;
        l2 = pk2(0.f, 0.f);
        rows = segs[ends % kSegs].rows;
      }
      const int valid = what & kValid;
      const bool both = rows > kRows;
      const bool live = 32 * (both ? warp : quarter) < rows;  // else: rows that nobody reads
      const uint32_t s_at = lanes + 64 * buf;
      if (live) {
        // before S is read: keys behind the last, -inf; large scales
        const bool scaled = a.scale.before != 1.f;
        if (valid < kKeys || scaled) {
#pragma unroll 1
          for (int c = scaled ? 0 : valid & ~15; c < kKeys; c += 16) {
            uint32_t x[16];
            tmem_ld16(s_at + c, x);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              x[i] = __float_as_uint(__uint_as_float(x[i]) * a.scale.before);
              if (c + i >= valid) x[i] = 0xFF800000u;
            }
            tmem_st16(s_at + c, x);
          }
          tmem_wait_st();
        }
        uint32_t x[32], y[32];
        tmem_ld32(s_at, x);
        tmem_ld32(s_at + 32, y);
        tmem_wait_ld();
        float v[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          v[0] = max3f(v[0], __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
          v[1] = max3f(v[1], __uint_as_float(x[16 + i]), __uint_as_float(x[17 + i]));
          v[2] = max3f(v[2], __uint_as_float(y[i]), __uint_as_float(y[i + 1]));
          v[3] = max3f(v[3], __uint_as_float(y[16 + i]), __uint_as_float(y[17 + i]));
        }
        // (a product of its own: fused with a difference from m it would be another number)
        const float mx = __fmul_rn(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])), a.scale.fused);
        const bool grows = mx > fmaxf(m, limit_of(m));  // -inf: always, where there is a key
        if (__any_sync(0xFFFFFFFFu, grows)) {
          const float c = grows ? ex2_f32(m - mx) : 1.f;
          if (grows) m = mx;
          l2 = mul2(l2, pk2(c, c));
          // raised behind the segment's first unit: O so far, which the stream's PV before has
          // finished
          if (!(what & kUnitStart)) {
            const uint32_t w = u - 2;
            if (!wait(&pv_done[w % 3], (w / 3) & 1, abort)) break;
            tc_fence_after();
#pragma unroll 1
            for (int z = 0; z < D; z += 8) {
              uint32_t t[8];
              tmem_ld8(o_at + z, t);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 8; ++i) t[i] = __float_as_uint(__uint_as_float(t[i]) * c);
              tmem_st8(o_at + z, t);
            }
          }
        }
        // ---- p = 2^(S log2e - m + kUp), over S
        const float ref = kUp - fmaxf(m, -3.4e38f);
        const uint64_t neg_m = pk2(ref, ref);
        uint32_t p[16];
        exponentials(x, scale2, neg_m, l2, p);
        tmem_st16(s_at, p);
        exponentials(y, scale2, neg_m, l2, p);
        tmem_st16(s_at + 16, p);
        tmem_wait_st();
      }
      tc_fence_before();
      mbar_arrive_warp(&p_full[buf]);
      if (!(what & kUnitEnd)) continue;
      // ---- the segment's end: what does not need O, while its last PV is on its way
      const Segment& sg = segs[ends % kSegs];
      float l0, l1;
      up2(l2, l0, l1);
      // back to p = 1 at the reference (exactly; a logarithm of larger numbers has fewer bits)
      constexpr float kDown = 1.f / (1 << static_cast<int>(kUp));
      float l = (l0 + l1) * kDown, own = kDown, other = 0.f;
      const int r = both ? threadIdx.x : threadIdx.x & (kRows - 1);  // row of the segment
      const int slot = sg.slot, row = sg.row0 + r, tok = row / a.G;
      const int64_t at = static_cast<int64_t>(sg.tok0 + tok) * a.H + sg.hk * a.G + row - tok * a.G;
      if (lane == 0) bulk_wait_group_read<0>();  // of the segment before
      if (!wait(&o_full[stream], ends++ & 1, abort)) break;
      tc_fence_after();
      if (!both) {  // the streams have halves of the keys: each takes half of the columns of both
        if (live) ml[kRows * stream + r] = make_float2(m, l);
        tc_fence_before();
        mbar_arrive_warp(&merge[4 * stream + quarter]);
        if (!wait(&merge[4 * (stream ^ 1) + quarter], joins++ & 1, abort)) break;
        tc_fence_after();
        const float2 v = ml[kRows * (stream ^ 1) + r];
        const float top = fmaxf(m, v.x), ref = fmaxf(top, -3.4e38f);
        own = ex2_f32(m - ref);
        other = ex2_f32(v.x - ref);
        l = fmaf(l, own, v.y * other);
        own *= kDown;
        other *= kDown;
        m = top;
      }
      if (slot < 0) {
        const float inv = l > 0.f ? __fdividef(1.f, l) : 0.f;
        own *= inv;
        other *= inv;
      }
      float* part = a.parts + max(slot, 0) * part_floats(a.part_rows, D);
      if (r < rows && (both || stream == 0)) {
        if (slot >= 0)
          *reinterpret_cast<float2*>(part + 2 * r) = make_float2(m, l);
        else if (a.lse != nullptr)
          a.lse[at] = row_lse(a, m, l);
      }
      // The warp's rows go through shared memory (16-byte pieces in the 128-byte swizzle): 32 whole
      // rows of o as tiles that one lane hands over, others a row at a time, 512 bytes a store;
      // bf16 rows at once, fp32 ones in two halves.  (Stores of 16 bytes of 32 rows kept the warp
      // for 9000 cycles a segment, more than two tiles' softmax, a bulk copy for each row for 2500,
      // the rows' stores for 2700, the tiles for 500.)
      const bool narrow = slot < 0 && a.o != nullptr;
      const int there = rows - (r - lane);  // rows of the warp's 32
      const int wide = both ? D : D / 2, x_end = both ? D : D / 2 + D / 2 * stream;
      const int cols = narrow ? wide : D / 2;  // at a time
      const bool tiles = narrow && a.tiles && there >= 32 && wide % 64 == 0;
      const uint32_t o_other = stream == 0 ? o_at + D : o_at - D;
      uint8_t* const area = smem + C::kOutAt + (4 * stream + quarter) * C::kOut;
      const auto piece = [&](int n, int c) {
        return reinterpret_cast<uint4*>(area + (c >> 3) * 4096 + n * 128 + (((c ^ n) & 7) << 4));
      };
#pragma unroll 1
      for (int x0 = x_end - wide; x0 < x_end; x0 += cols) {
        if (live) {
#pragma unroll 1
          for (int x = 0; x < cols; x += 32) {
            uint32_t v[32];
            tmem_ld32(o_at + x0 + x, v);
            tmem_wait_ld();
            const uint64_t own2 = pk2(own, own);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float z0, z1;
              up2(mul2(pk2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), own2), z0, z1);
              v[i] = __float_as_uint(z0);
              v[i + 1] = __float_as_uint(z1);
            }
            if (!both) {
#pragma unroll
              for (int h = 0; h < 32; h += 16) {
                uint32_t z[16];
                tmem_ld16(o_other + x0 + x + h, z);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  v[h + i] = __float_as_uint(
                      fmaf(__uint_as_float(z[i]), other, __uint_as_float(v[h + i])));
              }
            }
            if (narrow) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                *piece(lane, x / 8 + i) =
                    make_uint4(pack_bf16(v + 8 * i), pack_bf16(v + 8 * i + 2),
                               pack_bf16(v + 8 * i + 4), pack_bf16(v + 8 * i + 6));
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                *piece(lane, x / 4 + i) =
                    make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            }
          }
        }
        if (x0 + cols == x_end) {
          tc_fence_before();
          mbar_arrive_warp(&o_read[stream]);
          mbar_arrive_warp(&o_read[both ? stream : stream ^ 1]);
        }
        if (tiles) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
#pragma unroll 1
            for (int x = 0; x < cols; x += 64)
              tma_store_4d(&to, area + x * 64, x0 + x, sg.hk * a.G, sg.tok0 + tok, 0);
            bulk_commit_group();
          }
          break;
        }
        __syncwarp();
        float* const wide_row = slot < 0 ? a.o32 + at * D : part + 2 * a.part_rows + r * D;
        uint8_t* const out = narrow ? reinterpret_cast<uint8_t*>(a.o + at * D + x0)
                                    : reinterpret_cast<uint8_t*>(wide_row + x0);
        // a row's pieces: 16 or 8 of heads of 128, 8 or 4 of heads of 64
        constexpr int kLog = D == 128 ? 4 : 3;
        const int log = narrow && !both ? kLog - 1 : kLog;
        const int sub = lane >> log, c = lane & ((1 << log) - 1);
#pragma unroll 4
        for (int i = 0; i < 32; i += 32 >> log) {
          const unsigned long long dst =
              __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(out), i + sub);
          if (i + sub < there)
            reinterpret_cast<uint4*>(dst)[c] = *piece(i + sub, c);
        }
        __syncwarp();
      }
    }
    if (lane == 0) bulk_wait_group<0>();
  } else if (warp >= kQWarp && warp < kProducerWarp) {
    // ------------------------------------------------------------ q~
    const int t = threadIdx.x - 32 * kQWarp;
    int left = n_tiles > 0 ? n_tiles - (segs[0].i_end - segs[0].i) : 0;  // tiles behind the segment
#pragma unroll 1
    for (int seg = 1; left > 0; ++seg) {
      const Segment& sg = segs[seg % kSegs];
      if (t == 0) {  // (between the segments the walk lies in shared memory, not in registers)
        Walk w = walk();
        w.next(a);
        walk() = w;
        describe(a, w, run, u0, u1, all, segs[seg % kSegs], &described[seg % kSegs]);
      }
      if (!wait(&described[seg % kSegs], (seg / kSegs) & 1, abort)) break;
      left -= sg.i_end - sg.i;
      // all rows on their way to L2 at once: registers hold those of two loads a thread only
#pragma unroll 1
      for (int r = t; r < sg.rows; r += 128) {
        const int row = sg.row0 + r, tok = row / a.G;
        const uint16_t* src = a.q + (sg.tok0 + tok) * a.ld_q +
                              static_cast<int64_t>(sg.hk * a.G + row - tok * a.G) * D;
#pragma unroll
        for (int x = 0; x < D; x += 64)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(src + x));
      }
      QueryTile<D, 128> q;
      q.begin(a, sg, t);
      const int qb = seg & 1;
      if (!wait_segment(&q_empty[qb], ((seg >> 1) & 1) ^ 1, &abort_word, &begun)) break;
      q.quantize(a, smem + C::kQAt + 2 * qb * C::kQ, smem + C::kQScAt + 2 * qb * C::kQSc, t);
      fence_proxy_async_smem();
      mbar_arrive_warp(&q_full[qb]);
    }
    // ---- rows without keys, rows outside of all sequences: by their numbers over all these warps
    // (counted from each sequence's first one warp had all sequences of a row: 256 of them took
    // 52 us)
    const int first = 4 * run + warp - kQWarp, step = 4 * static_cast<int>(gridDim.x);
#pragma unroll 1
    for (int s0 = 0; s0 < a.B && empties; s0 += 32) {
      int wrong;
      Extent x{0, 0, 0, 0, 1};
      if (s0 + lane < a.B) x = extent(a, s0 + lane, &wrong);
      uint32_t none = __ballot_sync(0xFFFFFFFFu, x.toks > 0 && x.key_tiles == 0);
      if (none == 0) continue;
      int z0 = first - x.tok0 % step;  // the warp's first row of the sequence
      if (z0 < 0) z0 += step;
      none &= __ballot_sync(0xFFFFFFFFu, x.toks > z0);
#pragma unroll 1
      for (; none != 0; none &= none - 1) {
        const int i = __ffs(none) - 1;
        const int tok0 = __shfl_sync(0xFFFFFFFFu, x.tok0, i);
        const int toks = __shfl_sync(0xFFFFFFFFu, x.toks, i);
#pragma unroll 1
        for (int64_t z = __shfl_sync(0xFFFFFFFFu, z0, i); z < toks; z += step)
          empty_token<D>(a, tok0 + static_cast<int>(z), lane);
      }
    }
    if (a.cu != nullptr) {
      const int lo = falls ? 0 : min(max(a.cu[0], 0), a.T);
      const int hi = falls ? 0 : min(max(a.cu[a.B], 0), a.T);
      // rows [0, lo) and [hi, T), as one run of rows
#pragma unroll 1
      for (int64_t z = first; z < static_cast<int64_t>(lo) + a.T - hi; z += step)
        empty_token<D>(a, static_cast<int>(z < lo ? z : z - lo + hi), lane);
    }
  }

  tc_fence_before();
  __syncthreads();
  report_abort(&abort_word, a.err);
  if (warp == kPvWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the segments that cross runs, in run order.  Block (c, y): the segment that
// begins in run c, if any; a thread takes four elements of a row.
template <int D>
__global__ void __launch_bounds__(256) cross_join_kernel(const CrossArgs a) {
  constexpr int kLanes = D / 4, kBatch = 4;
  pdl_trigger();
  pdl_wait();
  const Split s = a.split[blockIdx.x];
  const int run = blockIdx.x;
  // end < 0: nothing to join; what else is out of range was never written, by a kernel that gave
  // up a wait and has reported it
  if (s.end < 0 || s.all <= s.end || s.slot < 0 || s.slot >= 2 * a.runs || s.rows > a.part_rows)
    return;
  // the run that holds tile u: the last c with all c / n <= u
  const int64_t n_runs = s.all < a.runs ? s.all : a.runs;
  const int last = static_cast<int>(((s.end + 1) * n_runs + s.all - 1) / s.all - 1);
  const int r = (blockIdx.y * 256 + threadIdx.x) / kLanes, x = threadIdx.x % kLanes;
  if (r >= s.rows) return;
  const int64_t stride = part_floats(a.part_rows, D);
  float mx = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  // loads of a few parts in flight: one after another they cost a memory latency each
  for (int c0 = run; c0 <= last; c0 += kBatch) {
    float2 ml[kBatch];
    float4 po[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int c = min(c0 + i, last);
      const float* part = a.parts + (c == run ? s.slot : 2 * c) * stride;
      ml[i] = *reinterpret_cast<const float2*>(part + 2 * r);
      po[i] = *reinterpret_cast<const float4*>(part + 2 * a.part_rows + r * D + 4 * x);
      if (c0 + i > last) ml[i] = make_float2(-INFINITY, 0.f);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float mn = fmaxf(mx, ml[i].x), ref = fmaxf(mn, -3.4e38f);
      const float co = ex2_f32(mx - ref), cn = ex2_f32(ml[i].x - ref);
      mx = mn;
      l = l * co + ml[i].y * cn;
      o = make_float4(o.x * co + po[i].x * cn, o.y * co + po[i].y * cn, o.z * co + po[i].z * cn,
                      o.w * co + po[i].w * cn);
    }
  }
  const int row = s.row0 + r, tok = row / a.G;
  const int64_t at = static_cast<int64_t>(s.tok0 + tok) * a.H + s.hk * a.G + row - tok * a.G;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  if (a.o != nullptr) {
    const __nv_bfloat162 h[2] = {__floats2bfloat162_rn(o.x * inv, o.y * inv),
                                 __floats2bfloat162_rn(o.z * inv, o.w * inv)};
    *reinterpret_cast<uint2*>(a.o + at * D + 4 * x) = *reinterpret_cast<const uint2*>(h);
  } else {
    *reinterpret_cast<float4*>(a.o32 + at * D + 4 * x) =
        make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  }
  if (x == 0 && a.lse != nullptr) a.lse[at] = row_lse(a, mx, l);
}

template <int D>
cudaError_t launch_cross_d(const CUtensorMap& tk, const CUtensorMap& to, const CrossArgs& a,
                           cudaStream_t stream) {
  using C = Cfg<D>;
  const cudaError_t e = cudaFuncSetAttribute(
      cross_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(a.runs));
  const cudaError_t k =
      launch_pdl(cross_kernel<D>, grid, dim3(kThreads), C::kSmem, stream, 1, tk, to, a);
  if (k != cudaSuccess) return k;
  return launch_pdl(cross_join_kernel<D>,
                    dim3(grid.x, static_cast<unsigned>(a.part_rows * (D / 4) / 256)), dim3(256), 0,
                    stream, 1, a);
}

struct Plan {
  int runs, part_rows;
  size_t parts, total;
};

Plan plan(int64_t T, int B, int H, int Hkv, int D, int max_pages) {
  const int64_t rows = T * (H / Hkv);
  const int64_t tiles = (rows / kPair + B) * Hkv * max_pages;  // at most
  Plan p;
  p.runs = static_cast<int>(std::min<int64_t>(std::max<int64_t>(tiles, 1), device_sms()));
  p.part_rows = static_cast<int>(std::min<int64_t>(kPair, (rows + 31) / 32 * 32));
  p.parts = (p.runs * sizeof(Split) + 255) / 256 * 256;
  p.total = p.parts + 2 * p.runs * part_floats(p.part_rows, D) * sizeof(float);
  return p;
}

}  // namespace

nvq_status check_cross(int64_t T, int B, int H, int Hkv, int D, int max_pages) {
  if (T < 1 || B < 1 || H < 1 || Hkv < 1 || H % Hkv != 0 || max_pages < 1 ||
      max_pages > 0x7FFFFFFF / kPage)
    return NVQ_ERR_INVALID;
  if (D != 64 && D != 128) return NVQ_ERR_UNSUPPORTED;
  if (B > 65535 || H > 65535 || T > (0x7FFFFF00 - 1) / H) return NVQ_ERR_UNSUPPORTED;
  // The line has at most (rows / 256 + B) Hkv max_pages tiles ((rows / 128 + B) Hkv < 2^24 + 2^32:
  // no overflow), of which a run counts its own in 29 bits (four units each).  The second holds
  // for 32 runs and more by the first.
  const int64_t tiles = (T * (H / Hkv) / kRows + B) * Hkv * max_pages;
  if (tiles >= int64_t{1} << 34) return NVQ_ERR_UNSUPPORTED;
  if (tiles >= 1 << 29 && tiles / device_sms() >= (1 << 29) - 1) return NVQ_ERR_UNSUPPORTED;
  return NVQ_OK;
}

size_t cross_workspace(int64_t T, int B, int H, int Hkv, int D, int max_pages) {
  return plan(T, B, H, Hkv, D, max_pages).total;
}

nvq_status launch_cross(const CrossCall& c, uint8_t* ws, cudaStream_t stream) {
  const Plan p = plan(c.T, c.B, c.H, c.Hkv, c.D, c.max_pages);
  if (c.num_pages > 0x7FFFFFFF / c.Hkv) return NVQ_ERR_UNSUPPORTED;  // tensor-map coordinates
  int* err = device_error_word();
  if (err == nullptr) return NVQ_ERR_CUDA;
  CUtensorMap tk;
  if (const int r = make_kv_codes_map(&tk, c.pool, c.num_pages * c.Hkv, c.D, kPage); r != 0)
    return fail_driver("cuTensorMapEncodeTiled", r);
  const int G = c.H / c.Hkv;
  CUtensorMap to = tk;
  if (c.o != nullptr && 32 % G == 0)
    if (const int r = make_rows_map(&to, c.o, c.T, c.H, c.D, G, 32 / G); r != 0)
      return fail_driver("cuTensorMapEncodeTiled", r);
  const CrossArgs a{static_cast<const uint16_t*>(c.q), c.ld_q, static_cast<int>(c.T),
                    static_cast<const uint8_t*>(c.pool), c.num_pages, c.page_table, c.ld_table,
                    c.max_pages, c.kv_lens, c.cu_tokens, static_cast<int>(c.T / c.B), c.B, c.H,
                    c.Hkv, G, c.o != nullptr && 32 % G == 0, scales_of(c.scale * kLog2e, c.D),
                    static_cast<__nv_bfloat16*>(c.o), c.o32,
                    c.lse, reinterpret_cast<Split*>(ws),
                    reinterpret_cast<float*>(ws + p.parts),
                    p.part_rows, p.runs, ~uint64_t{0} / p.runs + 1, err};
  const cudaError_t e = timed(NVQ_KERNEL_CROSS, stream, [&] {
    return c.D == 128 ? launch_cross_d<128>(tk, to, a, stream)
                      : launch_cross_d<64>(tk, to, a, stream);
  });
  return e == cudaSuccess ? NVQ_OK : fail_cuda("attn cross", e);
}

}  // namespace nvq

extern "C" {

size_t attn_qat_cross_workspace(int64_t T, int B, int H, int Hkv, int D, int max_pages) {
  if (nvq::check_cross(T, B, H, Hkv, D, max_pages) != NVQ_OK) return 0;
  const size_t n = nvq::cross_workspace(T, B, H, Hkv, D, max_pages);
  return T == B ? std::max(n, attn_qat_decode_workspace(B, H, Hkv, D, max_pages)) : n;
}

nvq_status attn_qat_cross(const void* q, int64_t ld_q, int64_t T, const void* pool,
                          int64_t num_pages, const int32_t* page_table, int64_t ld_table,
                          int max_pages, const int32_t* kv_lens, const int32_t* cu_tokens, int B,
                          int H, int Hkv, int D, float scale, void* o, float* lse, void* ws,
                          size_t ws_bytes, nvq_stream_t stream) {
  using namespace nvq;
  nvq_status st = check_cross(T, B, H, Hkv, D, max_pages);
  if (st != NVQ_OK) return st;
  const int64_t row = static_cast<int64_t>(H) * D;
  if (!(std::isfinite(scale) && scale > 0.f) || (cu_tokens == nullptr && T % B != 0) ||
      (reinterpret_cast<uintptr_t>(cu_tokens) & 3u) != 0)
    return NVQ_ERR_INVALID;
  if (q == nullptr || o == nullptr || (reinterpret_cast<uintptr_t>(q) & 15u) != 0 ||
      (reinterpret_cast<uintptr_t>(o) & 15u) != 0 || ld_q < row || ld_q % 8 != 0 ||
      (reinterpret_cast<uintptr_t>(lse) & 3u) != 0)
    return NVQ_ERR_INVALID;
  st = check_kv(pool, num_pages, page_table, ld_table, max_pages, kv_lens);
  if (st != NVQ_OK) return st;
  if (ws == nullptr || ws_bytes < attn_qat_cross_workspace(T, B, H, Hkv, D, max_pages) ||
      (reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
    return NVQ_ERR_WORKSPACE;
  // a row of q is read by one run after another, at whatever time: o elsewhere
  if (ranges_meet(q, 2 * static_cast<uint64_t>((T - 1) * ld_q + row), o,
                  2 * static_cast<uint64_t>(row * T)))
    return NVQ_ERR_INVALID;
  // One token a sequence goes to the single-token kernel, up to the 16 query heads of a KV head
  // that one of its runs takes: it reads every key again for each 16 more, and here 256 rows cost
  // little more than one.  64 sequences of 8192 keys, 8 KV heads of 128, there and here: 1 head a
  // KV head 102 and 220 us, 16 heads 149 and 263, 32 heads 279 and 279, 64 heads 537 and 290, 128
  // heads 1055 and 301; 8 sequences of 512 keys, one KV head of 64: 8.6 and 8.7, 9.4 and 8.6, 9.9
  // and 8.7, 11.3 and 8.7, 13.6 and 9.4.
  if (cu_tokens == nullptr && T == B && H / Hkv <= 16)
    return attn_qat_decode(q, ld_q, pool, num_pages, page_table, ld_table, max_pages, kv_lens, B,
                           H, Hkv, D, scale, 0, 0, o, lse, ws, ws_bytes, stream);
  return launch_cross({q, ld_q, T, pool, num_pages, page_table, ld_table, max_pages, kv_lens,
                       cu_tokens, B, H, Hkv, D, scale, o, nullptr, lse},
                      static_cast<uint8_t*>(ws), stream);
}

}  // extern "C"
