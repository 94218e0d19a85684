// Attention of one new token per sequence over the paged NVFP4 cache:
//   S_j = scale q~ . K~_j,  o = sum_j exp(S_j - lse) V~_j,  lse = ln sum exp S_j
// over the visible keys, in one pass with the running maximum and sum of every
// query head.
//
// Bound.  A key of one KV head is 9 D / 8 bytes (codes and scales of K and V) and
// 4 D operations per query head that shares it, so the cache's bytes bound the
// call; on-chip, the decode of 2 D codes per key is what has to hide under them.
//
// Work split.  The visible pages of every (sequence, KV head, group of query
// heads) lie one after another on one line of tiles (a tile: one page record, 128
// keys), which is cut into equal runs, whatever the lengths: nothing waits for the
// longest sequence.  A run that covers all tiles of a segment
// (one sequence, KV head and group) writes o itself; a segment that crosses runs
// leaves (m, l, sum p V~) per run in the workspace, and a second small kernel
// joins them in run order, so results do not vary from run to run.
//
// One run, six warps; three runs (two above 8 query heads, four of long work on heads of
// 64) make a CTA, one CTA an SM (as CTAs of their own the second and third of an SM
// started 2 us and more late):
//   producer  fetches records into a ring of stages (K codes by tensor-map loads
//             with the swizzle the MMA reads, the rest by bulk copies; only the
//             rows that hold tokens) and describes each tile beside it
//   MMA       quantizes q of a new segment, brings K's scales into the order of
//             the scale operand and issues S [128 keys x 16 heads] = K~ q~^T as
//             block-scaled FP4 tcgen05 MMAs on the stored codes: K is never
//             decoded.  (Decoding K in registers for mma.sync made the issue
//             slots the bound: 159 us for 8 x 131072 tokens, 8 KV heads of 128.)
//   4 x 32    keys: read S from tensor memory in the fragment layout of an
//             m16n8 product, exponentiate, and accumulate
//               O^T [D x 8 heads] += V~^T [D x 16 keys] P^T
//             with V decoded as the A operand of mma.sync.  (V's scales run along
//             D, so its codes cannot be the FP4 operand of a product over keys;
//             decoded values are wanted in registers, where mma.sync takes them.)
// The accumulator fragment of S becomes the B operand by an 8x8 transpose across
// lanes.  Codes become f16 by the hardware conversion times their scale, exactly;
// p is rounded to f16 (as in the training forward), its sum is taken before the
// rounding; all sums are fp32.  The maximum that p refers to is raised only when
// a score exceeds it by 8 (log2): p then stays below 2^8, far inside f16, and the
// cross-lane maximum and the rescaling of O leave the common path.
//
// Measured (calls in a CUDA graph): 8 x up to 131072 tokens, 64 heads on 8 of 128:
// 117 us, 87% of the copy rate in bytes of the cache; 64 sequences of up to 8192, 32
// heads on 8: 63 us, 69%; one sequence of 777 tokens: 10 us, the latency of two
// launches, the scan and a tile.  Short segments cost most: each begins with a
// quantization of q and ends with two barriers of its four warps.
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

constexpr int kWarps = 4;  // consumer warps of a run, 32 keys of a tile each
constexpr int kProducer = kWarps, kMma = kWarps + 1;
constexpr int kRunWarps = kWarps + 2;
constexpr float kSlack = 8.f;  // scores may exceed the reference maximum by this (log2)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Per shape: query heads per run (8 NT), runs per CTA, ring stages; shared memory and
// tensor memory of a run.
template <int D, int NT, int kRunsPerCta>
struct Cfg {
  static constexpr int kHeads = 8 * NT;
  static constexpr int kRuns = kRunsPerCta;  // one CTA per SM
  static constexpr int kThreads = kRuns * kRunWarps * 32;
  static constexpr int kStages = D == 64 ? (kRuns == 4 ? 4 : 5) : (NT == 1 ? 2 : 3);
  static constexpr int kRow = D + 4;  // floats of a head's row in the join area
  static constexpr uint32_t kRec = record_bytes(D);
  static constexpr uint32_t kQ = kHeads * D * 2;         // q of a segment that starts with the tile
  static constexpr uint32_t kStage = kRec + kQ;
  static constexpr uint32_t kQCodes = kStages * kStage;  // [2] q~ codes, 16 rows of D/2 bytes
  static constexpr uint32_t kQScales = kQCodes + 2 * 1024;               // [2][D/64] blocks of 512
  static constexpr uint32_t kJoin = kQScales + 2 * 1024;                 // float [4][kHeads][kRow]
  static constexpr uint32_t kMl = kJoin + kWarps * kHeads * kRow * 4;     // float2 [4][heads]
  static constexpr uint32_t kDesc = kMl + kWarps * kHeads * 8;           // TileDesc [stages]
  static constexpr uint32_t kBars = kDesc + kStages * 32;
  static constexpr uint32_t kRun = (kBars + (3 * kStages + 4) * 8 + 1023) / 1024 * 1024;
  static constexpr uint32_t kSmem = kRuns * kRun + 1024;  // + alignment
  // tensor memory columns: S of stage s, scales of K of stage s, of q~ of buffer b
  static constexpr uint32_t kSfa = 16 * kStages, kSfb = kSfa + kStages * (D / 16);
  static constexpr uint32_t kCols = 128, kAlloc = kRuns > 2 ? 512 : 256;
  static_assert(kSfb + 2 * (D / 16) <= kCols, "tensor memory");
  static_assert(apart_from_linear_small(kSmem), "tensor memory");
  static_assert(kStage % 1024 == 0, "swizzle atoms");
};

enum : int { kStart = 1, kEnd = 2, kMasked = 4, kAbsent = 8 };

struct TileDesc {
  int key0, len, wstart, flags;  // keys [key0, key0 + 128); visible: < len and (>= wstart or sink)
  int b, hg, slot, rows;         // slot: where the segment's part goes (-1: it is whole)
};

struct DecodeArgs {
  const uint16_t* q;
  int64_t ld_q;
  const uint8_t* pool;
  int64_t num_pages;
  const int32_t* table;
  int64_t ld_table;
  int max_pages;
  const int32_t* lens;
  int B, H, Hkv, G, chunks;  // G query heads per KV head in `chunks` groups
  float scale_log2;
  int window, sinks;
  __nv_bfloat16* o;
  float* lse;
  struct RunInfo* split;  // what crosses runs, by run or by segment (workspace)
  int by_segment;         // 1: entries by segment (there are fewer than runs)
  float* parts;           // [2 runs] parts (workspace)
  int runs;               // of the grid
  uint64_t runs_magic;    // 2^64 / runs, rounded up
  int* err;
};

// A segment that begins in a run and goes on in later ones; last < 0: none.
struct RunInfo {
  int b, hg, run, slot, last;  // its first run, that run's part, its last run
};

// Floats of one part: m (log2 units) and l per head, then the sums [heads][D].
__host__ __device__ constexpr int part_floats(int D, int heads) { return heads * (D + 2); }

// The line of `all` tiles is cut into n = min(all, runs) runs: run c is [all c / n,
// all (c + 1) / n), never empty; of the grid's runs those from n on have nothing.
// all c / n = (all / n) c + (all % n) c / n.  n is the grid's or all itself, so there is
// nothing to divide: the host gives 2^64 / runs, rounded up (all <= 2^53 and runs < 2^10
// keep the product's error below 1 / runs).
struct Runs {
  int64_t all, per;
  int n, rest;
  uint32_t magic;
  __device__ __forceinline__ Runs(int64_t all_, int runs, uint64_t magic_) : all(all_) {
    if (all < runs) {
      n = static_cast<int>(all);
      per = 1;
      rest = 0;
    } else {
      n = runs;
      per = static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(all), magic_));
      rest = static_cast<int>(all - per * runs);
    }
    magic = static_cast<uint32_t>(magic_ >> 32) + 1;  // rest c < 2^24: exact as well
  }
  __device__ __forceinline__ int64_t begin(int c) const {
    return c < n ? per * c + __umulhi(static_cast<uint32_t>(rest * c), magic) : all;
  }
};

// The tiles of a sequence: pages [0, sink_pages) and [first, pages).
struct Extent {
  int len, sink_pages, first, tiles, wstart;
};

__device__ __forceinline__ Extent extent(const DecodeArgs& a, int b, bool* over) {
  Extent e;
  const int cap = a.max_pages * kPage;
  const int n = a.lens[b];
  *over = n > cap;
  e.len = max(0, min(n, cap));
  const int pages = (e.len + kPage - 1) / kPage;
  e.wstart = a.window > 0 ? max(0, e.len - a.window) : 0;
  e.first = e.wstart / kPage;
  e.sink_pages = e.wstart > 0 ? min((min(a.sinks, e.len) + kPage - 1) / kPage, e.first) : 0;
  e.tiles = pages - e.first + e.sink_pages;
  return e;
}

// The KV head of a head group (a division only where there are several per KV head).
__device__ __forceinline__ int kv_head(const DecodeArgs& a, int hg) {
  return a.chunks == 1 ? hg : hg / a.chunks;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  return __byte_perm(a, b, sel);
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// tcgen05.ld of 16 lanes (keys) x 8 NT columns (heads): register 4 nt + e holds, as
// the accumulator of an m16n8 product, key g (e < 2) or g + 8, head 8 nt + 2t + e % 2.
template <int NT>
__device__ __forceinline__ void load_scores(uint32_t taddr, float (&v)[NT][4]) {
  uint32_t r[4 * NT];
  if constexpr (NT == 1)
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 4 * NT; ++i) v[i / 4][i % 4] = __uint_as_float(r[i]);
}

// Offsets in a record of what a lane (4 g + t) reads of V: of each 16 keys 2t, 2t + 1,
// 2t + 8, 2t + 9, elements [D/8 g, D/8 (g + 1)).  Lanes of odd t take the odd key
// first: keys of both parities in one load, whose rows lie in different banks.
template <int D>
struct VOffsets {
  int codes[2], scales[2];
  __device__ __forceinline__ VOffsets(int r0, int g, int t) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = r0 + 2 * t + (j ^ (t & 1));
      codes[j] = v_codes_at(D) + row * (D / 2) + g * (D / 16);
      scales[j] = v_scales_at(D) + row * (D / 16) + g * (D / 8) / 16;
    }
  }
};

// State of a consumer warp for the current segment.  Lane = 4 g + t.
template <int D, int NT>
struct State {
  float o[NT][D / 16][4];    // O^T: elements d = D/8 g + 2 i (+1: [2], [3]), heads 2t, 2t + 1
  float m[NT][2], l[NT][2];  // reference maximum (log2 units; all lanes) and this lane's sum

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }
  }
};

__device__ __forceinline__ bool sees(const TileDesc& td, int sinks, int key) {
  return key < td.len && (key >= td.wstart || key < sinks);
}

// Keys r0..r0 + 31 of the record at `rec`, scores at tensor memory address `tm`;
// arrives on `release` once the stage is read.
template <int D, int NT>
__device__ __forceinline__ void tile_keys(const DecodeArgs& a, const uint8_t* rec, int r0,
                                          uint32_t tm, uint64_t* release, const TileDesc& td,
                                          const VOffsets<D>& vo, State<D, NT>& st, int g, int t) {
  float s[2][NT][4];
  load_scores<NT>(tm, s[0]);
  load_scores<NT>(tm + (16u << 16), s[1]);
  // ---- codes and scales of V~
  uint32_t vc[2][4][D / 64], vs[2][2];
  const int odd = t & 1;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t sb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = 16 * i + 8 * (j >> 1);  // behind the lane's first
      const uint8_t* c = rec + vo.codes[j & 1] + row * (D / 2);
      if constexpr (D == 128) {
        const uint2 v = *reinterpret_cast<const uint2*>(c);
        vc[i][j][0] = v.x;
        vc[i][j][1] = v.y;
      } else {
        vc[i][j][0] = *reinterpret_cast<const uint32_t*>(c);
      }
      sb[j] = rec[vo.scales[j & 1] + row * (D / 16)];
    }
    if (td.flags & kMasked) {
      // rows that no visible key owns may hold anything, NaN scales among it: their p
      // becomes 0 below, their V~ here
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (!sees(td, a.sinks, td.key0 + r0 + 16 * i + 2 * t + ((j & 1) ^ odd) + 8 * (j >> 1)))
          sb[j] = 0;
    }
    vs[i][0] = e4m3x2_to_f16x2(prmt(sb[0], sb[1], 0x0040u));
    vs[i][1] = e4m3x2_to_f16x2(prmt(sb[2], sb[3], 0x0040u));
  }
  tmem_wait_ld();
  // everything of the stage is in registers: it is refilled under the arithmetic
  // (held until its end: 1 us more at 8 x 131072 tokens, 8 KV heads of 128)
  tc_fence_before();
  mbar_arrive_warp(release);
  // ---- p = 2^(S log2e - m)
  float mx[NT][2];
  bool grows = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    if (td.flags & kMasked) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (!sees(td, a.sinks, td.key0 + r0 + 16 * i + g + 8 * h))
            s[i][nt][2 * h] = s[i][nt][2 * h + 1] = -INFINITY;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mx[nt][h] = max3f(s[0][nt][h], s[0][nt][2 + h], fmaxf(s[1][nt][h], s[1][nt][2 + h]));
      mx[nt][h] *= a.scale_log2;
      grows |= mx[nt][h] > st.m[nt][h] + kSlack;
    }
  }
  if (__any_sync(0xFFFFFFFFu, grows)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mn = mx[nt][h];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
          mn = fmaxf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, off));
        mn = fmaxf(mn, st.m[nt][h]);
        // -inf: nothing seen yet, the sums are 0
        const float c = mn > -INFINITY ? ex2_f32(st.m[nt][h] - mn) : 1.f;
        st.m[nt][h] = mn;
        st.l[nt][h] *= c;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          st.o[nt][i][h] *= c;
          st.o[nt][i][2 + h] *= c;
        }
      }
  }
  uint32_t pb[2][NT][2];
  const uint32_t swap = odd ? 0x1032u : 0x3210u;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const uint64_t neg_m = pk2(-fmaxf(st.m[nt][0], -3.4e38f), -fmaxf(st.m[nt][1], -3.4e38f));
    const uint64_t scale2 = pk2(a.scale_log2, a.scale_log2);
    uint64_t l2 = pk2(st.l[nt][0], st.l[nt][1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float p0, p1, p2, p3;
      up2(fma2(pk2(s[i][nt][0], s[i][nt][1]), scale2, neg_m), p0, p1);
      up2(fma2(pk2(s[i][nt][2], s[i][nt][3]), scale2, neg_m), p2, p3);
      p0 = ex2_f32(p0);
      p1 = ex2_f32(p1);
      p2 = ex2_f32(p2);
      p3 = ex2_f32(p3);
      l2 = add2(l2, add2(pk2(p0, p1), pk2(p2, p3)));
      pb[i][nt][0] = movmatrix_trans(pack_f16x2_rn(p0, p1));
      pb[i][nt][1] = movmatrix_trans(pack_f16x2_rn(p2, p3));
      pb[i][nt][0] = prmt(pb[i][nt][0], 0u, swap);
      pb[i][nt][1] = prmt(pb[i][nt][1], 0u, swap);
    }
    up2(l2, st.l[nt][0], st.l[nt][1]);
  }
  // ---- O^T += V~^T P^T: codes of two keys interleaved, so that one conversion
  // gives a pair of keys of one element
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int w = 0; w < D / 64; ++w) {
      uint32_t ev[2][4], od[2][4];  // even and odd elements of the 4 bytes, the two pairs of keys
#pragma unroll
      for (int pr = 0; pr < 2; ++pr) {
        const uint32_t x = vc[i][2 * pr][w], y = vc[i][2 * pr + 1][w];
        e2m1x8_to_f16x2((x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u), ev[pr]);
        e2m1x8_to_f16x2(((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), od[pr]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t af[4] = {hmul2(ev[0][e], vs[i][0]), hmul2(od[0][e], vs[i][0]),
                                hmul2(ev[1][e], vs[i][1]), hmul2(od[1][e], vs[i][1])};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma16816(st.o[nt][4 * w + e], af, pb[i][nt][0], pb[i][nt][1]);
      }
    }
  }
}

// The MMA warp: q~ of the segment whose first tile holds q at `qraw` -- codes in the
// swizzled rows of the B operand, scales in the 512-byte blocks of the scale operand.
template <int D, int NT>
__device__ __forceinline__ void quantize_q(const uint8_t* qraw, int heads, uint8_t* codes,
                                           uint8_t* scales, int lane) {
  constexpr int kBlocks = D / 16;
#pragma unroll
  for (int x = lane; x < 8 * NT * kBlocks; x += 32) {
    const int n = x / kBlocks, j = x % kBlocks;
    uint2 c = make_uint2(0u, 0u);
    uint32_t sb = 0;
    if (n < heads) {
      const uint4* src = reinterpret_cast<const uint4*>(qraw + n * (D * 2) + j * 32);
      const uint4 lo = src[0], hi = src[1];
      const uint32_t v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      const Codes16 r = codes16_unit(v);
      c = make_uint2(r.codes[0], r.codes[1]);
      sb = r.sbyte;
    }
    const int swz = D == 128 ? (n >> 1) & 3 : (n >> 2) & 1;  // 64- and 32-byte swizzles
    *reinterpret_cast<uint2*>(codes + n * (D / 2) + (((j >> 1) ^ swz) << 4) + (j & 1) * 8) = c;
    scales[(j >> 2) * 512 + n * 16 + (j & 3)] = static_cast<uint8_t>(sb);
  }
}

// K's scales [128][D/16] to D/64 blocks of 512 bytes, in place: row r of a block holds
// the words (4 scales) of keys r, r + 32, r + 64, r + 96.
template <int D>
__device__ __forceinline__ void arrange_scales(uint8_t* sc, int lane) {
  uint32_t w[D / 64][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (D == 128) {
      const uint2 v = *reinterpret_cast<const uint2*>(sc + (lane + 32 * i) * 8);
      w[0][i] = v.x;
      w[1][i] = v.y;
    } else {
      w[0][i] = *reinterpret_cast<const uint32_t*>(sc + (lane + 32 * i) * 4);
    }
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < D / 64; ++k)
    *reinterpret_cast<uint4*>(sc + k * 512 + lane * 16) =
        make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
}

// Element of O at position `pos` of a stored row: the rows keep the order in which
// the lanes hold them, pos = 16 i + 2 g + e for d = D/8 g + 2 i + e.
template <int D>
__device__ __forceinline__ int element_of(int pos) {
  return (pos >> 1 & 7) * (D / 8) + (pos >> 4) * 2 + (pos & 1);
}

// Place in a ring of `stages`: stage and the parity of its use.
struct Ring {
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) {
      s = 0;
      phase ^= 1;
    }
  }
};

template <int D, int NT, int kRunsPerCta>
__global__ void __launch_bounds__(Cfg<D, NT, kRunsPerCta>::kThreads, 1)
    decode_kernel(const __grid_constant__ CUtensorMap tk,
                  const __grid_constant__ CUtensorMap tk32, const DecodeArgs a) {
  using C = Cfg<D, NT, kRunsPerCta>;
  constexpr int kThreads = C::kThreads;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int64_t warp_sum[kThreads / 32];
  __shared__ int64_t start_before[C::kRuns];
  __shared__ int start_b[C::kRuns];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  const int sub = threadIdx.x / (kRunWarps * 32);     // run of the CTA
  const int tid = threadIdx.x % (kRunWarps * 32);     // thread and warp of the run
  const int warp = tid >> 5, lane = threadIdx.x & 31;
  const int quarter = threadIdx.x >> 5 & 3;           // of tensor memory that this warp may read
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023u) &
                                             ~static_cast<uintptr_t>(1023u)) + sub * C::kRun;
  float* join = reinterpret_cast<float*>(smem + C::kJoin);
  float2* ml = reinterpret_cast<float2*>(smem + C::kMl);
  TileDesc* desc = reinterpret_cast<TileDesc*>(smem + C::kDesc);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBars);
  uint64_t* empty = full + C::kStages;
  uint64_t* scored = empty + C::kStages;   // S of the stage is in tensor memory
  uint64_t* q_free = scored + C::kStages;  // [2]: the MMAs that read q~ buffer b are done
  uint64_t* meet = q_free + 2;             // [2]: parts written, parts read
  volatile int* abort = &abort_word;
  pdl_trigger();

  if (threadIdx.x == 0) *abort = 0;
  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kWarps);
      mbar_init(&scored[s], 1);
    }
    mbar_init(&q_free[0], 1);
    mbar_init(&q_free[1], 1);
    mbar_init(&meet[0], kWarps);
    mbar_init(&meet[1], kWarps);
    fence_mbar_init();
  }
  for (uint32_t i = tid; i < 4096 / 16; i += kRunWarps * 32)  // unused rows of q~ stay 0
    *reinterpret_cast<uint4*>(smem + C::kQCodes + 16 * i) = make_uint4(0, 0, 0, 0);
  if (threadIdx.x < 32) {
    tmem_alloc(&tmem_slot, C::kAlloc);
    tmem_relinquish();
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tk32);
  }
  pdl_wait();  // before this nothing that another kernel may have written is read
  // ---- the runs of this CTA: a scan over the sequences
  const int hgs = a.Hkv * a.chunks;
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b_lo = min(a.B, static_cast<int>(threadIdx.x) * per), b_hi = min(a.B, b_lo + per);
  int64_t mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    bool over;
    mine += extent(a, b, &over).tiles;
    if (over && blockIdx.x == 0) atomicMax(a.err, kErrTable);
  }
  int64_t scan = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, scan, off);
    if (lane >= off) scan += v;
  }
  if (lane == 31) warp_sum[threadIdx.x >> 5] = scan;
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < static_cast<int>(threadIdx.x >> 5)) scan += warp_sum[w];
    total += warp_sum[w];
  }
  const int64_t before = scan - mine;  // tiles (of one head group) before this thread's sequences
  // consecutive runs lie on different SMs: a few tiles spread over all of them
  const int ctas = static_cast<int>(gridDim.x);
  const Runs line(total * hgs, a.runs, a.runs_magic);
  for (int i = 0; i < C::kRuns && mine > 0; ++i) {
    const int64_t u = line.begin(i * ctas + static_cast<int>(blockIdx.x));
    if (u < line.all && before * hgs <= u && u < (before + mine) * hgs) {
      int64_t at = before;
      int b = b_lo;
      for (;; ++b) {
        bool over;
        const int n = extent(a, b, &over).tiles;
        if (u < (at + n) * hgs) break;
        at += n;
      }
      start_b[i] = b;
      start_before[i] = at;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot + sub * C::kCols;
  const int run = sub * ctas + static_cast<int>(blockIdx.x);
  const int64_t u0 = line.begin(run), u1 = line.begin(run + 1);
  const int n_tiles = static_cast<int>(u1 - u0);
  if (!a.by_segment && warp == kProducer && lane == 0) a.split[run].last = -1;

  if (warp == kProducer && n_tiles > 0) {
    // ------------------------------------------------------------ producer
    int b = start_b[sub];
    bool over, ok = true;
    Extent e = extent(a, b, &over);
    int64_t seg0 = start_before[sub] * hgs;  // line position of the sequence's first tile
    const int64_t into = u0 - seg0;
    int hg;  // into / tiles, below 2^16
    if (into < (int64_t{1} << 23)) {  // the float quotient is off by less than 1
      const int n = static_cast<int>(into);
      hg = static_cast<int>(__fdividef(static_cast<float>(n), static_cast<float>(e.tiles)));
      if (static_cast<int64_t>(hg) * e.tiles > n) --hg;
      if (static_cast<int64_t>(hg + 1) * e.tiles <= n) ++hg;
    } else {
      hg = static_cast<int>(into / e.tiles);
    }
    int i = static_cast<int>(into - static_cast<int64_t>(hg) * e.tiles);
    int n = 0;
    Ring ring;
    while (n < n_tiles && ok) {
      // ---- one segment (the part of it that lies in the run: tiles i .. i_end - 1)
      const int64_t first = seg0 + static_cast<int64_t>(hg) * e.tiles;
      const int i_end = min(e.tiles, i + n_tiles - n);
      // whole segments are written directly; a part that begins with the run goes
      // to the run's slot 0, one that begins inside it to slot 1
      const bool whole = first >= u0 && first + e.tiles <= u1;
      TileDesc td;
      td.len = e.len;
      td.wstart = e.wstart;
      td.b = b;
      td.hg = hg;
      td.slot = whole ? -1 : 2 * run + (first > u0 ? 1 : 0);
      const int hk = kv_head(a, hg), g0 = (hg - hk * a.chunks) * C::kHeads;
      const uint8_t* q = reinterpret_cast<const uint8_t*>(
          a.q + b * a.ld_q + static_cast<int64_t>(hk * a.G + g0) * D);
      uint32_t q_bytes = min(C::kHeads, a.G - g0) * (D * 2);  // with the first tile
      const int32_t* table = a.table + b * a.ld_table;
      const int i0 = i;
      int pages = 0;  // this lane's page number: of tile i0 + 32 k + lane
      for (; i < i_end; ++i, ++n, ring.next(C::kStages)) {
        // everything about the tile first, then the wait for its stage: the loads go
        // out as soon as the stage is free
        if (((i - i0) & 31) == 0) {
          const int j = i + lane;
          pages = j < e.tiles ? table[j < e.sink_pages ? j : e.first + j - e.sink_pages] : -1;
        }
        const int page = __shfl_sync(0xFFFFFFFFu, pages, i - i0);
        td.key0 = (i < e.sink_pages ? i : e.first + i - e.sink_pages) * kPage;
        td.rows = min(kPage, e.len - td.key0);
        td.flags = (i == i0 ? kStart : 0) | (i == i_end - 1 ? kEnd : 0);
        const bool there = page >= 0 && page < a.num_pages;
        if (!there) {
          td.flags |= kAbsent;
          if (lane == 0) atomicMax(a.err, kErrTable);
        }
        if (td.rows < kPage || (td.key0 < e.wstart && td.key0 + kPage > a.sinks))
          td.flags |= kMasked;
        const int s = ring.s;
        uint8_t* dst = smem + s * C::kStage;
        const int rec = page * a.Hkv + hk;
        const uint8_t* src = a.pool + static_cast<int64_t>(rec) * record_bytes(D);
        if (!(ok = mbar_wait_warp(&empty[s], ring.phase ^ 1, abort))) break;
        if (lane == 0) desc[s] = td;
        __syncwarp();
        if (there && td.rows == kPage) {
          mbar_arrive_expect_tx_w(&full[s], q_bytes + C::kRec);
          tma_load_4d_w(dst, &tk, 0, 0, rec, 0, &full[s]);
          bulk_load_w(dst + v_codes_at(D), src + v_codes_at(D), C::kRec - v_codes_at(D), &full[s]);
        } else if (there) {
          const uint32_t boxes = (td.rows + 31) / 32;  // K codes in boxes of 32 keys
          const uint32_t rows = (td.rows + 3) & ~3;    // whole 16-byte units of scales
          const uint32_t cb = rows * (D / 2), sb = rows * (D / 16);
          mbar_arrive_expect_tx_w(&full[s], q_bytes + boxes * (16 * D) + cb + 2 * sb);
          for (uint32_t x = 0; x < boxes; ++x)
            tma_load_4d_w(dst + x * (16 * D), &tk32, 0, x * 32, rec, 0, &full[s]);
          bulk_load_w(dst + v_codes_at(D), src + v_codes_at(D), cb, &full[s]);
          bulk_load_w(dst + k_scales_at(D), src + k_scales_at(D), sb, &full[s]);
          bulk_load_w(dst + v_scales_at(D), src + v_scales_at(D), sb, &full[s]);
        } else {
          mbar_arrive_expect_tx_w(&full[s], q_bytes);
        }
        if (q_bytes > 0) bulk_load_w(dst + C::kRec, q, q_bytes, &full[s]);
        q_bytes = 0;
      }
      if (lane == 0 && first >= u0) {  // with the loads on their way
        RunInfo* info = a.split + (a.by_segment ? b * hgs + hg : run);
        if (first + e.tiles > u1) {
          // the run that holds tile u: the last c with all c / n <= u
          const int64_t u = first + e.tiles - 1;
          *info = {b, hg, run, td.slot,
                   static_cast<int>(((u + 1) * line.n + line.all - 1) / line.all - 1)};
        } else if (a.by_segment) {
          info->last = -1;
        }
      }
      if (n == n_tiles || !ok) break;
      i = 0;
      if (++hg == hgs) {
        hg = 0;
        seg0 += static_cast<int64_t>(e.tiles) * hgs;
        do {
          e = extent(a, ++b, &over);
        } while (e.tiles == 0);
      }
    }
    if (!ok) {  // let the copies already issued land before the block leaves
      for (int m = max(0, n - C::kStages); m < n; ++m)
        mbar_wait_warp(&full[m % C::kStages], (m / C::kStages) & 1, nullptr, 10000000ull);
    }
  } else if (warp == kMma) {
    // ----------------------------------------------------------------- MMA
    constexpr uint32_t idesc = idesc_mxf4nvf4(128, 16);
    constexpr uint32_t lay = D == 128 ? 4u : 6u, sbo = 4 * D;  // swizzle, bytes of 8 rows
    int seg = 0;  // segments begun
    bool ok = true;
    int n = 0;
    if (sub == 0) {  // sequences without visible keys, while the first tile is on its way
      for (int b = blockIdx.x; b < a.B; b += ctas) {
        bool over;
        if (extent(a, b, &over).tiles > 0) continue;
        for (int x = lane; a.by_segment && x < hgs; x += 32) a.split[b * hgs + x].last = -1;
        const int64_t row0 = static_cast<int64_t>(b) * a.H;
        for (int x = lane; x < a.H * (D / 8); x += 32)
          reinterpret_cast<uint4*>(a.o + row0 * D)[x] = make_uint4(0, 0, 0, 0);
        if (a.lse != nullptr)
          for (int x = lane; x < a.H; x += 32) a.lse[row0 + x] = -INFINITY;
      }
    }
    Ring ring;
    for (; n < n_tiles; ++n, ring.next(C::kStages)) {
      const int s = ring.s;
      if (!(ok = mbar_wait_warp(&full[s], ring.phase, abort))) break;
      tc_fence_after();  // the scores that were in this stage's columns have been read
      struct { int flags, hg; } td = {desc[s].flags, desc[s].hg};
      uint8_t* stage = smem + s * C::kStage;
      if (td.flags & kStart) {
        const int qb = seg & 1;
        if (!(ok = mbar_wait_warp(&q_free[qb], ((seg >> 1) & 1) ^ 1, abort))) break;
        const int g0 = (td.hg - kv_head(a, td.hg) * a.chunks) * C::kHeads;
        quantize_q<D, NT>(stage + C::kRec, min(C::kHeads, a.G - g0), smem + C::kQCodes + qb * 1024,
                          smem + C::kQScales + qb * 1024, lane);
        ++seg;
      }
      const int qb = (seg - 1) & 1;
      if (!(td.flags & kAbsent)) {
        arrange_scales<D>(stage + k_scales_at(D), lane);
        fence_proxy_async_smem();
        __syncwarp();
        const uint32_t sfa = tmem + C::kSfa + s * (D / 16), sfb = tmem + C::kSfb + qb * (D / 16);
        const uint32_t ka = smem_u32(stage), qa = smem_u32(smem + C::kQCodes + qb * 1024);
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
          tmem_cp_32x128_x4_w(sfa + 4 * k, smem_u32(stage + k_scales_at(D)) + 512 * k);
          if (td.flags & kStart)
            tmem_cp_32x128_x4_w(sfb + 4 * k, smem_u32(smem + C::kQScales + qb * 1024) + 512 * k);
        }
        const uint64_t kd[2] = {sdesc(ka, 16, sbo, lay), sdesc(ka, 16, sbo, lay) + 2};
        const uint64_t qd[2] = {sdesc(qa, 16, sbo, lay), sdesc(qa, 16, sbo, lay) + 2};
        umma_fp4_group_w<D / 64>(tmem + 16 * s, kd, qd, idesc, sfa, sfb, bar_u32(&scored[s]),
                                 td.flags & kEnd ? bar_u32(&q_free[qb]) : 0u);
      } else {
        if (td.flags & kStart) {  // later tiles of the segment read q~ all the same
          fence_proxy_async_smem();
          __syncwarp();
#pragma unroll
          for (int k = 0; k < D / 64; ++k)
            tmem_cp_32x128_x4_w(tmem + C::kSfb + qb * (D / 16) + 4 * k,
                                smem_u32(smem + C::kQScales + qb * 1024) + 512 * k);
        }
        umma_commit_w(&scored[s]);
        if (td.flags & kEnd) umma_commit_w(&q_free[qb]);
      }
    }
    for (int m = max(0, n - C::kStages); m < n; ++m)  // the MMAs in flight end before the block
      mbar_wait_warp(&scored[m % C::kStages], (m / C::kStages) & 1, nullptr, 10000000ull);
  } else if (warp < kWarps) {
    // ----------------------------------------------------------- consumers
    const int g = lane >> 2, t = lane & 3;
    const int r0 = quarter * 32;  // its keys of a tile
    const VOffsets<D> vo(r0, g, t);
    State<D, NT> st;
    uint32_t ends = 0;
    Ring ring;
    for (int n = 0; n < n_tiles; ++n, ring.next(C::kStages)) {
      const int s = ring.s;
      if (!mbar_wait_warp(&full[s], ring.phase, abort)) break;
      if (!mbar_wait_warp(&scored[s], ring.phase, abort)) break;
      tc_fence_after();
      const TileDesc td = desc[s];
      if (td.flags & kStart) st.clear();
      if (!(td.flags & kAbsent) && r0 < td.rows) {
        tile_keys<D, NT>(a, smem + s * C::kStage, r0,
                         tmem + 16 * s + (static_cast<uint32_t>(r0) << 16), &empty[s], td, vo, st,
                         g, t);
      } else {
        mbar_arrive_warp(&empty[s]);
      }
      if (!(td.flags & kEnd)) continue;
      // ---- the warps' parts meet in shared memory, a head per warp at a time.  (An area
      // for all heads costs a stage of the ring: 2 us more at 8 x 131072 tokens, but half
      // of the barriers at a segment's end: 46 -> 39 us at 256 x 512.  A seventh warp that
      // joins while the others go on leaves 80 registers a thread: 140 us.)
      if (ends > 0 && !mbar_wait_warp(&meet[1], (ends - 1) & 1, abort)) break;
      const int hk = kv_head(a, td.hg), g0 = (td.hg - hk * a.chunks) * C::kHeads;
      const int heads = min(C::kHeads, a.G - g0);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int head = nt * 8 + 2 * t + h;
          float l = st.l[nt][h];
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, off);
          if (g == 0) ml[warp * C::kHeads + head] = make_float2(st.m[nt][h], l);
          float* row = join + (warp * C::kHeads + head) * C::kRow + 2 * g;
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
            *reinterpret_cast<float2*>(row + 16 * i) =
                make_float2(st.o[nt][i][h], st.o[nt][i][2 + h]);
        }
      }
      mbar_arrive_warp(&meet[0]);
      if (!mbar_wait_warp(&meet[0], ends & 1, abort)) break;
      ++ends;
      for (int head = warp; head < heads; head += kWarps) {
        float c[kWarps], mx = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, ml[w * C::kHeads + head].x);
        const float ref = fmaxf(mx, -3.4e38f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 v = ml[w * C::kHeads + head];
          c[w] = ex2_f32(v.x - ref);
          l = fmaf(v.y, c[w], l);
        }
        const int64_t row = static_cast<int64_t>(td.b) * a.H + hk * a.G + g0 + head;
        const float inv = l > 0.f ? 1.f / l : 0.f;
        float* part = a.parts + static_cast<int64_t>(max(td.slot, 0)) * part_floats(D, C::kHeads);
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {
          const int pos = 2 * lane + 64 * x;
          float o0 = 0.f, o1 = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 ov = *reinterpret_cast<const float2*>(
                join + (w * C::kHeads + head) * C::kRow + pos);
            o0 = fmaf(ov.x, c[w], o0);
            o1 = fmaf(ov.y, c[w], o1);
          }
          if (td.slot < 0)
            *reinterpret_cast<__nv_bfloat162*>(a.o + row * D + element_of<D>(pos)) =
                __floats2bfloat162_rn(o0 * inv, o1 * inv);
          else
            *reinterpret_cast<float2*>(part + 2 * C::kHeads + head * D + pos) = make_float2(o0, o1);
        }
        if (lane == 0) {
          if (td.slot >= 0)
            *reinterpret_cast<float2*>(part + 2 * head) = make_float2(mx, l);
          else if (a.lse != nullptr)
            a.lse[row] = l > 0.f ? (mx + log2f(l)) * kLn2 : -INFINITY;
        }
      }
      mbar_arrive_warp(&meet[1]);
    }
  }

  tc_fence_before();
  __syncthreads();
  report_abort(abort, a.err);
  if (threadIdx.x < 32) {
    tc_fence_after();
    tmem_dealloc(tmem_slot, C::kAlloc);
  }
}

// Joins the parts of the segments that cross runs, in run order.  Block (c, y): entry c
// of what crosses runs, heads [y, y + 1) kHeads / gridDim.y.  Sixteen or 32 lanes of
// four stored positions take one head; where fewer heads than lane groups are left,
// the groups share the parts and meet in shared memory.
template <int D, int NT, int kThreads>
__global__ void __launch_bounds__(kThreads) join_kernel(const DecodeArgs a) {
  constexpr int kHeads = 8 * NT, kLanes = D / 4, kGroups = kThreads / kLanes;
  constexpr int kFloats = part_floats(D, kHeads);
  __shared__ float4 red[kGroups][kLanes];
  __shared__ float2 red_ml[kGroups];
  pdl_trigger();
  pdl_wait();
  const RunInfo r = a.split[blockIdx.x];
  // last < 0: nothing to join; what else is out of range was never written, by a
  // kernel that gave up a wait and has reported it
  if (r.run < 0 || r.last < r.run || r.last >= a.runs || r.slot < 0 || r.slot >= 2 * a.runs ||
      r.b < 0 || r.b >= a.B || r.hg < 0 || r.hg >= a.Hkv * a.chunks)
    return;
  const int per = kHeads / gridDim.y;  // heads of this block
  const int share = max(1, kGroups / per);
  const int x = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  const int g0 = r.hg % a.chunks * kHeads;
  for (int h0 = 0; h0 < per; h0 += kGroups / share) {
    const int head = blockIdx.y * per + h0 + grp / share, sub = grp % share;
    float mx = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    // eight parts' loads in flight: one after another they cost a memory latency each
    for (int c0 = r.run + sub; c0 <= r.last; c0 += 8 * share) {
      float2 pml[8];
      float4 po[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = min(c0 + i * share, r.last);
        const int slot = c == r.run ? r.slot : 2 * c;
        const float* part = a.parts + static_cast<int64_t>(slot) * kFloats;
        pml[i] = *reinterpret_cast<const float2*>(part + 2 * head);
        po[i] = *reinterpret_cast<const float4*>(part + 2 * kHeads + head * D + 4 * x);
        if (c0 + i * share > r.last) pml[i] = make_float2(-INFINITY, 0.f);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float mn = fmaxf(mx, pml[i].x), ref = fmaxf(mn, -3.4e38f);
        const float co = ex2_f32(mx - ref), cn = ex2_f32(pml[i].x - ref);
        mx = mn;
        l = l * co + pml[i].y * cn;
        o = make_float4(o.x * co + po[i].x * cn, o.y * co + po[i].y * cn, o.z * co + po[i].z * cn,
                        o.w * co + po[i].w * cn);
      }
    }
    if (share > 1) {
      red[grp][x] = o;
      if (x == 0) red_ml[grp] = make_float2(mx, l);
      __syncthreads();
      if (sub == 0) {
        for (int i = 1; i < share; ++i) mx = fmaxf(mx, red_ml[grp + i].x);
        const float ref = fmaxf(mx, -3.4e38f);
        l = 0.f;
        o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < share; ++i) {
          const float c = ex2_f32(red_ml[grp + i].x - ref);
          const float4 po = red[grp + i][x];
          l += red_ml[grp + i].y * c;
          o = make_float4(o.x + po.x * c, o.y + po.y * c, o.z + po.z * c, o.w + po.w * c);
        }
      }
      __syncthreads();
    }
    if (sub == 0 && g0 + head < a.G) {
      const int64_t row = static_cast<int64_t>(r.b) * a.H + r.hg / a.chunks * a.G + g0 + head;
      const float inv = l > 0.f ? 1.f / l : 0.f;
      __nv_bfloat16* dst = a.o + row * D;
      *reinterpret_cast<__nv_bfloat162*>(dst + element_of<D>(4 * x)) =
          __floats2bfloat162_rn(o.x * inv, o.y * inv);
      *reinterpret_cast<__nv_bfloat162*>(dst + element_of<D>(4 * x + 2)) =
          __floats2bfloat162_rn(o.z * inv, o.w * inv);
      if (x == 0 && a.lse != nullptr) a.lse[row] = l > 0.f ? (mx + log2f(l)) * kLn2 : -INFINITY;
    }
  }
}

nvq_status check_decode(int B, int H, int Hkv, int D, int max_pages) {
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv != 0 || max_pages < 1 ||
      max_pages > 0x7FFFFFFF / kPage)
    return NVQ_ERR_INVALID;
  if (D != 64 && D != 128) return NVQ_ERR_UNSUPPORTED;
  if (B > 65535 || H > 65535 || static_cast<int64_t>(B) * H > 0x7FFFFFFF ||
      static_cast<int64_t>(B) * H * max_pages > int64_t{1} << 53)
    return NVQ_ERR_UNSUPPORTED;
  return NVQ_OK;
}

// CTAs and runs, query heads per run and the workspace: what goes on from each run,
// then two parts per run.
struct Plan {
  int nt, chunks, ctas, per_cta, runs, by_segment, join_x, join_y, join_threads;
  size_t parts, total;
};

Plan plan(int B, int H, int Hkv, int D, int max_pages, int window, int sinks) {
  Plan p;
  const int G = H / Hkv;
  p.nt = G > 8 ? 2 : 1;  // 8 or 16 columns: V~ is decoded once for both
  p.chunks = (G + 8 * p.nt - 1) / (8 * p.nt);
  const int64_t segments = static_cast<int64_t>(B) * Hkv * p.chunks;
  p.ctas = static_cast<int>(std::min<int64_t>(segments * max_pages, device_sms()));
  int64_t pages = max_pages;  // that a sequence may show
  if (window > 0)
    pages = std::min(pages, (int64_t{window} + kPage - 2) / kPage + 1 +
                                (int64_t{sinks} + kPage - 1) / kPage);
  // Heads of 64: four runs a CTA from six tiles a run on (64 sequences of up to 8192, 32
  // heads on 8: 46 us, 48 with three; 8 of up to 131072: 76, 85); with fewer tiles the
  // fourth only adds a part to join and a larger block to start (32 of a window of 4100, 16
  // heads on 2: 16.6, 15.7).  Heads of 128 have no registers for it.
  p.per_cta = p.nt == 2 ? 2 : D == 64 && segments * pages >= 24 * p.ctas ? 4 : 3;
  p.runs = p.ctas * p.per_cta;
  // Fewer segments than runs: entries by segment, so the join has no idle blocks.
  p.by_segment = segments <= p.runs;
  p.join_x = p.by_segment ? static_cast<int>(segments) : p.runs;
  // Segments of more than two parts, as they fall on average, get a block per query
  // head, whose thread groups share the parts (64 sequences of up to 32768 tokens, 16
  // heads on one KV head: 49 us in all, 54 with one block per segment), and one of 1024
  // threads above 64 parts (one sequence of 131072 tokens: 23 us, 28 with 256).
  p.join_y = p.runs > 2 * segments ? 8 * p.nt : 1;
  p.join_threads = p.runs > 64 * segments ? 1024 : 256;
  p.parts = (static_cast<size_t>(p.runs) * sizeof(RunInfo) + 255) / 256 * 256;
  p.total = p.parts + static_cast<size_t>(2 * p.runs) * part_floats(D, 8 * p.nt) * 4;
  return p;
}

template <int D, int NT, int kRunsPerCta>
cudaError_t launch_decode(const CUtensorMap& tk, const CUtensorMap& tk32, const DecodeArgs& a,
                          const Plan& p, cudaStream_t stream) {
  using C = Cfg<D, NT, kRunsPerCta>;
  const auto kernel = decode_kernel<D, NT, kRunsPerCta>;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  if ((e = launch_pdl(kernel, dim3(p.ctas), dim3(C::kThreads), C::kSmem, stream, 1, tk, tk32, a)) !=
      cudaSuccess)
    return e;
  const dim3 grid(p.join_x, p.join_y);
  if (p.join_threads == 1024)
    return launch_pdl(join_kernel<D, NT, 1024>, grid, dim3(1024), 0, stream, 1, a);
  return launch_pdl(join_kernel<D, NT, 256>, grid, dim3(256), 0, stream, 1, a);
}

}  // namespace

}  // namespace nvq

extern "C" {

size_t attn_qat_decode_workspace(int B, int H, int Hkv, int D, int max_pages) {
  if (nvq::check_decode(B, H, Hkv, D, max_pages) != NVQ_OK) return 0;
  return nvq::plan(B, H, Hkv, D, max_pages, 0, 0).total;  // a window needs no more
}

nvq_status attn_qat_decode(const void* q, int64_t ld_q, const void* pool, int64_t num_pages,
                           const int32_t* page_table, int64_t ld_table, int max_pages,
                           const int32_t* seq_lens, int B, int H, int Hkv, int D, float scale,
                           int window, int sinks, void* o, float* lse, void* ws, size_t ws_bytes,
                           nvq_stream_t stream) {
  using namespace nvq;
  nvq_status st = check_decode(B, H, Hkv, D, max_pages);
  if (st != NVQ_OK) return st;
  if (!(std::isfinite(scale) && scale > 0.f) || window < 0 || sinks < 0) return NVQ_ERR_INVALID;
  if (q == nullptr || o == nullptr || (reinterpret_cast<uintptr_t>(q) & 15u) != 0 ||
      (reinterpret_cast<uintptr_t>(o) & 15u) != 0 || ld_q < static_cast<int64_t>(H) * D ||
      ld_q % 8 != 0 || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0)
    return NVQ_ERR_INVALID;
  st = check_kv(pool, num_pages, page_table, ld_table, max_pages, seq_lens);
  if (st != NVQ_OK) return st;
  const Plan p = plan(B, H, Hkv, D, max_pages, window, sinks);
  if (num_pages > 0x7FFFFFFF / Hkv) return NVQ_ERR_UNSUPPORTED;  // tensor-map coordinates
  // a run counts its tiles in 31 bits
  if (static_cast<int64_t>(B) * Hkv * p.chunks * max_pages / p.runs >= 0x7FFFFFFF)
    return NVQ_ERR_UNSUPPORTED;
  if (ws == nullptr || ws_bytes < p.total || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
    return NVQ_ERR_WORKSPACE;
  // q is read by every run of its sequence, at whatever time: o elsewhere
  const int64_t row = static_cast<int64_t>(H) * D;
  if (ranges_meet(q, 2 * static_cast<uint64_t>((B - 1) * ld_q + row), o,
                  2 * static_cast<uint64_t>(row * B)))
    return NVQ_ERR_INVALID;
  int* err = device_error_word();
  if (err == nullptr) return NVQ_ERR_CUDA;
  CUtensorMap tk, tk32;
  int r;
  if ((r = make_kv_codes_map(&tk, pool, num_pages * Hkv, D, kPage)) != 0 ||
      (r = make_kv_codes_map(&tk32, pool, num_pages * Hkv, D, 32)) != 0)
    return fail_driver("cuTensorMapEncodeTiled", r);
  uint8_t* wb = static_cast<uint8_t*>(ws);
  const DecodeArgs a{static_cast<const uint16_t*>(q), ld_q, static_cast<const uint8_t*>(pool),
                     num_pages, page_table, ld_table, max_pages, seq_lens, B, H, Hkv, H / Hkv,
                     p.chunks, scale * kLog2e, window, sinks, static_cast<__nv_bfloat16*>(o), lse,
                     reinterpret_cast<RunInfo*>(wb), p.by_segment,
                     reinterpret_cast<float*>(wb + p.parts), p.runs,
                     ~uint64_t{0} / p.runs + 1, err};
  const cudaError_t e = timed(NVQ_KERNEL_DECODE, stream, [&] {
    if (D == 128)
      return p.nt == 1 ? launch_decode<128, 1, 3>(tk, tk32, a, p, stream)
                       : launch_decode<128, 2, 2>(tk, tk32, a, p, stream);
    if (p.nt == 2) return launch_decode<64, 2, 2>(tk, tk32, a, p, stream);
    return p.per_cta == 4 ? launch_decode<64, 1, 4>(tk, tk32, a, p, stream)
                          : launch_decode<64, 1, 3>(tk, tk32, a, p, stream);
  });
  return e == cudaSuccess ? NVQ_OK : fail_cuda("attn decode", e);
}

}  // extern "C"
