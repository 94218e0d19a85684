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
// keys), and every CTA takes an equal run of that line, whatever the lengths: no
// CTA waits for the longest sequence.  A run that covers all tiles of a segment
// (one sequence, KV head and group) writes o itself; a segment that crosses runs
// leaves (m, l, sum p V~) per run in the workspace, and a second small kernel
// joins them in run order, so results do not vary from run to run.
//
// One CTA: a producer warp fetches records by bulk copies into a ring of stages
// (only the rows that hold tokens) and writes each tile's description beside it;
// eight consumer warps take 16 of a tile's keys each.  The products run on the
// tensor cores with the query heads as the 8-column side (mma.sync, not tcgen05:
// the operands are decoded in registers, where the fragments are wanted, and
// tcgen05 would need them written back to shared memory as f16; at 8 columns the
// products are 1/4 of the time that the bytes allow):
//   S^T [16 keys x 8 heads] = K~ [16 x D] q~^T      K~ decoded as the A operand
//   O^T [D x 8 heads] += V~^T [D x 16 keys] P^T     V~ decoded as the A operand
// The contraction of the first runs over D in an order of its own: lane t of four
// owns D/4 consecutive elements (one 16-byte load for D = 128), its q~ fragment
// likewise.  S's accumulator becomes the second product's B operand by an 8x8
// transpose across lanes.  Codes become f16 by the hardware conversion times
// their scale, which is exact; p is rounded to f16 (as in the training forward),
// its sum is taken before the rounding, all sums are fp32.
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

constexpr int kWarps = 8;                        // consumer warps
constexpr int kThreads = (kWarps + 1) * 32;      // and the producer
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Per shape: query heads per CTA (8 NT), CTAs per SM and ring stages.
template <int D, int NT>
struct Cfg {
  static constexpr int kHeads = 8 * NT;
  static constexpr int kPerSm = NT == 1 ? 2 : 1;
  static constexpr int kStages = D == 128 ? (NT == 1 ? 4 : 6) : 6;
  static constexpr int kRow = D + 4;  // floats of a head's row in the join area
  static constexpr uint32_t kRec = record_bytes(D);
  static constexpr uint32_t kJoin = kStages * kRec;                            // float [8][heads][kRow]
  static constexpr uint32_t kMl = kJoin + kWarps * kHeads * kRow * 4;          // float2 [8][heads]
  static constexpr uint32_t kDesc = kMl + kWarps * kHeads * 8;                 // TileDesc [stages]
  static constexpr uint32_t kBars = kDesc + kStages * 32;
  static constexpr uint32_t kSmem = kBars + (2 * kStages + 2) * 8 + 16;
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
  int64_t* prefix;  // [B + 1] tiles before each sequence (workspace)
  float* parts;     // [2 gridDim.x] parts (workspace)
  int* err;
};

// Floats of one part: m (log2 units) and l per head, then the sums [heads][D].
__host__ __device__ constexpr int part_floats(int D, int heads) { return heads * (D + 2); }

// The line of `all` tiles is cut into this many runs; run c is [all c / runs,
// all (c + 1) / runs).  No run is empty.
__device__ __forceinline__ int runs_of(int64_t all, int ctas) {
  return static_cast<int>(all < ctas ? all : ctas);
}

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

// State of a consumer warp for the current segment.  Lane = 4 g + t.
template <int D, int NT>
struct State {
  uint32_t q[NT][D / 8];      // q~ of head g (of each group of 8), elements [t D/4, (t + 1) D/4)
  float o[NT][D / 16][4];     // O^T: elements d = D/8 g + 2 i (+1: [2], [3]), heads 2t, 2t + 1
  float m[NT][2], l[NT][2];   // running maximum (log2 units; all lanes) and this lane's sum
};

template <int D, int NT>
__device__ __forceinline__ void start_segment(const DecodeArgs& a, const TileDesc& td,
                                              State<D, NT>& st, int g, int t) {
  const int hk = td.hg / a.chunks, g0 = (td.hg % a.chunks) * 8 * NT;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int gi = g0 + nt * 8 + g;
    if (gi < a.G) {
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + td.b * a.ld_q + static_cast<int64_t>(hk * a.G + gi) * D + t * (D / 4));
#pragma unroll
      for (int blk = 0; blk < D / 64; ++blk) {
        const uint4 lo = __ldg(src + 2 * blk), hi = __ldg(src + 2 * blk + 1);
        const uint32_t x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        const Q16 r = quant16_unit<true>(x);
#pragma unroll
        for (int j = 0; j < 8; ++j) st.q[nt][8 * blk + j] = r.out[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < D / 8; ++j) st.q[nt][j] = 0;
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[nt][i][e] = 0.f;
    st.m[nt][0] = st.m[nt][1] = -INFINITY;
    st.l[nt][0] = st.l[nt][1] = 0.f;
  }
}

// Sixteen keys, rows r0..r0 + 15 of the record at `rec`.  Row index rho of the
// first product's A operand is key r0 + key_of(rho): neighbouring lane groups and
// the second product's lanes then hit different banks.
__device__ __forceinline__ int key_of(int rho) { return rho ^ ((rho >> 1) & 1); }

template <int D, int NT>
__device__ __forceinline__ void sixteen_keys(const DecodeArgs& a, const uint8_t* rec, int r0,
                                             const TileDesc& td, bool masked, State<D, NT>& st,
                                             int g, int t) {
  constexpr int kSteps = D / 16;  // products over D; also tiles of 16 elements of O^T
  constexpr int kRowCodes = D / 2, kRowScales = D / 16;
  float s[NT][4];
  {
    // ---- S^T: codes and scales of keys rho = g and g + 8
    uint32_t kc[2][D / 32], ks[2][D / 64];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = r0 + key_of(g) + 8 * h;
      const uint8_t* c = rec + row * kRowCodes + t * (D / 8);
      const uint8_t* sc = rec + k_scales_at(D) + row * kRowScales + t * (D / 64);
      if constexpr (D == 128) {
        const uint4 v = *reinterpret_cast<const uint4*>(c);
        kc[h][0] = v.x; kc[h][1] = v.y; kc[h][2] = v.z; kc[h][3] = v.w;
        const uint32_t two = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(sc));
        ks[h][0] = prmt(two, two, 0x1010u);
        ks[h][1] = prmt(two, two, 0x3232u);
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(c);
        kc[h][0] = v.x; kc[h][1] = v.y;
        const uint32_t one = e4m3x2_to_f16x2(*sc);
        ks[h][0] = prmt(one, one, 0x1010u);
      }
    }
    float acc[NT][2][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][p][e] = 0.f;
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {  // 8 codes of each key: two steps
      uint32_t h0[4], h1[4];
      e2m1x8_to_f16x2(kc[0][w], h0);
      e2m1x8_to_f16x2(kc[1][w], h1);
      const uint32_t s0 = ks[0][w / 2], s1 = ks[1][w / 2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint32_t af[4] = {hmul2(h0[2 * p], s0), hmul2(h1[2 * p], s1),
                                hmul2(h0[2 * p + 1], s0), hmul2(h1[2 * p + 1], s1)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma16816(acc[nt][p], af, st.q[nt][4 * w + 2 * p], st.q[nt][4 * w + 2 * p + 1]);
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = (acc[nt][0][e] + acc[nt][1][e]) * a.scale_log2;
  }
  // ---- codes and scales of V~ (keys rho = 2t, 2t + 1, 2t + 8, 2t + 9), elements [D/8 g, D/8 (g + 1))
  uint32_t vc[4][D / 64], vs[2];
  {
    uint32_t sb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = r0 + key_of(2 * t + (j & 1)) + 8 * (j >> 1);
      const uint8_t* c = rec + v_codes_at(D) + row * kRowCodes + g * (D / 16);
      if constexpr (D == 128) {
        const uint2 v = *reinterpret_cast<const uint2*>(c);
        vc[j][0] = v.x; vc[j][1] = v.y;
      } else {
        vc[j][0] = *reinterpret_cast<const uint32_t*>(c);
      }
      sb[j] = rec[v_scales_at(D) + row * kRowScales + g * (D / 8) / 16];
    }
    if (masked) {
      // rows that no visible key owns may hold anything, NaN scales among it:
      // their p is 0, their V~ made 0 too
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = td.key0 + r0 + key_of(2 * t + (j & 1)) + 8 * (j >> 1);
        if (!(key < td.len && (key >= td.wstart || key < a.sinks))) sb[j] = 0;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int key = td.key0 + r0 + key_of(g) + 8 * h;
        if (!(key < td.len && (key >= td.wstart || key < a.sinks))) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) s[nt][2 * h] = s[nt][2 * h + 1] = -INFINITY;
        }
      }
    }
    vs[0] = e4m3x2_to_f16x2(sb[0] | (sb[1] << 8));
    vs[1] = e4m3x2_to_f16x2(sb[2] | (sb[3] << 8));
  }
  // ---- running maximum and sum; p as the B operand of the second product
  uint32_t p0[NT], p1[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float mx[2] = {fmaxf(s[nt][0], s[nt][2]), fmaxf(s[nt][1], s[nt][3])};
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xFFFFFFFFu, mx[0], off));
      mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xFFFFFFFFu, mx[1], off));
    }
    const bool grows = mx[0] > st.m[nt][0] || mx[1] > st.m[nt][1];
    if (__any_sync(0xFFFFFFFFu, grows)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float mn = fmaxf(st.m[nt][h], mx[h]);
        // both -inf: nothing seen yet, the factor of 0 does not matter
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
    float p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = ex2_f32(s[nt][e] - fmaxf(st.m[nt][e & 1], -3.4e38f));
    st.l[nt][0] += p[0] + p[2];
    st.l[nt][1] += p[1] + p[3];
    p0[nt] = movmatrix_trans(pack_f16x2_rn(p[0], p[1]));
    p1[nt] = movmatrix_trans(pack_f16x2_rn(p[2], p[3]));
  }
  // ---- O^T += V~^T P^T: codes of two keys interleaved, so that one conversion
  // gives the pair (key 2t, key 2t + 1) of an element
#pragma unroll
  for (int w = 0; w < D / 64; ++w) {
    uint32_t ev[2][4], od[2][4];  // even and odd elements of the 4 bytes, keys (0, 1) and (2, 3)
#pragma unroll
    for (int pr = 0; pr < 2; ++pr) {
      const uint32_t x = vc[2 * pr][w], y = vc[2 * pr + 1][w];
      e2m1x8_to_f16x2((x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u), ev[pr]);
      e2m1x8_to_f16x2(((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), od[pr]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t af[4] = {hmul2(ev[0][i], vs[0]), hmul2(od[0][i], vs[0]),
                              hmul2(ev[1][i], vs[1]), hmul2(od[1][i], vs[1])};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma16816(st.o[nt][4 * w + i], af, p0[nt], p1[nt]);
    }
  }
  static_assert(kSteps == 4 * (D / 64), "tiles of O^T");
}

// Element of O at position `pos` of a stored row: the rows keep the order in which
// the lanes hold them, pos = 16 i + 2 g + e for d = D/8 g + 2 i + e.
template <int D>
__device__ __forceinline__ int element_of(int pos) {
  return (pos >> 1 & 7) * (D / 8) + (pos >> 4) * 2 + (pos & 1);
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT>::kPerSm) decode_kernel(const DecodeArgs a) {
  using C = Cfg<D, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  float* join = reinterpret_cast<float*>(smem + C::kJoin);
  float2* ml = reinterpret_cast<float2*>(smem + C::kMl);
  TileDesc* desc = reinterpret_cast<TileDesc*>(smem + C::kDesc);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBars);
  uint64_t* empty = full + C::kStages;
  uint64_t* meet = empty + C::kStages;  // [2]: parts written, parts read
  volatile int* abort = reinterpret_cast<volatile int*>(meet + 2);
  __shared__ int64_t warp_sum[kWarps + 1];
  __shared__ int64_t start_before;
  __shared__ int start_b;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    *abort = 0;
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kWarps);
    }
    mbar_init(&meet[0], kWarps);
    mbar_init(&meet[1], kWarps);
    fence_mbar_init();
  }
  // ---- this CTA's run of the line of tiles: a scan over the sequences
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
  if (lane == 31) warp_sum[warp] = scan;
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w <= kWarps; ++w) {
    if (w < warp) scan += warp_sum[w];
    total += warp_sum[w];
  }
  int64_t before = scan - mine;  // tiles (of one head group) before this thread's sequences
  const int64_t all = total * hgs;
  const int runs = runs_of(all, static_cast<int>(gridDim.x)), run = static_cast<int>(blockIdx.x);
  const int64_t u0 = run < runs ? all * run / runs : all;
  const int64_t u1 = run < runs ? all * (run + 1) / runs : all;
  if (blockIdx.x == 0) {
    int64_t at = before;
    for (int b = b_lo; b < b_hi; ++b) {
      bool over;
      a.prefix[b] = at;
      at += extent(a, b, &over).tiles;
    }
    if (threadIdx.x == 0) a.prefix[a.B] = total;
  }
  if (u0 < u1 && before * hgs <= u0 && u0 < (before + mine) * hgs) {
    int b = b_lo;
    for (;; ++b) {
      bool over;
      const int n = extent(a, b, &over).tiles;
      if (u0 < (before + n) * hgs) break;
      before += n;
    }
    start_b = b;
    start_before = before;
  }
  __syncthreads();
  if (u0 >= u1) return;
  const int n_tiles = static_cast<int>(u1 - u0);

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer
    int b = start_b;
    bool over;
    Extent e = extent(a, b, &over);
    int64_t seg0 = start_before * hgs;  // line position of the sequence's first tile
    int hg = static_cast<int>((u0 - seg0) / e.tiles);
    int i = static_cast<int>((u0 - seg0) - static_cast<int64_t>(hg) * e.tiles);
    int pages = 0, pages_at = -1;  // this lane's page number of the 32 tiles from pages_at
    bool ok = true;
    int issued = 0;
    for (int n = 0; n < n_tiles; ++n) {
      const int s = n % C::kStages;
      if (!(ok = mbar_wait_warp(&empty[s], ((n / C::kStages) & 1) ^ 1, abort))) break;
      if (pages_at < 0 || i >= pages_at + 32 || i < pages_at) {
        const int j = i + lane;
        const int p = j < e.sink_pages ? j : e.first + j - e.sink_pages;
        pages = j < e.tiles ? a.table[b * a.ld_table + p] : -1;
        pages_at = i;
      }
      const int page = __shfl_sync(0xFFFFFFFFu, pages, i - pages_at);
      const int p = i < e.sink_pages ? i : e.first + i - e.sink_pages;
      const int64_t first = seg0 + static_cast<int64_t>(hg) * e.tiles;
      TileDesc td;
      td.key0 = p * kPage;
      td.len = e.len;
      td.wstart = e.wstart;
      td.b = b;
      td.hg = hg;
      td.rows = min(kPage, e.len - td.key0);
      td.flags = 0;
      if (n == 0 || i == 0) td.flags |= kStart;
      if (n == n_tiles - 1 || i == e.tiles - 1) td.flags |= kEnd;
      if (td.rows < kPage || (td.key0 < e.wstart && td.key0 + kPage > a.sinks)) td.flags |= kMasked;
      // whole segments are written directly; a part that begins with the run goes
      // to the run's slot 0, one that begins inside it to slot 1
      const bool whole = first >= u0 && first + e.tiles <= u1;
      td.slot = whole ? -1 : 2 * run + (first > u0 ? 1 : 0);
      const bool there = page >= 0 && page < a.num_pages;
      if (!there) {
        td.flags |= kAbsent;
        if (lane == 0) atomicMax(a.err, kErrTable);
      }
      if (lane == 0) desc[s] = td;
      __syncwarp();
      uint8_t* dst = smem + s * C::kRec;
      const uint8_t* src =
          a.pool + (static_cast<int64_t>(page) * a.Hkv + hg / a.chunks) * record_bytes(D);
      if (!there) {
        mbar_arrive_expect_tx_w(&full[s], 0);
      } else if (td.rows == kPage) {
        mbar_arrive_expect_tx_w(&full[s], C::kRec);
        bulk_load_w(dst, src, C::kRec, &full[s]);
      } else {
        const uint32_t rows = (td.rows + 3) & ~3;  // whole 16-byte units of scales
        const uint32_t cb = rows * (D / 2), sb = rows * (D / 16);
        mbar_arrive_expect_tx_w(&full[s], 2 * (cb + sb));
        bulk_load_w(dst, src, cb, &full[s]);
        bulk_load_w(dst + v_codes_at(D), src + v_codes_at(D), cb, &full[s]);
        bulk_load_w(dst + k_scales_at(D), src + k_scales_at(D), sb, &full[s]);
        bulk_load_w(dst + v_scales_at(D), src + v_scales_at(D), sb, &full[s]);
      }
      issued = n + 1;
      if (++i == e.tiles && n + 1 < n_tiles) {
        i = 0;
        pages_at = -1;
        if (++hg == hgs) {
          hg = 0;
          seg0 += static_cast<int64_t>(e.tiles) * hgs;
          do {
            e = extent(a, ++b, &over);
          } while (e.tiles == 0);
        }
      }
    }
    if (!ok) {  // let the copies already issued land before the block leaves
      for (int n = max(0, issued - C::kStages); n < issued; ++n)
        mbar_wait_warp(&full[n % C::kStages], (n / C::kStages) & 1, nullptr, 10000000ull);
    }
  } else {
    // ----------------------------------------------------------- consumers
    const int g = lane >> 2, t = lane & 3;
    State<D, NT> st;
    uint32_t meets = 0;
    for (int n = 0; n < n_tiles; ++n) {
      const int s = n % C::kStages;
      if (!mbar_wait_warp(&full[s], (n / C::kStages) & 1, abort)) break;
      const TileDesc td = desc[s];
      if (td.flags & kStart) start_segment<D, NT>(a, td, st, g, t);
      if (!(td.flags & kAbsent) && warp * 16 < td.rows)
        sixteen_keys<D, NT>(a, smem + s * C::kRec, warp * 16, td, td.flags & kMasked, st, g, t);
      mbar_arrive_warp(&empty[s]);
      if (!(td.flags & kEnd)) continue;
      // ---- the warps' parts meet in shared memory
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float l = st.l[nt][h];
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, off);
          const int head = nt * 8 + 2 * t + h;
          if (g == 0) ml[warp * C::kHeads + head] = make_float2(st.m[nt][h], l);
          float* row = join + (warp * C::kHeads + head) * C::kRow + 2 * g;
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
            *reinterpret_cast<float2*>(row + 16 * i) =
                make_float2(st.o[nt][i][h], st.o[nt][i][2 + h]);
        }
      }
      mbar_arrive_warp(&meet[0]);
      if (!mbar_wait_warp(&meet[0], meets & 1, abort)) break;
      const int hk = td.hg / a.chunks, g0 = (td.hg % a.chunks) * C::kHeads;
      const int heads = min(C::kHeads, a.G - g0);
      for (int x = threadIdx.x; x < heads * (D / 2); x += kWarps * 32) {
        const int head = x / (D / 2), pos = 2 * (x % (D / 2));
        float mx = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, ml[w * C::kHeads + head].x);
        const float ref = fmaxf(mx, -3.4e38f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 v = ml[w * C::kHeads + head];
          const float c = ex2_f32(v.x - ref);
          const float2 ov = *reinterpret_cast<const float2*>(
              join + (w * C::kHeads + head) * C::kRow + pos);
          l = fmaf(v.y, c, l);
          o0 = fmaf(ov.x, c, o0);
          o1 = fmaf(ov.y, c, o1);
        }
        if (td.slot < 0) {
          const int64_t row = static_cast<int64_t>(td.b) * a.H + hk * a.G + g0 + head;
          const float inv = l > 0.f ? 1.f / l : 0.f;
          *reinterpret_cast<__nv_bfloat162*>(a.o + row * D + element_of<D>(pos)) =
              __floats2bfloat162_rn(o0 * inv, o1 * inv);
          if (pos == 0 && a.lse != nullptr)
            a.lse[row] = l > 0.f ? (mx + log2f(l)) * kLn2 : -INFINITY;
        } else {
          float* part = a.parts + static_cast<int64_t>(td.slot) * part_floats(D, C::kHeads);
          if (pos == 0) {
            part[2 * head] = mx;
            part[2 * head + 1] = l;
          }
          *reinterpret_cast<float2*>(part + 2 * C::kHeads + head * D + pos) = make_float2(o0, o1);
        }
      }
      mbar_arrive_warp(&meet[1]);
      if (!mbar_wait_warp(&meet[1], meets & 1, abort)) break;
      ++meets;
    }
  }
  __syncthreads();
  report_abort(abort, a.err);
}

// Joins the parts of one sequence and query head, in run order; writes the empty
// rows.  Thread x of the first D takes the stored position x; groups of D threads
// take every kGroups-th part.
template <int D, int NT>
__global__ void __launch_bounds__(256) join_kernel(const DecodeArgs a, int ctas) {
  constexpr int kHeads = 8 * NT, kGroups = 256 / D, kFloats = part_floats(D, kHeads);
  __shared__ float red[kGroups][D + 2];
  const int b = blockIdx.x / a.H, h = blockIdx.x % a.H;
  const int hk = h / a.G, gi = h % a.G, head = gi % kHeads;
  const int hgs = a.Hkv * a.chunks, hg = hk * a.chunks + gi / kHeads;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t p0 = a.prefix[b], tiles = a.prefix[b + 1] - p0, all = a.prefix[a.B] * hgs;
  const int64_t row = static_cast<int64_t>(b) * a.H + h;
  if (tiles == 0) {
    if (threadIdx.x < D) a.o[row * D + threadIdx.x] = __float2bfloat16_rn(0.f);
    if (threadIdx.x == 0 && a.lse != nullptr) a.lse[row] = -INFINITY;
    return;
  }
  const int runs = runs_of(all, ctas);
  const int64_t s0 = p0 * hgs + hg * tiles, s1 = s0 + tiles;
  // the run that holds tile u
  auto run_of = [&](int64_t u) { return static_cast<int>(((u + 1) * runs + all - 1) / all - 1); };
  const int c0 = run_of(s0), c1 = run_of(s1 - 1);
  if (c0 == c1) return;  // written by its run
  const int x = threadIdx.x % D, grp = threadIdx.x / D;
  float mx = -INFINITY, l = 0.f, o = 0.f;
  for (int c = c0 + grp; c <= c1; c += kGroups) {
    const int slot = 2 * c + (c == c0 && all * c / runs < s0 ? 1 : 0);
    const float* part = a.parts + static_cast<int64_t>(slot) * kFloats;
    const float pm = part[2 * head], pl = part[2 * head + 1];
    const float po = part[2 * kHeads + head * D + x];
    const float mn = fmaxf(mx, pm), ref = fmaxf(mn, -3.4e38f);
    const float c_old = ex2_f32(mx - ref), c_new = ex2_f32(pm - ref);
    mx = mn;
    l = l * c_old + pl * c_new;
    o = o * c_old + po * c_new;
  }
  red[grp][x] = o;
  if (x == 0) {
    red[grp][D] = mx;
    red[grp][D + 1] = l;
  }
  __syncthreads();
  if (grp != 0) return;
  mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) mx = fmaxf(mx, red[i][D]);
  const float ref = fmaxf(mx, -3.4e38f);
  l = 0.f;
  o = 0.f;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const float c = ex2_f32(red[i][D] - ref);
    l += red[i][D + 1] * c;
    o += red[i][x] * c;
  }
  a.o[row * D + element_of<D>(x)] = __float2bfloat16_rn(l > 0.f ? o / l : 0.f);
  if (x == 0 && a.lse != nullptr) a.lse[row] = l > 0.f ? (mx + log2f(l)) * kLn2 : -INFINITY;
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return 152;
  return sms;
}

nvq_status check_decode(int B, int H, int Hkv, int D, int max_pages) {
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv != 0 || max_pages < 1 ||
      max_pages > 0x7FFFFFFF / kPage)
    return NVQ_ERR_INVALID;
  if (D != 64 && D != 128) return NVQ_ERR_UNSUPPORTED;
  if (B > 65535 || H > 65535 || static_cast<int64_t>(B) * H > 0x7FFFFFFF) return NVQ_ERR_UNSUPPORTED;
  return NVQ_OK;
}

// Runs (CTAs), query heads per CTA and the workspace: the prefix, then two parts
// per run.
struct Plan {
  int nt, chunks, runs;
  size_t parts, total;
};

Plan plan(int B, int H, int Hkv, int D, int max_pages) {
  Plan p;
  const int G = H / Hkv;
  p.nt = G > 8 ? 2 : 1;  // 8 or 16 columns: K~ and V~ are decoded once for both
  p.chunks = (G + 8 * p.nt - 1) / (8 * p.nt);
  const int64_t most = static_cast<int64_t>(B) * Hkv * p.chunks * max_pages;
  p.runs = static_cast<int>(std::min<int64_t>(most, sm_count() * (p.nt == 1 ? 2 : 1)));
  p.parts = (static_cast<size_t>(B + 1) * 8 + 255) / 256 * 256;
  p.total = p.parts + static_cast<size_t>(2 * p.runs) * part_floats(D, 8 * p.nt) * 4;
  return p;
}

template <int D, int NT>
cudaError_t launch_decode(const DecodeArgs& a, int runs, cudaStream_t stream) {
  using C = Cfg<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(decode_kernel<D, NT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  decode_kernel<D, NT><<<runs, kThreads, C::kSmem, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // the join's blocks come up while the last runs finish
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B * a.H));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<D, NT>, a, runs);
}

}  // namespace

}  // namespace nvq

extern "C" {

size_t attn_qat_decode_workspace(int B, int H, int Hkv, int D, int max_pages) {
  if (nvq::check_decode(B, H, Hkv, D, max_pages) != NVQ_OK) return 0;
  return nvq::plan(B, H, Hkv, D, max_pages).total;
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
  const Plan p = plan(B, H, Hkv, D, max_pages);
  if (ws == nullptr || ws_bytes < p.total || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
    return NVQ_ERR_WORKSPACE;
  int* err = device_error_word();
  if (err == nullptr) return NVQ_ERR_CUDA;
  uint8_t* wb = static_cast<uint8_t*>(ws);
  const DecodeArgs a{static_cast<const uint16_t*>(q), ld_q, static_cast<const uint8_t*>(pool),
                     num_pages, page_table, ld_table, max_pages, seq_lens, B, H, Hkv, H / Hkv,
                     p.chunks, scale * kLog2e, window, sinks, static_cast<__nv_bfloat16*>(o), lse,
                     reinterpret_cast<int64_t*>(wb), reinterpret_cast<float*>(wb + p.parts), err};
  const cudaError_t e = timed(NVQ_KERNEL_ATTN_FWD, stream, [&] {
    if (D == 128)
      return p.nt == 1 ? launch_decode<128, 1>(a, p.runs, stream)
                       : launch_decode<128, 2>(a, p.runs, stream);
    return p.nt == 1 ? launch_decode<64, 1>(a, p.runs, stream)
                     : launch_decode<64, 2>(a, p.runs, stream);
  });
  return e == cudaSuccess ? NVQ_OK : fail_cuda("attn decode", e);
}

}  // extern "C"
