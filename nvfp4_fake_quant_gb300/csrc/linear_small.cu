// The packed NVFP4 linear of a few rows (a decode step's tokens):
//   out[m, n] = alpha sum_k x~[m, k] w~[n, k] + bias[n],  M <= 64.
//
// Bound.  Every weight is read once, 9/16 byte each (codes and scales): the call is
// a stream of w through the chip.  The weights are the 128-row side of the
// block-scaled FP4 MMAs (tcgen05 kind::mxf4nvf4) and are never decoded; the rows of
// x are the narrow side (M rounded up to 16 columns).
//
// Work split.  Units are (128-row tile of w, 256-element stage of K).
//   Up to one tile per SM: 1 to 8 CTAs share a tile, each a range of K, as one cluster;
//   they leave their sums in the first one's shared memory, which adds them in order.
//   (Through the workspace, as below, the same sum costs 2 us more: 7.8 against 5.9 us
//   for 1 x 4608 x 1536.)
//   More tiles: the line of units is cut into equal runs, one CTA each, so that every
//   SM streams the same bytes.  A tile that crosses runs leaves fp32 parts in the
//   workspace; whichever warp arrives last at the tile's ticket adds the parts in run
//   order (the sum does not depend on who that is).
//
// Measured (calls in a CUDA graph): 53248 x 16384 82 us for one row, 88% of the copy
// rate, 87 for 64; 28672 x 8192 27 us for 1 to 32 rows, 73%; one row of 1536 x 8960 6.8
// us and of 4608 x 1536 5.2, the latency of a launch, of the first loads and of the
// cluster's sum.  Addresses count here: 64-bit products for the outputs' rows cost 28672
// x 8192 2 us at 64 rows, 65536 x 1024 4.
//
// Launches.  With few blocks of x per CTA the clusters quantize x themselves, each CTA
// its range of K, while the first weights arrive.  Else there are two: x is quantized
// (and the tickets cleared) by a small kernel, while the main kernel, launched behind
// it programmatically, already fills its ring with weights, which do not depend on x.
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "nvq_internal.h"
#include "nvq_ptx.cuh"
#include "nvq_quant.cuh"

namespace nvq {

namespace {

constexpr int kThreads = 192;  // producer, MMA, 4 epilogue warps
constexpr int kSteps = 4;      // MMA steps (64 elements) per stage
constexpr int kFusedBlocks = 4;  // of x per thread, at most, where the kernel quantizes x itself
constexpr int kStages = 6;     // of the ring (8: 1 us slower at 32 x 28672 x 8192)
// bytes of a stage: w codes, w scales, x scales
constexpr uint32_t kW = 128 * 128, kSc = kSteps * 512, kXs = 1024;
constexpr uint32_t kScCol = 128;  // tensor memory: two accumulators of 64 columns, then scales
static_assert(kScCol + 32 * kStages <= 512 && kScCol + 32 * 4 <= 256, "tensor memory");

struct SmallArgs {
  int M, N, cols, stages;   // cols: M rounded up to 16; stages of the ring
  int tiles, k_stages, k_steps;
  int runs, per_run, rest;  // runs, units / runs, units % runs
  int split;                // CTAs per tile (clusters)
  uint32_t sums_at;         // of their sums in the first one's shared memory
  const uint16_t* x;        // x itself (kFused)
  int64_t ld_x;
  const uint8_t* sx;        // x scales (stage blocks), w scales (tiled layout)
  const uint8_t* sw;
  const float* gx;          // device scalars; gw nullptr: 1
  const float* gw;
  const __nv_bfloat16* bias;
  __nv_bfloat16* out;
  unsigned int* tickets;    // [4 tiles], zero at the start
  float* parts;             // [2 runs][cols][128]
  int* err;
};

// One 16-element block of x, quantized.
__device__ __forceinline__ Q16 quant_block(const uint4& lo, const uint4& hi, float g) {
  const uint32_t v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  Q16 q = quant16_static_fast<false>(v, g, __frcp_rn(g));
  code_signs(v, q.codes);
  return q;
}

// Where the scale of x's block (row r, K block cb) lies.  The scales of a stage (4 MMA
// steps) are two blocks of 512 bytes: row r % 32 of block i holds 4 words (of 4 scales),
// those of (step 2 i, r / 32 = 0), (2 i, 1), (2 i + 1, 0), (2 i + 1, 1).  One copy of a
// block then brings the scales of two steps to 4 columns of tensor memory, where the
// tiled layout, made for 128 rows, takes a copy per step.  The scales of rows M and up
// are not written: the products of those rows are never stored.
__device__ __forceinline__ int x_scale_at(int r, int cb) {
  const int step = cb >> 2, w = (step & 1) * 2 + (r >> 5);
  return (step >> 1) * 512 + (r & 31) * 16 + w * 4 + (cb & 3);
}

// x [M, K] to codes and scales, one 16-element block per thread; clears the tickets.
__global__ void __launch_bounds__(128) quant_rows_kernel(const uint16_t* __restrict__ x, int64_t ld,
                                                         int M, int nbc,
                                                         const float* __restrict__ gsf,
                                                         uint8_t* __restrict__ codes,
                                                         uint8_t* __restrict__ scales,
                                                         unsigned int* __restrict__ tickets,
                                                         int n_tickets) {
  // the kernels before this one are done when the next one starts: it may read w early
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x * 128 + threadIdx.x;
  if (i < n_tickets) tickets[i] = 0;
  if (i >= M * nbc) return;
  const int r = i / nbc, cb = i - r * nbc;
  const float g = *gsf;
  const uint4* src = reinterpret_cast<const uint4*>(x + r * ld + static_cast<int64_t>(cb) * 16);
  const uint4 lo = __ldg(src), hi = __ldg(src + 1);
  const Q16 q = quant_block(lo, hi, g);
  *reinterpret_cast<uint2*>(codes + static_cast<int64_t>(i) * 8) =
      make_uint2(q.codes[0], q.codes[1]);
  scales[x_scale_at(r, cb)] = static_cast<uint8_t>(q.sbyte);
}

// Run c covers units [units c / runs, units (c + 1) / runs) of the line.
__device__ __forceinline__ int run_begin(const SmallArgs& p, int c) {
  return p.per_run * c + p.rest * c / p.runs;
}
// The run that holds unit u: the last c with units c / runs <= u.
__device__ __forceinline__ int run_of(const SmallArgs& p, int u) {
  const int64_t units = static_cast<int64_t>(p.tiles) * p.k_stages;
  return static_cast<int>((static_cast<int64_t>(u + 1) * p.runs + units - 1) / units - 1);
}

// Place of a unit in the line (tile, stage of K) and in the ring (stage, parity).
struct Place {
  int tile, ks, s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ Place(const SmallArgs& p, int u)
      : tile(u / p.k_stages), ks(u - tile * p.k_stages) {}
  __device__ __forceinline__ void next(const SmallArgs& p) {
    if (++ks == p.k_stages) {
      ks = 0;
      ++tile;
    }
    if (++s == p.stages) {
      s = 0;
      phase ^= 1;
    }
  }
};

// One whole stage from one elected lane: the copies of its scales, four MMAs, the
// commit.  wd, xd: descriptors of the scale blocks; a, b: of the codes; w_col, x_col:
// tensor memory columns of the scales (4 a step; 2 a step).
__device__ __forceinline__ void issue_stage(uint32_t d, uint32_t idesc, uint32_t acc, uint64_t a,
                                            uint64_t b, uint64_t wd, uint64_t xd, uint32_t w_col,
                                            uint32_t x_col, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred p, e, t;\n\t"
      "setp.ne.b32 p, %2, 0;\n\t"
      "setp.eq.u32 t, 0, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%11], %3;\n\t"
      "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%15], %7;\n\t"
      "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%17], %8;\n\t"
      "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%12], %4;\n\t"
      "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%13], %5;\n\t"
      "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%14], %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %9, %10, %1, "
      "[%11], [%15], p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %19, %20, %1, "
      "[%12], [%16], t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %21, %22, %1, "
      "[%13], [%17], t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %24, %25, %1, "
      "[%14], [%18], t;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%23];\n\t}" ::"r"(d),
      "r"(idesc), "r"(acc), "l"(wd), "l"(wd + 32), "l"(wd + 64), "l"(wd + 96), "l"(xd),
      "l"(xd + 32), "l"(a), "l"(b), "r"(w_col), "r"(w_col + 4), "r"(w_col + 8), "r"(w_col + 12),
      "r"(x_col), "r"(x_col + 2), "r"(x_col + 4), "r"(x_col + 6), "l"(a + 2), "l"(b + 2),
      "l"(a + 4), "l"(b + 4), "r"(smem_u32(bar)), "l"(a + 6), "l"(b + 6)
      : "memory");
}

// Wait on a barrier that other CTAs of the cluster arrive on, whose writes into this
// CTA's shared memory are then visible.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, volatile int* abort) {
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], 0;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar))
        : "memory");
    if (__all_sync(0xFFFFFFFFu, ok != 0)) return true;
    const bool late = globaltimer_ns() - t0 > NVQ_WAIT_LIMIT_NS;
    if (late) *abort = 1;
    if (__any_sync(0xFFFFFFFFu, late || *abort)) return false;
  }
}

// Address in shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}

// kClusters: one tile per cluster of p.split CTAs; else runs.  kFused (clusters only): the
// epilogue's warps quantize the CTA's part of x into shared memory first.
template <bool kClusters, bool kFused>
__global__ void __launch_bounds__(kThreads)
    linear_small_kernel(const __grid_constant__ CUtensorMap tx,
                        const __grid_constant__ CUtensorMap tw, const SmallArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023u) &
                                             ~static_cast<uintptr_t>(1023u));
  __shared__ uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2];
  __shared__ uint64_t sums_full, x_full;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  volatile int* abort = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t x_bytes = static_cast<uint32_t>(p.cols) * 128;
  // a stage: w codes, x codes, w scales, x scales; fused: without x, whose stages follow
  // the ring (all codes, then all scales)
  const uint32_t sx_at = kW + (kFused ? 0u : x_bytes);
  const uint32_t stage_bytes = (sx_at + kSc + (kFused ? 0u : kXs) + 1023) & ~1023u;
  constexpr uint32_t kAlloc = kClusters ? 256 : 512;
  pdl_trigger();
  if (threadIdx.x == 0) {
    *abort = 0;
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
    }
    if (kClusters) mbar_init(&sums_full, max(4 * (p.split - 1), 1));
    if (kFused) mbar_init(&x_full, 4);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, kAlloc);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  if (kClusters && p.split > 1) cluster_arrive();  // waited for before the first remote write
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  int u0, u1;
  if constexpr (kClusters) {
    const int tile = blockIdx.x / p.split, rank = blockIdx.x - tile * p.split;
    u0 = tile * p.k_stages + p.k_stages * rank / p.split;
    u1 = tile * p.k_stages + p.k_stages * (rank + 1) / p.split;
  } else {
    u0 = run_begin(p, blockIdx.x);
    u1 = run_begin(p, blockIdx.x + 1);
  }
  const int count = u1 - u0;
  uint8_t* xc = smem + p.stages * stage_bytes;  // fused: x codes and scales of the CTA's part
  uint8_t* xs = xc + count * x_bytes;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    tma_prefetch_desc(&tx);
    tma_prefetch_desc(&tw);
    // Places are counted on, not divided out: a warp alone waits 0.2 us for a division
    // on its own, and five in a stage held the loads back (1 x 14336 x 16384: 37 us, 29
    // without them).
    auto load_w = [&](const Place& at) {
      const int ns = min(kSteps, p.k_steps - at.ks * kSteps);
      uint8_t* st = smem + at.s * stage_bytes;
      mbar_arrive_expect_tx_w(&full[at.s],
                              sx_at + (kFused ? 0u : kXs) + static_cast<uint32_t>(ns) * 512u);
      tma_load_4d_w(st, &tw, at.ks * 128, at.tile * 128, 0, 0, &full[at.s]);
      bulk_load_w(st + sx_at,
                  p.sw + (static_cast<int64_t>(at.tile) * p.k_steps + at.ks * kSteps) * 512,
                  ns * 512, &full[at.s]);
    };
    auto load_x = [&](const Place& at) {
      uint8_t* st = smem + at.s * stage_bytes;
      tma_load_4d_w(st + kW, &tx, at.ks * 128, 0, 0, 0, &full[at.s]);
      bulk_load_w(st + sx_at + kSc, p.sx + static_cast<int64_t>(at.ks) * kXs, kXs,
                  &full[at.s]);
    };
    const int head = min(count, p.stages);
    Place at(p, u0), at_x(p, u0);
    if (kFused) pdl_wait();  // no kernel of this call stands between w's writer and this one
    for (int i = 0; i < head; ++i, at.next(p)) load_w(at);
    if (!kFused) {
      pdl_wait();  // x~
      for (int i = 0; i < head; ++i, at_x.next(p)) load_x(at_x);
    }
    int i = head;
    bool ok = true;
    for (; i < count; ++i, at.next(p)) {
      if (!(ok = mbar_wait_warp(&empty[at.s], at.phase ^ 1, abort))) break;
      load_w(at);
      if (!kFused) load_x(at);
    }
    if (!ok) {  // let the copies already issued land before the block leaves
      for (int k = max(0, i - p.stages); k < i; ++k)
        mbar_wait_warp(&full[k % p.stages], (k / p.stages) & 1, nullptr, 10000000ull);
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    const uint32_t idesc = idesc_mxf4nvf4(128, 0) | (static_cast<uint32_t>(p.cols >> 3) << 17);
    int part = 0, i = 0;
    Place at(p, u0);
    const bool x_there = !kFused || mbar_wait_warp(&x_full, 0, abort);
    for (; i < count && x_there; ++i, at.next(p)) {
      const int s = at.s, ks = at.ks;
      const int ns = min(kSteps, p.k_steps - ks * kSteps);
      const bool first = i == 0 || ks == 0;
      const uint32_t d = tmem + 64 * (part & 1);
      if (first && !mbar_wait_warp(&acc_empty[part & 1], ((part >> 1) & 1) ^ 1, abort)) break;
      if (!mbar_wait_warp(&full[s], at.phase, abort)) break;
      tc_fence_after();
      const uint32_t a = smem_u32(smem + s * stage_bytes), sa = a + sx_at;
      const uint32_t b = kFused ? smem_u32(xc + i * x_bytes) : a + kW;
      const uint32_t sb = kFused ? smem_u32(xs + i * kXs) : sa + kSc;
      const uint32_t col = tmem + kScCol + 32 * s;
      const uint64_t ad = sdesc_sw128(a, 16, 1024), bd = sdesc_sw128(b, 16, 1024);
      const uint64_t wd = sdesc(sa, 128, 128, 0), xd = sdesc(sb, 128, 128, 0);
      if (ns == kSteps) {
        issue_stage(d, idesc, first ? 0u : 1u, ad, bd, wd, xd, col, col + 16, &empty[s]);
      } else {  // the last stage of a K that is no multiple of 256
        for (int w = 0; w < 2; ++w) tmem_cp_32x128_x4_w(col + 16 + 4 * w, sb + 512 * w);
        for (int j = 0; j < ns; ++j) {
          tmem_cp_32x128_x4_w(col + 4 * j, sa + 512 * j);
          umma_fp4_ss_w(d, ad + 2 * j, bd + 2 * j, idesc, col + 4 * j, col + 16 + 2 * j,
                        (!first || j > 0) ? 1u : 0u);
        }
        umma_commit_w(&empty[s]);
      }
      if (ks == p.k_stages - 1 || i == count - 1) {
        umma_commit_w(&acc_full[part & 1]);
        ++part;
      }
    }
    // the MMAs in flight end before the block does
    for (int k = max(0, i - p.stages); k < i; ++k)
      mbar_wait_warp(&empty[k % p.stages], (k / p.stages) & 1, nullptr, 10000000ull);
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, row = quarter * 32 + lane;
    pdl_wait();
    if constexpr (kFused) {
      // the CTA's part of x: codes in the swizzled rows of the B operand
      const int tile = blockIdx.x / p.split, ks0 = u0 - tile * p.k_stages;
      const int nb = min(16 * count, 4 * p.k_steps - 16 * ks0), all = p.M * nb;
      const uint16_t* x = p.x + 256 * static_cast<int64_t>(ks0);
      const float g = *p.gx;
      auto source = [&](int i, int& r, int& cb) {
        r = i / nb;
        cb = i - r * nb;
        return reinterpret_cast<const uint4*>(x + r * p.ld_x + cb * 16);
      };
      for (int i0 = threadIdx.x - 64; i0 < all; i0 += 128 * kFusedBlocks) {
        uint4 lo[kFusedBlocks], hi[kFusedBlocks];
        int r[kFusedBlocks], cb[kFusedBlocks];
#pragma unroll
        for (int j = 0; j < kFusedBlocks; ++j) {
          if (i0 + 128 * j >= all) break;
          const uint4* src = source(i0 + 128 * j, r[j], cb[j]);
          lo[j] = __ldg(src);
          hi[j] = __ldg(src + 1);
        }
#pragma unroll
        for (int j = 0; j < kFusedBlocks; ++j) {
          if (i0 + 128 * j >= all) break;
          const Q16 q = quant_block(lo[j], hi[j], g);
          const int c = cb[j] & 15;  // of its stage: 16-byte units c / 2, swizzled by the row
          uint8_t* row = xc + (cb[j] >> 4) * x_bytes + r[j] * 128;
          *reinterpret_cast<uint2*>(row + (((c >> 1) ^ (r[j] & 7)) << 4) + (c & 1) * 8) =
              make_uint2(q.codes[0], q.codes[1]);
          xs[x_scale_at(r[j], cb[j])] = static_cast<uint8_t>(q.sbyte);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive_warp(&x_full);
    }
    const float alpha = 1.0f / (*p.gx * (p.gw != nullptr ? *p.gw : 1.0f));
    if constexpr (kClusters) {
      const int tile = blockIdx.x / p.split, rank = blockIdx.x - tile * p.split;
      const int n = tile * 128 + row;
      const float bias = p.bias != nullptr && n < p.N ? __bfloat162float(p.bias[n]) : 0.f;
      float* sums = reinterpret_cast<float*>(smem + p.sums_at);  // [split - 1][cols][128]
      if (p.split > 1) cluster_wait();
      const uint32_t acc = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
      bool ok = mbar_wait_warp(&acc_full[0], 0, abort);
      tc_fence_after();
      if (rank > 0) {
        const uint32_t to = map_rank(sums + (rank - 1) * p.cols * 128 + row, 0);
        for (int c = 0; c < p.M && ok; c += 16) {
          uint32_t v[16];
          tmem_ld16(acc + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(to + (c + j) * 512), "r"(v[j])
                         : "memory");
        }
        __syncwarp();
        if (lane == 0)
          asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                           map_rank(&sums_full, 0))
                       : "memory");
      } else {
        if (ok && p.split > 1) ok = mbar_wait_cluster(&sums_full, abort);
        for (int c = 0; c < p.M && ok; c += 16) {
          uint32_t v[16];
          tmem_ld16(acc + c, v);
          tmem_wait_ld();
          float f[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) f[j] = __uint_as_float(v[j]);
          const float* theirs = sums + c * 128 + row;
          for (int r = 0; r < p.split - 1; ++r, theirs += p.cols * 128)
#pragma unroll
            for (int j = 0; j < 16; ++j) f[j] += theirs[j * 128];
          __nv_bfloat16* o = p.out + static_cast<int64_t>(c) * p.N + n;
#pragma unroll
          for (int j = 0; j < 16; ++j, o += p.N)
            if (c + j < p.M && n < p.N) *o = __float2bfloat16_rn(fmaf(alpha, f[j], bias));
        }
      }
    } else {
      int part = 0;
      for (int u = u0; u < u1; ++part) {
        const int tile = u / p.k_stages, t0 = tile * p.k_stages;
        const int from = u;
        u = min(u1, t0 + p.k_stages);
        const int n = tile * 128 + row;
        const bool whole = from == t0 && u == t0 + p.k_stages;
        const float bias = p.bias != nullptr && n < p.N ? __bfloat162float(p.bias[n]) : 0.f;
        // the tile's parts are those of runs c0 .. c1; slot 0 of a run: the part that
        // begins with it; slot 1: one that begins inside
        const int c0 = whole ? 0 : run_of(p, t0), c1 = whole ? 0 : run_of(p, t0 + p.k_stages - 1);
        const int me = whole ? 0 : static_cast<int>(blockIdx.x);
        auto part_of = [&](int c) {
          const int slot = 2 * c + (c == c0 && run_begin(p, c) < t0 ? 1 : 0);
          return p.parts + static_cast<int64_t>(slot) * p.cols * 128 + row;
        };
        unsigned int* ticket = &p.tickets[4 * tile + quarter];
        const unsigned int others = static_cast<unsigned int>(c1 - c0);
        auto all_there = [&] {  // acquired by every lane: the parts may be read
          unsigned int seen;
          asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(ticket) : "memory");
          return __all_sync(0xFFFFFFFFu, seen == others) != 0;
        };
        // Usually a run's last part finds its one other there (that run began with it):
        // its values are fetched while the MMAs still run, and added to the accumulator,
        // which is never written out.
        float other[32];
        const bool early = others == 1 && all_there();
        const float* theirs = part_of(me == c0 ? c1 : c0);
        if (early) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            other[j] = j < p.cols ? __ldcg(theirs + j * 128) : 0.f;
        }
        if (!mbar_wait_warp(&acc_full[part & 1], (part >> 1) & 1, abort)) break;
        tc_fence_after();
        const uint32_t acc = tmem + 64 * (part & 1) + (static_cast<uint32_t>(quarter * 32) << 16);
        if (whole || early) {
          for (int m0 = 0; m0 < p.M; m0 += 32) {
            uint32_t own[32];
            tmem_ld32(acc + m0, own);
            if (early && m0 > 0) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                other[j] = m0 + j < p.cols ? __ldcg(theirs + (m0 + j) * 128) : 0.f;
            }
            tmem_wait_ld();
            __nv_bfloat16* o = p.out + static_cast<int64_t>(m0) * p.N + n;
#pragma unroll
            for (int j = 0; j < 32; ++j, o += p.N) {
              const float f = __uint_as_float(own[j]) + (early ? other[j] : 0.f);
              if (m0 + j < p.M && n < p.N) *o = __float2bfloat16_rn(fmaf(alpha, f, bias));
            }
          }
        } else {
          bool last = all_there();
          if (!last) {
            float* mine = part_of(me);
            for (int c = 0; c < p.M; c += 16) {
              uint32_t v[16];
              tmem_ld16(acc + c, v);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) mine[(c + j) * 128] = __uint_as_float(v[j]);
            }
            __threadfence();
            __syncwarp();
            unsigned int before = 0;
            if (lane == 0) before = atomicAdd(ticket, 1u);
            last = __shfl_sync(0xFFFFFFFFu, before, 0) == others;
            if (last) __threadfence();
          }
          for (int m0 = 0; m0 < p.M && last; m0 += 16) {  // in run order
            uint32_t own[16];
            tmem_ld16(acc + m0, own);
            tmem_wait_ld();
            float f[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) f[j] = 0.f;
#pragma unroll 2
            for (int c = c0; c <= c1; ++c) {
              const float* from_c = part_of(c) + m0 * 128;
              float v[16];
#pragma unroll
              for (int j = 0; j < 16; ++j)
                v[j] = c == me ? __uint_as_float(own[j]) : __ldcg(from_c + j * 128);
#pragma unroll
              for (int j = 0; j < 16; ++j) f[j] += v[j];
            }
            __nv_bfloat16* o = p.out + static_cast<int64_t>(m0) * p.N + n;
#pragma unroll
            for (int j = 0; j < 16; ++j, o += p.N)
              if (m0 + j < p.M && n < p.N) *o = __float2bfloat16_rn(fmaf(alpha, f[j], bias));
          }
        }
        tc_fence_before();
        mbar_arrive_warp(&acc_empty[part & 1]);
        __syncwarp();
      }
    }
  }
  if (kClusters && p.split > 1 && !(warp >= 2)) cluster_wait();
  tc_fence_before();
  __syncthreads();
  if (kClusters && p.split > 1) cluster_sync_all();  // no CTA leaves while a peer may write into it
  report_abort(abort, p.err);
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kAlloc);
  }
}

size_t rup(size_t v, size_t a) { return (v + a - 1) / a * a; }

// Workspace, each region 256-byte aligned.
struct SmallPlan {
  int cols, tiles, k_stages, split, runs;  // split 0: runs
  bool fused;
  size_t cx, sx, tickets, parts, total;
};

SmallPlan small_plan(int64_t M, int64_t N, int64_t K) {
  SmallPlan p{};
  p.cols = static_cast<int>((M + 15) / 16 * 16);
  p.tiles = static_cast<int>((N + 127) / 128);
  p.k_stages = static_cast<int>((K + 255) / 256);
  const int sms = device_sms();
  if (p.tiles <= sms) {
    // As many CTAs a tile as there are SMs and stages of K for, and half as many again, two
    // to an SM, for few rows: up to 16 (1 x 10240 x 8192 12 us, 15 without; 1 x 12800 x 4096
    // 7.3, 9.9), and up to 32 where each CTA has 16 stages and more (32 x 10240 x 8192 13.0,
    // 15.6).  With more rows or shorter parts the second sum costs more (32 x 10240 x 2048
    // 7.9, 7.2; 64 x 14336 x 16384 33, 30).
    // The sums are at most 112 KB, and 56 KB where the clusters need two CTAs per SM: those
    // of more than 128 SMs' worth, of which the chip's groups of SMs do not hold all at once
    // with one CTA per SM (64 x 4864 x 8192 in four, one per SM: 21 us, in two: 13).  Of 7
    // and 8, few fit a group (32 x 2304 x 4096, 18 tiles: 15 us in seven, 8.3 in four; 32 x
    // 2048 x 4096, 16 tiles: 15 us in eight, 7.9 in seven).
    p.split = 1;
    for (int x = 2; x <= 8 && x <= p.k_stages; ++x) {
      const int ctas = x * p.tiles, sum_rows = (x - 1) * p.cols;
      const bool pairs = p.cols == 16 || (p.cols == 32 && p.k_stages >= 16 * x);
      if (ctas <= 128 ? sum_rows <= 224 && (x < 7 || p.tiles <= (sum_rows <= 112 ? 16 : 12))
                      : ctas <= (pairs ? 3 * sms / 2 : sms) && sum_rows <= 112 && x <= 4)
        p.split = x;
    }
    p.runs = p.split * p.tiles;
    // x quantized in place, by every CTA its part, saves the other launch (2 us of the
    // host's time), and time on the device up to 3.5 blocks a thread: 1 x 4608 x 1536 5.2
    // us (5.9 in two launches), 5 x 1536 x 8960 (3.1 blocks) 7.4 (7.7); 8 x 4096 x 4096 (4
    // blocks) 7.3 (7.1).  Eight stages of x, at most, lie beside the ring.
    const int64_t part = (p.k_stages + p.split - 1) / p.split;
    p.fused = part <= 8 && 16 * M * part <= 448;  // of 128 kFusedBlocks
  } else {
    p.runs = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(p.tiles) * p.k_stages, sms));
  }
  p.cx = 0;
  p.sx = rup(static_cast<size_t>(M) * (K / 2), 256);
  p.tickets = p.sx + static_cast<size_t>(p.k_stages) * kXs;
  p.parts = p.tickets + (p.split > 0 ? 0 : rup(static_cast<size_t>(p.tiles) * 16, 256));
  p.total = p.parts + (p.split > 0 ? 0 : static_cast<size_t>(2 * p.runs) * p.cols * 128 * 4);
  return p;
}

}  // namespace

// The M K / 16 blocks of x and N K / 256 units have to fit 31 bits (weights of up to 2^39
// elements do).
bool linear_small_takes(int64_t M, int64_t N, int64_t K) {
  return M <= kLinearSmallRows && N <= (int64_t{1} << 30) && K <= (int64_t{1} << 30) &&
         M * (K / 16) < (int64_t{1} << 31) - 128 &&
         (N + 127) / 128 * ((K + 255) / 256) < (int64_t{1} << 31) / 4 - 1;
}

size_t linear_small_workspace(int64_t M, int64_t N, int64_t K) { return small_plan(M, N, K).total; }

cudaError_t launch_linear_small(const void* x, int64_t ld_x, const float* gx,
                                const CUtensorMap& tx, const CUtensorMap& tw, const uint8_t* sw,
                                const float* gw, const void* bias, int64_t M, int64_t N, int64_t K,
                                void* out, uint8_t* ws, int* err, cudaStream_t stream) {
  const SmallPlan q = small_plan(M, N, K);
  unsigned int* tickets = reinterpret_cast<unsigned int*>(ws + q.tickets);
  cudaError_t e = cudaSuccess;
  if (!q.fused) {
    const int nbc = static_cast<int>(K / 16), blocks = static_cast<int>(M) * nbc;
    const int n_tickets = q.split == 0 ? 4 * q.tiles : 0;
    e = launch_pdl(quant_rows_kernel, dim3((std::max(blocks, n_tickets) + 127) / 128), dim3(128), 0,
                   stream, 1, static_cast<const uint16_t*>(x), ld_x, static_cast<int>(M), nbc, gx,
                   ws + q.cx, ws + q.sx, tickets, n_tickets);
    if (e != cudaSuccess) return e;
  }
  const uint32_t x_stage = q.cols * 128u + kXs;
  const uint32_t stage = (kW + kSc + (q.fused ? 0 : x_stage) + 1023) / 1024 * 1024;
  SmallArgs a{};
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.cols = q.cols;
  a.stages = std::min<int>(kStages, (220 * 1024) / stage);
  a.split = q.split;
  a.tiles = q.tiles;
  a.k_stages = q.k_stages;
  a.k_steps = static_cast<int>(K / 64);
  a.runs = q.runs;
  a.per_run = static_cast<int>(static_cast<int64_t>(q.tiles) * q.k_stages / q.runs);
  a.rest = static_cast<int>(static_cast<int64_t>(q.tiles) * q.k_stages % q.runs);
  a.x = static_cast<const uint16_t*>(x);
  a.ld_x = ld_x;
  a.sx = ws + q.sx;
  a.sw = sw;
  a.gx = gx;
  a.gw = gw;
  a.bias = static_cast<const __nv_bfloat16*>(bias);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.tickets = tickets;
  a.parts = reinterpret_cast<float*>(ws + q.parts);
  a.err = err;
  size_t smem = a.stages * stage + 1024;
  if (q.split == 0) {
    e = cudaFuncSetAttribute(linear_small_kernel<false, false>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, 226 * 1024);
    if (e != cudaSuccess) return e;
    return launch_pdl(linear_small_kernel<false, false>, dim3(q.runs), dim3(kThreads), smem, stream,
                      1, tx, tw, a);
  }
  // At most four stages, and 112 KB where there are more CTAs than one per SM leaves room
  // for: two fit an SM then.  At least 78 KB: no three do, whose 256 tensor-memory
  // columns each would not fit, so that no CTA waits for columns that a cluster holds
  // which in its turn waits for that CTA's cluster.  (The library's other kernels whose
  // CTAs wait for one another or hold tensor memory long take over 149 KB: they share no
  // SM with these.)
  const int part = (q.k_stages + q.split - 1) / q.split;  // stages of a CTA, at most
  const size_t sums = static_cast<size_t>(q.split - 1) * q.cols * 512;
  const size_t xs = q.fused ? static_cast<size_t>(part) * x_stage : 0;
  const size_t room = (q.runs > 128 ? 112 : 222) * 1024;
  a.stages = std::min<int>({4, part, static_cast<int>((room - 1024 - sums - xs) / stage)});
  a.sums_at = static_cast<uint32_t>(a.stages * stage + xs);
  smem = std::max<size_t>(a.sums_at + sums + 1024, 78 * 1024);
  auto* kernel = q.fused ? linear_small_kernel<true, true> : linear_small_kernel<true, false>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 226 * 1024);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(q.runs), dim3(kThreads), smem, stream, q.split, tx, tw, a);
}

}  // namespace nvq
