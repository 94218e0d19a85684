// The packed NVFP4 linear of a few rows (a decode step's tokens):
//   out[m, n] = alpha sum_k x~[m, k] w~[n, k] + bias[n],  M <= 64.
//
// Bound.  Every weight is read once, 9/16 byte each (codes and scales): the call is
// a stream of w through the chip.  The weights are the 128-row side of the
// block-scaled FP4 MMAs (tcgen05 kind::mxf4nvf4) and are never decoded; the rows of
// x are the narrow side (M rounded up to 16 columns).
//
// Work split.  A tile of 128 weight rows belongs to one CTA, or, where there are few
// tiles, to a cluster of up to eight, each with a range of K; they leave their sums in
// the first one's shared memory, which adds them in order.  (Through the workspace and a
// ticket the same sum costs 2 us more: 7.8 against 5.9 us for 1 x 4608 x 1536.)  Two CTAs
// fit an SM, so that one's stream goes on under the other's start and end: whole tiles
// beat equal runs of all tiles, whose ends cross tiles, by 5 to 40% up to 304 tiles and
// by up to 20% from 400 on (28672 x 1024 4.9 us, 8.9; 65536 x 1024 9.1, 11.7); between
// them the second wave is short (40960 x 8192 39 us, 35).
//
// Measured (calls in a CUDA graph): 53248 x 16384 78 us for one row, 93% of the copy
// rate, 82 for 64; 28672 x 8192 25 us for one row, 78%, 26 for 32 and 64; one row of 1536
// x 8960 6.4 us and of 4608 x 1536 4.9, the latency of a launch, of the first loads and of the
// cluster's sum.  What a lone warp computes counts here: divisions per stage in the
// producer cost 1 x 14336 x 16384 8 us, 64-bit products for the outputs' rows 28672 x
// 8192 2 us at 64 rows.
//
// Launches.  With few blocks of x per CTA the clusters quantize x themselves, each CTA
// its range of K, while the first weights arrive.  Else there are two: x is quantized by
// a small kernel, while the main kernel, launched behind it programmatically, already
// fills its ring with weights, which do not depend on x.
#include <algorithm>
#include <cstdint>
#include <iterator>

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
constexpr int kStages = 4;     // of the ring, at most (six or eight: 0 to 6% slower)
// bytes of a stage: w codes, w scales, x scales
constexpr uint32_t kW = 128 * 128, kSc = kSteps * 512, kXs = 1024;
constexpr uint32_t kScCol = 64, kCols = 256;  // tensor memory: the sums of 64 columns, then scales
static_assert(kScCol + 32 * kStages <= kCols, "tensor memory");

struct SmallArgs {
  int M, N, cols, stages;   // cols: M rounded up to 16; stages of the ring
  int k_stages, k_steps;
  int split;                // CTAs per tile
  uint32_t sums_at;         // of their sums in the first one's shared memory
  const uint16_t* x;        // x itself (kFused)
  int64_t ld_x;
  const uint8_t* sx;        // x scales (stage blocks), w scales (tiled layout)
  const uint8_t* sw;
  const float* gx;          // device scalars; gw nullptr: 1
  const float* gw;
  const __nv_bfloat16* bias;
  __nv_bfloat16* out;
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
// are not written: the products of those rows are never stored.  (Four bytes an element of
// K, which the host admits up to 2^30: the offset needs more than 32 bits.)
__host__ __device__ __forceinline__ int64_t x_scale_at(int r, int cb) {
  const int step = cb >> 2, w = (step & 1) * 2 + (r >> 5);
  return static_cast<int64_t>(step >> 1) * 512 + ((r & 31) * 16 + w * 4 + (cb & 3));
}

// x [M, K] to codes and scales, one 16-element block per thread.
__global__ void __launch_bounds__(128)
    quant_rows_kernel(const uint16_t* x, int64_t ld, int M, int nbc, const float* gsf,
                      uint8_t* codes, uint8_t* scales) {
  // the kernels before this one are done when the next one starts: it may read w early
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x * 128 + threadIdx.x;
  if (i >= M * nbc) return;
  const int r = i / nbc, cb = i - r * nbc;
  const float g = *gsf;
  const uint4* src = reinterpret_cast<const uint4*>(x + r * ld + static_cast<int64_t>(cb) * 16);
  const uint4 lo = ld16(src), hi = ld16(src + 1);
  const Q16 q = quant_block(lo, hi, g);
  *reinterpret_cast<uint2*>(codes + static_cast<int64_t>(i) * 8) =
      make_uint2(q.codes[0], q.codes[1]);
  scales[x_scale_at(r, cb)] = static_cast<uint8_t>(q.sbyte);
}

// Place in the ring: stage and the parity of its use.
struct Place {
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) {
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

// One tile per cluster of p.split CTAs, stages [ks0, ks0 + count) of K each.  kFused: the
// epilogue's warps quantize the CTA's part of x into shared memory first.
template <bool kFused>
__global__ void __launch_bounds__(kThreads)
    linear_small_kernel(const __grid_constant__ CUtensorMap tx,
                        const __grid_constant__ CUtensorMap tw, const SmallArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023u) &
                                             ~static_cast<uintptr_t>(1023u));
  __shared__ uint64_t full[kStages], empty[kStages], acc_full, sums_full, x_full;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  volatile int* abort = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t x_bytes = static_cast<uint32_t>(p.cols) * 128;
  // a stage: w codes, x codes, w scales, x scales; fused: without x, whose stages follow
  // the ring (all codes, then all scales)
  const uint32_t sx_at = kW + (kFused ? 0u : x_bytes);
  const uint32_t stage_bytes = (sx_at + kSc + (kFused ? 0u : kXs) + 1023) & ~1023u;
  pdl_trigger();
  if (threadIdx.x == 0) {
    *abort = 0;
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_full, 1);
    mbar_init(&sums_full, max(4 * (p.split - 1), 1));
    if (kFused) mbar_init(&x_full, 4);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  if (p.split > 1) cluster_arrive();  // waited for before the first remote write
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int tile = blockIdx.x / p.split, rank = blockIdx.x - tile * p.split;
  const int ks0 = p.k_stages * rank / p.split;
  const int count = p.k_stages * (rank + 1) / p.split - ks0;
  uint8_t* xc = smem + p.stages * stage_bytes;  // fused: x codes and scales of the CTA's part
  uint8_t* xs = xc + count * x_bytes;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    tma_prefetch_desc(&tx);
    tma_prefetch_desc(&tw);
    // (places are counted on, not divided out: a warp alone waits 0.1 us for a division)
    auto load_w = [&](int i, int s) {
      const int ks = ks0 + i, ns = min(kSteps, p.k_steps - ks * kSteps);
      uint8_t* st = smem + s * stage_bytes;
      mbar_arrive_expect_tx_w(&full[s],
                              sx_at + (kFused ? 0u : kXs) + static_cast<uint32_t>(ns) * 512u);
      tma_load_4d_w(st, &tw, ks * 128, tile * 128, 0, 0, &full[s]);
      bulk_load_w(st + sx_at,
                  p.sw + (static_cast<int64_t>(tile) * p.k_steps + ks * kSteps) * 512, ns * 512,
                  &full[s]);
    };
    auto load_x = [&](int i, int s) {
      uint8_t* st = smem + s * stage_bytes;
      tma_load_4d_w(st + kW, &tx, (ks0 + i) * 128, 0, 0, 0, &full[s]);
      bulk_load_w(st + sx_at + kSc, p.sx + static_cast<int64_t>(ks0 + i) * kXs, kXs, &full[s]);
    };
    const int head = min(count, p.stages);
    if (kFused) pdl_wait();  // no kernel of this call stands between w's writer and this one
    for (int i = 0; i < head; ++i) load_w(i, i);
    if (!kFused) {
      pdl_wait();  // x~
      for (int i = 0; i < head; ++i) load_x(i, i);
    }
    Place at;  // head stages on: once around the ring
    at.phase = 1;
    int i = head;
    bool ok = true;
    for (; i < count; ++i, at.next(p.stages)) {
      if (!(ok = mbar_wait_warp(&empty[at.s], at.phase ^ 1, abort))) break;
      load_w(i, at.s);
      if (!kFused) load_x(i, at.s);
    }
    if (!ok) {  // let the copies already issued land before the block leaves
      for (int k = max(0, i - p.stages); k < i; ++k)
        mbar_wait_warp(&full[k % p.stages], (k / p.stages) & 1, nullptr, 10000000ull);
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    const uint32_t idesc = idesc_mxf4nvf4(128, 0) | (static_cast<uint32_t>(p.cols >> 3) << 17);
    int i = 0;
    Place at;
    const bool x_there = !kFused || mbar_wait_warp(&x_full, 0, abort);
    for (; i < count && x_there; ++i, at.next(p.stages)) {
      const int s = at.s, ns = min(kSteps, p.k_steps - (ks0 + i) * kSteps);
      if (!mbar_wait_warp(&full[s], at.phase, abort)) break;
      tc_fence_after();
      const uint32_t a = smem_u32(smem + s * stage_bytes), sa = a + sx_at;
      const uint32_t b = kFused ? smem_u32(xc + i * x_bytes) : a + kW;
      const uint32_t sb = kFused ? smem_u32(xs + i * kXs) : sa + kSc;
      const uint32_t col = tmem + kScCol + 32 * s;
      const uint64_t ad = sdesc_sw128(a, 16, 1024), bd = sdesc_sw128(b, 16, 1024);
      const uint64_t wd = sdesc(sa, 128, 128, 0), xd = sdesc(sb, 128, 128, 0);
      if (ns == kSteps) {
        issue_stage(tmem, idesc, i > 0 ? 1u : 0u, ad, bd, wd, xd, col, col + 16, &empty[s]);
      } else {  // the last stage of a K that is no multiple of 256
        for (int w = 0; w < 2; ++w) tmem_cp_32x128_x4_w(col + 16 + 4 * w, sb + 512 * w);
        for (int j = 0; j < ns; ++j) {
          tmem_cp_32x128_x4_w(col + 4 * j, sa + 512 * j);
          umma_fp4_ss_w(tmem, ad + 2 * j, bd + 2 * j, idesc, col + 4 * j, col + 16 + 2 * j,
                        (i > 0 || j > 0) ? 1u : 0u);
        }
        umma_commit_w(&empty[s]);
      }
      if (i == count - 1) umma_commit_w(&acc_full);
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
          lo[j] = ld16(src);
          hi[j] = ld16(src + 1);
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
    const int n = tile * 128 + row;
    const float bias = p.bias != nullptr && n < p.N ? __bfloat162float(p.bias[n]) : 0.f;
    float* sums = reinterpret_cast<float*>(smem + p.sums_at);  // [split - 1][cols][128]
    if (p.split > 1) cluster_wait();
    const uint32_t acc = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    bool ok = mbar_wait_warp(&acc_full, 0, abort);
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
  }
  if (p.split > 1 && warp < 2) cluster_wait();
  tc_fence_before();
  __syncthreads();
  if (p.split > 1) cluster_sync_all();  // no CTA leaves while a peer may write into it
  report_abort(abort, p.err);
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

size_t rup(size_t v, size_t a) { return (v + a - 1) / a * a; }

// The workspace: codes of x, its scales at a 256-byte boundary.
size_t scales_at(int64_t M, int64_t K) { return rup(static_cast<size_t>(M) * (K / 2), 256); }
size_t scale_bytes(int64_t K) { return static_cast<size_t>((K + 255) / 256) * kXs; }

// CTAs and their shared memory.
struct SmallPlan {
  int cols, tiles, k_stages, split, ctas;
  bool fused;
  int part, stages;   // stages of K of a CTA, at most; of its ring
  uint32_t sums_at;   // in shared memory: the other CTAs' sums
  size_t smem;
};

SmallPlan small_plan(int64_t M, int64_t N, int64_t K) {
  SmallPlan p{};
  p.cols = static_cast<int>((M + 15) / 16 * 16);
  p.tiles = static_cast<int>((N + 127) / 128);
  p.k_stages = static_cast<int>((K + 255) / 256);
  const int sms = device_sms();
  // As many CTAs a tile as there are SMs and stages of K for, and half as many again, two
  // to an SM, for few rows: up to 16 (1 x 10240 x 8192 12 us, 15 without; 1 x 12800 x 4096
  // 7.3, 9.9), and up to 32 where each CTA has 16 stages and more (32 x 10240 x 8192 13.0,
  // 15.6).  With more rows or shorter parts the second sum costs more (32 x 10240 x 2048
  // 7.9, 7.2; 64 x 14336 x 16384 33, 30).
  // The sums are at most 112 KB, and 56 KB where the clusters need two CTAs per SM: those
  // of more than 128 SMs' worth, of which the chip's groups of SMs do not hold all at once
  // with one CTA per SM (64 x 4864 x 8192 in four, one per SM: 21 us, in two: 13).  Of
  // clusters of 7 and 8, 15 run at once with one CTA per SM, 16 do not: 16 x 1920 x 8192, 15
  // tiles, 7.0 us in eight (6.8 in six), 16 x 2048 x 8192, 16 tiles, 12.0 (6.8); x 28672 9.9
  // (10.8) and 18.1 (10.9).  With sums over 56 KB they pay from K of 16384 on, up to 12 tiles
  // by 0 to 9% (32 x 1536 x 28672 11.5 us, 12.1 in six; x 8192 8.5, 7.9; x 2048 7.3, 6.6); at
  // 13 to 15 tiles, in six, they would win as little and lose as much (32 x 1664 x 28672 12.3
  // us, 11.6 in eight; x 8192 7.9, 8.5; x 2048 6.6, 7.4).
  p.split = 1;
  for (int x = 2; x <= 8 && x <= p.k_stages; ++x) {
    const int64_t ctas = static_cast<int64_t>(x) * p.tiles;
    const int sum_rows = (x - 1) * p.cols;
    const bool pairs = p.cols == 16 || (p.cols == 32 && p.k_stages >= 16 * x);
    if (ctas <= 128 ? sum_rows <= 224 && (x < 7 || p.tiles <= (sum_rows <= 112 ? 15 : 12))
                    : ctas <= (pairs ? 3 * sms / 2 : sms) && sum_rows <= 112 && x <= 4)
      p.split = x;
  }
  p.ctas = p.split * p.tiles;
  // x quantized in place, by every CTA its part, saves the other launch (2 us of the
  // host's time), and time on the device up to 3.5 blocks a thread: 1 x 4608 x 1536 5.2
  // us (5.9 in two launches), 5 x 1536 x 8960 (3.1 blocks) 7.4 (7.7); 8 x 4096 x 4096 (4
  // blocks) 7.3 (7.1).  Eight stages of x, at most, lie beside the ring.
  p.part = (p.k_stages + p.split - 1) / p.split;
  p.fused = p.part <= 8 && 16 * M * p.part <= 448;  // of 128 kFusedBlocks
  // At most four stages, and 112 KB where there are more CTAs than one per SM leaves room
  // for: two fit an SM then.  At least kLinearSmallSmem: no three do, whose 256 tensor-memory
  // columns each would not fit, so that no CTA waits for columns that a cluster holds
  // which in its turn waits for that CTA's cluster.  (The library's other kernels that hold
  // tensor memory assert that they share no SM with these, or that their CTAs wait for
  // nobody.)
  const uint32_t x_stage = p.cols * 128u + kXs;
  const uint32_t stage = (kW + kSc + (p.fused ? 0 : x_stage) + 1023) / 1024 * 1024;
  const int sums = (p.split - 1) * p.cols * 512;
  const int xs = p.fused ? p.part * static_cast<int>(x_stage) : 0;
  const int room = (p.ctas > 128 ? 112 : 222) * 1024 - 1024 - sums - xs;
  p.stages = std::min({kStages, p.part, room / static_cast<int>(stage)});
  p.sums_at = p.stages * stage + xs;
  p.smem = std::max<size_t>(p.sums_at + sums + 1024, kLinearSmallSmem);
  return p;
}

}  // namespace

// The M K / 16 blocks of x have to fit 31 bits.
bool linear_small_takes(int64_t M, int64_t N, int64_t K) {
  return M <= kLinearSmallRows && N <= (int64_t{1} << 30) && K <= (int64_t{1} << 30) &&
         M * (K / 16) < (int64_t{1} << 31) - 128;
}

size_t linear_small_workspace(int64_t M, int64_t K) { return scales_at(M, K) + scale_bytes(K); }

cudaError_t launch_linear_small(const void* x, int64_t ld_x, const float* gx,
                                const CUtensorMap& tx, const CUtensorMap& tw, const uint8_t* sw,
                                const float* gw, const void* bias, int64_t M, int64_t N, int64_t K,
                                void* out, uint8_t* ws, int* err, cudaStream_t stream) {
  const SmallPlan q = small_plan(M, N, K);
  uint8_t* const sx = ws + scales_at(M, K);
  cudaError_t e = cudaSuccess;
  if (!q.fused) {
    const int nbc = static_cast<int>(K / 16), blocks = static_cast<int>(M) * nbc;
    e = launch_pdl(quant_rows_kernel, dim3((blocks + 127) / 128), dim3(128), 0, stream, 1,
                   static_cast<const uint16_t*>(x), ld_x, static_cast<int>(M), nbc, gx, ws, sx);
    if (e != cudaSuccess) return e;
  }
  if (q.stages < 1) return cudaErrorInvalidConfiguration;  // the plan leaves room for one and more
  SmallArgs a{};
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.cols = q.cols;
  a.stages = q.stages;
  a.k_stages = q.k_stages;
  a.k_steps = static_cast<int>(K / 64);
  a.split = q.split;
  a.sums_at = q.sums_at;
  a.x = static_cast<const uint16_t*>(x);
  a.ld_x = ld_x;
  a.sx = sx;
  a.sw = sw;
  a.gx = gx;
  a.gw = gw;
  a.bias = static_cast<const __nv_bfloat16*>(bias);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.err = err;
  const auto kernel = q.fused ? linear_small_kernel<true> : linear_small_kernel<false>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 226 * 1024);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(q.ctas), dim3(kThreads), q.smem, stream, q.split, tx, tw, a);
}

}  // namespace nvq

extern "C" nvq_status nvq_selftest_linear_plan(int64_t M, int64_t N, int64_t K, int64_t* plan) {
  using namespace nvq;
  if (plan == nullptr || M < 1 || N < 1 || N % 16 != 0 || K < 1 || K % 64 != 0)
    return NVQ_ERR_INVALID;
  if (!linear_small_takes(M, N, K)) return NVQ_ERR_UNSUPPORTED;
  const SmallPlan p = small_plan(M, N, K);
  int64_t end = 0;  // the last block's scales lie furthest
  for (int r = 0; r < M; ++r)
    end = std::max(end, x_scale_at(r, static_cast<int>(K / 16) - 1) + 1);
  const int64_t got[] = {p.split, p.ctas, p.fused, p.part, p.stages,
                         static_cast<int64_t>(p.smem), static_cast<int64_t>(scale_bytes(K)), end};
  std::copy(std::begin(got), std::end(got), plan);
  return NVQ_OK;
}
