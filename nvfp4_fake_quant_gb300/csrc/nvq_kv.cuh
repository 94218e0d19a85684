// Layout of a page record of the paged NVFP4 cache (include/nvfp4attn.h), the argument checks its
// calls share, and what the attention kernels over it (attn_decode.cu, attn_cross.cu) share.
#pragma once
#include <cstdint>

#include "nvfp4attn.h"

namespace nvq {

constexpr int kPage = NVQ_KV_PAGE;

// K codes | V codes | K scales | V scales, kPage rows each.
__host__ __device__ constexpr int record_bytes(int D) { return kPage * D * 9 / 8; }
__host__ __device__ constexpr int v_codes_at(int D) { return kPage * D / 2; }
__host__ __device__ constexpr int k_scales_at(int D) { return kPage * D; }
__host__ __device__ constexpr int v_scales_at(int D) { return kPage * D + kPage * D / 16; }

// How the kernels multiply the scores S by scale (in log2 units).  p = 2^(S scale - m) is one fused
// product and difference, while the reference m is a score times scale, rounded: up to half a step
// of m may come on top of kSlack, for |m| < 2^28 at most 8.  |S| <= 2688^2 D (codes of 6, scales of
// 448), so any scale up to 25.7 / D, more than twice D^-0.5, keeps S scale below 2^28.  For a
// larger one S is first replaced by S scale, rounded as m is; the difference is then exact.
struct Scales {
  float before, fused;  // S before (1: not at all); in the fused product
};
inline Scales scales_of(float scale_log2, int D) {
  if (scale_log2 * (2688.f * 2688.f * static_cast<float>(D)) < 0x1p28f) return {1.f, scale_log2};
  return {scale_log2, 1.f};
}

inline nvq_status check_kv(const void* pool, int64_t num_pages, const int32_t* page_table,
                           int64_t ld_table, int max_pages, const int32_t* seq_lens) {
  if (pool == nullptr || (reinterpret_cast<uintptr_t>(pool) & 15u) != 0 || num_pages < 1 ||
      num_pages > 0x7FFFFFFF || page_table == nullptr ||
      (reinterpret_cast<uintptr_t>(page_table) & 3u) != 0 || max_pages < 1 ||
      max_pages > 0x7FFFFFFF / kPage || ld_table < max_pages || seq_lens == nullptr ||
      (reinterpret_cast<uintptr_t>(seq_lens) & 3u) != 0)
    return NVQ_ERR_INVALID;
  return NVQ_OK;
}

constexpr float kSlack = 8.f;  // scores may exceed the reference maximum by this (log2)
// The largest score for which m stays the reference.  m's rounding adds to kSlack: from steps of
// 1/8 (2^20) on less is left, from 2^24 on nothing (the result is then m or below it).
__device__ __forceinline__ float limit_of(float m) {
  return fmaf(fabsf(m), -0x1p-21f, m + kSlack);
}
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// The line of `all` tiles is cut into n = min(all, runs) runs: run c is [all c / n,
// all (c + 1) / n), never empty; of the grid's runs those from n on have nothing.
// all c / n = (all / n) c + (all % n) c / n.  n is the grid's or all itself, so there is
// nothing to divide: the host gives 2^64 / runs, rounded up (all <= 2^53 and runs < 2^10
// keep the product's error below 1 / runs; for one run 2^64 is kept as 0, and begin asks for no
// product).
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

}  // namespace nvq
