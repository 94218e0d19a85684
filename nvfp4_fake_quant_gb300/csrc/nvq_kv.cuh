// Layout of a page record of the paged NVFP4 cache (include/nvfp4attn.h) and the
// argument checks its calls share.
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

}  // namespace nvq
