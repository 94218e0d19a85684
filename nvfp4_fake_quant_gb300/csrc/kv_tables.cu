// Tables of the paged cache, kept on the device: pages for new tokens (with the place and the
// position of each), and the pages of finished sequences back.
//
// Free pages are a stack: free_pages[0 .. free_count).  The new pages of a call, numbered in the
// order of (sequence, page), are taken from its top: number k is free_pages[count - 1 - k]; those
// given back are pushed in the same order.  So the tables follow from the inputs alone, whatever
// the order in which threads run.
//
// Both are exclusive sums over the sequences (tokens, pages), then independent work per token
// and page.  One block of 1024 threads takes the sums: each thread a chunk of consecutive
// sequences, whose sums stay in shared memory; a token's or page's sequence is found by a binary
// search over the chunks and a walk inside one.  Few tokens are placed by the same block; many by
// a second kernel over the whole chip, which takes the sums again from the first one's outputs
// (so nothing has to be kept between them, and no workspace is needed).
//
// Bound by latency: a launch, two dependent loads, the scan's barriers.
#include <algorithm>
#include <cstdint>
#include <initializer_list>

#include <cuda_runtime.h>

#include "nvq_internal.h"
#include "nvq_kv.cuh"
#include "nvq_ptx.cuh"

namespace nvq {

namespace {

constexpr int kThreads = 1024;
// Tokens that the summing block places itself.
constexpr int64_t kOneBlock = 2048;

// Exclusive sums over chunks of consecutive sequences: tokens and pages before chunk c, for
// c = 0 .. chunks (the last entry: all of them).
struct Sums {
  int tokens[kThreads + 1];
  int pages[kThreads + 1];
};

struct Total {
  int64_t tokens, pages;
};

// Sums of (tokens, pages) over the block, and those before this thread.  `warps`: 32 entries.
__device__ __forceinline__ Total block_scan(int64_t t, int64_t p, Total* warps, Total* before) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t st = t, sp = p;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t a = __shfl_up_sync(0xFFFFFFFFu, st, off),
                  b = __shfl_up_sync(0xFFFFFFFFu, sp, off);
    if (lane >= off) {
      st += a;
      sp += b;
    }
  }
  if (lane == 31) warps[warp] = {st, sp};
  __syncthreads();
  if (warp == 0) {
    Total w = warps[lane];
    int64_t wt = w.tokens, wp = w.pages;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t a = __shfl_up_sync(0xFFFFFFFFu, wt, off),
                    b = __shfl_up_sync(0xFFFFFFFFu, wp, off);
      if (lane >= off) {
        wt += a;
        wp += b;
      }
    }
    warps[lane] = {wt, wp};
  }
  __syncthreads();
  const Total base = warp == 0 ? Total{0, 0} : warps[warp - 1];
  *before = {base.tokens + st - t, base.pages + sp - p};
  return warps[31];
}

// The chunk whose run of `sums` holds x: the last c in [0, n) with sums[c] <= x < sums[n].
__device__ __forceinline__ int find_chunk(const int* sums, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int pages_of(int n) { return (n + kPage - 1) / kPage; }

struct ExtendArgs {
  const int32_t* fresh;  // new tokens
  const int32_t* lens;
  const int32_t* start;
  int B;
  int32_t* table;
  int64_t ld_table;
  int max_pages;
  const int32_t* free_pages;
  const int32_t* free_count;
  int64_t num_pages;
  int64_t T;
  int32_t* lens_out;
  int32_t* count_out;
  int32_t* cu;
  int32_t* positions;
  int64_t* slots;
  int* err;
};

// A sequence's new tokens and its length before them.  kAfter: from the outputs of the planning
// kernel (a refused call has no new tokens there).
template <bool kAfter>
__device__ __forceinline__ int2 growth(const ExtendArgs& a, int b) {
  if constexpr (kAfter) {
    const int t = a.cu[b + 1] - a.cu[b];
    return make_int2(t, max(a.lens_out[b] - t, 0));
  } else {
    return make_int2(max(a.fresh[b], 0), max(a.lens[b], 0));
  }
}

// kPlan: lengths, offsets, the free pages' count (one block).  kPlace: table entries, positions
// and slots.
template <bool kPlan, bool kPlace>
__global__ void __launch_bounds__(kThreads) extend_kernel(const ExtendArgs a) {
  constexpr bool kAfter = !kPlan;
  __shared__ Total warps[32];
  __shared__ Sums sums;
  pdl_trigger();
  pdl_wait();
  const int per = (a.B + kThreads - 1) / kThreads;
  const int chunks = (a.B + per - 1) / per;
  const int b_lo = min(a.B, static_cast<int>(threadIdx.x) * per), b_hi = min(a.B, b_lo + per);
  const int64_t cap = static_cast<int64_t>(a.max_pages) * kPage;
  int count = kAfter ? *a.count_out : *a.free_count;
  int64_t t = 0, p = 0;
  bool bad = false;
  for (int b = b_lo; b < b_hi; ++b) {
    const int2 g = growth<kAfter>(a, b);
    const int64_t end = static_cast<int64_t>(g.y) + g.x;
    bad |= end > cap;
    t += g.x;
    p += (end + kPage - 1) / kPage - (g.y + static_cast<int64_t>(kPage) - 1) / kPage;
  }
  Total before;
  Total all = block_scan(t, p, warps, &before);
  if constexpr (kPlan) {
    bad |= count < 0 || count > a.num_pages || all.pages > count || all.tokens > a.T;
    bad = __syncthreads_or(bad);
    if (bad) {
      all = before = {0, 0};
      t = p = 0;
      if (threadIdx.x == 0) atomicMax(a.err, kErrTable);
    }
  } else {
    count += static_cast<int>(all.pages);  // as before the call
  }
  if constexpr (kPlace) {
    if (b_lo < b_hi) {
      sums.tokens[threadIdx.x] = static_cast<int>(before.tokens);
      sums.pages[threadIdx.x] = static_cast<int>(before.pages);
    }
    if (threadIdx.x == 0) {
      sums.tokens[chunks] = static_cast<int>(all.tokens);
      sums.pages[chunks] = static_cast<int>(all.pages);
    }
    __syncthreads();
    const int64_t step = static_cast<int64_t>(kThreads) * gridDim.x;
    const int64_t first = static_cast<int64_t>(kThreads) * blockIdx.x + threadIdx.x;
    // ---- table entries of the new pages
    for (int64_t i = first; i < all.pages; i += step) {
      const int k = static_cast<int>(i);
      const int c = find_chunk(sums.pages, chunks, k);
      int at = sums.pages[c], b = c * per, held;
      for (;; ++b) {
        const int2 g = growth<kAfter>(a, b);
        held = pages_of(g.y);
        const int n = pages_of(g.y + g.x) - held;
        if (k < at + n) break;
        at += n;
      }
      a.table[b * a.ld_table + held + (k - at)] = a.free_pages[count - 1 - k];
    }
    // ---- positions and slots of the new tokens
    for (int64_t r = first; r < a.T; r += step) {
      int64_t slot = -1;
      int pos = -1;
      if (r < all.tokens) {
        const int row = static_cast<int>(r);
        const int c = find_chunk(sums.tokens, chunks, row);
        int at = sums.tokens[c], k = sums.pages[c], b = c * per;
        int2 g;
        for (;; ++b) {
          g = growth<kAfter>(a, b);
          if (row < at + g.x) break;
          at += g.x;
          k += pages_of(g.y + g.x) - pages_of(g.y);
        }
        const int tok = g.y + (row - at), held = pages_of(g.y);
        const int i = tok / kPage;
        const int page = i < held ? a.table[b * a.ld_table + i]
                                  : a.free_pages[count - 1 - (k + i - held)];
        pos = tok + (a.start == nullptr ? 0 : a.start[b]);
        if (page >= 0 && page < a.num_pages)
          slot = static_cast<int64_t>(page) * kPage + tok % kPage;
        else
          atomicMax(a.err, kErrTable);
      }
      a.positions[r] = pos;
      a.slots[r] = slot;
    }
  }
  if constexpr (kPlan) {
    // the outputs may be the inputs: every read of them is done
    if constexpr (kPlace) __syncthreads();
    int at = static_cast<int>(before.tokens);
    for (int b = b_lo; b < b_hi; ++b) {
      const int2 g = growth<false>(a, b);
      a.cu[b] = at;
      a.lens_out[b] = bad ? a.lens[b] : g.y + g.x;
      if (!bad) at += g.x;
    }
    if (threadIdx.x == 0) {
      a.cu[a.B] = static_cast<int>(all.tokens);
      *a.count_out = count - static_cast<int>(all.pages);
    }
  }
}

struct ReleaseArgs {
  const uint8_t* done;
  const int32_t* lens;
  int B;
  const int32_t* table;
  int64_t ld_table;
  int max_pages;
  int32_t* free_pages;
  const int32_t* free_count;
  int64_t num_pages;
  int32_t* lens_out;
  int32_t* count_out;
  int* err;
};

// One block: sums, a pass over the pages that checks them, one that pushes them.
__global__ void __launch_bounds__(kThreads) release_kernel(const ReleaseArgs a) {
  __shared__ Total warps[32];
  __shared__ int before_chunk[kThreads + 1];
  pdl_trigger();
  pdl_wait();
  const int per = (a.B + kThreads - 1) / kThreads;
  const int chunks = (a.B + per - 1) / per;
  const int b_lo = min(a.B, static_cast<int>(threadIdx.x) * per), b_hi = min(a.B, b_lo + per);
  const int count = *a.free_count;
  auto held = [&](int b) -> int64_t {
    return a.done[b] ? (static_cast<int64_t>(max(a.lens[b], 0)) + kPage - 1) / kPage : 0;
  };
  int64_t p = 0;
  bool bad = count < 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const int64_t n = held(b);
    bad |= n > a.max_pages;
    p += n;
  }
  Total before;
  const Total all = block_scan(0, p, warps, &before);
  bad = __syncthreads_or(bad || all.pages > a.num_pages - count);
  if (!bad) {
    if (b_lo < b_hi) before_chunk[threadIdx.x] = static_cast<int>(before.pages);
    if (threadIdx.x == 0) before_chunk[chunks] = static_cast<int>(all.pages);
    __syncthreads();
    auto page_of = [&](int k) {
      const int c = find_chunk(before_chunk, chunks, k);
      int at = before_chunk[c], b = c * per;
      for (;; ++b) {
        const int n = static_cast<int>(held(b));
        if (k < at + n) break;
        at += n;
      }
      return a.table[b * a.ld_table + (k - at)];
    };
    for (int64_t k = threadIdx.x; k < all.pages; k += kThreads) {
      const int page = page_of(static_cast<int>(k));
      bad |= page < 0 || page >= a.num_pages;
    }
    bad = __syncthreads_or(bad);
    if (!bad)
      for (int64_t k = threadIdx.x; k < all.pages; k += kThreads)
        a.free_pages[count + k] = page_of(static_cast<int>(k));
  }
  __syncthreads();  // the outputs may be the inputs
  for (int b = b_lo; b < b_hi; ++b) {
    const int n = a.lens[b];
    a.lens_out[b] = !bad && a.done[b] ? 0 : n;
  }
  if (threadIdx.x == 0) {
    *a.count_out = bad ? count : count + static_cast<int>(all.pages);
    if (bad) atomicMax(a.err, kErrTable);
  }
}

bool aligned(const void* p, unsigned n) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

nvq_status check_tables(int B, const int32_t* seq_lens, const int32_t* page_table, int64_t ld_table,
                        int max_pages, const int32_t* free_pages, const int32_t* free_count,
                        int64_t num_pages, const int32_t* lens_out, const int32_t* count_out) {
  if (B < 1 || max_pages < 1 || max_pages > 0x7FFFFFFF / kPage || ld_table < max_pages ||
      num_pages < 1 || num_pages > 0x7FFFFFFF)
    return NVQ_ERR_INVALID;
  if (!aligned(seq_lens, 4) || !aligned(page_table, 4) || !aligned(free_pages, 4) ||
      !aligned(free_count, 4) || !aligned(lens_out, 4) || !aligned(count_out, 4))
    return NVQ_ERR_INVALID;
  return B > 65535 ? NVQ_ERR_UNSUPPORTED : NVQ_OK;
}

struct Range {
  const void* p;
  uint64_t n;  // bytes
};

// What is written lies apart from everything else: threads read their inputs at any time until the
// block's last barrier, and of many tokens in a second kernel.
bool apart(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
  const auto meet = [](const Range& a, const Range& b) {
    return a.n > 0 && b.n > 0 && ranges_meet(a.p, a.n, b.p, b.n);
  };
  for (const Range* o = outs.begin(); o != outs.end(); ++o) {
    for (const Range* x = o + 1; x != outs.end(); ++x)
      if (meet(*o, *x)) return false;
    for (const Range& x : ins)
      if (meet(*o, x)) return false;
  }
  return true;
}

uint64_t table_bytes(int B, int64_t ld, int max_pages) {
  return 4 * static_cast<uint64_t>((B - 1) * ld + max_pages);
}

}  // namespace

}  // namespace nvq

extern "C" {

nvq_status nvfp4_kv_extend(const int32_t* new_tokens, const int32_t* seq_lens,
                           const int32_t* start, int B, int32_t* page_table, int64_t ld_table,
                           int max_pages, const int32_t* free_pages, const int32_t* free_count,
                           int64_t num_pages, int64_t T, int32_t* seq_lens_out,
                           int32_t* free_count_out, int32_t* cu_tokens, int32_t* positions,
                           int64_t* slots, nvq_stream_t stream) {
  using namespace nvq;
  nvq_status st = check_tables(B, seq_lens, page_table, ld_table, max_pages, free_pages, free_count,
                               num_pages, seq_lens_out, free_count_out);
  if (st != NVQ_OK) return st;
  if (!aligned(new_tokens, 4) || !aligned(cu_tokens, 4) ||
      (reinterpret_cast<uintptr_t>(start) & 3u) != 0 || T < 0 ||
      (T > 0 && (!aligned(positions, 4) || !aligned(slots, 8))))
    return NVQ_ERR_INVALID;
  if (T > 0x7FFFFFFF) return NVQ_ERR_UNSUPPORTED;
  const uint64_t seqs = 4 * static_cast<uint64_t>(B), none = 0;
  const uint64_t rows = static_cast<uint64_t>(T);
  if (!apart({{seq_lens_out, seqs}, {free_count_out, 4}, {cu_tokens, seqs + 4},
              {positions, 4 * rows}, {slots, 8 * rows},
              {page_table, table_bytes(B, ld_table, max_pages)}},
             {{new_tokens, seqs}, {start, start != nullptr ? seqs : none},
              {seq_lens, seq_lens != seq_lens_out ? seqs : none},
              {free_count, free_count != free_count_out ? 4 : none},
              {free_pages, 4 * static_cast<uint64_t>(num_pages)}}))
    return NVQ_ERR_INVALID;
  int* err = device_error_word();
  if (err == nullptr) return NVQ_ERR_CUDA;
  const ExtendArgs a{new_tokens, seq_lens, start, B, page_table, ld_table, max_pages, free_pages,
                     free_count, num_pages, T, seq_lens_out, free_count_out, cu_tokens, positions,
                     slots, err};
  const cudaError_t e = timed(NVQ_KERNEL_KV_TABLES, stream, [&] {
    if (T <= kOneBlock)
      return launch_pdl(extend_kernel<true, true>, dim3(1), dim3(kThreads), 0, stream, 1, a);
    const cudaError_t r =
        launch_pdl(extend_kernel<true, false>, dim3(1), dim3(kThreads), 0, stream, 1, a);
    if (r != cudaSuccess) return r;
    const int64_t blocks = std::min<int64_t>((T + kThreads - 1) / kThreads, 2 * device_sms());
    return launch_pdl(extend_kernel<false, true>, dim3(static_cast<unsigned>(blocks)),
                      dim3(kThreads), 0, stream, 1, a);
  });
  return e == cudaSuccess ? NVQ_OK : fail_cuda("kv extend", e);
}

nvq_status nvfp4_kv_release(const uint8_t* done, const int32_t* seq_lens, int B,
                            const int32_t* page_table, int64_t ld_table, int max_pages,
                            int32_t* free_pages, const int32_t* free_count, int64_t num_pages,
                            int32_t* seq_lens_out, int32_t* free_count_out, nvq_stream_t stream) {
  using namespace nvq;
  nvq_status st = check_tables(B, seq_lens, page_table, ld_table, max_pages, free_pages, free_count,
                               num_pages, seq_lens_out, free_count_out);
  if (st != NVQ_OK) return st;
  if (done == nullptr) return NVQ_ERR_INVALID;
  const uint64_t seqs = 4 * static_cast<uint64_t>(B), none = 0;
  if (!apart({{seq_lens_out, seqs}, {free_count_out, 4},
              {free_pages, 4 * static_cast<uint64_t>(num_pages)}},
             {{done, static_cast<uint64_t>(B)}, {seq_lens, seq_lens != seq_lens_out ? seqs : none},
              {free_count, free_count != free_count_out ? 4 : none},
              {page_table, table_bytes(B, ld_table, max_pages)}}))
    return NVQ_ERR_INVALID;
  int* err = device_error_word();
  if (err == nullptr) return NVQ_ERR_CUDA;
  const ReleaseArgs a{done, seq_lens, B, page_table, ld_table, max_pages, free_pages, free_count,
                      num_pages, seq_lens_out, free_count_out, err};
  const cudaError_t e = timed(NVQ_KERNEL_KV_TABLES, stream, [&] {
    return launch_pdl(release_kernel, dim3(1), dim3(kThreads), 0, stream, 1, a);
  });
  return e == cudaSuccess ? NVQ_OK : fail_cuda("kv release", e);
}

}  // extern "C"
