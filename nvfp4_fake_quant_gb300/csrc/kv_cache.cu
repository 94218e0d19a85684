// The paged NVFP4 key-value cache: new tokens quantized into pages.
//
// The record of one page (128 tokens) and KV head is contiguous: K codes, V
// codes, K scales, V scales, token rows in order.  One record is one attention
// tile: a decode kernel fetches it with a few bulk copies, and a page's records
// are one contiguous run for whoever copies pages.
//
// Append: per token and head, D/16 blocks of K and of V are read (32 bytes each)
// and written as 8 code bytes and one scale byte.  A block of threads takes 8 tokens
// and walks over the heads; consecutive lanes take the blocks of one token's row, then
// the next token, so that a prompt's reads are whole head rows and its writes of one
// head contiguous runs of 8 D / 2 bytes.  (16 tokens in 256 threads: 1 us more; the
// smaller block leaves more of them to hide the loads.)  Where tokens are few their
// heads are spread over more blocks instead, so that a decode step fills the chip.
//
// Bound by HBM: reads 4 D, writes 9 D / 8 bytes per token and head.  Measured (calls in
// a CUDA graph): 25088 tokens of 12 heads of 128 36.6 us, 80% of the copy rate; 64 single
// tokens 2.1 us, the latency of a launch and of two dependent loads (length, page), under
// which the first head's values arrive (2.4 us when they were asked for behind them).
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "nvq_internal.h"
#include "nvq_kv.cuh"
#include "nvq_ptx.cuh"
#include "nvq_quant.cuh"

namespace nvq {

namespace {

constexpr int kThreads = 128;
constexpr int kTokens = 8;  // tokens per block

struct AppendArgs {
  const uint16_t* k;
  const uint16_t* v;
  int64_t ld_k, ld_v, T;
  int B, Hkv;
  const int64_t* slots;  // places given (lens, table, cu unused), or nullptr
  const int32_t* cu;  // nullptr: one token per sequence
  const int32_t* lens;
  const int32_t* table;
  int64_t ld_table;
  int max_pages;
  uint8_t* pool;
  int64_t num_pages;
  int* err;
};

// Where token t goes: its page's first record and its row there; nullptr if it
// is not written.
__device__ __forceinline__ uint8_t* find_row(const AppendArgs& a, int64_t t, int D, int* row) {
  if (a.slots != nullptr) {
    const int64_t slot = a.slots[t];
    if (slot < 0) return nullptr;
    if (slot / kPage >= a.num_pages) {
      atomicMax(a.err, kErrTable);
      return nullptr;
    }
    *row = static_cast<int>(slot % kPage);
    return a.pool + slot / kPage * a.Hkv * record_bytes(D);
  }
  int b = 0;
  int64_t end = t + 1;
  if (a.cu == nullptr) {
    b = static_cast<int>(t);
  } else {
    // the last b with cu[b] <= t (cu does not decrease: empty sequences share a bound)
    if (t < a.cu[0] || t >= a.cu[a.B]) return nullptr;
    int lo = 0, hi = a.B;  // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu[mid] <= t) lo = mid; else hi = mid;
    }
    b = lo;
    end = a.cu[b + 1];
  }
  const int64_t pos = a.lens[b] - (end - t);
  if (pos < 0) return nullptr;
  if (pos >= static_cast<int64_t>(a.max_pages) * kPage) {
    atomicMax(a.err, kErrTable);
    return nullptr;
  }
  const int page = a.table[b * a.ld_table + pos / kPage];
  if (page < 0 || page >= a.num_pages) {
    atomicMax(a.err, kErrTable);
    return nullptr;
  }
  *row = static_cast<int>(pos % kPage);
  return a.pool + static_cast<int64_t>(page) * a.Hkv * record_bytes(D);
}

// Grid: token groups along x; K and V heads (2 Hkv of them) split along y.
template <int D>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendArgs a) {
  constexpr int kBlocks = D / 16;  // per row
  __shared__ uint8_t* page[kTokens];
  __shared__ int row[kTokens];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens;
  pdl_trigger();
  pdl_wait();
  const int cb = threadIdx.x % kBlocks, tok = threadIdx.x / kBlocks % kTokens;
  constexpr int kRows = kThreads / (kBlocks * kTokens);  // heads per pass
  const int step = gridDim.y * kRows;
  int hv = blockIdx.y * kRows + threadIdx.x / (kBlocks * kTokens);
  const uint16_t* const k = a.k + (t0 + tok) * a.ld_k + cb * 16;
  const uint16_t* const v = a.v + (t0 + tok) * a.ld_v + cb * 16 - static_cast<int64_t>(a.Hkv) * D;
  uint4 lo, hi;
  auto load = [&](int i) {
    const uint4* s4 = reinterpret_cast<const uint4*>((i >= a.Hkv ? v : k) + i * D);
    lo = ld16(s4);
    hi = ld16(s4 + 1);
  };
  // the first head's loads do not wait for the tokens' places
  if (t0 + tok < a.T && hv < 2 * a.Hkv) load(hv);
  if (threadIdx.x < kTokens) {
    const int64_t t = t0 + threadIdx.x;
    page[threadIdx.x] = t < a.T ? find_row(a, t, D, &row[threadIdx.x]) : nullptr;
  }
  __syncthreads();
  uint8_t* const base = page[tok];
  if (base == nullptr) return;
  const int r = row[tok];
  for (; hv < 2 * a.Hkv; hv += step) {
    const uint32_t x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    if (hv + step < 2 * a.Hkv) load(hv + step);
    const bool is_v = hv >= a.Hkv;
    const Codes16 q = codes16_unit(x);
    uint8_t* rec = base + static_cast<int64_t>(is_v ? hv - a.Hkv : hv) * record_bytes(D);
    *reinterpret_cast<uint2*>(rec + (is_v ? v_codes_at(D) : 0) + r * (D / 2) + cb * 8) =
        make_uint2(q.codes[0], q.codes[1]);
    rec[(is_v ? v_scales_at(D) : k_scales_at(D)) + r * kBlocks + cb] =
        static_cast<uint8_t>(q.sbyte);
  }
}

// The checks of k and v that both append calls make (T tokens of Hkv heads; nothing of a call
// without tokens is looked at).
nvq_status check_rows(const void* k, int64_t ld_k, const void* v, int64_t ld_v, int Hkv, int D,
                      int64_t T) {
  if (D != 64 && D != 128) return NVQ_ERR_UNSUPPORTED;
  if (Hkv > 65535) return NVQ_ERR_UNSUPPORTED;
  if (T == 0) return NVQ_OK;
  const int64_t row = static_cast<int64_t>(Hkv) * D;
  if (k == nullptr || v == nullptr || (reinterpret_cast<uintptr_t>(k) & 15u) != 0 ||
      (reinterpret_cast<uintptr_t>(v) & 15u) != 0 || ld_k < row || ld_v < row || ld_k % 8 != 0 ||
      ld_v % 8 != 0)
    return NVQ_ERR_INVALID;
  return NVQ_OK;
}

nvq_status launch_append(AppendArgs a, int D, cudaStream_t stream) {
  const int64_t groups = (a.T + kTokens - 1) / kTokens;
  if (groups > 0x7FFFFFFF) return NVQ_ERR_UNSUPPORTED;
  if ((a.err = device_error_word()) == nullptr) return NVQ_ERR_CUDA;
  // a few tokens: spread their heads over the SMs
  const int rows = kThreads / (D / 16 * kTokens);
  const int64_t want = std::max<int64_t>(1, (2 * device_sms() + groups - 1) / groups);
  const int y = static_cast<int>(std::min<int64_t>(want, (2 * a.Hkv + rows - 1) / rows));
  const cudaError_t e = timed(NVQ_KERNEL_KV_APPEND, stream, [&] {
    const dim3 grid(static_cast<unsigned>(groups), static_cast<unsigned>(y));
    return launch_pdl(D == 128 ? kv_append_kernel<128> : kv_append_kernel<64>, grid, dim3(kThreads),
                      0, stream, 1, a);
  });
  return e == cudaSuccess ? NVQ_OK : fail_cuda("kv append", e);
}

}  // namespace

}  // namespace nvq

extern "C" {

size_t nvfp4_kv_page_bytes(int Hkv, int D) {
  if (Hkv < 1 || (D != 64 && D != 128)) return 0;
  return static_cast<size_t>(Hkv) * nvq::record_bytes(D);
}

nvq_status nvfp4_kv_append(const void* k, int64_t ld_k, const void* v, int64_t ld_v, int64_t T,
                           int B, int Hkv, int D, const int32_t* cu_tokens,
                           const int32_t* seq_lens, const int32_t* page_table, int64_t ld_table,
                           int max_pages, void* pool, int64_t num_pages, nvq_stream_t stream) {
  using namespace nvq;
  if (T < 0 || B < 1 || Hkv < 1 || (cu_tokens == nullptr && T != B && T != 0))
    return NVQ_ERR_INVALID;
  nvq_status st = check_rows(k, ld_k, v, ld_v, Hkv, D, T);
  if (st != NVQ_OK || T == 0) return st;
  if ((reinterpret_cast<uintptr_t>(cu_tokens) & 3u) != 0) return NVQ_ERR_INVALID;
  st = check_kv(pool, num_pages, page_table, ld_table, max_pages, seq_lens);
  if (st != NVQ_OK) return st;
  return launch_append({static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), ld_k,
                        ld_v, T, B, Hkv, nullptr, cu_tokens, seq_lens, page_table, ld_table,
                        max_pages, static_cast<uint8_t*>(pool), num_pages, nullptr},
                       D, stream);
}

nvq_status nvfp4_kv_append_slots(const void* k, int64_t ld_k, const void* v, int64_t ld_v,
                                 int64_t T, int Hkv, int D, const int64_t* slots, void* pool,
                                 int64_t num_pages, nvq_stream_t stream) {
  using namespace nvq;
  if (T < 0 || Hkv < 1) return NVQ_ERR_INVALID;
  const nvq_status st = check_rows(k, ld_k, v, ld_v, Hkv, D, T);
  if (st != NVQ_OK || T == 0) return st;
  if (slots == nullptr || (reinterpret_cast<uintptr_t>(slots) & 7u) != 0 || pool == nullptr ||
      (reinterpret_cast<uintptr_t>(pool) & 15u) != 0 || num_pages < 1 || num_pages > 0x7FFFFFFF)
    return NVQ_ERR_INVALID;
  return launch_append({static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), ld_k,
                        ld_v, T, 0, Hkv, slots, nullptr, nullptr, nullptr, 0, 0,
                        static_cast<uint8_t*>(pool), num_pages, nullptr},
                       D, stream);
}

}  // extern "C"
