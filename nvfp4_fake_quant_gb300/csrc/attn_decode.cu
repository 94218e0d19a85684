// Attention of one new token per sequence over the paged NVFP4 cache:
//   S_j = scale q~ . K~_j,  o = sum_j exp(S_j - lse) V~_j,  lse = ln sum exp S_j
// over the visible keys.  One pass with the running maximum and sum.
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "nvq_internal.h"
#include "nvq_kv.cuh"
#include "nvq_quant.cuh"

namespace nvq {

namespace {

constexpr int kWarps = 8;
constexpr int kHeads = 8;  // query heads per block

struct DecodeArgs {
  const uint16_t* q;
  int64_t ld_q;
  const uint8_t* pool;
  int64_t num_pages;
  const int32_t* table;
  int64_t ld_table;
  int max_pages;
  const int32_t* lens;
  int H, Hkv;
  float scale;
  int window, sinks;
  __nv_bfloat16* o;
  float* lse;
  int* err;
};

__device__ __forceinline__ float4 codes4(uint32_t packed, float s) {
  uint32_t h[4];
  e2m1x8_to_f16x2(packed, h);
  return make_float4(f16lo_to_f32(h[0]) * s, f16hi_to_f32(h[0]) * s, f16lo_to_f32(h[1]) * s,
                     f16hi_to_f32(h[1]) * s);
}

// One block per sequence, KV head and group of kHeads query heads; warps take
// keys in turn, a lane D / 32 elements.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) decode_kernel(const DecodeArgs a) {
  constexpr int kE = D / 32;
  __shared__ float sq[kHeads][D];
  __shared__ float sm[kWarps][kHeads], sl[kWarps][kHeads];
  __shared__ float so[kWarps][kHeads][D];
  const int b = blockIdx.z, hk = blockIdx.y, G = a.H / a.Hkv;
  const int g0 = blockIdx.x * kHeads, ng = min(kHeads, G - g0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < ng * (D / 16); i += kWarps * 32) {
    const int g = i / (D / 16), c = i % (D / 16);
    const uint16_t* src = a.q + b * a.ld_q + static_cast<int64_t>(hk * G + g0 + g) * D + c * 16;
    uint32_t x[8];
    for (int j = 0; j < 8; ++j) x[j] = reinterpret_cast<const uint32_t*>(src)[j];
    const Q16 r = quant16_unit<true>(x);
    for (int j = 0; j < 8; ++j) {
      sq[g][c * 16 + 2 * j] = f16lo_to_f32(r.out[j]);
      sq[g][c * 16 + 2 * j + 1] = f16hi_to_f32(r.out[j]);
    }
  }
  __syncthreads();
  int len = max(a.lens[b], 0);
  if (len > static_cast<int64_t>(a.max_pages) * kPage) {
    if (threadIdx.x == 0) atomicMax(a.err, kErrTable);
    len = a.max_pages * kPage;
  }
  float m[kHeads], l[kHeads], acc[kHeads][kE];
  for (int g = 0; g < kHeads; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
    for (int e = 0; e < kE; ++e) acc[g][e] = 0.f;
  }
  for (int j = warp; j < len; j += kWarps) {
    if (a.window > 0 && j < len - a.window && j >= a.sinks) continue;
    const int page = a.table[b * a.ld_table + j / kPage];
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) atomicMax(a.err, kErrTable);
      continue;
    }
    const uint8_t* rec = a.pool + (static_cast<int64_t>(page) * a.Hkv + hk) * record_bytes(D);
    const int r = j % kPage, byte = r * (D / 2) + lane * kE / 2, sc = r * (D / 16) + lane * kE / 16;
    uint32_t kc, vc;
    if constexpr (kE == 4) {
      kc = *reinterpret_cast<const uint16_t*>(rec + byte);
      vc = *reinterpret_cast<const uint16_t*>(rec + v_codes_at(D) + byte);
    } else {
      kc = rec[byte];
      vc = rec[v_codes_at(D) + byte];
    }
    const float4 kv = codes4(kc, f16lo_to_f32(e4m3_to_f16x2(rec[k_scales_at(D) + sc])));
    const float4 vv = codes4(vc, f16lo_to_f32(e4m3_to_f16x2(rec[v_scales_at(D) + sc])));
    const float kk[4] = {kv.x, kv.y, kv.z, kv.w}, vx[4] = {vv.x, vv.y, vv.z, vv.w};
    for (int g = 0; g < kHeads; ++g) {
      if (g >= ng) break;
      float s = 0.f;
      for (int e = 0; e < kE; ++e) s += sq[g][lane * kE + e] * kk[e];
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
      s *= a.scale;
      const float mn = fmaxf(m[g], s), c = __expf(m[g] - mn), p = __expf(s - mn);
      m[g] = mn;
      l[g] = l[g] * c + p;
      for (int e = 0; e < kE; ++e) acc[g][e] = acc[g][e] * c + p * vx[e];
    }
  }
  for (int g = 0; g < kHeads; ++g) {
    if (lane == 0) {
      sm[warp][g] = m[g];
      sl[warp][g] = l[g];
    }
    for (int e = 0; e < kE; ++e) so[warp][g][lane * kE + e] = acc[g][e];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < ng * D; i += kWarps * 32) {
    const int g = i / D, d = i % D;
    float mx = -INFINITY, ls = 0.f, os = 0.f;
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm[w][g]);
    for (int w = 0; w < kWarps; ++w) {
      if (sl[w][g] == 0.f) continue;
      const float c = __expf(sm[w][g] - mx);
      ls += sl[w][g] * c;
      os += so[w][g][d] * c;
    }
    const int64_t row = static_cast<int64_t>(b) * a.H + hk * G + g0 + g;
    a.o[row * D + d] = __float2bfloat16_rn(ls > 0.f ? os / ls : 0.f);
    if (d == 0 && a.lse != nullptr) a.lse[row] = ls > 0.f ? mx + logf(ls) : -INFINITY;
  }
}

nvq_status check_decode(int B, int H, int Hkv, int D, int max_pages) {
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv != 0 || max_pages < 1 ||
      max_pages > 0x7FFFFFFF / kPage)
    return NVQ_ERR_INVALID;
  if (D != 64 && D != 128) return NVQ_ERR_UNSUPPORTED;
  if (B > 65535 || H > 65535) return NVQ_ERR_UNSUPPORTED;
  return NVQ_OK;
}

}  // namespace

}  // namespace nvq

extern "C" {

size_t attn_qat_decode_workspace(int B, int H, int Hkv, int D, int max_pages) {
  if (nvq::check_decode(B, H, Hkv, D, max_pages) != NVQ_OK) return 0;
  return 256;
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
  if (ws == nullptr || ws_bytes < attn_qat_decode_workspace(B, H, Hkv, D, max_pages) ||
      (reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
    return NVQ_ERR_WORKSPACE;
  int* err = device_error_word();
  if (err == nullptr) return NVQ_ERR_CUDA;
  const DecodeArgs a{static_cast<const uint16_t*>(q), ld_q, static_cast<const uint8_t*>(pool),
                     num_pages, page_table, ld_table, max_pages, seq_lens, H, Hkv, scale, window,
                     sinks, static_cast<__nv_bfloat16*>(o), lse, err};
  const cudaError_t e = timed(NVQ_KERNEL_ATTN_FWD, stream, [&] {
    const dim3 grid((H / Hkv + kHeads - 1) / kHeads, Hkv, B);
    if (D == 128)
      decode_kernel<128><<<grid, kWarps * 32, 0, stream>>>(a);
    else
      decode_kernel<64><<<grid, kWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
  });
  return e == cudaSuccess ? NVQ_OK : fail_cuda("attn decode", e);
}

}  // extern "C"
