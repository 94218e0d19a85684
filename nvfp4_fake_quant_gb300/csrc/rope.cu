// Rotary positions of Q and K: element pairs (x1, x2) of a head turn by the angle
// a = position * inv_freq[pair],
//   y1 = mscale (x1 cos a - x2 sin a),   y2 = mscale (x1 sin a + x2 cos a);
// the gradient with respect to x is the rotation by -a.
//
// The angle.  Only its fraction of a turn matters: with f = inv_freq / 2 pi
// (turns per position, whole turns dropped) held as a 64-bit fixed-point
// fraction F = rint(f 2^64), position * F modulo 2^64 IS the fraction of the
// turn, exact but for F's own rounding.  fp32 products would be off by whole
// radians at far positions, fp64 sines cost more than the copy (the FP64 rate is
// a few operations per clock and SM).  F is formed once per block and pair, the
// sine and cosine once per (token, pair) and shared by all heads through shared
// memory; what is left is a copy of Q and K, bound by HBM.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "nvq_internal.h"

namespace nvq {

namespace {

constexpr int kMaxD = 256;
constexpr int kMaxTokens = 16;  // tokens per block
constexpr int kThreads = 256;

struct RopeTensor {
  const __nv_bfloat16* in;
  __nv_bfloat16* out;
  int64_t ld_in, ld_out;
};

struct RopeArgs {
  RopeTensor q, k;
  int Hq, heads;  // heads of q, of q and k
  int64_t T;
  int D, rot, tokens;  // tokens per block
  const int32_t* positions;
  int axes, end0, end1;  // pairs [0, end0) turn by axis 0, [end0, end1) by axis 1
  const double* inv_freq;
  float mscale, sign;
};

// (x1, x2) of one pair turned by (cos, sin).
__device__ __forceinline__ float2 turn(float x1, float x2, float c, float s) {
  return make_float2(fmaf(x1, c, -x2 * s), fmaf(x1, s, x2 * c));
}

__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A block takes a.tokens consecutive tokens, all heads.  The work item of a
// thread is 16 bytes of a head (interleaved: 4 whole pairs) or, in the half
// layout, the two 16-byte vectors that hold 8 pairs; the unrotated tail of a
// head is copied in 16-byte items.
template <bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a) {
  constexpr int kPairs = kInterleaved ? 4 : 8;  // pairs per item
  __shared__ uint64_t turns[kMaxD / 2];
  // cos and sin of (token, pair p = kPairs u + e) at float4 (e / 2) * units + u of
  // the token's part: the float4 loads of a warp, whose lanes take consecutive
  // items u, touch consecutive addresses
  __shared__ float4 cs4[kMaxTokens * kMaxD / 4];
  const int pairs = a.rot / 2, units = pairs / kPairs;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens;
  const int tokens = static_cast<int>(a.T - t0 < a.tokens ? a.T - t0 : a.tokens);
  for (int p = threadIdx.x; p < pairs; p += kThreads) {
    double f = a.inv_freq[p] * 0.15915494309189533577;  // 1 / (2 pi)
    f -= rint(f);
    turns[p] = static_cast<uint64_t>(__double2ll_rn(f * 18446744073709551616.0));  // 2^64
  }
  __syncthreads();
  for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
    const int tok = i / pairs, p = i - tok * pairs;
    const int axis = p < a.end0 ? 0 : (p < a.end1 ? 1 : 2);
    const int64_t pos = a.positions[(t0 + tok) * a.axes + axis];
    const uint64_t u = static_cast<uint64_t>(pos) * turns[p] + 0x80000000u;
    const float half_turns = static_cast<float>(static_cast<int32_t>(u >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(half_turns, &s, &c);
    float2* at = reinterpret_cast<float2*>(cs4 + tok * (pairs / 2));
    at[((p % kPairs) / 2 * units + p / kPairs) * 2 + (p & 1)] =
        make_float2(c * a.mscale, s * (a.mscale * a.sign));
  }
  __syncthreads();
  const int tail = (a.D - a.rot) / 8;  // 16-byte items copied behind the rotated ones
  const int per_head = units + tail, per_token = per_head * a.heads;
  for (int i = threadIdx.x; i < tokens * per_token; i += kThreads) {
    const int tok = i / per_token, r = i - tok * per_token;
    const int h = r / per_head, u = r - h * per_head;
    const bool is_q = h < a.Hq;
    const RopeTensor& x = is_q ? a.q : a.k;
    const int hh = is_q ? h : h - a.Hq;
    const __nv_bfloat16* src = x.in + (t0 + tok) * x.ld_in + hh * a.D;
    __nv_bfloat16* dst = x.out + (t0 + tok) * x.ld_out + hh * a.D;
    if (u >= units) {
      const int d = a.rot + (u - units) * 8;
      *reinterpret_cast<uint4*>(dst + d) = *reinterpret_cast<const uint4*>(src + d);
      continue;
    }
    const float4* cs = cs4 + tok * (pairs / 2) + u;
    if constexpr (kInterleaved) {
      const uint4 v = *reinterpret_cast<const uint4*>(src + 8 * u);
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 c = cs[e * units];
        const float2 y0 = turn(lo_f32(w[2 * e]), hi_f32(w[2 * e]), c.x, c.y);
        const float2 y1 = turn(lo_f32(w[2 * e + 1]), hi_f32(w[2 * e + 1]), c.z, c.w);
        w[2 * e] = pack(y0.x, y0.y);
        w[2 * e + 1] = pack(y1.x, y1.y);
      }
      *reinterpret_cast<uint4*>(dst + 8 * u) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      const uint4 v1 = *reinterpret_cast<const uint4*>(src + 8 * u);
      const uint4 v2 = *reinterpret_cast<const uint4*>(src + pairs + 8 * u);
      uint32_t w1[4] = {v1.x, v1.y, v1.z, v1.w}, w2[4] = {v2.x, v2.y, v2.z, v2.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 c = cs[e * units];
        const float2 y0 = turn(lo_f32(w1[e]), lo_f32(w2[e]), c.x, c.y);
        const float2 y1 = turn(hi_f32(w1[e]), hi_f32(w2[e]), c.z, c.w);
        w1[e] = pack(y0.x, y1.x);
        w2[e] = pack(y0.y, y1.y);
      }
      *reinterpret_cast<uint4*>(dst + 8 * u) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
      *reinterpret_cast<uint4*>(dst + pairs + 8 * u) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
    }
  }
}

bool bad_tensor(const void* in, int64_t ld_in, const void* out, int64_t ld_out, int H, int D) {
  const int64_t row = static_cast<int64_t>(H) * D;
  return in == nullptr || out == nullptr || (reinterpret_cast<uintptr_t>(in) & 15u) != 0 ||
         (reinterpret_cast<uintptr_t>(out) & 15u) != 0 || ld_in < row || ld_out < row ||
         ld_in % 8 != 0 || ld_out % 8 != 0 || (in == out && ld_in != ld_out);
}

}  // namespace

}  // namespace nvq

extern "C" nvq_status rope_apply(const void* q, int64_t ld_q, void* q_out, int64_t ld_qo, int Hq,
                                 const void* k, int64_t ld_k, void* k_out, int64_t ld_ko, int Hk,
                                 int64_t T, int D, int rot_dim, int interleaved,
                                 const int32_t* positions, int axes, const int* axis_pairs,
                                 const double* inv_freq, float mscale, int inverse,
                                 nvq_stream_t stream) {
  using namespace nvq;
  if (T < 0 || Hq < 1 || Hk < 0 || D < 16 || rot_dim < 16 || rot_dim > D) return NVQ_ERR_INVALID;
  if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1))
    return NVQ_ERR_INVALID;
  if (!(std::isfinite(mscale) && mscale > 0.f)) return NVQ_ERR_INVALID;
  if (D % 16 != 0 || D > kMaxD || rot_dim % 16 != 0) return NVQ_ERR_UNSUPPORTED;
  if (Hq > 65535 || Hk > 65535) return NVQ_ERR_UNSUPPORTED;
  if (axes < 1 || axes > 3 || axis_pairs == nullptr) return NVQ_ERR_INVALID;
  int64_t sum = 0;
  for (int i = 0; i < axes; ++i) {
    if (axis_pairs[i] < 0) return NVQ_ERR_INVALID;
    sum += axis_pairs[i];
  }
  if (sum != rot_dim / 2) return NVQ_ERR_INVALID;
  if (T == 0) return NVQ_OK;
  if (bad_tensor(q, ld_q, q_out, ld_qo, Hq, D) ||
      (Hk > 0 && bad_tensor(k, ld_k, k_out, ld_ko, Hk, D)))
    return NVQ_ERR_INVALID;
  if (positions == nullptr || (reinterpret_cast<uintptr_t>(positions) & 3u) != 0 ||
      inv_freq == nullptr || (reinterpret_cast<uintptr_t>(inv_freq) & 7u) != 0)
    return NVQ_ERR_INVALID;
  RopeArgs a{};
  a.q = {static_cast<const __nv_bfloat16*>(q), static_cast<__nv_bfloat16*>(q_out), ld_q, ld_qo};
  a.k = {static_cast<const __nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(k_out), ld_k, ld_ko};
  a.Hq = Hq;
  a.heads = Hq + Hk;
  a.T = T;
  a.D = D;
  a.rot = rot_dim;
  a.positions = positions;
  a.axes = axes;
  a.end0 = axis_pairs[0];
  a.end1 = a.end0 + (axes > 1 ? axis_pairs[1] : 0);
  a.inv_freq = inv_freq;
  a.mscale = mscale;
  a.sign = inverse ? -1.0f : 1.0f;
  // enough blocks for eight on every SM first, then more tokens per block
  a.tokens = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kMaxTokens, T / (152 * 8))));
  const int64_t blocks = (T + a.tokens - 1) / a.tokens;
  if (blocks > 0x7FFFFFFF) return NVQ_ERR_UNSUPPORTED;
  const cudaError_t e = timed(NVQ_KERNEL_VSA, stream, [&] {
    const dim3 grid(static_cast<unsigned>(blocks));
    if (interleaved)
      rope_kernel<true><<<grid, kThreads, 0, stream>>>(a);
    else
      rope_kernel<false><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
  });
  return e == cudaSuccess ? NVQ_OK : fail_cuda("rope", e);
}
