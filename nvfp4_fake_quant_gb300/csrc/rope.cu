// Rotary positions of Q and K: element pairs (x1, x2) of a head turn by the angle
// a = position * inv_freq[pair],
//   y1 = mscale (x1 cos a - x2 sin a),   y2 = mscale (x1 sin a + x2 cos a);
// the gradient with respect to x is the rotation by -a.
//
// The angle.  Only its fraction of a turn matters: with f = inv_freq / 2 pi
// (turns per position, whole turns dropped) held as a 64-bit fixed-point
// fraction F = rint(f 2^64), position * F modulo 2^64 IS the fraction of the
// turn, exact but for the roundings of f (fp64) and F; its upper 32 bits, rounded to fp32
// (2^-26 of a turn at most, at any position), go to the sine.  fp32 products would be off by
// whole radians at far positions, fp64 sines cost more than the copy (the FP64 rate is a few
// operations per clock and SM).  F is formed once per block and pair, the
// sine and cosine once per (token, pair) and shared by all heads through shared
// memory; what is left is a copy of Q and K, bound by HBM.
//
// Measured (calls in a CUDA graph): 25088 tokens of 12 + 12 heads of 128 54 us (half
// layout, one axis) and 56 us (interleaved, three axes), 85 and 81% of the copy rate;
// 32760 tokens of 12 + 12 heads, half of each head rotated, 72 us, 82%; 64 tokens of 32 +
// 8 heads 3 us, the latency of a launch and of the loads behind one another.  With few
// heads the sines are no longer shared by enough of them: 25088 tokens of 1 + 1 heads
// take 16 us (half layout) and 14 us (interleaved), 4 of them for the copy; of 8 + 1 heads
// 21 and 23, 17 of them.  The half layout spills 12 bytes at the cap of 64 registers that
// four blocks an SM leave.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "nvq_internal.h"
#include "nvq_ptx.cuh"

namespace nvq {

namespace {

constexpr int kMaxD = 256;
constexpr int kMaxTokens = 16;  // tokens per block
constexpr int kThreads = 256, kPerSm = 4;  // blocks per SM

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

// Blocks take groups of a.tokens consecutive tokens, all heads, in turn (one wave of
// blocks: F is formed once each).  The work item of a thread is 16 bytes of a head
// (interleaved: 4 whole pairs) or, in the half layout, the two 16-byte vectors that
// hold 8 pairs; the unrotated tail of a head is copied in 16-byte items.  A thread
// keeps its item of the head and walks over the group's (token, head) rows, four rows'
// loads in flight.
template <bool kInterleaved>
__global__ void __launch_bounds__(kThreads, kPerSm) rope_kernel(const RopeArgs a) {
  constexpr int kPairs = kInterleaved ? 4 : 8;  // pairs per item
  constexpr int kUnroll = 4;
  __shared__ uint64_t turns[kMaxD / 2];
  // cos and sin of (token, pair p = kPairs u + e) at float4 (e / 2) * units + u of
  // the token's part: the float4 loads of a warp, whose lanes take consecutive
  // items u, touch consecutive addresses
  __shared__ float4 cs4[kMaxTokens * kMaxD / 4];
  pdl_trigger();
  const int pairs = a.rot / 2, units = pairs / kPairs;
  const int per_head = units + (a.D - a.rot) / 8;      // items of a head
  const int rows_at_once = kThreads / per_head;        // rows of a pass
  const int row0 = threadIdx.x / per_head, u = threadIdx.x - row0 * per_head;
  const int first = u < units ? 8 * u : a.rot + (u - units) * 8;  // element of the head
  pdl_wait();
  for (int p = threadIdx.x; p < pairs; p += kThreads) {
    double f = a.inv_freq[p] * 0.15915494309189533577;  // 1 / (2 pi)
    f -= rint(f);
    turns[p] = static_cast<uint64_t>(__double2ll_rn(f * 18446744073709551616.0));  // 2^64
  }
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens; t0 < a.T;
       t0 += static_cast<int64_t>(gridDim.x) * a.tokens) {
    const int tokens = static_cast<int>(a.T - t0 < a.tokens ? a.T - t0 : a.tokens);
    __syncthreads();  // turns are there; the last group's cs4 has been read
    for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
      const int tok = i / pairs, p = i - tok * pairs;
      const int axis = p < a.end0 ? 0 : (p < a.end1 ? 1 : 2);
      const int64_t pos = a.positions[(t0 + tok) * a.axes + axis];
      const uint64_t turn = static_cast<uint64_t>(pos) * turns[p] + 0x80000000u;
      const float half_turns = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
      float s, c;
      sincospif(half_turns, &s, &c);
      float2* at = reinterpret_cast<float2*>(cs4 + tok * (pairs / 2));
      at[((p % kPairs) / 2 * units + p / kPairs) * 2 + (p & 1)] =
          make_float2(c * a.mscale, s * (a.mscale * a.sign));
    }
    __syncthreads();
    if (row0 >= rows_at_once) continue;  // threads left over
    const int rows = tokens * a.heads;
    int tok = row0 / a.heads, h = row0 - tok * a.heads;
    for (int r = row0; r < rows; r += kUnroll * rows_at_once) {
      uint4 v1[kUnroll], v2[kUnroll];
      __nv_bfloat16* dst[kUnroll];
      const float4* cs[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        if (r + i * rows_at_once < rows) {
          const bool is_q = h < a.Hq;
          const RopeTensor& x = is_q ? a.q : a.k;
          const int at = (is_q ? h : h - a.Hq) * a.D + first;
          const __nv_bfloat16* src = x.in + (t0 + tok) * x.ld_in + at;
          dst[i] = x.out + (t0 + tok) * x.ld_out + at;
          cs[i] = cs4 + tok * (pairs / 2) + u;
          v1[i] = ld16(src);
          if (!kInterleaved && u < units) v2[i] = ld16(src + pairs);
        }
        h += rows_at_once;
        while (h >= a.heads) {
          h -= a.heads;
          ++tok;
        }
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        if (r + i * rows_at_once >= rows) break;
        if (u < units) {
          uint32_t w1[4] = {v1[i].x, v1[i].y, v1[i].z, v1[i].w};
          if constexpr (kInterleaved) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float4 c = cs[i][e * units];
              const float2 y0 = turn(lo_f32(w1[2 * e]), hi_f32(w1[2 * e]), c.x, c.y);
              const float2 y1 = turn(lo_f32(w1[2 * e + 1]), hi_f32(w1[2 * e + 1]), c.z, c.w);
              w1[2 * e] = pack(y0.x, y0.y);
              w1[2 * e + 1] = pack(y1.x, y1.y);
            }
          } else {
            uint32_t w2[4] = {v2[i].x, v2[i].y, v2[i].z, v2[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 c = cs[i][e * units];
              const float2 y0 = turn(lo_f32(w1[e]), lo_f32(w2[e]), c.x, c.y);
              const float2 y1 = turn(hi_f32(w1[e]), hi_f32(w2[e]), c.z, c.w);
              w1[e] = pack(y0.x, y1.x);
              w2[e] = pack(y0.y, y1.y);
            }
            *reinterpret_cast<uint4*>(dst[i] + pairs) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
          }
          v1[i] = make_uint4(w1[0], w1[1], w1[2], w1[3]);
        }
        *reinterpret_cast<uint4*>(dst[i]) = v1[i];
      }
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
  // one wave of blocks; as few rounds of groups as kMaxTokens allows, all full
  const int64_t wave = static_cast<int64_t>(kPerSm) * device_sms();
  const int64_t rounds = (T + kMaxTokens * wave - 1) / (kMaxTokens * wave);
  a.tokens = static_cast<int>((T + rounds * wave - 1) / (rounds * wave));
  const int64_t groups = (T + a.tokens - 1) / a.tokens;
  const cudaError_t e = timed(NVQ_KERNEL_ROPE, stream, [&] {
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(groups, wave)));
    return launch_pdl(interleaved ? rope_kernel<true> : rope_kernel<false>, grid, dim3(kThreads), 0,
                      stream, 1, a);
  });
  return e == cudaSuccess ? NVQ_OK : fail_cuda("rope", e);
}
