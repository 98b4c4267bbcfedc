// A cache row's rotated part and its 8-bit codes: what the two appends share.
#pragma once

#include <cuda_runtime.h>

#include "vmla_device.cuh"

namespace vmla {
namespace rope {

constexpr int kRopeDim = kDqk - kDv;  // 64
constexpr int kLatentU4 = kDv / 8;    // 64 granules of 16 bytes
constexpr int kHeadsPerPass = 8;      // heads a warp instruction covers (4 lanes each)

// cos and sin of the lane's eight pairs: those of granule g (first four when the pairs are
// neighbours) and of granule g + 4; with pairs (i, i + 32) granule g holds the a's of pairs
// 8g .. 8g + 7 and granule g + 4 their b's.
struct Angles {
  float c[8], s[8];
};

__device__ __forceinline__ Angles load_angles(const float* __restrict__ row, int g, bool neighbours) {
  const float4* t = reinterpret_cast<const float4*>(row);
  const int first = neighbours ? g : 2 * g, second = neighbours ? g + 4 : 2 * g + 1;
  Angles a;
  const float4 c0 = __ldg(t + first), c1 = __ldg(t + second), s0 = __ldg(t + 8 + first), s1 = __ldg(t + 8 + second);
  a.c[0] = c0.x; a.c[1] = c0.y; a.c[2] = c0.z; a.c[3] = c0.w;
  a.c[4] = c1.x; a.c[5] = c1.y; a.c[6] = c1.z; a.c[7] = c1.w;
  a.s[0] = s0.x; a.s[1] = s0.y; a.s[2] = s0.z; a.s[3] = s0.w;
  a.s[4] = s1.x; a.s[5] = s1.y; a.s[6] = s1.z; a.s[7] = s1.w;
  return a;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = bf16_lo(w[k]);
    x[2 * k + 1] = bf16_hi(w[k]);
  }
}

__device__ __forceinline__ void turn(float& x, float& y, float c, float s) {
  const float xr = fmaf(x, c, -(y * s)), yr = fmaf(x, s, y * c);
  x = xr;
  y = yr;
}

// The granules g (lo) and g + 4 (hi) of a 64-wide part, turned.
__device__ __forceinline__ void rotate(const uint4& vlo, const uint4& vhi, const Angles& a, bool neighbours,
                                       float (&lo)[8], float (&hi)[8]) {
  unpack8(vlo, lo);
  unpack8(vhi, hi);
  if (neighbours) {
#pragma unroll
    for (int k = 0; k < 4; ++k) turn(lo[2 * k], lo[2 * k + 1], a.c[k], a.s[k]);
#pragma unroll
    for (int k = 0; k < 4; ++k) turn(hi[2 * k], hi[2 * k + 1], a.c[4 + k], a.s[4 + k]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) turn(lo[k], hi[k], a.c[k], a.s[k]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// x / scale of two values, correctly rounded, given r = 1 / scale correctly rounded: the estimate x r is moved
// twice by the exact remainder times r (Markstein, IBM J. Res. Dev. 34, 1990).  For scales from 2^-60 to 2^60,
// where no remainder that a code could show falls below the smallest float; estimates that are not below 1024
// (infinities and NaN too) are left as they are, beyond the largest code.  (Remainders are taken as
// q scale - x, so that a zero keeps its sign.)
__device__ __forceinline__ float2 quotients(float2 x, float scale, float r) {
  float2 q0, q;
  asm("{.reg .b64 x, n, s, m, q, e;\n\tmov.b64 x, {%4, %5};\n\tmov.b64 s, {%6, %6};\n\tmov.b64 m, {%7, %7};\n\t"
      "mov.b64 q, {%8, %8};\n\tmul.rn.f32x2 q, x, q;\n\tmov.b64 {%0, %1}, q;\n\t"
      "mov.b64 n, {%9, %9};\n\tmul.rn.f32x2 n, x, n;\n\t"
      "fma.rn.f32x2 e, q, s, n;\n\tfma.rn.f32x2 q, e, m, q;\n\t"
      "fma.rn.f32x2 e, q, s, n;\n\tfma.rn.f32x2 q, e, m, q;\n\tmov.b64 {%2, %3}, q;}"
      : "=f"(q0.x), "=f"(q0.y), "=f"(q.x), "=f"(q.y)
      : "f"(x.x), "f"(x.y), "f"(scale), "f"(-r), "f"(r), "f"(-1.f));
  return make_float2(fabsf(q0.x) < 1024.f ? q.x : q0.x, fabsf(q0.y) < 1024.f ? q.y : q0.y);
}

// Eight values -> eight e4m3 codes of value / scale (nearest even, beyond 448 the largest code).
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float scale) {
  uint32_t w[4];
  const float r = __frcp_rn(scale);
  const bool usual = scale >= 0x1p-60f && scale <= 0x1p60f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 v = make_float2(x[2 * k], x[2 * k + 1]);
    const float2 q =
        usual ? quotients(v, scale, r) : make_float2(__fdiv_rn(v.x, scale), __fdiv_rn(v.y, scale));
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(q.y), "f"(q.x));
    w[k] = c;
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// The rotated parts of 8 kPasses heads (the part-th so many) of token t's queries, by one warp; row: the
// token's angles, read only if `use`.
template <int kPasses>
__device__ __forceinline__ void turn_heads(const AppendArgs& a, int64_t t, int part, int lane, bool use,
                                           const float* __restrict__ row) {
  // a head takes four lanes
  const int g = lane & 3, h0 = part * kHeadsPerPass * kPasses + (lane >> 2);
  const bool neighbours = a.neighbours != 0;
  uint4 v0[kPasses], v1[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int h = h0 + p * kHeadsPerPass;
    if (h < a.num_heads) {
      // (plain loads: q_rope may be the same memory as q's last columns, each element read and
      // written by one lane)
      const uint4* src = reinterpret_cast<const uint4*>(a.q_rope + t * a.q_rope_stride_t + h * a.q_rope_stride_h);
      v0[p] = src[g];
      v1[p] = src[g + 4];
    }
  }
  if (!use) return;
  const Angles ang = load_angles(row, g, neighbours);
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int h = h0 + p * kHeadsPerPass;
    if (h < a.num_heads) {
      float lo[8], hi[8];
      rotate(v0[p], v1[p], ang, neighbours, lo, hi);
      uint4* dst = reinterpret_cast<uint4*>(a.q + (t * a.num_heads + h) * kDqk + kDv);
      dst[g] = pack8(lo);
      dst[g + 4] = pack8(hi);
    }
  }
}

}  // namespace rope
}  // namespace vmla
