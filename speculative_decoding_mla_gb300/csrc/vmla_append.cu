// Append of new tokens' rows to the latent pool, with the position rotation.
//
// A cache row is [latent (512) | rotated part (64)].  The model hands over the
// latent and the unrotated part of each new token; the 32 pairs (a, b) of the
// latter are turned by the token's position, with (c, s) = (cos, sin) of
// position x frequency from the caller's table:
//   (a, b) -> (a c - b s, a s + b c),
// pairs being (2i, 2i + 1) or (i, i + 32).  The query heads' rotated parts are
// turned by the same angles, so one launch serves both: the row goes to the
// token's slot (bf16, or e4m3 codes of value / scale), the queries into the
// last 64 columns of q.  Products and sums are fp32, rounded once at the store;
// quotients by the scale are correctly rounded, since a reciprocal's rounding
// would move values across code borders.
//
// A token costs 1152 bytes in, 256 of table, 1152 (or 576) out and 256 per
// head, and nothing is read twice, so the kernel is bound by memory for many
// tokens and by one chain of loads (slot and position, table, store) for few.
// One warp takes one token's row, or 16 or 32 of its heads: a lane holds the
// 16-byte granules g and g + 4 of a 64-wide part (g = lane & 3), which contain
// whole pairs in either pairing, and its 8 cosines and sines serve every head of
// the warp.  The data loads do not depend on the slot or the position and are
// issued with them.  32 heads (eight loads per lane in flight, 32 warps on an
// SM) pay off where there are many tokens of more than 16 heads: 16,384 x 64
// heads took 55.5 us against 57.5 with 16; 16,001 x 16 heads, e4m3, 28.9 against
// 26.0 us; 144 x 64 heads 4.2 against 3.8 us.  Blocks of four warps leave an SM
// in smaller steps than blocks of eight: 53.6 us (5.8 TB/s) against 55.4, and 5,000
// x 16 heads, e4m3, 8.7 against 10.2; of two warps, or 48 warps on an SM, gain
// nothing.  16,001 x 16 heads take 22.6 us in both types (4.7 and 4.3 TB/s), of which
// 10.4 to 12.4 are the cache rows'; rows two or four to a warp took longer.
#include <cuda_runtime.h>

#include "vmla_device.cuh"

namespace vmla {
namespace {

constexpr int kAppendWarps = 4;                               // of a block
constexpr int kHeadsPerPass = 8;                              // heads a warp instruction covers (4 lanes each)
constexpr int kRopeDim = kDqk - kDv;                          // 64
constexpr int kLatentU4 = kDv / 8;                            // 64 granules

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

// The granules g (lo) and g + 4 (hi) of a 64-wide part, turned.
__device__ __forceinline__ void rotate(const uint4& vlo, const uint4& vhi, const Angles& a, bool neighbours,
                                       float (&lo)[8], float (&hi)[8]) {
  unpack8(vlo, lo);
  unpack8(vhi, hi);
  auto turn = [](float& x, float& y, float c, float s) {
    const float xr = fmaf(x, c, -(y * s)), yr = fmaf(x, s, y * c);
    x = xr;
    y = yr;
  };
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

template <int kPasses>
__global__ void __launch_bounds__(kAppendWarps * 32, kPasses == 4 ? 8 : 10)
append_kernel(const AppendArgs a, int parts) {
  constexpr int kHeadsPerWarp = kHeadsPerPass * kPasses;
  const int lane = threadIdx.x & 31, g = lane & 3;
  const int64_t unit = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);  // warp-uniform
  const int64_t t = a.tokens * parts <= UINT32_MAX ? (int64_t)((uint32_t)unit / (uint32_t)parts) : unit / parts;
  const int part = (int)(unit - t * parts);  // 0: the cache row; p > 0: heads from (p - 1) kHeadsPerWarp on
  if (t >= a.tokens) return;
  const int32_t slot = __ldg(a.slots + t), pos = __ldg(a.positions + t);
  const bool neighbours = a.neighbours != 0;
  const bool use = slot >= 0 && (int64_t)slot < a.pool_slots && pos >= 0 && (int64_t)pos < a.table_rows;
  const float* row = a.cos_sin + (int64_t)(use ? pos : 0) * kRopeDim;
  if (part == 0) {
    const bool fp8 = a.kv_scale > 0.f;
    const uint4* lat = reinterpret_cast<const uint4*>(a.latent + t * a.latent_stride);
    const uint4* rope = reinterpret_cast<const uint4*>(a.k_rope + t * a.k_rope_stride);
    // e4m3: granules 2 lane, 2 lane + 1, the sources of code granule `lane`
    const uint4 v0 = __ldg(lat + (fp8 ? 2 * lane : lane)), v1 = __ldg(lat + (fp8 ? 2 * lane + 1 : lane + 32));
    uint4 r0 = make_uint4(0, 0, 0, 0), r1 = r0;
    if (lane < 4) {
      r0 = __ldg(rope + g);
      r1 = __ldg(rope + g + 4);
    }
    if (!use) {
      // -1 is padding; anything else out of range is reported and left out
      if (lane == 0 && slot != -1) record_status(a.status, VMLA_ERR_INDEX, (uint32_t)t);
      return;
    }
    float lo[8], hi[8];
    if (lane < 4) rotate(r0, r1, load_angles(row, g, neighbours), neighbours, lo, hi);
    if (fp8) {
      uint8_t* dst = reinterpret_cast<uint8_t*>(a.pool) + (int64_t)slot * kDqk;
      float x0[8], x1[8];
      unpack8(v0, x0);
      unpack8(v1, x1);
      const uint2 c0 = codes8(x0, a.kv_scale), c1 = codes8(x1, a.kv_scale);
      reinterpret_cast<uint4*>(dst)[lane] = make_uint4(c0.x, c0.y, c1.x, c1.y);
      if (lane < 4) {
        *reinterpret_cast<uint2*>(dst + kDv + 8 * g) = codes8(lo, a.kv_scale);
        *reinterpret_cast<uint2*>(dst + kDv + 8 * (g + 4)) = codes8(hi, a.kv_scale);
      }
    } else {
      uint4* dst = reinterpret_cast<uint4*>(a.pool) + (int64_t)slot * (kDqk / 8);
      dst[lane] = v0;
      dst[lane + 32] = v1;
      if (lane < 4) {
        dst[kLatentU4 + g] = pack8(lo);
        dst[kLatentU4 + g + 4] = pack8(hi);
      }
    }
    return;
  }
  // the queries' rotated parts: a head takes four lanes
  const int h0 = (part - 1) * kHeadsPerWarp + (lane >> 2);
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

}  // namespace

int launch_append(const AppendArgs& a, void* stream) {
  if (a.tokens == 0) return VMLA_OK;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) !=
                                                cudaSuccess)
    return VMLA_ERR_CUDA;
  // 32 heads per warp once they fill the SMs' warps twice over
  const bool wide = a.num_heads > 2 * kHeadsPerPass && a.tokens * ((a.num_heads + 31) / 32) >= (int64_t)sms * 64;
  const int heads = (wide ? 4 : 2) * kHeadsPerPass;
  const int parts = 1 + (a.num_heads + heads - 1) / heads;
  const int64_t blocks = (a.tokens * parts + kAppendWarps - 1) / kAppendWarps;
  if (blocks > INT32_MAX) return VMLA_ERR_SHAPE;
  const auto kernel = wide ? append_kernel<4> : append_kernel<2>;
  kernel<<<(unsigned)blocks, kAppendWarps * 32, 0, (cudaStream_t)stream>>>(a, parts);
  return cudaGetLastError() == cudaSuccess ? VMLA_OK : VMLA_ERR_CUDA;
}

}  // namespace vmla
