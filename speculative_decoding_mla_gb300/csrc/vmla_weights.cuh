// A token's weight exp((x - max) / T) to about 2^-37, in whole units of 2^-45: sums of them are exact in
// any order.  Shared by the sampling and the beams' selection.
#pragma once

#include <cuda_runtime.h>

#include <cmath>

#include "vmla_device.cuh"

namespace vmla {
namespace weights {

constexpr float kOctaves = 46.f;             // weights below 2^-kOctaves count as zero
constexpr int kUnitBits = 45;                // weights in units of 2^-45
static_assert((uint64_t)VMLA_MAX_VOCAB << kUnitBits == 1ull << 63, "a sum of weights, times the root of two, fits 64 bits");

// 2^(k/64) as a pair of floats, filled by the host.
struct ExpTable {
  float2 t[64];
};

// The table, made at the first call (host).
inline const ExpTable& exp_table() {
  static const ExpTable table = [] {
    ExpTable t;
    for (int k = 0; k < 64; ++k) {
      const double v = std::exp2(k / 64.0);
      t.t[k].x = (float)v;
      t.t[k].y = (float)(v - (double)t.t[k].x);
    }
    return t;
  }();
  return table;
}

// Two floats in one instruction, each as by itself.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 sum2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 less2(float2 a, float2 b) { return fma2(b, both(-1.f), a); }  // a - b, rounded once

// log2(e) / temperature in two floats, and the row's maximum.
struct Exponent {
  float max, hi, lo;
};

// 2^-a, a = (max - x) c, in units of 2^-45, as high (2^-23) and low parts: value = high 2^22 + low.
// a = ph + pl in two floats; ph = n / 64 + r; 2^-a = 2^(-n/64) e^z with z = -(r + pl) ln 2, |z| < 2^-7.5,
// e^z - 1 = z + z^2 (1/2 + z (1/6 + z/24)) up to 2^-44 (z in two floats, zl below 2^-18: its square is
// left out); the table's factor times e^z in two floats.
__device__ __forceinline__ void weights_of(float2 x, const Exponent& e, const float2* table, int32_t (&high)[2],
                                           int32_t (&low)[2]) {
  const float2 mx = both(e.max), hi = both(e.hi);
  const float2 s = less2(mx, x);
  const float2 bb = less2(s, mx);
  const float2 err = less2(less2(mx, less2(s, bb)), sum2(x, bb));
  const float2 ph = mul2(s, hi);
  float2 pl = fma2(s, hi, mul2(s, both(-e.hi)));
  pl = fma2(s, both(e.lo), pl);
  pl = fma2(err, hi, pl);
  constexpr float kRound = 196608.f;  // 1.5 x 2^17: a sum with it is rounded to a multiple of 1/64
  const float2 t = sum2(ph, both(kRound));
  const int n[2] = {(int)(__float_as_uint(kRound) - __float_as_uint(t.x)),
                    (int)(__float_as_uint(kRound) - __float_as_uint(t.y))};
  const float2 r = less2(sum2(t, both(-kRound)), ph);  // (of the other sign)
  constexpr float kLn2Hi = 0.693147182464599609375f, kLn2Lo = -1.904654299957767e-9f;
  const float2 zh = mul2(r, both(kLn2Hi)), minus_zh = mul2(r, both(-kLn2Hi));
  float2 zl = fma2(r, both(kLn2Hi), minus_zh);
  zl = fma2(r, both(kLn2Lo), zl);
  zl = fma2(pl, both(-kLn2Hi), zl);
  const float2 p2 = fma2(zh, fma2(zh, both(1.f / 24), both(1.f / 6)), both(0.5f));
  const float2 q = fma2(mul2(zh, zh), p2, fma2(zh, zl, zl));
  const float2 sh = sum2(zh, q), sl = less2(q, sum2(sh, minus_zh));  // e^z - 1
  const float2 f0 = table[n[0] & 63], f1 = table[n[1] & 63];
  const float2 fx = make_float2(f0.x, f1.x), fy = make_float2(f0.y, f1.y);
  const float2 p = mul2(fx, sh);
  const float2 pe = fma2(fx, sh, mul2(p, both(-1.f)));
  const float2 rest = fma2(fy, sh, fma2(fx, sl, sum2(fy, pe)));
  const float2 wh = sum2(fx, p);
  const float2 wl = sum2(less2(p, less2(wh, fx)), rest);
  const float2 scale = make_float2(__uint_as_float((uint32_t)(127 + 23 + (n[0] >> 6)) << 23),   // 2^23 x 2^floor(-a)
                                   __uint_as_float((uint32_t)(127 + 23 + (n[1] >> 6)) << 23));
  constexpr float kWhole = 8388608.f, kHalf = 12582912.f;  // 2^23, 1.5 x 2^23
  const float2 hf = fma2(wh, scale, both(kWhole));
  const float2 res = fma2(wl, scale, fma2(wh, scale, less2(both(kWhole), hf)));
  const float2 lf = fma2(res, both(4194304.f), both(kHalf));
  // (no branch above: the weights of a thread's tokens are worked out side by side)
  const bool some0 = ph.x < kOctaves, some1 = ph.y < kOctaves;  // not where x is -inf
  high[0] = some0 ? (int)(__float_as_uint(hf.x) - __float_as_uint(kWhole)) : 0;
  high[1] = some1 ? (int)(__float_as_uint(hf.y) - __float_as_uint(kWhole)) : 0;
  low[0] = some0 ? (int)(__float_as_uint(lf.x) - __float_as_uint(kHalf)) : 0;
  low[1] = some1 ? (int)(__float_as_uint(lf.y) - __float_as_uint(kHalf)) : 0;
}
// One token's weight, by the same steps.
__device__ __forceinline__ void weight_of(float x, const Exponent& e, const float2* table, int32_t* high,
                                          int32_t* low) {
  int32_t h[2], l[2];
  weights_of(make_float2(x, e.max), e, table, h, l);
  *high = h[0], *low = l[0];
}

__device__ __forceinline__ uint64_t units(int64_t high, int64_t low) { return (uint64_t)((high << 22) + low); }

__device__ __forceinline__ uint64_t weight_units(float x, const Exponent& e, const float2* table) {
  int32_t h, l;
  weight_of(x, e, table, &h, &l);
  return units(h, l);
}

}  // namespace weights
}  // namespace vmla
