// Sampling of the target's tokens from the verified logits.
//
// For one row of logits x with temperature T > 0 the weight of token i is
//   w_i = exp((x_i - max x) / T),
// the tokens are ordered by value (descending, ties by index), top-k keeps the
// first k of that order, top-p the shortest prefix of what top-k leaves with at
// least p of its mass, min-p the tokens with w_i >= min_p.  All three keep
// prefixes of the one order, so what is kept is the shortest of them: the
// tokens above a value x*, and of those equal to it the ones up to an index.
// The token drawn is the smallest index i with
//   sum_{j <= i, kept} w_j > u sum_kept w_j.
//
// The result is a whole number, so the sums that decide it must not depend on
// the order of summation or on single precision: among 10^5 tokens a relative
// error of 2^-20 would move the draw in one row of ten.  A weight is computed in
// pairs of floats to about 2^-37 (weight_of) and added as a 64-bit integer in
// units of 2^-45; integer sums are exact in any order.  Weights below 2^-46 of
// the largest count as zero.
//
// One cluster of one to eight CTAs takes one row and keeps it in shared memory,
// so the logits are read from memory once; a thread only ever reads back its own
// elements until the last step.  Where a filter needs the order, the cut is
// found without sorting:
//   1. a histogram of counts over 44.5 buckets per factor of two in weight;
//      counts give top-k's bucket, and bounds of each bucket's mass bracket the
//      bucket of top-p's cut;
//   2. for top-p, one pass that adds the exact masses of all tokens and of those
//      above the bracket;
//   3. inside the bracket, histograms over 1024 equal ranges of the values' bit
//      patterns in their order (count, and exact mass for top-p), each narrowing the range to one
//      bucket, down to one value: one or two rounds, over the few tokens left.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cmath>
#include <mutex>

#include "vmla_device.cuh"

namespace vmla {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kChunkBytes = kThreads * 16;   // shared memory per iteration: 16 bytes per thread
constexpr int kMaxIters = 17;                // 8 x 17 x 2048 floats hold VMLA_MAX_VOCAB and a misaligned start
constexpr int kRoomyIters = 8;               // 64 KB: three CTAs per SM
constexpr int kBuckets = 2048;               // of the weight histogram; the last one holds what counts as zero
constexpr float kOctaves = 46.f;             // weights below 2^-kOctaves count as zero
constexpr int kRanges = 1024;                // of the bit-pattern histograms
constexpr int kUnitBits = 45;                // weights in units of 2^-45: 2^18 tokens' sum stays below 2^63
static_assert((int64_t)VMLA_MAX_VOCAB << kUnitBits <= INT64_MAX, "sums of weights fit 63 bits");
static_assert((int64_t)kMaxCluster * kMaxIters * (kChunkBytes / 4) >= VMLA_MAX_VOCAB + 3, "every vocabulary fits");
static_assert((1 << 23) / 1 * 1ll * kMaxIters * 8 < (1ll << 31), "a thread's sum of high parts fits 32 bits");

// 2^(k/64) as a pair of floats, filled by the host.
struct ExpTable {
  float2 t[64];
};

struct Shared {
  union {
    uint32_t hist[kBuckets];
    struct {
      uint32_t count[kRanges], mass_lo[kRanges], mass_hi[kRanges];
    } r;
  };
  float2 table[64];
  uint64_t warp_u64[kWarps], warp_u64b[kWarps];
  uint32_t warp_u32[kWarps];
  float warp_f[kWarps], warp_g[kWarps];
  // x_max, the sums, keys, count and index are read by the other CTAs of the cluster; each is written once per phase, with a cluster barrier
  // between a phase's reads and its slot's next write
  float x_max;
  float exp_hi, exp_lo;    // log2(e) / temperature (written and read within the CTA)
  double min_p_offset;     // temperature x ln(min_p)
  uint64_t sum_a, sum_b;
  uint32_t key_lo, key_hi, count;
  int32_t index;
  // results of a search, the same in every CTA
  int32_t bucket_k, bucket_first, bucket_last;
  uint32_t before_k;
  int32_t range;
  uint32_t range_before, range_count;
  uint64_t range_mass_before;
  uint64_t chunk[kMaxIters];
};

// Whole numbers in the order of the values, without the low bits that a type's values never use.
template <int kLowBits>
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // one zero
  return (b & 0x80000000u ? ~b : b | 0x80000000u) >> kLowBits;
}
template <int kLowBits>
__device__ __forceinline__ float order_value(uint32_t key) {
  const uint32_t k = key << kLowBits;
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~(k | ((1u << kLowBits) - 1u)));
}

// log2(e) / temperature in two floats, and the row's maximum.
struct Exponent {
  float max, hi, lo;
};

// 2^-a, a = (max - x) c, in units of 2^-45, as high (2^-23) and low parts: value = high 2^22 + low.
// a = ph + pl in two floats; ph = n / 64 + r; 2^-a = 2^(-n/64) e^z with z = -(r + pl) ln 2, |z| < 2^-7.5,
// e^z - 1 = z + z^2 (1/2 + z (1/6 + z/24)) up to 2^-44 (z in two floats, zl below 2^-18: its square is
// left out); the table's factor times e^z in two floats.
__device__ __forceinline__ void weight_of(float x, const Exponent& e, const float2* table, int32_t* high,
                                          int32_t* low) {
  const float s = __fsub_rn(e.max, x);
  const float bb = __fsub_rn(s, e.max);
  const float err = __fsub_rn(__fsub_rn(e.max, __fsub_rn(s, bb)), __fadd_rn(x, bb));
  const float ph = __fmul_rn(s, e.hi);
  *high = *low = 0;
  if (!(ph < kOctaves)) return;  // also where x is -inf
  float pl = __fmaf_rn(s, e.hi, -ph);
  pl = __fmaf_rn(s, e.lo, pl);
  pl = __fmaf_rn(err, e.hi, pl);
  constexpr float kRound = 196608.f;  // 1.5 x 2^17: a sum with it is rounded to a multiple of 1/64
  const float t = __fadd_rn(ph, kRound);
  const int n = -(int)(__float_as_uint(t) - __float_as_uint(kRound));
  const float r = __fsub_rn(ph, __fsub_rn(t, kRound));
  constexpr float kLn2Hi = 0.693147182464599609375f, kLn2Lo = -1.904654299957767e-9f;
  const float zh = __fmul_rn(-r, kLn2Hi);
  float zl = __fmaf_rn(-r, kLn2Hi, -zh);
  zl = __fmaf_rn(-r, kLn2Lo, zl);
  zl = __fmaf_rn(-pl, kLn2Hi, zl);
  const float p2 = __fmaf_rn(zh, __fmaf_rn(zh, 1.f / 24, 1.f / 6), 0.5f);
  const float q = __fmaf_rn(__fmul_rn(zh, zh), p2, __fmaf_rn(zh, zl, zl));
  const float sh = __fadd_rn(zh, q), sl = __fsub_rn(q, __fsub_rn(sh, zh));  // e^z - 1
  const float2 f = table[n & 63];
  const float p = __fmul_rn(f.x, sh);
  const float pe = __fmaf_rn(f.x, sh, -p);
  const float rest = __fmaf_rn(f.y, sh, __fmaf_rn(f.x, sl, __fadd_rn(f.y, pe)));
  const float wh = __fadd_rn(f.x, p);
  const float wl = __fadd_rn(__fsub_rn(p, __fsub_rn(wh, f.x)), rest);
  const float scale = __uint_as_float((uint32_t)(127 + 23 + (n >> 6)) << 23);  // 2^23 x 2^floor(-a)
  constexpr float kWhole = 8388608.f, kHalf = 12582912.f;                      // 2^23, 1.5 x 2^23
  const float hf = __fmaf_rn(wh, scale, kWhole);
  const float res = __fmaf_rn(wl, scale, __fmaf_rn(wh, scale, -__fsub_rn(hf, kWhole)));
  const float lf = __fmaf_rn(res, 4194304.f, kHalf);
  *high = (int)(__float_as_uint(hf) - __float_as_uint(kWhole));
  *low = (int)(__float_as_uint(lf) - __float_as_uint(kHalf));
}

__device__ __forceinline__ uint64_t units(int64_t high, int64_t low) { return (uint64_t)((high << 22) + low); }

__device__ __forceinline__ uint64_t weight_units(float x, const Exponent& e, const float2* table) {
  int32_t h, l;
  weight_of(x, e, table, &h, &l);
  return units(h, l);
}

template <typename V>
__device__ __forceinline__ V warp_add(V v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <typename V>
__device__ __forceinline__ V warp_scan(V v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
// Exclusive prefix of v over the block's threads, and the total; `buf` holds kWarps values.
template <typename V>
__device__ __forceinline__ V block_scan(V v, V* buf, V* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const V inc = warp_scan(v, lane);
  __syncthreads();  // earlier readers of buf are done
  if (lane == 31) buf[warp] = inc;
  __syncthreads();
  V before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const V x = buf[w];
    if (w < warp) before += x;
    all += x;
  }
  *total = all;
  return before + inc - v;
}
template <typename V>
__device__ __forceinline__ V block_add(V v, V* buf) {
  V total;
  block_scan(v, buf, &total);
  return total;
}

template <typename T>
struct Elems;
template <>
struct Elems<float> {
  static constexpr int kVec = 4;
  static constexpr int kLowBits = 0;  // low bits of the fp32 pattern that are always zero
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <>
struct Elems<uint16_t> {  // bf16
  static constexpr int kVec = 8;
  static constexpr int kLowBits = 16;
  static __device__ __forceinline__ float one(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) x[2 * k] = bf16_lo(w[k]), x[2 * k + 1] = bf16_hi(w[k]);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {  // of bf16 values: exact
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
  }
};

// One row on one cluster.  Element v of the "shifted" row is token v - shift, shift being the
// elements between the row's start and the 16-byte boundary below it, so that whole granules load
// as vectors whatever the row's alignment; places outside the row read as -inf.  CTA r holds
// places [r S, (r + 1) S), its warp w the w-th of kWarps equal runs of them.
template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
sample_kernel(const SampleArgs a, const __grid_constant__ ExpTable exp_table, int iters) {
  using E = Elems<T>;
  constexpr int kVec = E::kVec;
  constexpr int kStep = 32 * kVec;  // places of one warp iteration
  extern __shared__ __align__(16) uint8_t slice_raw[];
  __shared__ Shared sm;
  const cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = (int64_t)blockIdx.x / C;
  const T* src = static_cast<const T*>(a.logits) + row * a.stride;
  const int shift = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
  const T* base = src - shift;
  const int end = a.vocab + shift;  // places [shift, end) are tokens
  const int seg = iters * kStep;    // a warp's places
  const int first = (rank * kWarps + warp) * seg;
  uint4* mine = reinterpret_cast<uint4*>(slice_raw) + (size_t)warp * iters * 32 + lane;  // granule of iteration i: mine[32 i]

  // settings; a row with a bad one draws nothing
  const float temp = a.temperature ? __ldg(a.temperature + row) : 1.f;
  const int top_k = a.top_k ? __ldg(a.top_k + row) : 0;
  const float top_p = a.top_p ? __ldg(a.top_p + row) : 1.f;
  const float min_p = a.min_p ? __ldg(a.min_p + row) : 0.f;
  const float u = __ldg(a.uniform + row);
  const bool good = (temp == 0.f || (temp >= kSampleMinTemp && temp <= kSampleMaxTemp)) && top_p > 0.f &&
                    top_p <= 1.f && min_p >= 0.f && min_p <= 1.f && u >= 0.f && u <= 1.f;
  if (!good) {  // the same in every thread of the cluster
    if (rank == 0 && tid == 0) {
      record_status(a.status, VMLA_ERR_PARAM, (uint32_t)row);
      a.token[row] = -1;
    }
    return;
  }

  if (tid == 0 && temp > 0.f) {
    // one thread: 64-bit arithmetic is some 60 times slower than 32-bit here
    const double c = 1.4426950408889634 / (double)temp;
    sm.exp_hi = (float)c;
    sm.exp_lo = (float)(c - (double)sm.exp_hi);
    sm.min_p_offset = min_p > 0.f && min_p < 1.f ? (double)temp * log((double)min_p) : 0.0;
  }
  // ---- the row into shared memory, and its maximum
  float mx = -INFINITY;
  constexpr int kFlight = 4;
  for (int i0 = 0; i0 < iters; i0 += kFlight) {
    uint4 v[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int p = first + (i0 + f) * kStep + lane * kVec;
      if (i0 + f < iters) {
        if (p >= shift && p + kVec <= end) {
          asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(v[f].x), "=r"(v[f].y), "=r"(v[f].z), "=r"(v[f].w)
                       : "l"(base + p));
        } else {
          float x[kVec];
#pragma unroll
          for (int k = 0; k < kVec; ++k) x[k] = p + k >= shift && p + k < end ? E::one(base + p + k) : -INFINITY;
          v[f] = E::pack(x);
        }
      }
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      if (i0 + f < iters) {
        float x[kVec];
        E::unpack(v[f], x);
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
          x[k] = fmaxf(x[k], -INFINITY);  // NaN counts as -inf
          mx = fmaxf(mx, x[k]);
        }
        mine[32 * (i0 + f)] = E::pack(x);
      }
    }
  }
  if (tid < 64) sm.table[tid] = exp_table.t[tid];
  mx = warp_max(mx);
  if (lane == 0) sm.warp_f[warp] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm.warp_f[w]);
  if (tid == 0) sm.x_max = mx;
  cluster.sync();
  for (int r = 0; r < C; ++r) mx = fmaxf(mx, *cluster.map_shared_rank(&sm.x_max, r));

  // f(x, place) for every element of this thread
  auto each = [&](auto&& f) {
#pragma unroll 1
    for (int i = 0; i < iters; ++i) {
      float x[kVec];
      E::unpack(mine[32 * i], x);
      const int p = first + i * kStep + lane * kVec;
#pragma unroll
      for (int k = 0; k < kVec; ++k) f(x[k], p + k);
    }
  };

  if (temp == 0.f || mx == -INFINITY) {
    // the first token of the largest value; none where every logit is -inf or NaN
    int at = INT32_MAX;
    if (mx != -INFINITY) each([&](float x, int p) { at = x == mx && p < at ? p : at; });
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == 0) sm.warp_u32[warp] = (uint32_t)at;
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < kWarps; ++w) at = min(at, (int)sm.warp_u32[w]);
      sm.index = at;
    }
    cluster.sync();
    if (rank == 0 && tid == 0) {
      for (int r = 0; r < C; ++r) at = min(at, *cluster.map_shared_rank(&sm.index, r));
      a.token[row] = at == INT32_MAX ? -1 : at - shift;
    }
    cluster.sync();
    return;
  }
  if (mx == INFINITY) {
    // tokens at +inf share the draw evenly: they become 0, all others -inf
#pragma unroll 1
    for (int i = 0; i < iters; ++i) {
      float x[kVec];
      E::unpack(mine[32 * i], x);
#pragma unroll
      for (int k = 0; k < kVec; ++k) x[k] = x[k] == INFINITY ? 0.f : -INFINITY;
      mine[32 * i] = E::pack(x);
    }
    mx = 0.f;
  }
  const Exponent ex = {mx, sm.exp_hi, sm.exp_lo};
  const float per_octave = (kBuckets - 2) / kOctaves;
  const float to_bucket = ex.hi * per_octave;
  auto bucket_of = [&](float x) {  // non-increasing in x; kBuckets - 1: counts as zero
    const float b = (mx - x) * to_bucket;
    return b < (float)(kBuckets - 1) ? (int)b : kBuckets - 1;
  };

  // ---- what is kept: x > cut_x, and x == cut_x up to place cut_place
  float cut_x = -INFINITY;
  int cut_place = INT32_MAX;
  uint32_t cut_keep = 0, cut_equal = 0;  // of the tokens equal to cut_x, the first cut_keep of cut_equal
  bool with_k = top_k > 0 && top_k < a.vocab;
  bool with_p = top_p < 1.f;
  if (with_k || with_p) {
    for (int b = tid; b < kBuckets; b += kThreads) sm.hist[b] = 0;
    __syncthreads();
    each([&](float x, int) {
      const int b = bucket_of(x);
      if (b < kBuckets - 1) atomicAdd(&sm.hist[b], 1u);
    });
    if (tid == 0) sm.bucket_k = -1, sm.bucket_first = sm.bucket_last = kBuckets - 1;
    cluster.sync();
    constexpr int kOwn = kBuckets / kThreads;
    uint32_t n[kOwn], mine_n = 0;
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      n[j] = 0;
      for (int r = 0; r < C; ++r) n[j] += cluster.map_shared_rank(sm.hist, r)[kOwn * tid + j];
      mine_n += n[j];
    }
    uint32_t total;
    uint32_t before = block_scan(mine_n, sm.warp_u32, &total);
    if (with_k && (uint32_t)top_k >= total) with_k = false;  // nothing of weight is past the k-th
    if (with_k) {
      uint32_t at = before;
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        if (at < (uint32_t)top_k && at + n[j] >= (uint32_t)top_k) sm.bucket_k = kOwn * tid + j, sm.before_k = at;
        at += n[j];
      }
    }
    if (with_p) {
      // bounds of the mass up to each bucket, of what top-k leaves; 10^-3 covers the rounding of
      // bounds, sums and bucket borders
      float lo[kOwn], hi[kOwn], sum_lo = 0.f, sum_hi = 0.f;
      uint32_t at = before;
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        const uint32_t left = with_k ? (at < (uint32_t)top_k ? (uint32_t)top_k - at : 0u) : UINT32_MAX;
        const float m = (float)(n[j] < left ? n[j] : left);
        const float b = (float)(kOwn * tid + j);
        lo[j] = m * ex2_approx(-(b + 1.f) / per_octave) * 0.999f;
        hi[j] = m * ex2_approx(-b / per_octave) * 1.001f;
        sum_lo += lo[j];
        sum_hi += hi[j];
        at += n[j];
      }
      float all_lo, all_hi;
      float cum_lo = block_scan(sum_lo, sm.warp_f, &all_lo), cum_hi = block_scan(sum_hi, sm.warp_g, &all_hi);
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        cum_lo += lo[j];
        cum_hi += hi[j];
        if (cum_hi >= top_p * all_lo * 0.999f) atomicMin(&sm.bucket_first, kOwn * tid + j);
        if (cum_lo >= top_p * all_hi * 1.001f) atomicMin(&sm.bucket_last, kOwn * tid + j);
      }
    }
    __syncthreads();
    cluster.sync();  // the histograms have been read

    // The value at which a running count (or mass) over the tokens with bucket in [b_lo, b_hi] and
    // pattern at or above `floor_key`, in descending order, reaches `target`: its pattern, the
    // count and mass before it, and how many tokens have it.
    auto refine = [&](int b_lo, int b_hi, uint32_t floor_key, bool by_mass, uint64_t target, uint32_t* key,
                      uint32_t* equal, uint64_t* left) {
      uint32_t klo = UINT32_MAX, khi = 0;
      each([&](float x, int) {
        const int b = bucket_of(x);
        const uint32_t k = order_key<E::kLowBits>(x);
        if (b >= b_lo && b <= b_hi && b < kBuckets - 1 && k >= floor_key) klo = min(klo, k), khi = max(khi, k);
      });
      klo = __reduce_min_sync(0xffffffffu, klo);
      khi = __reduce_max_sync(0xffffffffu, khi);
      if (tid == 0) sm.key_lo = UINT32_MAX, sm.key_hi = 0;
      __syncthreads();
      if (lane == 0) atomicMin(&sm.key_lo, klo), atomicMax(&sm.key_hi, khi);
      cluster.sync();
      for (int r = 0; r < C; ++r) {
        klo = min(klo, *cluster.map_shared_rank(&sm.key_lo, r));
        khi = max(khi, *cluster.map_shared_rank(&sm.key_hi, r));
      }
      // (a round leaves 10 bits fewer: 32, 22, 12, 2)
      for (int round = 0; round < 4; ++round) {
        // ranges of equal width, a power of two
        int width = 32 - __clz((khi - klo) | 1) - 10;
        width = width < 0 ? 0 : width;
        for (int b = tid; b < kRanges; b += kThreads) sm.r.count[b] = sm.r.mass_lo[b] = sm.r.mass_hi[b] = 0;
        __syncthreads();
        each([&](float x, int) {
          const uint32_t k = order_key<E::kLowBits>(x);
          if (k >= klo && k <= khi) {
            const uint32_t g = (k - klo) >> width;
            atomicAdd(&sm.r.count[g], 1u);
            if (by_mass) {
              const uint64_t w = weight_units(x, ex, sm.table);
              const uint32_t wl = (uint32_t)w, old = atomicAdd(&sm.r.mass_lo[g], wl);
              atomicAdd(&sm.r.mass_hi[g], (uint32_t)(w >> 32) + (old + wl < old ? 1u : 0u));
            }
          }
        });
        cluster.sync();
        constexpr int kPer = kRanges / kThreads;
        uint32_t n2[kPer], sum_n = 0;
        uint64_t m2[kPer], sum_m = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int g = kRanges - 1 - (kPer * tid + j);  // descending
          n2[j] = 0, m2[j] = 0;
          for (int r = 0; r < C; ++r) {
            const Shared* o = cluster.map_shared_rank(&sm, r);
            n2[j] += o->r.count[g];
            if (by_mass) m2[j] += ((uint64_t)o->r.mass_hi[g] << 32) + o->r.mass_lo[g];
          }
          sum_n += n2[j], sum_m += m2[j];
        }
        uint32_t all_n;
        uint64_t all_m = 0, cum_m = 0;
        uint32_t cum_n = block_scan(sum_n, sm.warp_u32, &all_n);
        if (by_mass) cum_m = block_scan(sum_m, sm.warp_u64, &all_m);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const uint64_t was = by_mass ? cum_m : cum_n;
          cum_n += n2[j], cum_m += m2[j];
          const uint64_t now = by_mass ? cum_m : cum_n;
          if (was < target && now >= target) {  // one range of one thread
            sm.range = kRanges - 1 - (kPer * tid + j);
            sm.range_count = n2[j];
            sm.range_mass_before = was;
          }
        }
        __syncthreads();
        target -= sm.range_mass_before;
        const uint32_t lo2 = klo + ((uint32_t)sm.range << width);
        const uint32_t hi2 = lo2 + ((1u << width) - 1u);
        *equal = sm.range_count;
        klo = lo2;
        khi = hi2 < khi ? hi2 : khi;
        cluster.sync();  // the histograms have been read
        if (width == 0) break;
      }
      *key = klo;
      *left = target;
    };

    uint32_t floor_key = 0;
    if (with_k) {
      uint64_t left;
      refine(sm.bucket_k, sm.bucket_k, 0, false, (uint64_t)top_k - sm.before_k, &floor_key, &cut_equal, &left);
      cut_x = order_value<E::kLowBits>(floor_key);
      cut_keep = (uint32_t)left;
    }
    if (with_p) {
      // exact masses of what top-k leaves: all of it, and the part above the bracket
      const int b_lo = sm.bucket_first, b_hi = sm.bucket_last;
      uint32_t all_h = 0, top_h = 0;
      int32_t all_l = 0, top_l = 0;
      each([&](float x, int) {
        if (x > cut_x) {
          int32_t h, l;
          weight_of(x, ex, sm.table, &h, &l);
          all_h += h, all_l += l;
          if (bucket_of(x) < b_lo) top_h += h, top_l += l;
        }
      });
      uint64_t all = warp_add(units(all_h, all_l)), top = warp_add(units(top_h, top_l));
      if (lane == 0) sm.warp_u64[warp] = all, sm.warp_u64b[warp] = top;
      __syncthreads();
      if (tid == 0) {
        all = top = 0;
        for (int w = 0; w < kWarps; ++w) all += sm.warp_u64[w], top += sm.warp_u64b[w];
        sm.sum_a = all, sm.sum_b = top;
      }
      cluster.sync();
      all = with_k ? (uint64_t)cut_keep * weight_units(cut_x, ex, sm.table) : 0, top = 0;
      for (int r = 0; r < C; ++r)
        all += *cluster.map_shared_rank(&sm.sum_a, r), top += *cluster.map_shared_rank(&sm.sum_b, r);
      // the least mass that reaches p of all: p has 24 bits, so p 2^64 is whole for p >= 2^-40
      const uint64_t p64 = (uint64_t)(top_p * 18446744073709551616.f);
      uint64_t target = __umul64hi(p64, all) + (p64 * all != 0 ? 1 : 0);
      target = target > top ? target - top : 1;
      uint32_t key, equal;
      uint64_t left;
      refine(b_lo, b_hi, floor_key, true, target, &key, &equal, &left);
      const float x = order_value<E::kLowBits>(key);
      const uint64_t w = weight_units(x, ex, sm.table);
      uint32_t keep = w > 0 ? (uint32_t)min((left + w - 1) / w, (uint64_t)equal) : equal;
      if (with_k && x == cut_x) {
        cut_keep = min(cut_keep, keep);
      } else {
        cut_x = x, cut_keep = keep, cut_equal = equal;
      }
    }
  }
  if (min_p > 0.f) {
    // w >= min_p  <=>  x >= max + T ln(min_p)
    const float x = __double2float_ru((double)mx + sm.min_p_offset);
    if (x > cut_x) cut_x = x, cut_keep = cut_equal = 0;
  }
  if (cut_keep < cut_equal) {
    // the place of the cut_keep-th token equal to cut_x, in the order of the places
    uint32_t here = 0;
    each([&](float x, int) { here += x == cut_x ? 1u : 0u; });
    here = warp_add(here);
    if (lane == 0) sm.warp_u32[warp] = here;
    __syncthreads();
    uint32_t block = 0, skip = 0;
    for (int w = 0; w < kWarps; ++w) {
      block += sm.warp_u32[w];
      if (w < warp) skip += sm.warp_u32[w];
    }
    if (tid == 0) sm.count = block;
    cluster.sync();
    for (int r = 0; r < rank; ++r) skip += *cluster.map_shared_rank(&sm.count, r);
    if (skip < cut_keep && skip + here >= cut_keep) {  // one warp of the cluster
      for (int i = 0; i < iters; ++i) {
        float x[kVec];
        E::unpack(mine[32 * i], x);
        uint32_t own = 0;
#pragma unroll
        for (int k = 0; k < kVec; ++k) own += x[k] == cut_x ? 1u : 0u;
        const uint32_t inc = warp_scan(own, lane);
        uint32_t at = skip + inc - own;
        if (at < cut_keep && at + own >= cut_keep) {
#pragma unroll
          for (int k = 0; k < kVec; ++k) {
            if (x[k] == cut_x && ++at == cut_keep)
              for (int r = 0; r < C; ++r) *cluster.map_shared_rank(&sm.index, r) = first + i * kStep + lane * kVec + k;
          }
        }
        skip += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
    cluster.sync();
    cut_place = sm.index;
  }

  // ---- the draw, in the order of the places
  auto kept_units = [&](float x, int p) {
    return x > cut_x || (x == cut_x && p <= cut_place) ? weight_units(x, ex, sm.table) : 0ull;
  };
  uint32_t sum_h = 0;
  int32_t sum_l = 0;
  each([&](float x, int p) {
    if (x > cut_x || (x == cut_x && p <= cut_place)) {
      int32_t h, l;
      weight_of(x, ex, sm.table, &h, &l);
      sum_h += h, sum_l += l;
    }
  });
  uint64_t sum = warp_add(units(sum_h, sum_l));
  __syncthreads();
  if (lane == 0) sm.warp_u64[warp] = sum;
  __syncthreads();
  uint64_t block = 0;
  for (int w = 0; w < kWarps; ++w) block += sm.warp_u64[w];
  if (tid == 0) sm.sum_a = block;
  cluster.sync();
  uint64_t all = 0, before = 0;
  for (int r = 0; r < C; ++r) {
    const uint64_t s = *cluster.map_shared_rank(&sm.sum_a, r);
    if (r < rank) before += s;
    all += s;
  }
  // the token's running sum is the first above `goal` = floor(u all)
  const uint64_t goal = u < 1.f ? __umul64hi((uint64_t)(u * 18446744073709551616.f), all) : all - 1;
  if (before <= goal && goal < before + block) {  // one CTA of the cluster
    int w0 = 0;
    while (w0 < kWarps - 1 && before + sm.warp_u64[w0] <= goal) before += sm.warp_u64[w0++];
    // that warp's places, one iteration's per warp of this CTA
    const uint4* theirs = reinterpret_cast<const uint4*>(slice_raw) + (size_t)w0 * iters * 32 + lane;
    const int start = (rank * kWarps + w0) * seg + lane * kVec;
    for (int i = warp; i < iters; i += kWarps) {
      float x[kVec];
      E::unpack(theirs[32 * i], x);
      uint64_t s = 0;
#pragma unroll 1
      for (int k = 0; k < kVec; ++k) s += kept_units(x[k], start + i * kStep + k);
      s = warp_add(s);
      if (lane == 0) sm.chunk[i] = s;
    }
    __syncthreads();
    if (warp == 0) {
      int i = 0;
      while (i < iters - 1 && before + sm.chunk[i] <= goal) before += sm.chunk[i++];
      float x[kVec];
      uint64_t s = 0, w[kVec];
      E::unpack(theirs[32 * i], x);
#pragma unroll
      for (int k = 0; k < kVec; ++k) s += w[k] = kept_units(x[k], start + i * kStep + k);
      uint64_t at = before + warp_scan(s, lane) - s;
      if (at <= goal && goal < at + s) {
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
          if (at <= goal && goal < at + w[k]) a.token[row] = start + i * kStep + k - shift;
          at += w[k];
        }
      }
    }
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
}

// CTAs per row: the smallest power of two whose slice leaves room for three CTAs on an SM (or the
// largest cluster), then more while the rows leave SMs idle.
template <typename T>
int choose_cluster(int64_t rows, int vocab, int sms, int* iters) {
  const int64_t places = (int64_t)vocab + Elems<T>::kVec - 1;
  auto need = [&](int c) {
    const int64_t per = (int64_t)c * (kChunkBytes / sizeof(T));
    return (int)((places + per - 1) / per);
  };
  int c = 1;
  while (c < kMaxCluster && need(c) > kRoomyIters) c *= 2;
  while (c < kMaxCluster && rows * c * 2 <= sms && need(c) > 1) c *= 2;
  *iters = need(c);
  return c;
}

template <typename T>
int launch(const SampleArgs& a, int sms, int dev, cudaStream_t stream) {
  static const ExpTable table = [] {
    ExpTable t;
    for (int k = 0; k < 64; ++k) {
      const double v = std::exp2(k / 64.0);
      t.t[k].x = (float)v;
      t.t[k].y = (float)(v - (double)t.t[k].x);
    }
    return t;
  }();
  int iters = 0;
  const int c = choose_cluster<T>(a.rows, a.vocab, sms, &iters);
  if (iters > kMaxIters || a.rows * c > INT32_MAX) return VMLA_ERR_SHAPE;
  {
    static bool ready[64] = {};
    static std::mutex mu;
    std::lock_guard<std::mutex> g(mu);
    if (dev >= 64 || !ready[dev]) {
      if (cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kMaxIters * kChunkBytes) != cudaSuccess)
        return VMLA_ERR_CUDA;
      if (dev < 64) ready[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)c;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(a.rows * c), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)iters * kChunkBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a, table, iters) == cudaSuccess ? VMLA_OK : VMLA_ERR_CUDA;
}

}  // namespace

int launch_sample(const SampleArgs& a, bool fp32, void* stream) {
  if (a.rows == 0) return VMLA_OK;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) !=
                                                cudaSuccess)
    return VMLA_ERR_CUDA;
  return fp32 ? launch<float>(a, sms, dev, (cudaStream_t)stream) : launch<uint16_t>(a, sms, dev, (cudaStream_t)stream);
}

}  // namespace vmla
