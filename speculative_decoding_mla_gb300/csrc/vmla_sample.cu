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
// pairs of floats to about 2^-37 (weight_of), rounded to whole units of 2^-45 of
// the largest and added as a 64-bit integer; integer sums are exact in any order.
// Weights below 2^-46 of the largest count as zero.
//
// One cluster of one to eight CTAs takes one row.  With few rows a row is kept in
// shared memory; with many, its later passes read it again, from L2, which lets
// more rows be in work at once.  Where a filter needs the order, the cut is
// found without sorting, from a histogram of counts over the leading 16 bits of
// the values (bins_of): one shared-memory atomic per token, in the pass that finds
// the maximum.
//   bf16: a bin holds one value (but for the bin of the values next to zero), so
//      the masses are counts times exact weights of some thousand values, and the
//      histogram alone gives both cuts exactly;
//   few tokens: where top-k's bins hold at most 1024 tokens (or the vocabulary does)
//      one CTA sorts them and does the rest: order, masses, cuts and draw;
//   fp32: counts give top-k's bin, and, with each bin's middle value, the few bins that
//      can hold top-p's cut; one pass adds the masses of all tokens and of those above
//      these bins, in single precision (where its error could move the cut, again
//      exactly), and lists the keys in them; inside the bin or bins, histograms over 1024
//      equal ranges of the values' bit patterns in their order (count, and exact mass for
//      top-p) narrow it down to one value: one to three rounds, over the few tokens left.
// The draw first sums weights in single precision with a known error (about_of);
// only where the random number falls so near a running sum that this could decide
// it, the sums are taken again exactly: by the same cluster, or, for calls without
// any filter (which read a row once, in a kernel of their own), by a second launch.
//
// What bounds it: 512 rows of 131,072 bf16 (134 MB, 20 us of reading) take 80 us without a
// filter, instructions (22 a token: the weight 13, the loop 5, the rest the search), and
// 130 us with top-p.  There a row is one CTA's, two on an SM, for 53 us: maximum and
// histogram 18 (its shared-memory atomics, 3.8 cycles a warp for their banks' conflicts,
// take 28 us of the whole call, and make the other CTA's shared memory slow meanwhile;
// maximum and histogram in two passes: 145 us), values next to zero 5, cuts 7, the sums of
// the draw 14, its search 6, barriers.  A row that the draw's first sums do not decide (one
// in some hundred) takes 20 us more, 45 if all its tokens and not the kept ones are
// weighed.  128 rows of 151,001 fp32 take 125 to 139 us with top-p and 85 to 93 with all filters
// (of which most have top-k): 225 and 130 where all masses for top-p are exact.  At 64 registers a
// thread the filtered kernel spills 588 (bf16) and 572 (fp32) bytes, 136 and 128 where the row is in
// shared memory; the kernel without filters, at 40, 28 and 40.
// Times depend on the values.  Rows of one or two values, or of a spread far below the temperature,
// have many tokens in top-p's bin: their keys pass the list, each round reads the row again, and the
// atomics go to few addresses.  128 rows of 151,001 with top-p 0.9 take 155 us (fp32) and 76 (bf16)
// for normal logits of deviation 2, 340 and 410 of 10^-4, 670 and 500 for two values, 290 to 460 and
// 66 to 515 for one value.
// Tried and not kept: whole rows in shared memory for 512 rows (216 us), undecided rows of
// the filtered kernel by a second launch (203 -> 215 us), more loads in flight.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "vmla_device.cuh"
#include "vmla_weights.cuh"

namespace vmla {
using namespace weights;
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kChunkBytes = kThreads * 16;   // shared memory per iteration: 16 bytes per thread
constexpr int kKeepIters = 8;                // a row kept in shared memory takes up to 64 KB of each CTA
constexpr int kMaxElems = 264;               // logits of one thread
constexpr int kMaxChunks = kMaxElems / 4;    // iterations of one warp
constexpr int kNearZero = 0x3A80;            // leading 16 bits of 2^-10: smaller values share one bin
constexpr int kBins = 18 * kThreads;         // 9216: see number_of
constexpr int kRanges = 1024;                // of the bit-pattern histograms
constexpr int kKeys = kBins - 3 * kRanges;   // of the keys that they count, listed for the next round
constexpr int kList = 2 * kThreads;          // tokens that one CTA sorts
static_assert((int64_t)kMaxCluster * kThreads * kMaxElems >= VMLA_MAX_VOCAB + 7, "every vocabulary fits");
static_assert(kChunkBytes / 4 >= kList + 3, "one iteration of one CTA holds a list's worth of logits");
static_assert((int64_t)kMaxElems << 23 < (1ll << 32) && kKeepIters * 8 <= kMaxElems, "a thread's sum of high parts fits 32 bits");

struct Shared {
  union {
    uint32_t hist[kBins];
    struct {
      uint32_t count[kRanges], mass_lo[kRanges], mass_hi[kRanges];
      uint32_t key[kKeys];  // of this CTA's tokens that they count
    } r;
    struct {
      uint64_t key[kList], weight[kList], by_place[kList], spare[kList];
    } list;
    float kept[kWarps][64 + 32 * 8];  // of each warp, tokens to weigh
  };
  float2 table[64];
  uint64_t warp_u64[kWarps], warp_u64b[kWarps];
  uint32_t warp_u32[kWarps];
  float warp_f[kWarps], warp_g[kWarps];
  float exp_hi, exp_lo;    // log2(e) / temperature
  float ln_hi, ln_lo;      // temperature x ln(min_p)
  // read by the other CTAs of the cluster; a cluster barrier lies between a phase's reads and the
  // slot's next write
  float x_max, first_max;
  uint64_t sum_a, sum_b, tiny;
  float sum_f, sum_g;
  uint32_t key_lo, key_hi, count, bin_count;
  int32_t index, bin_first, bin_last;
  // written by the one thread of the cluster that finds them, into every CTA
  int32_t bin_k, bin_p, sure;
  uint32_t bin_k_rank, bin_k_count, bin_p_keep;
  // results of a search, the same in every CTA
  uint32_t listed;         // (in the first CTA) tokens in its list
  uint32_t keys;           // (of each CTA its own) keys in its list, more than kKeys where it is not whole
  uint32_t few[32], few_keys;
  int32_t range;
  uint32_t range_key;
  uint32_t range_count;
  uint64_t range_before;
  uint64_t chunk[kMaxChunks];
  uint32_t chunk_same[kMaxChunks];
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

// Signed number of a value's leading 16 bits, not decreasing in the value: 0 next to zero, then one
// step per pattern.  The bin of a value is a number not below the row's maximum's (kAbove) less its own.  A weight of at
// least 2^-46 means a value within 46 ln 2 T < 2^25 of the maximum, T being at most 2^20, and that
// window holds at most 2 (25 + 10) 128 + 1 numbers (when zero is in its middle).
__device__ __forceinline__ int number_of(float x) {
  const uint32_t b = __float_as_uint(x);
  const int n = max((int)((b & 0x7FFFFFFFu) >> 16) - (kNearZero - 1), 0);
  return (int)b < 0 ? -n : n;
}
// The value of a bf16's number other than 0, and the smallest magnitude of an fp32 with it.
__device__ __forceinline__ float number_value(int n) {
  const uint32_t b = (uint32_t)((n < 0 ? -n : n) + (kNearZero - 1)) << 16;
  return __uint_as_float(n < 0 ? b | 0x80000000u : b);
}
constexpr int kAbove = 128;    // numbers above the largest of the first logits
constexpr int kLastBins = 32;  // what counts as zero is thrown into these, one for each lane
static_assert(2 * (25 + 10) * 128 + 1 + kAbove <= kBins - kLastBins, "every token of weight has a bin");

__device__ __forceinline__ uint32_t add2(uint32_t a, uint32_t b) {  // 16-bit halves
  uint32_t r;
  asm("add.s16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Bins of a granule's values by their leading 16 bits, two values at a time in 16-bit halves, top being the
// number of the row's maximum and last this lane's bin for what counts as zero; whether a value is next to
// zero.  With d = max(magnitude bits - (kNearZero - 1), 0) and m = -1 where the sign is set, the number is
// (d ^ m) - m, so the bin is top + m + 1 + ~(d ^ m) (all modulo 2^16: a bin is below 2 x 17,666).
template <int N>
__device__ __forceinline__ bool bins_of(const uint32_t (&word)[N], int top, int last, uint32_t (&bin)[2 * N]) {
  const uint32_t top1 = ((uint32_t)(top + 1) & 0xFFFFu) * 0x10001u, last2 = (uint32_t)last * 0x10001u;
  constexpr uint32_t kFrom = ((uint32_t)(-(kNearZero - 1)) & 0xFFFFu) * 0x10001u;
  uint32_t zero_halves = 0;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    uint32_t d = add2(word[k] & 0x7FFF7FFFu, kFrom), b;
    asm("max.s16x2 %0, %1, %2;" : "=r"(d) : "r"(d), "r"(0u));
    uint32_t m;  // each half's sign over its 16 bits
    asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(m) : "r"(word[k]));
    b = add2(add2(top1, m), ~(d ^ m));
    asm("min.u16x2 %0, %1, %2;" : "=r"(b) : "r"(b), "r"(last2));
    bin[2 * k] = b & 0xFFFFu;
    bin[2 * k + 1] = b >> 16;
    zero_halves |= (d - 0x00010001u) & ~d;  // (d is at most 0x4501 in either half: the sign bits tell)
  }
  return (zero_halves & 0x80008000u) != 0;
}
__device__ __forceinline__ bool bins_of(const float (&)[8], const uint4& v, int top, int last, uint32_t (&bin)[8]) {
  const uint32_t word[4] = {v.x, v.y, v.z, v.w};
  return bins_of(word, top, last, bin);
}
__device__ __forceinline__ bool bins_of(const float (&)[4], const uint4& v, int top, int last, uint32_t (&bin)[4]) {
  const uint32_t word[2] = {__byte_perm(v.x, v.y, 0x7632), __byte_perm(v.z, v.w, 0x7632)};
  return bins_of(word, top, last, bin);
}

// The weight in single precision, times a factor that all of a row's weights share: 2^(x c + bias),
// bias being the whole number next to -max c (below 2^20).  The exponent is split into a whole
// number n = t - 1.5 x 2^23 and f, |f| <= 1/2 (and what x lo adds, below 2^-4): bias - n is exact, f is off by at
// most 2^-26 + 2^-25, which moves the weight by 3.1e-8; ex2.approx on such f is off by -1.43e-7 to 1.46e-7 (every
// float of that range, on this GPU); sums of eight in a tree add 3 x 2^-24 = 1.79e-7, their running sum in two
// floats nothing that counts: kAboutError in all.  For x c + bias > -100 only.
//
// Whether a border, the running sum C of the exact weights, lies above u W is told by C' and W', both taken from
// sums of the same approximate weights: with e_i token i's error, W' - W = sum e_i w_i and C' - C = sum_(i <= j)
// e_i w_i, so u W' - C' is off by u sum_(i > j) e_i w_i - (1 - u) sum_(i <= j) e_i w_i, which at a border near u W
// is at most 2 u (1 - u) kAboutError W.  Only a sum C' made of the very numbers that make W' has these e_i.  The
// last part of C', S up to the border, is summed anew, token by token, which gives its tokens other errors than
// they have in W', by up to kTreeError where only the tree differs, or kAnewError where the bias does too (the
// whole e_i, and 3.1e-8 + 1.46e-7): that much of S comes on top, whatever u is.
struct About {
  float hi, lo, magic;
};
constexpr float kAboutMax = 1048576.f;  // of |max c|
constexpr float kAboutError = 3.6e-7f;  // 3.1e-8 + 1.46e-7 + 1.79e-7
constexpr float kTreeError = 1.8e-7f;
constexpr float kAnewError = 5.4e-7f;   // kAboutError + 3.1e-8 + 1.46e-7

// How near to u W a border may lie and still be decided by single-precision sums, `anew` being what was summed
// anew up to the border (roundings to whole units, at most one a token, by the 2^18).
constexpr uint64_t kAboutUnits = VMLA_MAX_VOCAB;
__device__ __forceinline__ uint64_t about_margin(float u, uint64_t all, uint64_t anew, float anew_error) {
  return (uint64_t)(2.f * u * (1.f - u) * kAboutError * (float)all + anew_error * (float)anew) + kAboutUnits;
}

__device__ __forceinline__ About about(const Exponent& e) {
  return {e.hi, e.lo, __fadd_rn(12582912.f, rintf(-e.max * e.hi))};  // 1.5 x 2^23 + bias
}
__device__ __forceinline__ float about_of(float x, const About& a) {
  const float t = __fmaf_rn(x, a.hi, a.magic);
  const float f = __fmaf_rn(x, a.lo, __fmaf_rn(x, a.hi, __fsub_rn(a.magic, t)));  // magic - t = bias - n
  return __uint_as_float(__float_as_uint(ex2_approx(f)) + (__float_as_uint(t) << 23));
}
// about_of of a granule's values, in pairs (t - magic by an exact product with -1).
template <int N>
__device__ __forceinline__ void about_all(const float (&x)[N], const About& a, float (&w)[N]) {
  const float2 hi = make_float2(a.hi, a.hi), lo = make_float2(a.lo, a.lo), magic = make_float2(a.magic, a.magic);
#pragma unroll
  for (int k = 0; k < N; k += 2) {
    const float2 v = make_float2(x[k], x[k + 1]);
    const float2 t = fma2(v, hi, magic);
    const float2 f = fma2(v, lo, fma2(v, hi, fma2(t, make_float2(-1.f, -1.f), magic)));
    w[k] = __uint_as_float(__float_as_uint(ex2_approx(f.x)) + (__float_as_uint(t.x) << 23));
    w[k + 1] = __uint_as_float(__float_as_uint(ex2_approx(f.y)) + (__float_as_uint(t.y) << 23));
  }
}
// Their sum, in a tree.
__device__ __forceinline__ float tree_sum(const float (&w)[8]) {
  const float2 a = sum2(make_float2(w[0], w[1]), make_float2(w[4], w[5]));
  const float2 b = sum2(make_float2(w[2], w[3]), make_float2(w[6], w[7]));
  const float2 c = sum2(a, b);
  return __fadd_rn(c.x, c.y);
}
__device__ __forceinline__ float tree_sum(const float (&w)[4]) {
  const float2 c = sum2(make_float2(w[0], w[1]), make_float2(w[2], w[3]));
  return __fadd_rn(c.x, c.y);
}
// A float's value v >= 0 in units of 2^-kBits, v 2^kBits < 2^64, rounded down.  (By shifts: the conversion
// to 64 bits runs at two lanes a cycle on an SM, which 512 threads at once would feel.)
template <int kBits>
__device__ __forceinline__ uint64_t fixed(float v) {
  const uint32_t b = __float_as_uint(v), m = (b & 0x7FFFFFu) | 0x800000u;
  const int up = (int)(b >> 23) - (150 - kBits);
  return up >= 0 ? (uint64_t)m << min(up, 63) : m >> min(-up, 31);
}
__device__ __forceinline__ uint64_t about_units(float v) { return fixed<kUnitBits>(v); }
__device__ __forceinline__ uint64_t about_units(float s, float e) {
  const uint64_t rest = about_units(fabsf(e));
  return about_units(s) + (e < 0.f ? 0 - rest : rest);
}
// 2^d of a whole number d, zero below 2^-126 and one above 2^0.
__device__ __forceinline__ float power_of_two(float d) {
  return d < -126.f ? 0.f : __uint_as_float((uint32_t)(127 + (int)fminf(d, 0.f)) << 23);
}
// a + (b + c), c far below b, rounded up to a float.
__device__ __forceinline__ float sum_rounded_up(float a, float b, float c) {
  const float t = __fadd_rn(a, b), v = __fsub_rn(t, a);
  const float e = __fadd_rn(__fsub_rn(a, __fsub_rn(t, v)), __fsub_rn(b, v));
  return __fadd_ru(t, __fadd_rn(e, c));
}
// v into a sum held in two floats.
__device__ __forceinline__ void add_in_two(float v, float* s, float* e) {
  const float t = __fadd_rn(*s, v), b = __fsub_rn(t, *s);
  *e = __fadd_rn(*e, __fadd_rn(__fsub_rn(*s, __fsub_rn(t, b)), __fsub_rn(v, b)));
  *s = t;
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
  typedef float Max;
  static __device__ __forceinline__ Max lowest() { return -INFINITY; }
  static __device__ __forceinline__ float largest(Max m) { return m; }
  // The granule with NaN made -inf; also with its values taken into the running maximum.
  static __device__ __forceinline__ uint4 numbers(const uint4& v) {
    float x[4];
    unpack(v, x);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = fmaxf(x[k], -INFINITY);
    return pack(x);
  }
  static __device__ __forceinline__ uint4 settle(const uint4& v, Max& m) {
    const uint4 r = numbers(v);
    float x[4];
    unpack(r, x);
#pragma unroll
    for (int k = 0; k < 4; ++k) m = fmaxf(m, x[k]);
    return r;
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
  typedef uint32_t Max;  // two bf16 maxima
  static __device__ __forceinline__ Max lowest() { return 0xFF80FF80u; }
  static __device__ __forceinline__ float largest(Max m) { return fmaxf(bf16_lo(m), bf16_hi(m)); }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {  // of a NaN and a number: the number
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ uint4 numbers(const uint4& v) {
    return make_uint4(max2(v.x, lowest()), max2(v.y, lowest()), max2(v.z, lowest()), max2(v.w, lowest()));
  }
  static __device__ __forceinline__ uint4 settle(const uint4& v, Max& m) {
    const uint4 r = numbers(v);
    m = max2(m, max2(max2(r.x, r.y), max2(r.z, r.w)));
    return r;
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {  // of bf16 values: exact
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
  }
};

// Descending order of these keys is that of the tokens: by value, then by place.
__device__ __forceinline__ uint64_t sort_key(float x, int place) {
  return ((uint64_t)order_key<0>(x) << 32) | (uint32_t)~place;
}

// keys[0, n), n a power of two from 64 to kList, in descending order (a permutation: equal keys by their
// place).  Up to 256 keys each one's rank is counted, by 2 to 8 threads, into `spare`; more are sorted in
// place by exchanges (45 or 55 block-wide steps).  Returns the array that holds them.
__device__ __forceinline__ uint64_t* in_descending_order(uint64_t* keys, uint64_t* spare, int n) {
  const int t = threadIdx.x;
  __syncthreads();
  if (n <= kThreads / 2) {
    const int group = kThreads / n, e = t / group, part = t % group;
    const uint64_t mine = keys[e];
    int rank = 0;
#pragma unroll 4
    for (int j = part; j < n; j += group) {
      const uint64_t other = keys[j];
      rank += other > mine || (other == mine && j < e) ? 1 : 0;
    }
    for (int o = group >> 1; o > 0; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (part == 0) spare[rank] = mine;
    __syncthreads();
    return spare;
  }
  for (int run = 2; run <= n; run <<= 1) {
    for (int gap = run >> 1; gap > 0; gap >>= 1) {
      if (t < n >> 1) {
        const int i = 2 * t - (t & (gap - 1)), j = i + gap;
        const uint64_t x = keys[i], y = keys[j];
        if ((x < y) == ((i & run) == 0)) keys[i] = y, keys[j] = x;
      }
      __syncthreads();
    }
  }
  return keys;
}

// The place of the token drawn from the `listed` tokens of sm.list, which hold the row's top-k first
// ones: in their order exact weights, whose running sums give top-p's cut; then by place, for the draw.
__device__ __noinline__ int draw_listed(Shared& sm, const Exponent& ex, uint32_t listed, uint32_t top_k, bool with_p,
                                        uint64_t p64, float min_p, uint64_t u64) {
  const int tid = threadIdx.x;
  int n = 64;
  while (n < (int)listed) n <<= 1;
  for (int i = listed + tid; i < n; i += kThreads) sm.list.key[i] = 0;
  const uint64_t* order = in_descending_order(sm.list.key, sm.list.spare, n);
  const float least = min_p > 0.f ? sum_rounded_up(ex.max, sm.ln_hi, sm.ln_lo) : -INFINITY;
  // this thread's two tokens of the order
  float x[2];
  uint64_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t i = 2 * tid + j;
    const bool in = i < listed && i < top_k;
    x[j] = in ? order_value<0>((uint32_t)(order[i] >> 32)) : -INFINITY;
    w[j] = weight_units(x[j], ex, sm.table);
  }
  uint64_t all;
  const uint64_t before = block_scan(w[0] + w[1], sm.warp_u64, &all);
  // (the token itself is kept while the mass ahead of it does not reach p of all)
  const uint64_t reach = with_p ? __umul64hi(p64, all) + (p64 * all != 0 ? 1 : 0) : ~0ull;
  uint64_t at = before;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t i = 2 * tid + j;
    const bool kept = w[j] > 0 && x[j] >= least && (at < reach || i == 0);
    at += w[j];
    if (!kept) w[j] = 0;
    if (i < (uint32_t)n) {
      // places ascend as these keys descend; a token left out comes last
      sm.list.by_place[i] = kept ? (order[i] << 32) | i : 0;
      sm.list.weight[i] = w[j];
    }
  }
  // (with few keys `order` is the spare array, and the first one is free)
  const uint64_t* places = in_descending_order(sm.list.by_place, sm.list.key, n);
  uint64_t key[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = 2 * tid + j;
    key[j] = i < n ? places[i] : 0;
    w[j] = key[j] ? sm.list.weight[(uint32_t)key[j]] : 0;
  }
  at = block_scan(w[0] + w[1], sm.warp_u64, &all);
  const uint64_t goal = __umul64hi(u64, all);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (at <= goal && goal < at + w[j]) sm.index = (int)~(uint32_t)(key[j] >> 32);
    at += w[j];
  }
  __syncthreads();
  return sm.index;
}

// One row on one cluster.  Element v of the "shifted" row is token v - shift, shift being the
// elements between the row's start and the 16-byte boundary below it, so that whole granules load
// as vectors whatever the row's alignment; places outside the row read as -inf.  CTA r takes
// places [r S, (r + 1) S), its warp w the w-th of kWarps equal runs of them.
template <typename T, bool kKeep>
__global__ void __launch_bounds__(kThreads, 2)
sample_kernel(const SampleArgs a, const __grid_constant__ ExpTable exp_table, int iters) {
  using E = Elems<T>;
  constexpr int kVec = E::kVec;
  constexpr int kStep = 32 * kVec;  // places of one warp iteration
  extern __shared__ __align__(16) uint8_t slice_raw[];
  __shared__ Shared sm;
  const cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  auto sync_all = [&] {
    if (C > 1) cluster.sync();
    else __syncthreads();
  };
  auto of = [&](int r) -> Shared& { return C > 1 ? *cluster.map_shared_rank(&sm, r) : sm; };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = (int64_t)blockIdx.x / C;
  const T* src = static_cast<const T*>(a.logits) + row * a.stride;
  const int shift = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
  const T* base = src - shift;
  const int end = a.vocab + shift;  // places [shift, end) are tokens
  const int seg = iters * kStep;    // a warp's places
  const int first = (rank * kWarps + warp) * seg;
  uint4* slice = reinterpret_cast<uint4*>(slice_raw) + lane;  // granule of warp w, iteration i: slice[32 (w iters + i)]
  // the granule at place p as it lies in memory; `whole`: no part of this warp's run is outside the row
  const bool whole = (rank * kWarps + warp) * seg >= shift && (rank * kWarps + warp + 1) * seg <= end;
  auto granule = [&](int p, bool inside) {
    uint4 v;
    if (inside || (p >= shift && p + kVec <= end)) {
      asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                   : "l"(base + p));
    } else {
      float x[kVec];
#pragma unroll
      for (int k = 0; k < kVec; ++k) x[k] = p + k >= shift && p + k < end ? E::one(base + p + k) : -INFINITY;
      v = E::pack(x);
    }
    return v;
  };
  // the logits of warp w's iteration i that fall to this lane, NaN made -inf
  auto fetch = [&](int w, int i) {
    if (kKeep) return slice[32 * (w * iters + i)];
    return granule((rank * kWarps + w) * seg + i * kStep + lane * kVec, whole && w == warp);
  };
  auto values = [&](const uint4& v, float (&x)[kVec]) { E::unpack(kKeep ? v : E::numbers(v), x); };

  // the first granules on their way, then the settings; a row with a bad one draws nothing
  constexpr int kFlight = 4;
  uint4 flight[kFlight];
#pragma unroll
  for (int f = 0; f < kFlight; ++f)
    if (f < iters) flight[f] = granule(first + f * kStep + lane * kVec, whole);
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

  // one thread each: 64-bit arithmetic is some 60 times slower than 32-bit here
  if (tid == 0 && temp > 0.f) {
    const double c = 1.4426950408889634 / (double)temp;
    sm.exp_hi = (float)c;
    sm.exp_lo = (float)(c - (double)sm.exp_hi);
  }
  if (tid == 32) {
    const double l = min_p > 0.f && min_p < 1.f ? (double)temp * log((double)min_p) : 0.0;
    sm.ln_hi = (float)l;
    sm.ln_lo = (float)(l - (double)sm.ln_hi);
  }
  // ---- the row's maximum, and in the same pass the histogram, where a filter needs the order.  Its bins are
  // counted from a number an octave above the largest logit of the first granules (an eighth of 131,072
  // logits, spread over the row): only a row whose maximum is greater still is counted again.
  bool with_k = top_k > 0 && top_k < a.vocab;
  const bool with_p = top_p < 1.f, counted = temp > 0.f && (with_k || with_p) && a.vocab > kList;
  typename E::Max run = E::lowest();
  int top_number = 0;
  const int last_bin = kBins - kLastBins + lane;
  auto clear_bins = [&] {
    for (int b = tid; b < kBins - kLastBins; b += kThreads) sm.hist[b] = 0;
  };
  uint32_t nears = 0;  // bit min(i, 31): iteration i's granule of this lane has a value next to zero
  auto count = [&](const uint4& v, const float (&x)[kVec], int i) {
    uint32_t bin[kVec];
    const bool near = bins_of(x, v, top_number, last_bin, bin);
#pragma unroll
    for (int k = 0; k < kVec; ++k) atomicAdd(&sm.hist[bin[k]], 1u);
    if (E::kLowBits && near) nears |= 1u << min(i, 31);
  };
  if (counted) {
    clear_bins();
#pragma unroll
    for (int f = 0; f < kFlight; ++f)
      if (f < iters) E::settle(flight[f], run);
    float m = warp_max(E::largest(run));
    if (lane == 0) sm.warp_f[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm.warp_f[w]);
    if (C > 1) {
      if (tid == 0) sm.first_max = m;
      sync_all();
      for (int r = 0; r < C; ++r) m = fmaxf(m, of(r).first_max);
    }
    top_number = number_of(m) + kAbove;
  }
#pragma unroll 1
  for (int i0 = 0; i0 < iters; i0 += kFlight) {
    uint4 v[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) v[f] = flight[f];
#pragma unroll
    for (int f = 0; f < kFlight; ++f)
      if (i0 + kFlight + f < iters) flight[f] = granule(first + (i0 + kFlight + f) * kStep + lane * kVec, whole);
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      if (i0 + f < iters) {
        const uint4 now = E::settle(v[f], run);  // NaN counts as -inf
        if (kKeep) slice[32 * (warp * iters + i0 + f)] = now;
        if (counted) {
          float x[kVec];
          E::unpack(now, x);
          count(now, x, i0 + f);
        }
      }
    }
  }
  __syncthreads();  // (warp_f is written again)
  float mx = E::largest(run);
  if (tid == 0) sm.sure = 0, sm.listed = 0, sm.tiny = 0;  // (written from other CTAs only past the barriers below)
  if (tid < 64) sm.table[tid] = exp_table.t[tid];
  mx = warp_max(mx);
  if (lane == 0) sm.warp_f[warp] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm.warp_f[w]);
  if (tid == 0) sm.x_max = mx;
  sync_all();
  for (int r = 0; r < C; ++r) mx = fmaxf(mx, of(r).x_max);

  // g(granule, values, first place) for every granule of this thread, the next ones on their way
  auto each_raw = [&](auto&& g) {
    constexpr int kAhead = kKeep ? 1 : 2;
    uint4 v[kAhead];
#pragma unroll
    for (int h = 0; h < kAhead; ++h)
      if (h < iters) v[h] = fetch(warp, h);
#pragma unroll 1
    for (int i0 = 0; i0 < iters; i0 += kAhead) {
#pragma unroll
      for (int h = 0; h < kAhead; ++h) {
        const int i = i0 + h;
        if (i >= iters) break;
        const uint4 now = kKeep ? v[h] : E::numbers(v[h]);
        if (i + kAhead < iters) v[h] = fetch(warp, i + kAhead);
        float x[kVec];
        E::unpack(now, x);
        g(now, x, first + i * kStep + lane * kVec);
      }
    }
  };
  // g(values, first place)
  auto each_granule = [&](auto&& g) {
    each_raw([&](const uint4&, const float (&x)[kVec], int p) { g(x, p); });
  };
  // f(x) for every element of this thread, its code once and not once per element of a granule: for
  // passes that few rows take, whose instructions would otherwise come from memory each time
  auto each_small = [&](auto&& f) {
    each_granule([&](const float (&x)[kVec], int) {
#pragma unroll 1
      for (int k = 0; k < kVec; ++k) f(x[k]);
    });
  };
  // f(x, place) for every element of this thread
  auto each = [&](auto&& f) {
    each_granule([&](const float (&x)[kVec], int p) {
#pragma unroll
      for (int k = 0; k < kVec; ++k) f(x[k], p + k);
    });
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
    sync_all();
    if (rank == 0 && tid == 0) {
      for (int r = 0; r < C; ++r) at = min(at, of(r).index);
      a.token[row] = at == INT32_MAX ? -1 : at - shift;
    }
    sync_all();
    return;
  }
  const uint64_t p64 = top_p < 1.f ? fixed<64>(top_p) : ~0ull;  // p 2^64: whole for p >= 2^-40
  const uint64_t u64 = u < 1.f ? fixed<64>(u) : ~0ull;
  if (mx == INFINITY) {
    // the tokens at +inf have equal weights, and all others none: of the first kept ones by place, the
    // one numbered floor(u kept)
    uint32_t here = 0;
    each_small([&](float x) { here += x == INFINITY ? 1u : 0u; });
    here = warp_add(here);
    __syncthreads();
    if (lane == 0) sm.warp_u32[warp] = here;
    __syncthreads();
    uint32_t block = 0, ahead = 0, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      block += sm.warp_u32[w];
      if (w < warp) ahead += sm.warp_u32[w];
    }
    if (tid == 0) sm.count = block;
    sync_all();
    for (int r = 0; r < C; ++r) {
      const uint32_t n = of(r).count;
      if (r < rank) ahead += n;
      all += n;
    }
    if (top_k > 0) all = min(all, (uint32_t)top_k);
    if (top_p < 1.f) all = max((uint32_t)(__umul64hi(p64, all) + (p64 * all != 0 ? 1 : 0)), 1u);
    uint32_t nth = (uint32_t)__umul64hi(u64, all);  // (u = 1: the last)
    if (ahead <= nth && nth < ahead + here) {       // one warp of the cluster
      for (int i = 0; i < iters; ++i) {
        float x[kVec];
        values(fetch(warp, i), x);
        uint32_t n = 0;
#pragma unroll
        for (int k = 0; k < kVec; ++k) n += x[k] == INFINITY ? 1u : 0u;
        uint32_t at = ahead + warp_scan(n, lane) - n;
#pragma unroll
        for (int k = 0; k < kVec; ++k)
          if (x[k] == INFINITY && at++ == nth) a.token[row] = first + i * kStep + lane * kVec + k - shift;
        ahead += warp_add(n);
      }
    }
    sync_all();
    return;
  }
  const Exponent ex = {mx, sm.exp_hi, sm.exp_lo};
  auto to_all = [&](auto member, auto value) {  // into every CTA's copy of a result
    for (int r = 0; r < C; ++r) of(r).*member = value;
  };

  // ---- what is kept: x > cut_x, and of the tokens equal to cut_x the first cut_keep
  constexpr uint32_t kAllEqual = UINT32_MAX;
  float cut_x = -INFINITY;
  uint32_t cut_keep = kAllEqual;
  if ((with_k || with_p) && a.vocab <= kList) {
    // the whole row goes into a list (of one CTA: its cluster has no other)
    each([&](float x, int p) {
      if (x > -INFINITY) sm.list.key[atomicAdd(&sm.listed, 1u) % kList] = sort_key(x, p);
    });
    __syncthreads();
    const int place = draw_listed(sm, ex, sm.listed, with_k ? (uint32_t)top_k : kList, with_p, p64, min_p, u64);
    if (tid == 0) a.token[row] = place - shift;
    return;
  }
  if (with_k || with_p) {
    if (number_of(mx) > top_number) {  // the same in every thread of the cluster
      top_number = number_of(mx);
      clear_bins();
      __syncthreads();
      nears = 0;
      each_raw([&](const uint4& v, const float (&x)[kVec], int p) { count(v, x, (p - first) / kStep); });
      sync_all();
    }
    // tokens of weight lie above
    const float x_low = fminf(mx, fmaxf(mx - kOctaves * 0.6931472f * temp * 1.0001f, -3.402823466e38f));
    // the bins in use; every CTA sums up an equal run of them
    const int bins = min(kBins - kLastBins, top_number - number_of(x_low) + 1);
    const int per = (bins + C * kThreads - 1) / (C * kThreads);  // consecutive bins of one thread
    const int bin0 = (rank * kThreads + tid) * per;
    const int tiny_bin = top_number;  // of number 0, where it is in use (0 <= top_number < bins)
    if (E::kLowBits && with_p && tiny_bin >= 0 && tiny_bin < bins) {
      // exact mass of the values that share the bin next to zero (one in 2,500 for logits of deviation 2):
      // their granules are read again, each lane its own
      uint64_t tiny = 0;
      for (uint32_t left = nears; left != 0; left &= left - 1) {
        const int at = __ffs(left) - 1;
        for (int i = at; i < (at < 31 ? at + 1 : iters); ++i) {
          const uint4 v = kKeep ? fetch(warp, i) : E::numbers(fetch(warp, i));
          float x[kVec];
          E::unpack(v, x);
          uint32_t which = 0;
#pragma unroll
          for (int k = 0; k < kVec; ++k) which |= number_of(x[k]) == 0 ? 1u << k : 0u;
          for (; which != 0; which &= which - 1) {
            float y = 0.f;
#pragma unroll
            for (int k = 0; k < kVec; ++k) y = __ffs(which) - 1 == k ? x[k] : y;
            tiny += weight_units(y, ex, sm.table);
          }
        }
      }
      if (tiny != 0) atomicAdd(reinterpret_cast<unsigned long long*>(&sm.tiny), (unsigned long long)tiny);
      sync_all();
    }
    // this thread's bins, summed over the CTAs (into this CTA's copy: no other CTA reads these bins
    // of it), and the tokens ahead of them
    uint32_t before = 0;
    if (C > 1 || with_k)
      for (int j = 0; j < per && bin0 + j < bins; ++j) {
        uint32_t n = 0;
        for (int r = 0; r < C; ++r) n += of(r).hist[bin0 + j];
        if (C > 1) sm.hist[bin0 + j] = n;
        before += n;
      }
    if (with_k) {
      uint32_t total;
      before = block_scan(before, sm.warp_u32, &total);
      if (tid == 0) sm.bin_count = total;
      sync_all();
      total = 0;
      for (int r = 0; r < C; ++r) {
        const uint32_t n = of(r).bin_count;
        if (r < rank) before += n;
        total += n;
      }
      if ((uint32_t)top_k >= total) with_k = false;  // nothing of weight is past the k-th
    }

    // Histograms of counts (and masses) over the 1024 equal ranges of keys from klo on, each 2^width
    // keys wide, of this CTA's tokens; the keys are clear when all CTAs have passed the next barrier.
    auto range_width = [](uint32_t klo, uint32_t khi) { return max(32 - __clz((khi - klo) | 1) - 10, 0); };
    auto clear_ranges = [&](bool list) {
      for (int b = tid; b < kRanges; b += kThreads) sm.r.count[b] = sm.r.mass_lo[b] = sm.r.mass_hi[b] = 0;
      if (tid == 0) {
        sm.few_keys = 0;
        if (list) sm.keys = 0;
      }
      __syncthreads();
    };
    auto list_key = [&](uint32_t k) {
      const uint32_t at = atomicAdd(&sm.keys, 1u);
      if (at < kKeys) sm.r.key[at] = k;
    };
    auto add_mass = [&](uint32_t g, uint64_t w) {
      const uint32_t wl = (uint32_t)w, old = atomicAdd(&sm.r.mass_lo[g], wl);
      atomicAdd(&sm.r.mass_hi[g], (uint32_t)(w >> 32) + (old + wl < old ? 1u : 0u));
    };
    // The range in which the running count (or mass), in descending order, reaches `target`: [klo, khi]
    // becomes it; its count; and what is left of the target.  False where it is not reached.
    auto pick = [&](bool by_mass, int width, uint32_t* klo, uint32_t* khi, uint64_t* target, uint32_t* equal) {
      constexpr int kPer = kRanges / kThreads;
      uint32_t n2[kPer], sum_n = 0;
      uint64_t m2[kPer], sum_m = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int g = kRanges - 1 - (kPer * tid + j);  // descending
        n2[j] = 0, m2[j] = 0;
        for (int r = 0; r < C; ++r) {
          const Shared* o = &of(r);
          n2[j] += o->r.count[g];
          if (by_mass) m2[j] += ((uint64_t)o->r.mass_hi[g] << 32) + o->r.mass_lo[g];
        }
        sum_n += n2[j], sum_m += m2[j];
      }
      uint32_t all_n;
      uint64_t all_m = 0, cum_m = 0;
      uint32_t cum_n = block_scan(sum_n, sm.warp_u32, &all_n);
      if (by_mass) cum_m = block_scan(sum_m, sm.warp_u64, &all_m);
      if (by_mass && *target - 1 >= all_m) {  // (0 too) the same in every thread of the cluster
        sync_all();
        return false;
      }
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const uint64_t was = by_mass ? cum_m : cum_n;
        cum_n += n2[j], cum_m += m2[j];
        const uint64_t now = by_mass ? cum_m : cum_n;
        if (was < *target && now >= *target) {  // one range of one thread
          sm.range = kRanges - 1 - (kPer * tid + j);
          sm.range_count = n2[j];
          sm.range_before = was;
        }
      }
      __syncthreads();
      *target -= sm.range_before;
      *equal = sm.range_count;
      *klo += (uint32_t)sm.range << width;
      *khi = min(*khi, *klo + ((1u << width) - 1u));
      sync_all();  // the histograms have been read
      return true;
    };
    // The value at which a running count (or mass) over the tokens with a key in [klo, khi], in
    // descending order, reaches `target`: its key, how many tokens have it, and what is left of the
    // target for them; false where it is not reached.  (A round leaves 10 bits fewer: 32, 22, 12, 2.)  The
    // keys come from the list, or, where there is none yet or too many, from the row.
    auto refine = [&](uint32_t klo, uint32_t khi, bool by_mass, bool listed, uint64_t* target, uint32_t* equal,
                      uint32_t* key) {
      *equal = UINT32_MAX;
#pragma unroll 1
      for (int round = 0; round < 4; ++round) {
        const int width = range_width(klo, khi);
        const uint32_t keys = listed ? sm.keys : kKeys + 1u;
        const bool few = listed && *equal <= 32;
        clear_ranges(!listed);
        auto take = [&](uint32_t k) {
          if (k < klo || k > khi) return;
          if (few) {
            sm.few[atomicAdd(&sm.few_keys, 1u) & 31u] = k;
            return;
          }
          const uint32_t g = (k - klo) >> width;
          atomicAdd(&sm.r.count[g], 1u);
          if (by_mass) add_mass(g, weight_units(order_value<E::kLowBits>(k), ex, sm.table));
          if (!listed) list_key(k);
        };
        if (keys <= kKeys) {
          for (uint32_t i = tid; i < keys; i += kThreads) take(sm.r.key[i]);
        } else {
          each([&](float x, int) { take(order_key<E::kLowBits>(x)); });
        }
        listed = true;
        if (few) {
          // one warp of each CTA takes the cluster's few keys, one to a lane
          sync_all();
          if (warp == 0) {
            uint32_t k = 0, n = 0, same = 0;
            for (int r = 0; r < C; ++r) {
              const uint32_t here = of(r).few_keys;
              if (lane >= n && lane < n + here) k = of(r).few[lane - n];
              n += here;
            }
            const uint64_t w = by_mass ? weight_units(order_value<E::kLowBits>(k), ex, sm.table) : 1;
            uint64_t ahead = 0;
            for (int j = 0; j < (int)n; ++j) {
              const uint32_t other = __shfl_sync(0xffffffffu, k, j);
              const uint64_t its = __shfl_sync(0xffffffffu, w, j);
              if (other > k) ahead += its;
              if (other == k) ++same;
            }
            if (lane < n && ahead < *target && *target <= ahead + same * w)  // (the same in equal keys' lanes)
              sm.range_key = k, sm.range_count = same, sm.range_before = ahead;
          }
          __syncthreads();
          *target -= sm.range_before;
          *equal = sm.range_count;
          klo = sm.range_key;
          sync_all();  // the keys have been read
          break;
        }
        sync_all();
        if (!pick(by_mass, width, &klo, &khi, target, equal)) return false;
        if (width == 0) break;
      }
      *key = klo;
      return true;
    };
    // Keys of the values in bins [b_first, b_last].
    auto bin_keys = [&](int b_first, int b_last, uint32_t* klo, uint32_t* khi) {
      constexpr int kL = E::kLowBits;
      const uint32_t rest = (1u << (16 - kL)) - 1u;  // an fp32's patterns of one number
      const int n_hi = top_number - b_first, n_lo = top_number - b_last;
      // numbers above 0 start at their own value's key, those below end at it
      const uint32_t zero = order_key<kL>(0.f), near = ((uint32_t)kNearZero << (16 - kL)) - 1u;
      if (n_hi >= number_of(mx)) *khi = order_key<kL>(mx);  // (the bins may begin beyond the largest number)
      else *khi = n_hi > 0 ? order_key<kL>(number_value(n_hi)) + rest
                           : n_hi == 0 ? zero + near : order_key<kL>(number_value(n_hi));
      *klo = n_lo > 0 ? order_key<kL>(number_value(n_lo))
                      : n_lo == 0 ? zero - 1u - near : order_key<kL>(number_value(n_lo)) - rest;
    };
    if (with_k) {
      uint32_t at = before;
      for (int j = 0; j < per && bin0 + j < bins; ++j) {
        const uint32_t n = sm.hist[bin0 + j];
        if (at < (uint32_t)top_k && at + n >= (uint32_t)top_k) {  // one bin of the cluster
          to_all(&Shared::bin_k, bin0 + j);
          to_all(&Shared::bin_k_rank, (uint32_t)top_k - at);
          to_all(&Shared::bin_k_count, n);
        }
        at += n;
      }
      sync_all();
    }
    // top-k leaves the bins up to bin_k, of that one the first k_rank tokens
    const int bin_k = with_k ? sm.bin_k : bins - 1;
    const uint32_t k_rank = with_k ? sm.bin_k_rank : UINT32_MAX;
    auto least_mass = [&](uint64_t all) {
      return max((uint64_t)__umul64hi(p64, all) + (p64 * all != 0 ? 1 : 0), (uint64_t)1);
    };

    const uint32_t top_listed = with_k ? (uint32_t)top_k - k_rank + sm.bin_k_count : UINT32_MAX;
    if (top_listed <= kList) {
      // Few tokens are in the bins that hold top-k's: they go into the first CTA's list (where its
      // histogram was: all have read it), and that CTA does the rest by sorting them.
      uint32_t klo, khi;
      bin_keys(bin_k, bin_k, &klo, &khi);
      const float least = order_value<E::kLowBits>(klo);
      Shared* to = &of(0);
      each_granule([&](const float (&x)[kVec], int p) {
        bool any = false;
#pragma unroll
        for (int k = 0; k < kVec; ++k) any |= x[k] >= least;
        if (any)
#pragma unroll
          for (int k = 0; k < kVec; ++k)
            if (x[k] >= least) to->list.key[atomicAdd(&to->listed, 1u) % kList] = sort_key(x[k], p + k);
      });
      sync_all();
      if (rank == 0) {
        const int place = draw_listed(sm, ex, top_listed, (uint32_t)top_k, with_p, p64, min_p, u64);
        if (tid == 0) a.token[row] = place - shift;
      }
      return;
    }
    bool found = false;
    if (E::kLowBits && !(with_k && bin_k == tiny_bin)) {
      // bf16: bins are values
      if (with_k) cut_x = number_value(top_number - bin_k), cut_keep = k_rank;
      found = !with_p;
      if (with_p) {
        uint64_t all = 0, tiny_all = 0, own = 0, block;
        for (int r = 0; r < C; ++r) tiny_all += of(r).tiny;
        const int stop = min(bin0 + per, bin_k + 1);
        for (int b = bin0; b < stop; b += 2) {
          // (of a row with one bin less than two, or of number 0, the value is not looked at)
          int32_t h[2], l[2];
          weights_of(make_float2(number_value(top_number - b), number_value(top_number - b - 1)), ex, sm.table, h, l);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (b + j < stop)
              own += b + j == tiny_bin ? tiny_all
                                       : units(h[j], l[j]) * (b + j == bin_k ? min(sm.hist[b + j], k_rank) : sm.hist[b + j]);
        }
        uint64_t ahead = block_scan(own, sm.warp_u64, &block);
        if (tid == 0) sm.sum_a = block;
        sync_all();
        for (int r = 0; r < C; ++r) {
          const uint64_t m = of(r).sum_a;
          if (r < rank) ahead += m;
          all += m;
        }
        const uint64_t target = least_mass(all);
        // one thread of the cluster has the bin; its warp looks at that thread's bins
        const uint32_t who = __ballot_sync(0xffffffffu, ahead < target && ahead + own >= target);
        if (who) {
          const int owner = __ffs(who) - 1;
          const int b = __shfl_sync(0xffffffffu, bin0, owner) + lane;
          const uint64_t w = b == tiny_bin ? 0 : weight_units(number_value(top_number - b), ex, sm.table);
          const bool mine = lane < per && b <= bin_k;
          const uint64_t m = !mine ? 0 : b == tiny_bin ? tiny_all : w * (b == bin_k ? min(sm.hist[b], k_rank) : sm.hist[b]);
          const uint64_t upto = __shfl_sync(0xffffffffu, ahead, owner) + warp_scan(m, lane);
          if (lane == __ffs(__ballot_sync(0xffffffffu, upto >= target)) - 1) {
            to_all(&Shared::bin_p, b);
            to_all(&Shared::bin_p_keep, w > 0 ? (uint32_t)((target - (upto - m) + w - 1) / w) : sm.hist[b]);
          }
        }
        sync_all();
        if (sm.bin_p != tiny_bin) {
          if (!with_k || sm.bin_p != bin_k || sm.bin_p_keep < cut_keep)
            cut_x = number_value(top_number - sm.bin_p), cut_keep = sm.bin_p_keep;
          found = true;
        }
      }
    }
    if (!found) {
      // The bins where top-p's mass can be reached: every token of a bin is taken for the bin's middle value,
      // which is off by at most a factor 2^h, and p all - cum, cum being the mass up to a bin, then by the error
      // of p (all - cum) + (1 - p) cum: a few bins.
      int b_lo = 0, b_hi = bin_k;
      if (with_p) {
        auto bin_mass = [&](int b, float* off) {
          const uint32_t n = b > bin_k ? 0 : b == bin_k ? min(sm.hist[b], k_rank) : sm.hist[b];
          *off = 0.f;
          if (n == 0) return 0.f;
          const int v = top_number - b;
          const uint32_t bits = __float_as_uint(number_value(v));
          const float middle = v == 0 ? 0.f : __uint_as_float(bits | (E::kLowBits ? 0u : 0x8000u));
          const float reach = v == 0 ? __uint_as_float((uint32_t)kNearZero << 16)
                                     : E::kLowBits ? 0.f : fabsf(middle - __uint_as_float(bits));
          const float m = (float)n * ex2_approx(fminf((middle - mx) * ex.hi, 0.f));
          *off = m * (ex2_approx(fminf(reach * ex.hi, 64.f)) - 1.f + 1e-4f);
          return m;
        };
        float own = 0.f, own_off = 0.f, off, all, all_off;
        for (int b = bin0; b < bin0 + per && b < bins; ++b) own += bin_mass(b, &off), own_off += off;
        float cum = block_scan(own, sm.warp_f, &all), cum_off = block_scan(own_off, sm.warp_g, &all_off);
        if (tid == 0) sm.sum_f = all, sm.sum_g = all_off, sm.bin_first = sm.bin_last = bin_k;
        sync_all();
        all = all_off = 0.f;
        for (int r = 0; r < C; ++r) {
          const float m = of(r).sum_f, e = of(r).sum_g;
          if (r < rank) cum += m, cum_off += e;
          all += m, all_off += e;
        }
        // (bins far before or past it need no second look)
        if (cum + own >= top_p * all - all_off && cum <= top_p * all + all_off)
          for (int b = bin0; b < bin0 + per && b < bins; ++b) {
            const float m = bin_mass(b, &off);
            if (m == 0.f) continue;
            cum += m, cum_off += off;
            const float over = cum - top_p * all, error = top_p * (all_off - cum_off) + (1.f - top_p) * cum_off;
            if (over >= -error) atomicMin(&sm.bin_first, b);
            if (over >= error) atomicMin(&sm.bin_last, b);
          }
        sync_all();
        b_lo = b_hi;
        for (int r = 0; r < C; ++r) b_lo = min(b_lo, of(r).bin_first), b_hi = min(b_hi, of(r).bin_last);
      }
      sync_all();  // the histograms and what was found in them have been read
      uint32_t floor_key = 0, klo, khi, equal;
      if (with_k) {
        uint64_t left = k_rank;
        bin_keys(bin_k, bin_k, &klo, &khi);
        refine(klo, khi, false, false, &left, &equal, &floor_key);
        cut_x = order_value<E::kLowBits>(floor_key);
        cut_keep = (uint32_t)left;
      }
      if (with_p) {
        // In one pass the masses of what top-k leaves and of its part above these bins, whose own tokens (of
        // those equal to top-k's cut, all: they come last) are listed.  First in single precision: where
        // the cut then lies too near a border, again with exact masses; where it is not in these bins,
        // among all.
        const float floor_x = with_k ? cut_x : -INFINITY;
        bool exact = !(fabsf(mx * ex.hi) < kAboutMax);
#pragma unroll 1
        for (int attempt = 0; attempt < 3; ++attempt) {
          bin_keys(b_lo, b_hi, &klo, &khi);
          klo = max(klo, floor_key);
          const float x_lo = order_value<E::kLowBits>(klo), x_hi = order_value<E::kLowBits>(khi);
          if (tid == 0) sm.keys = 0;
          __syncthreads();
          uint64_t all, top;
          auto list = [&](const float (&x)[kVec]) {
#pragma unroll
            for (int j = 0; j < kVec; ++j)
              if (x[j] >= x_lo && x[j] <= x_hi) list_key(order_key<E::kLowBits>(x[j]));
          };
          if (exact) {
            uint32_t all_h = 0, top_h = 0;
            int32_t all_l = 0, top_l = 0;
            each_granule([&](const float (&x)[kVec], int) {
              bool any = false;
#pragma unroll
              for (int j = 0; j < kVec; ++j) any |= x[j] >= floor_x;
              if (!any) return;  // (most, where there is a top-k cut)
#pragma unroll
              for (int j = 0; j < kVec; j += 2) {
                int32_t h[2], l[2];
                weights_of(make_float2(x[j], x[j + 1]), ex, sm.table, h, l);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  if (x[j + i] > floor_x) all_h += h[i], all_l += l[i];
                  if (x[j + i] > x_hi) top_h += h[i], top_l += l[i];
                }
              }
              list(x);
            });
            all = units(all_h, all_l), top = units(top_h, top_l);
          } else {
            const About ab = about(ex);
            const float x_least = fmaxf(floor_x, mx - kOctaves * 0.6931472f * temp);
            const float x_top = fmaxf(x_hi, x_least);
            // (`all` is made of the numbers that make `top`, and those of the rest: their errors are the same in
            // both; a tree over all of a granule would round a large token's sum with its small neighbours again)
            float rest_s = 0.f, rest_e = 0.f, top_s = 0.f, top_e = 0.f;
            each_granule([&](const float (&x)[kVec], int) {
              float w[kVec], high[kVec];
              about_all(x, ab, w);
#pragma unroll
              for (int j = 0; j < kVec; ++j) {
                high[j] = x[j] > x_top ? w[j] : 0.f;
                w[j] = x[j] > x_least && !(x[j] > x_top) ? w[j] : 0.f;
              }
              add_in_two(tree_sum(w), &rest_s, &rest_e);
              add_in_two(tree_sum(high), &top_s, &top_e);
              list(x);
            });
            top = about_units(top_s, top_e), all = about_units(rest_s, rest_e) + top;
          }
          all = warp_add(all), top = warp_add(top);
          if (lane == 0) sm.warp_u64[warp] = all, sm.warp_u64b[warp] = top;
          __syncthreads();
          if (tid == 0) {
            all = top = 0;
            for (int w = 0; w < kWarps; ++w) all += sm.warp_u64[w], top += sm.warp_u64b[w];
            sm.sum_a = all, sm.sum_b = top;
          }
          sync_all();
          const uint64_t last = with_k ? (uint64_t)cut_keep * weight_units(cut_x, ex, sm.table) : 0;
          all = last, top = 0;
          if (exact) {
            for (int r = 0; r < C; ++r) all += of(r).sum_a, top += of(r).sum_b;
          } else {
            // without the factor that about_of's weights share, a power of two from -1/2 to 1/2
            const About ab = about(ex);
            const float d = __fmaf_rn(-mx, ab.lo, __fmaf_rn(-mx, ab.hi, -__fsub_rn(ab.magic, 12582912.f)));
            const uint64_t by = fixed<63>(ex2_approx(d));
            for (int r = 0; r < C; ++r)
              all += __umul64hi(of(r).sum_a, by) << 1, top += __umul64hi(of(r).sum_b, by) << 1;
          }
          // (0, or over 2^63, where the cut lies above these bins)
          const uint64_t within = least_mass(all) - top;
          uint64_t left = within;
          if (!refine(klo, khi, true, true, &left, &equal, &klo)) {
            if (exact) b_lo = 0, b_hi = bin_k;
            exact = true;
            continue;
          }
          const float x = order_value<E::kLowBits>(klo);
          const uint64_t w = weight_units(x, ex, sm.table);
          const uint32_t keep = w > 0 ? (uint32_t)min((left + w - 1) / w, (uint64_t)equal) : equal;
          if (!exact) {
            // p all - top is off by at most the error of p (all - top) + (1 - p) top, and by that of the
            // factor (1.7e-7) in what is left of it, or in what the tokens at top-k's cut add to it
            const float off = top_p * (float)(all - top) + (1.f - top_p) * (float)top;
            const uint64_t margin =
                (uint64_t)(off * (1.01f * kAboutError) + ((float)within + (float)last) * 1.8e-7f) + 2 * kAboutUnits;
            exact = true;
            if (left <= (keep - 1) * w + margin || left + margin > keep * w) continue;
          }
          if (with_k && x == cut_x) cut_keep = min(cut_keep, keep);
          else cut_x = x, cut_keep = keep;
          break;
        }
      }
    }
  }
  if (min_p > 0.f) {
    // w >= min_p  <=>  x >= max + T ln(min_p)
    const float x = sum_rounded_up(mx, sm.ln_hi, sm.ln_lo);
    if (x > cut_x) cut_x = x, cut_keep = kAllEqual;
  }

  // ---- the draw, in the order of the places: sums of the weights above cut_x and counts of the tokens
  // equal to it, per warp, per CTA, and in the one warp whose run holds the token, per iteration, lane
  // and place.  With `exact` false in single precision: sm.sure tells whether that decides the token.
  const bool partial = cut_keep != kAllEqual;
  const float over = partial ? cut_x : nextafterf(cut_x, -INFINITY);  // kept whole: x > over
  const About ab = about(ex);
  const float x_zero = mx - kOctaves * 0.6931472f * temp;  // the single-precision sums leave out what lies below
  const float over_about = fmaxf(over, x_zero);  // (x_zero < mx where |max c| < kAboutMax)
  auto draw = [&](auto exactly) {
    constexpr bool exact = decltype(exactly)::value;
    // the weights of a granule's tokens above the cut: each in units, or their sum, and how many are equal to it
    auto about_weights = [&](const float (&x)[kVec], float (&w)[kVec]) {
      about_all(x, ab, w);
#pragma unroll
      for (int k = 0; k < kVec; ++k) w[k] = x[k] > over_about ? w[k] : 0.f;
    };
    auto mass = [&](const float (&x)[kVec], uint32_t* equal) -> uint64_t {
      *equal = 0;
      if (partial)
#pragma unroll
        for (int k = 0; k < kVec; ++k) *equal += x[k] == cut_x ? 1u : 0u;
      if (exact) {
        uint64_t m = 0;
#pragma unroll 1
        for (int k = 0; k < kVec; ++k) m += x[k] > over ? weight_units(x[k], ex, sm.table) : 0;
        return m;
      }
      float w[kVec];
      about_weights(x, w);
      return about_units(tree_sum(w));
    };
    const uint64_t w_cut =
        !partial ? 0 : exact ? weight_units(cut_x, ex, sm.table) : cut_x >= x_zero ? about_units(about_of(cut_x, ab)) : 0;
    // what the tokens numbered [from, to) of those equal to cut_x add
    auto equals = [&](uint32_t from, uint32_t to) { return w_cut * (min(to, cut_keep) - min(from, cut_keep)); };
    uint64_t sum;
    uint32_t same = 0;
    if (exact) {
      // the kept tokens, a quarter or less of many rows, are gathered first (in the histogram's place) and
      // weighed 64 at a time by a warp
      uint32_t h = 0;
      int32_t l = 0;
      float* kept = sm.kept[warp];
      int n = 0;
      auto weigh = [&](float2 x) {
        int32_t wh[2], wl[2];
        weights_of(x, ex, sm.table, wh, wl);
        h += wh[0] + wh[1];
        l += wl[0] + wl[1];
      };
      each_granule([&](const float (&x)[kVec], int) {
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
          const bool keep = x[k] > over;
          const uint32_t who = __ballot_sync(0xffffffffu, keep);
          if (keep) kept[n + __popc(who & ((1u << lane) - 1u))] = x[k];
          n += __popc(who);
          if (partial) same += x[k] == cut_x ? 1u : 0u;
        }
        __syncwarp();
        for (; n >= 64; n -= 64) weigh(make_float2(kept[n - 64 + lane], kept[n - 32 + lane]));
        __syncwarp();
      });
      weigh(make_float2(lane < n ? kept[lane] : -INFINITY, lane + 32 < n ? kept[lane + 32] : -INFINITY));
      sum = units(h, l);
    } else {
      float s = 0.f, e = 0.f;  // the sum in two floats
      each_granule([&](const float (&x)[kVec], int) {
        float w[kVec];
        about_weights(x, w);
        if (partial)
#pragma unroll
          for (int k = 0; k < kVec; ++k) same += x[k] == cut_x ? 1u : 0u;
        add_in_two(tree_sum(w), &s, &e);
      });
      sum = about_units(s, e);
    }
    sum = warp_add(sum);
    same = warp_add(same);
    __syncthreads();
    if (lane == 0) sm.warp_u64[warp] = sum, sm.warp_u32[warp] = same;
    __syncthreads();
    if (tid == 0) {
      uint64_t s = 0;
      uint32_t n = 0;
      for (int w = 0; w < kWarps; ++w) s += sm.warp_u64[w], n += sm.warp_u32[w];
      sm.sum_a = s, sm.count = n;
    }
    sync_all();
    uint64_t all = 0, before = 0, here = 0;  // mass of the row, of the CTAs before this one, and of this one
    uint32_t ahead = 0, seen = 0;            // tokens equal to cut_x before this CTA; before CTA r
    for (int r = 0; r < C; ++r) {
      const uint32_t n = of(r).count;
      const uint64_t m = of(r).sum_a + equals(seen, seen + n);
      if (r == rank) before = all, here = m, ahead = seen;
      all += m;
      seen += n;
    }
    // the token's running sum is the first above `goal` = floor(u all)
    const uint64_t goal = __umul64hi(u64, all);
    if (before <= goal && goal < before + here) {  // one CTA of the cluster
      // Of 32 runs of places, this lane's of mass m with n tokens equal to cut_x, the one that holds the
      // goal, or -1: the last one that begins at or before it.  `before` and `ahead` move to its start.
      auto run_of = [&](uint64_t m, uint32_t n) {
        const uint32_t nth = ahead + warp_scan(n, lane) - n;
        m += equals(nth, nth + n);
        const uint64_t upto = before + warp_scan(m, lane);
        const uint32_t past = __ballot_sync(0xffffffffu, upto > goal);
        const int at = past ? __ffs(past) - 1 : 31;
        before = __shfl_sync(0xffffffffu, past ? upto - m : upto, at);
        ahead = __shfl_sync(0xffffffffu, past ? nth : nth + n, at);
        return past ? at : -1;
      };
      const int w0 = max(run_of(lane < kWarps ? sm.warp_u64[lane] : 0, lane < kWarps ? sm.warp_u32[lane] : 0), 0);
      // that warp's places, one iteration's per warp of this CTA
      for (int i = warp; iters > 1 && i < iters; i += kWarps) {
        float x[kVec];
        values(fetch(w0, i), x);
        uint32_t n;
        uint64_t m = mass(x, &n);
        m = warp_add(m);
        n = warp_add(n);
        if (lane == 0) sm.chunk[i] = m, sm.chunk_same[i] = n;
      }
      __syncthreads();
      if (warp == 0) {
        int i = iters > 1 ? -1 : 0;
        for (int i0 = 0; i < 0 && i0 < iters; i0 += 32) {
          const bool in = i0 + lane < iters;
          const int at = run_of(in ? sm.chunk[i0 + lane] : 0, in ? sm.chunk_same[i0 + lane] : 0);
          if (at >= 0) i = i0 + at;
        }
        i = max(i, 0);  // (in single precision the parts can miss the sum of the whole)
        float x[kVec];
        values(fetch(w0, i), x);
        uint32_t n;
        const uint64_t m = mass(x, &n);
        const int lane_at = run_of(m, n);
        if (lane == lane_at) {
          // (before and ahead are this lane's now: `before` is made of the numbers that make `all`)
          const uint64_t start = before;
          float w[kVec];
          if (!exact) about_weights(x, w);
#pragma unroll(exact ? 1 : kVec)
          for (int k = 0; k < kVec; ++k) {
            const bool eq = partial && x[k] == cut_x;
            const uint64_t own = eq ? equals(ahead, ahead + 1)
                                    : !exact ? about_units(w[k]) : x[k] > over ? weight_units(x[k], ex, sm.table) : 0;
            if (eq) ++ahead;
            if (before <= goal && goal < before + own) {
              a.token[row] = (rank * kWarps + w0) * seg + i * kStep + lane * kVec + k - shift;
              if (!exact && goal - before >= about_margin(u, all, before - start, kTreeError) &&
                  before + own - goal > about_margin(u, all, before + own - start, kTreeError))
                to_all(&Shared::sure, 1);
            }
            before += own;
          }
        }
      }
    }
    sync_all();  // sm.sure is settled, and no CTA leaves while another reads its shared memory
  };
  bool sure = false;
  if (fabsf(mx * ex.hi) < kAboutMax) {
    draw(std::false_type{});
    sure = sm.sure != 0;
  }
  if (!sure) draw(std::true_type{});
}

// A row that single-precision sums did not decide, until the exact ones have.
constexpr int32_t kUndecided = INT32_MIN;

// Temperature alone (no filter given): one pass over the row.  A thread sums its weights in single
// precision (about_of) against a bias of its own, from its first logits, which powers of two bring to
// the row's later; the token's run is read again, from L2.  A greedy row needs its maximum and place.
// Rows that this does not decide (and rows with +inf, or of logits beyond about_of's range) are marked
// for the launch after it.
struct PlainShared {
  float2 table[64];
  uint64_t warp_u64[kWarps], chunk[kMaxChunks];
  float warp_f[kWarps];
  uint32_t marked[kWarps];
  float exp_hi, exp_lo;
  // read by the other CTAs of the cluster
  uint64_t sum, best;
  float x_max;
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 3)
sample_plain_kernel(const SampleArgs a, int iters) {
  using E = Elems<T>;
  constexpr int kVec = E::kVec;
  constexpr int kStep = 32 * kVec;
  __shared__ PlainShared sm;
  grid_dependents_launch();
  const cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = (int64_t)blockIdx.x / C;
  const T* src = static_cast<const T*>(a.logits) + row * a.stride;
  const int shift = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
  const T* base = src - shift;
  const int end = a.vocab + shift, seg = iters * kStep;
  const int first = (rank * kWarps + warp) * seg + lane * kVec;
  const bool whole = (rank * kWarps + warp) * seg >= shift && (rank * kWarps + warp + 1) * seg <= end;
  auto granule = [&](int p, bool inside = false) {
    uint4 v;
    if (inside || (p >= shift && p + kVec <= end)) {
      asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                   : "l"(base + p));
    } else {
      float x[kVec];
#pragma unroll
      for (int k = 0; k < kVec; ++k) x[k] = p + k >= shift && p + k < end ? E::one(base + p + k) : -INFINITY;
      v = E::pack(x);
    }
    return v;
  };
  constexpr int kAhead = 2;
  uint4 ahead[kAhead];
#pragma unroll
  for (int h = 0; h < kAhead; ++h)
    if (h < iters) ahead[h] = granule(first + h * kStep, whole);
  const float temp = a.temperature ? __ldg(a.temperature + row) : 1.f;
  const float u = __ldg(a.uniform + row);
  const bool good = (temp == 0.f || (temp >= kSampleMinTemp && temp <= kSampleMaxTemp)) && u >= 0.f && u <= 1.f;
  if (!good) {  // the same in every thread of the cluster
    if (rank == 0 && tid == 0) {
      record_status(a.status, VMLA_ERR_PARAM, (uint32_t)row);
      a.token[row] = -1;
    }
    return;
  }
  const bool greedy = temp == 0.f;
  if (tid == 0 && !greedy) {
    const double c = 1.4426950408889634 / (double)temp;
    sm.exp_hi = (float)c;
    sm.exp_lo = (float)(c - (double)sm.exp_hi);
  }
  __syncthreads();
  About ab;
  ab.hi = greedy ? 0.f : sm.exp_hi, ab.lo = greedy ? 0.f : sm.exp_lo, ab.magic = 12582912.f;
  float mx = -INFINITY, s = 0.f, e = 0.f, low = 0.f, high = -INFINITY;
  int at = 0;  // iteration of the first granule with this thread's maximum
#pragma unroll 1
  for (int i0 = 0; i0 < iters; i0 += kAhead) {
#pragma unroll
    for (int h = 0; h < kAhead; ++h) {
      const int i = i0 + h;
      if (i >= iters) break;
      float x[kVec];
      E::unpack(ahead[h], x);
      typename E::Max gm = E::lowest();
      E::settle(ahead[h], gm);
      const float g = E::largest(gm);
      if (i + kAhead < iters) ahead[h] = granule(first + (i + kAhead) * kStep, whole);
      if (g > mx) mx = g, at = i;
      if (greedy) continue;
      if (g > high && fabsf(g * ab.hi) < kAboutMax) {
        // a bias for this thread's first numbers, or for weights over 2^64 times what it is for
        const float magic = __fadd_rn(12582912.f, rintf(-g * ab.hi));
        const float by = power_of_two(magic - ab.magic);  // (at the first, of a sum of zero)
        s *= by, e *= by;
        ab.magic = magic;
        high = g + 64.f / ab.hi;
        low = g - 100.f / ab.hi;
      }
      float w[kVec];
#pragma unroll
      for (int k = 0; k < kVec; ++k) w[k] = about_of(fmaxf(x[k], low), ab);  // NaN and what lies 2^-100 below: next to nothing
#pragma unroll
      for (int o = kVec / 2; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < o; ++k) w[k] = __fadd_rn(w[k], w[k + o]);
      if (high > -INFINITY) add_in_two(w[0], &s, &e);
    }
  }
  const float own_max = mx;
  mx = warp_max(mx);
  if (lane == 0) sm.warp_f[warp] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm.warp_f[w]);
  if (greedy) {
    // the first place of the largest value: its thread reads the granule again
    uint64_t best = 0;
    if (own_max == mx && mx > -INFINITY) {
      float x[kVec];
      E::unpack(granule(first + at * kStep), x);
      int place = 0;
#pragma unroll
      for (int k = kVec - 1; k >= 0; --k) place = x[k] == mx ? first + at * kStep + k : place;
      best = ((uint64_t)order_key<0>(mx) << 32) | (uint32_t)~place;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    if (lane == 0) sm.warp_u64[warp] = best;
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < kWarps; ++w) best = max(best, sm.warp_u64[w]);
      sm.best = best;
    }
    cluster.sync();
    if (rank == 0 && tid == 0) {
      for (int r = 0; r < C; ++r) best = max(best, *cluster.map_shared_rank(&sm.best, r));
      a.token[row] = best == 0 ? -1 : (int32_t)~(uint32_t)best - shift;
    }
    cluster.sync();
    return;
  }
  // this thread's sum at the CTA's bias, and the CTA's at its own
  const float magic = __fadd_rn(12582912.f, rintf(-mx * ab.hi));
  uint64_t sum = 0;
  if (high > -INFINITY && fabsf(mx * ab.hi) < kAboutMax) {
    const float by = power_of_two(magic - ab.magic);
    sum = about_units(s * by, e * by);
  }
  sum = warp_add(sum);
  if (lane == 0) sm.warp_u64[warp] = sum;
  __syncthreads();
  if (tid == 0) {
    sum = 0;
    for (int w = 0; w < kWarps; ++w) sum += sm.warp_u64[w];
    sm.sum = sum;
    sm.x_max = mx;
  }
  cluster.sync();
  const float cta_max = mx;
  for (int r = 0; r < C; ++r) mx = fmaxf(mx, *cluster.map_shared_rank(&sm.x_max, r));
  // A thread (and a CTA) whose largest exponent is not below kAboutMax in magnitude has no bias and adds nothing:
  // with the row's at least 64 inside, what such a thread has is infinite, or below 2^-63 of the row's largest.
  if (!(mx > -INFINITY && fabsf(mx * ab.hi) < kAboutMax - 64.f)) {
    if (rank == 0 && tid == 0) a.token[row] = mx == -INFINITY ? -1 : kUndecided;
    cluster.sync();
    return;
  }
  // everything at the row's bias: a CTA's units by a power of two
  const Exponent ex = {mx, ab.hi, ab.lo};
  ab = about(ex);
  auto shift_of = [&](float m) {
    const float d = m > -INFINITY ? rintf(-m * ab.hi) - rintf(-mx * ab.hi) : 63.f;
    return (int)fminf(fmaxf(d, 0.f), 63.f);
  };
  uint64_t all = 0, before = 0, here = 0;
  for (int r = 0; r < C; ++r) {
    const uint64_t m = *cluster.map_shared_rank(&sm.sum, r) >> shift_of(*cluster.map_shared_rank(&sm.x_max, r));
    if (r == rank) before = all, here = m;
    all += m;
  }
  const uint64_t goal = u < 1.f ? __umul64hi((uint64_t)(u * 18446744073709551616.f), all) : all - 1;
  if (before <= goal && goal < before + here) {  // one CTA of the cluster
    const int down = shift_of(cta_max);
    const float x_zero = mx - kOctaves * 0.6931472f * temp;
    auto weight = [&](float x) -> uint64_t { return x > x_zero ? about_units(about_of(x, ab)) : 0; };
    int w0 = 0;
    for (; w0 < kWarps - 1; ++w0) {
      const uint64_t m = sm.warp_u64[w0] >> down;
      if (goal < before + m) break;
      before += m;
    }
    const uint64_t run = before;  // (up to here made of the numbers that make `all`)
    const int start = (rank * kWarps + w0) * seg + lane * kVec;
    for (int i = warp; i < iters; i += kWarps) {
      float x[kVec];
      E::unpack(granule(start + i * kStep), x);
      uint64_t m = 0;
#pragma unroll
      for (int k = 0; k < kVec; ++k) m += weight(x[k]);
      m = warp_add(m);
      if (lane == 0) sm.chunk[i] = m;
    }
    __syncthreads();
    if (warp == 0) {
      int i = 0;
      for (; i < iters - 1 && before + sm.chunk[i] <= goal; ++i) before += sm.chunk[i];
      float x[kVec];
      uint64_t m = 0, w[kVec];
      E::unpack(granule(start + i * kStep), x);
#pragma unroll
      for (int k = 0; k < kVec; ++k) m += w[k] = weight(x[k]);
      uint64_t upto = before + warp_scan(m, lane) - m;
      // the token, or a mark where no sum, or one next to the goal, decides
      int token = kUndecided;
      uint64_t low = 0, high = 0;  // its borders
#pragma unroll
      for (int k = 0; k < kVec; ++k) {
        if (upto <= goal && goal < upto + w[k]) token = start + i * kStep + k - shift, low = upto, high = upto + w[k];
        upto += w[k];
      }
      if (token != kUndecided && (goal - low < about_margin(u, all, low - run, kAnewError) ||
                                  high - goal <= about_margin(u, all, high - run, kAnewError)))
        token = kUndecided;
      const uint32_t found = __ballot_sync(0xffffffffu, token != kUndecided);
      if (found ? lane == __ffs(found) - 1 : lane == 0) a.token[row] = token;
    }
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
}

// The rows that the launch before left undecided, by exact sums: cluster c takes rows c, c + (clusters),
// and so on.  (Loops over a granule's elements are rolled: few rows come here, and the time of their
// instructions' first fetch would outweigh that of running them.)
template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
sample_plain_exact_kernel(const SampleArgs a, const __grid_constant__ ExpTable exp_table, int iters) {
  using E = Elems<T>;
  constexpr int kVec = E::kVec;
  constexpr int kStep = 32 * kVec;
  __shared__ PlainShared sm;
  const cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t clusters = gridDim.x / C;
  if (tid < 64) sm.table[tid] = exp_table.t[tid];
  grid_dependency_wait();
  for (int64_t first_row = blockIdx.x / C; first_row < a.rows; first_row += clusters * kThreads) {
    // the marks of the next kThreads of this cluster's rows, read by every CTA before one is cleared
    const int64_t my_row = first_row + tid * clusters;
    const bool mark = my_row < a.rows && *reinterpret_cast<volatile int32_t*>(a.token + my_row) == kUndecided;
    const uint32_t word = __ballot_sync(0xffffffffu, mark);
    __syncthreads();
    if (lane == 0) sm.marked[warp] = word;
    cluster.sync();
    for (int mw = 0; mw < kWarps; ++mw) {
      for (uint32_t left = sm.marked[mw]; left != 0; left &= left - 1) {
        const int64_t row = first_row + (32 * mw + __ffs(left) - 1) * clusters;
        const T* src = static_cast<const T*>(a.logits) + row * a.stride;
        const int shift = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
        const int seg = iters * kStep;
        // the logit at a place, -inf outside the row
        auto logit = [&](int p) {
          return p >= shift && p < a.vocab + shift ? fmaxf(E::one(src - shift + p), -INFINITY) : -INFINITY;
        };
        const int first = (rank * kWarps + warp) * seg + lane * kVec;
        float mx = -INFINITY;
        for (int i = 0; i < iters; ++i)
#pragma unroll
          for (int k = 0; k < kVec; ++k) mx = fmaxf(mx, logit(first + i * kStep + k));
        mx = warp_max(mx);
        if (lane == 0) sm.warp_f[warp] = mx;
        const float temp = a.temperature ? __ldg(a.temperature + row) : 1.f, u = __ldg(a.uniform + row);
        if (tid == 0) {
          const double c = 1.4426950408889634 / (double)temp;
          sm.exp_hi = (float)c;
          sm.exp_lo = (float)(c - (double)sm.exp_hi);
        }
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm.warp_f[w]);
        if (tid == 0) sm.x_max = mx;
        cluster.sync();
        for (int r = 0; r < C; ++r) mx = fmaxf(mx, *cluster.map_shared_rank(&sm.x_max, r));
        const bool only_inf = mx == INFINITY;  // tokens at +inf share the draw evenly
        const Exponent ex = {only_inf ? 0.f : mx, sm.exp_hi, sm.exp_lo};
        auto scaled = [&](int p) {
          const float x = logit(p);
          return !only_inf ? x : x == INFINITY ? 0.f : -INFINITY;
        };
        auto weight = [&](int p) { return weight_units(scaled(p), ex, sm.table); };
        auto weight2 = [&](int p) {  // of two places
          int32_t h[2], l[2];
          weights_of(make_float2(scaled(p), scaled(p + 1)), ex, sm.table, h, l);
          return units((int64_t)h[0] + h[1], (int64_t)l[0] + l[1]);
        };
        uint64_t sum = 0;
        for (int i = 0; i < iters; ++i)
#pragma unroll 1
          for (int k = 0; k < kVec; k += 2) sum += weight2(first + i * kStep + k);
        sum = warp_add(sum);
        if (lane == 0) sm.warp_u64[warp] = sum;
        __syncthreads();
        if (tid == 0) {
          sum = 0;
          for (int w = 0; w < kWarps; ++w) sum += sm.warp_u64[w];
          sm.sum = sum;
        }
        cluster.sync();
        uint64_t all = 0, before = 0, here = 0;
        for (int r = 0; r < C; ++r) {
          const uint64_t m = *cluster.map_shared_rank(&sm.sum, r);
          if (r == rank) before = all, here = m;
          all += m;
        }
        const uint64_t goal = u < 1.f ? __umul64hi((uint64_t)(u * 18446744073709551616.f), all) : all - 1;
        if (before <= goal && goal < before + here) {
          int w0 = 0;
          for (; w0 < kWarps - 1 && before + sm.warp_u64[w0] <= goal; ++w0) before += sm.warp_u64[w0];
          const int start = (rank * kWarps + w0) * seg + lane * kVec;
          for (int i = warp; i < iters; i += kWarps) {
            uint64_t m = 0;
#pragma unroll 1
            for (int k = 0; k < kVec; k += 2) m += weight2(start + i * kStep + k);
            m = warp_add(m);
            if (lane == 0) sm.chunk[i] = m;
          }
          __syncthreads();
          if (warp == 0) {
            int i = 0;
            for (; i < iters - 1 && before + sm.chunk[i] <= goal; ++i) before += sm.chunk[i];
            uint64_t m = 0;
#pragma unroll 1
            for (int k = 0; k < kVec; k += 2) m += weight2(start + i * kStep + k);
            uint64_t upto = before + warp_scan(m, lane) - m;
            if (upto <= goal && goal < upto + m) {
              int k = 0;
              for (uint64_t w; k < kVec - 1 && upto + (w = weight(start + i * kStep + k)) <= goal; ++k) upto += w;
              a.token[row] = start + i * kStep + k - shift;
            }
          }
        }
        cluster.sync();  // every CTA has read the others' sums; this row's shared memory may be written again
      }
    }
  }
}

// CTAs per row: more while that leaves SMs idle, or while rows are long (over 8 iterations of 8 KB a CTA) and
// most of the CTAs still find room at once (clusters do not fill every SM: 76 rows by four did not fit), or while
// they are longer (over 20) and the CTAs take at most two rounds; eight only while SMs idle.  More too while
// one CTA's share of a row is over 40 iterations (bf16: 33, what kMaxElems allows: 135,168 tokens); the row stays in
// shared memory where a share is at most 64 KB.  The rule does not look at which filters are given: 128 rows of
// 151,001 fp32 get four CTAs, 85 us with all filters (91 by two), 139 with top-p alone (140 by two), but
// 125 (108 by two) with top-p alone where many tokens are at -inf.
// Measured, us by cluster size 1 / 2 / 4 / 8, top-p of 131,072 bf16: 512 rows 130 / 148 / 190 / 336, 300 rows 100 / 94 /
// 123 / 202, 150 rows 55 / 50 / 72 / 110, 76 rows 53 / 37 / 47 / 66, 64 rows 53 / 35 / 31 / 51, 16 rows 51 / 35 / 24 / 26; all
// filters of 151,001 fp32: 512 rows - / 205 / 245 / 390, 300 rows - / 146 / 157 / 240, 128 rows - / 89 / 83 / 116, 76 rows
// - / 89 / 73 / 91, 16 rows - / 53 / 42 / 39; of 64,000: 512 rows 116 / 126 / 155 / 293, 128 rows 65 / 56 / 56 / 95; all filters
// of 32,000 bf16: 400 rows 42 / 61 / 93 / 171, 100 rows 24 / 27 / 34 / 51, 8 rows 23 / 23 / 20 / 19.
struct Shape {
  int cluster, iters;
  bool keep;
};
template <typename T>
int iterations(const SampleArgs& a, int cluster) {
  const bool aligned = (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0 && a.stride * sizeof(T) % 16 == 0;
  const int64_t places = (int64_t)a.vocab + (aligned ? 0 : Elems<T>::kVec - 1);
  const int64_t per = (int64_t)cluster * (kChunkBytes / sizeof(T));
  return (int)((places + per - 1) / per);
}
template <typename T>
Shape choose_shape(const SampleArgs& a, int sms) {
  auto need = [&](int c) { return iterations<T>(a, c); };
  constexpr int kMost = std::min(40, kMaxElems / Elems<T>::kVec);
  Shape s;
  s.cluster = 1;  // (a vocabulary of up to kList tokens stays in one CTA: one iteration holds it)
  while (s.cluster < kMaxCluster && need(s.cluster) > 1) {
    const int64_t ctas = a.rows * s.cluster * 2;
    const int n = need(s.cluster), room = s.cluster == 4 ? sms : n > 20 ? 4 * sms : sms + sms * 3 / 4;
    if (!(n > kMost || ctas <= sms / 2 || (n > 8 && ctas <= room))) break;
    s.cluster *= 2;
  }
  s.iters = need(s.cluster);
  s.keep = s.iters <= kKeepIters;
  return s;
}
// Without filters a CTA does one pass and two more barriers: more CTAs per row pay off only while all are
// resident.  Us by cluster size 1 / 2 / 4 / 8, both launches: 512 rows of 131,072 bf16 81 / 80 / 95 / 141, 150
// rows 37 / 34 / 40 / 51, 64 rows 37 / 29 / 28 / 35, one row 23 / 17 / 14 / 13; 400 rows of 32,000 25 / 32 / 42 / 79.
template <typename T>
Shape choose_plain_shape(const SampleArgs& a, int sms) {
  auto need = [&](int c) { return iterations<T>(a, c); };
  Shape s;
  s.cluster = 1;
  while (s.cluster < kMaxCluster && need(s.cluster) > 1 &&
         (a.rows * s.cluster * 2 <= 2 * sms || need(s.cluster) > 20 ||
          need(s.cluster) > kMaxElems / Elems<T>::kVec))
    s.cluster *= 2;
  s.iters = need(s.cluster);
  s.keep = false;
  return s;
}

template <typename... Params, typename... Args>
bool launch_clusters(void (*kernel)(Params...), int64_t rows, int cluster, size_t smem, bool early, cudaStream_t stream,
                     const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1] = early_start_attribute();
  cfg.gridDim = dim3((unsigned)(rows * cluster), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

template <typename T>
int launch(const SampleArgs& a, int sms, int dev, cudaStream_t stream) {
  const ExpTable& table = exp_table();
  const bool plain = !a.top_k && !a.top_p && !a.min_p;
  const Shape shape = plain ? choose_plain_shape<T>(a, sms) : choose_shape<T>(a, sms);
  if (shape.iters > kMaxElems / Elems<T>::kVec || a.rows * shape.cluster > INT32_MAX) return VMLA_ERR_SHAPE;
  if (plain) {
    // then its undecided rows, on clusters of eight that are all resident (two CTAs on an SM, and some
    // SMs of a GPC left over)
    const int64_t room = sms / 5 > 0 ? sms / 5 : 1, clusters = a.rows < room ? a.rows : room;
    if (!launch_clusters(sample_plain_kernel<T>, a.rows, shape.cluster, 0, false, stream, a, shape.iters) ||
        !launch_clusters(sample_plain_exact_kernel<T>, clusters, kMaxCluster, 0, true, stream, a, table,
                         iterations<T>(a, kMaxCluster)))
      return VMLA_ERR_CUDA;
    return VMLA_OK;
  }
  if (shape.keep) {
    static bool ready[64] = {};
    static std::mutex mu;
    std::lock_guard<std::mutex> g(mu);
    // (all of the SM's memory as shared memory, so that two CTAs fit)
    if (dev >= 64 || !ready[dev]) {
      if (cudaFuncSetAttribute(sample_kernel<T, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kKeepIters * kChunkBytes) != cudaSuccess ||
          cudaFuncSetAttribute(sample_kernel<T, true>, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared) != cudaSuccess)
        return VMLA_ERR_CUDA;
      if (dev < 64) ready[dev] = true;
    }
  }
  const auto kernel = shape.keep ? sample_kernel<T, true> : sample_kernel<T, false>;
  const size_t smem = shape.keep ? (size_t)shape.iters * kChunkBytes : 0;
  if (!launch_clusters(kernel, a.rows, shape.cluster, smem, false, stream, a, table, shape.iters)) return VMLA_ERR_CUDA;
  return VMLA_OK;
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
