// Beam search: the best continuations over a request's beams and the vocabulary, and the reordering of the beams'
// states.
//
// Beam w of a request (score c_w, logits x) continues with token v at the score
//   c_w + x_v - lse_w,   lse_w = ln sum_v exp(x_v),
// and the K best over all (w, v) are kept, in descending order, equal ones by the index w vocab + v.
//
// Within a beam the order is the logits' own, so a row's first K tokens by (logit, index) are all that can be kept.
// The first kernel reads each row once: a thread sums exp(x - r) against a reference r of its own, a logit (raised when
// a granule's maximum passes it by 8) and remembers its largest granule, (maximum, place).  The K-th largest of
// the threads' granules bounds the row's K-th token from below, and no token above the bound lies outside the K
// threads that have these granules: only their granules are read again (from L2), the tokens above the bound listed,
// and the list ranked.  Rows are cut into parts, one CTA each, while that is needed to fill the GPU.
// The second kernel, a CTA per request, joins the parts' sums and merges the sorted lists: the lists' heads are ranked,
// which leaves at most K (K + 1) / 2 entries, and one warp takes the best of them K times, a lane per list.
//
// Scores of different beams are compared through lse_w, and the single-precision terms put it off by up to about
// 4e-6 (kMargin).  Where two neighbours of the merged order, or the last of it and one that is left out, are of
// different beams and lie closer than that, the request's CTA sums the beams concerned again in whole units
// (weight_units, exact in any order: equal rows have equal sums wherever they lie) and merges anew, until no beam is
// left in doubt.  Scores closer than about 2^-27 are not told apart for certain.  A CTA takes 0.6 to 0.9 ns a token for
// this, the requests side by side: with two equal beams a call takes 75 us instead of 15 (4 beams of 32 000 tokens) or 234
// instead of 39 (64 x 8 of 131 072), with all equal 130 and 822, and 16 equal ones of 262 144 tokens 2.6 ms.
//
// Sums are kept as two floats (an exact sum of two): doubles cost more than all the rest, at their rate on this GPU.
//
// What bounds it: for many rows the logits, 2 or 4 bytes a token in, and the exponentials, 16 a clock and SM.  Measured:
// 64 x 8 beams of 131 072 tokens in bf16 (134 MB) 45 us, the rows' kernel 31 of them (4.3 TB/s; 60 % of the issue slots),
// the join 9, the reordering of tables of 4000 slots 7; 9 x 15 beams, 30 kept, of 151 001 tokens in fp32 (82 MB) 49 us:
// 24, 14 and 11; one request of four beams 16 us: 7, 8 and 4, all latency.  (Doubles in the loop, every thread ranked
// against all and the entries ranked against each other: 60, 77 and 18.4 us.)
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "vmla_device.cuh"
#include "vmla_weights.cuh"

namespace vmla {
using namespace weights;
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBeams = VMLA_MAX_BEAMS, kMaxKeep = VMLA_MAX_BEAM_KEEP;
constexpr int kMaxParts = 16;
constexpr int kList = 2048;      // tokens above the bound that are ranked at once
constexpr float kLowest = -3.402823466e38f;
constexpr float kAbove = 8.f;    // how far a thread's terms may lie above its reference (see kMargin)
constexpr float kLog2e = 1.44269504088896340736f;
constexpr double kLn2 = 0.69314718055994530942;
static_assert(kMaxKeep <= kThreads && kMaxBeams * kMaxParts <= kThreads, "a thread per place and per list");

// One part of a row: the sum of exp(x - ref), tokens at +inf, and the first n tokens as sorted keys.
struct alignas(16) RowPart {
  double sum;
  float ref;
  uint32_t infinite;
  uint32_t n;
  uint32_t pad[3];
  uint64_t key[kMaxKeep];
};

// Order of the logits as whole numbers (-0 like 0); -inf and NaN below every other, as 0.
__device__ __forceinline__ uint32_t ordered(float x) {
  if (!(x > -INFINITY)) return 0;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float ordered_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
// Larger keys first: by logit, then by the lower index.
__device__ __forceinline__ uint64_t key_of(uint32_t order, uint32_t index) { return (uint64_t)order << 32 | (uint32_t)~index; }

template <typename T>
struct Row {
  static constexpr int kVec = 16 / (int)sizeof(T);
  const T* first;    // aligned to 16 bytes, at or before the row's first element
  int lead;          // elements in front of the row
  int vocab;
  __device__ __forceinline__ Row(const void* logits, int64_t stride, int64_t row, int v) {
    const T* p = static_cast<const T*>(logits) + row * stride;
    lead = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    first = p - lead;
    vocab = v;
  }
  __device__ __forceinline__ int granules() const { return (vocab + lead + kVec - 1) / kVec; }
  // whether granule g lies in the row as a whole
  __device__ __forceinline__ bool whole(int g) const { return g * kVec >= lead && (g + 1) * kVec <= vocab + lead; }
  __device__ __forceinline__ static float value(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
  __device__ __forceinline__ static float value(float v) { return v; }
  // granule g's logits, -inf outside the row
  __device__ __forceinline__ void get(int g, float (&x)[kVec]) const {
    if (whole(g)) {
      unpack(__ldg(reinterpret_cast<const uint4*>(first) + g), x);
      return;
    }
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      const int i = g * kVec + k - lead;
      x[k] = i >= 0 && i < vocab ? value(__ldg(first + g * kVec + k)) : -INFINITY;
    }
  }
  __device__ __forceinline__ static void unpack(const uint4& v, float (&x)[kVec]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[2 * k] = bf16_lo(w[k]);
        x[2 * k + 1] = bf16_hi(w[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = __uint_as_float(w[k]);
    }
  }
};

// A granule's logits in pairs, and the largest of them (NaN left out, unless there is nothing else).
__device__ __forceinline__ float pairs_of(const uint4& v, float2 (&x)[4], uint16_t) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t m = w[0];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[k] = make_float2(bf16_lo(w[k]), bf16_hi(w[k]));
    if (k > 0) asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[k]));
  }
  return fmaxf(bf16_lo(m), bf16_hi(m));
}
__device__ __forceinline__ float pairs_of(const uint4& v, float2 (&x)[2], float) {
  x[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
  x[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
  return fmaxf(fmaxf(x[0].x, x[0].y), fmaxf(x[1].x, x[1].y));
}

// A thread's sum, as high + low + sum, and its largest granule.
struct Acc {
  float ref = kLowest, limit = -INFINITY, sum = 0.f, high = 0.f, low = 0.f, best = -INFINITY;
  int place = -1;
  uint32_t infinite = 0;

  template <int N>
  __device__ __forceinline__ void add(const float2 (&x)[N], float m, int g) {
    if (m > best) {
      best = m;
      place = g;
    }
    if (m > limit) {
      if (m == INFINITY) {  // those tokens share the row evenly
#pragma unroll
        for (int k = 0; k < N; ++k) infinite += (x[k].x == INFINITY) + (x[k].y == INFINITY);
        return;
      }
      const float f = ex2_approx((ref - m) * kLog2e);
      high *= f;
      low *= f;
      sum *= f;
      ref = m;
      limit = m + kAbove;
    }
    const float2 r = make_float2(-ref, -ref), scale = make_float2(kLog2e, kLog2e);
    float2 e[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float2 d = mul2(sum2(x[k], r), scale);
      e[k] = make_float2(ex2_approx(d.x), ex2_approx(d.y));
    }
#pragma unroll
    for (int s = N / 2; s > 0; s >>= 1)
#pragma unroll
      for (int k = 0; k < s; ++k) e[k] = sum2(e[k], e[k + s]);
    float t = e[0].x + e[0].y;
    if (t != t) {  // NaN counts as -inf
      t = 0.f;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        t += x[k].x > -INFINITY ? ex2_approx((x[k].x - ref) * kLog2e) : 0.f;
        t += x[k].y > -INFINITY ? ex2_approx((x[k].y - ref) * kLog2e) : 0.f;
      }
    }
    sum += t;
  }
  // (two-sum: high + low holds what single precision would drop)
  __device__ __forceinline__ void flush() {
    const float to = high + sum, part = to - high;
    low += (high - (to - part)) + (sum - part);
    high = to;
    sum = 0.f;
  }
  __device__ __forceinline__ double total() const { return (double)high + (double)low; }
};

struct RowShared {
  uint64_t list[kList];
  uint64_t warp_key[kWarps];
  uint8_t thread_of[kThreads];
  uint32_t warp_low[kWarps];
  int32_t thread[kMaxKeep];
  float warp_f[kWarps];
  double warp_d[kWarps];
  uint32_t warp_u[kWarps];
  uint64_t bound;
  uint32_t listed;
};
static_assert(kThreads <= 256 && kThreads <= kList, "the threads' list");

template <typename T>
__global__ void __launch_bounds__(kThreads, 4)
beam_rows_kernel(const BeamArgs a, RowPart* __restrict__ out, int parts) {
  constexpr int kVec = Row<T>::kVec;
  __shared__ RowShared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dependents_launch();
  const int64_t row_at = blockIdx.x / (unsigned)parts;
  const int part = (int)(blockIdx.x % (unsigned)parts);
  RowPart& r = out[blockIdx.x];
  const Row<T> row(a.logits, a.stride, row_at, a.vocab);
  const int all = row.granules(), per = (all + parts - 1) / parts;
  const int g0 = part * per, g1 = min(all, g0 + per);
  // four granules at a time, the next four on their way meanwhile
  constexpr int kAhead = 4, kRound = kAhead * kThreads;
  const int w0 = row.lead ? 1 : 0, w1 = min(g1, (a.vocab + row.lead) / kVec);  // granules in the row as a whole
  uint4 next[kAhead];
  auto fetch = [&](int g) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int h = g + k * kThreads;
      if (h >= w0 && h < w1) next[k] = __ldg(reinterpret_cast<const uint4*>(row.first) + h);
    }
  };
  fetch(g0 + tid);
  const float score = a.score[row_at];
  if (!(score > -INFINITY) || (a.finished && a.finished[row_at])) {  // nothing of its logits counts
    if (tid == 0) {
      r.n = 0;
      r.sum = 0.0;
      r.ref = -INFINITY;
      r.infinite = 0;
    }
    return;
  }
  Acc acc;
#pragma unroll 1
  for (int base = g0; base < g1; base += kRound) {
    const int g = base + tid;
    uint4 v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) v[k] = next[k];
    fetch(g + kRound);
    if (base >= w0 && base + kRound <= w1) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        float2 x[kVec / 2];
        const float m = pairs_of(v[k], x, T());
        acc.add(x, m, g + k * kThreads);
      }
    } else {
#pragma unroll 1
      for (int k = 0; k < kAhead; ++k) {
        const int h = g + k * kThreads;
        const uint4 q = k == 0 ? v[0] : k == 1 ? v[1] : k == 2 ? v[2] : v[3];
        if (h >= g1) break;
        float2 x[kVec / 2];
        float m;
        if (h >= w0 && h < w1) {
          m = pairs_of(q, x, T());
        } else {
          float y[kVec];
          row.get(h, y);
          m = y[0];
#pragma unroll
          for (int i = 1; i < kVec; ++i) m = fmaxf(m, y[i]);
#pragma unroll
          for (int i = 0; i < kVec / 2; ++i) x[i] = make_float2(y[2 * i], y[2 * i + 1]);
        }
        acc.add(x, m, h);
      }
    }
    acc.flush();
  }
  // the part's sum against its largest reference
  float ref = warp_max(acc.place >= 0 ? acc.ref : -INFINITY);
  if (lane == 0) s.warp_f[warp] = ref;
  const uint64_t mine = acc.place >= 0 ? key_of(ordered(acc.best), (uint32_t)acc.place) : 0;
  if (tid == 0) s.listed = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) ref = fmaxf(ref, s.warp_f[w]);
  double total = acc.place >= 0 ? acc.total() * (double)ex2_approx((acc.ref - ref) * kLog2e) : 0.0;
  uint32_t infinite = acc.infinite;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    infinite += __shfl_xor_sync(0xffffffffu, infinite, o);
  }
  if (lane == 0) {
    s.warp_d[warp] = total;
    s.warp_u[warp] = infinite;
  }
  // The K threads with the largest granules, and the K-th of these: each warp's ceil(K / warps)-th value bounds them
  // together, the threads at or above the least of these bounds are listed, and the list ranked.
  const int keep = a.keep;
  const uint32_t order = (uint32_t)(mine >> 32);
  uint32_t rest = order, low = 0;
  for (int n = (keep + kWarps - 1) / kWarps; n > 0; --n) {
    low = __reduce_max_sync(0xffffffffu, rest);
    if (rest == low) rest = 0;
  }
  if (lane == 0) s.warp_low[warp] = low;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) low = min(low, s.warp_low[w]);
  if (mine != 0 && order >= low) {
    const uint32_t at = atomicAdd(&s.listed, 1u);
    s.list[at] = mine;
    s.thread_of[at] = (uint8_t)tid;
  }
  __syncthreads();
  const int top = (int)s.listed;
  if (tid < top) {
    const uint64_t k = s.list[tid];
    int above = 0;
#pragma unroll 4
    for (int i = 0; i < top; ++i) above += s.list[i] > k;
    if (above < keep) {
      s.thread[above] = s.thread_of[tid];
      if (above == keep - 1) s.bound = k;
    }
  }
  __syncthreads();
  if (tid == 0) s.listed = 0;
  const int chosen = min(top, keep);
  const uint64_t bound = chosen == keep ? s.bound : 1;
  const uint32_t least = (uint32_t)(bound >> 32), last_place = ~(uint32_t)bound;
  __syncthreads();
  // their tokens at or above the bound (of the bound's own value, those up to its granule)
  const int rounds = (g1 - g0 + kThreads - 1) / kThreads;
  for (int i = tid; i < chosen * rounds; i += kThreads) {
    const int g = g0 + s.thread[i / rounds] + (i % rounds) * kThreads;
    if (g >= g1) continue;
    float x[kVec];
    row.get(g, x);
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      const uint32_t o = ordered(x[k]);
      if (o != 0 && (o > least || (o == least && (uint32_t)g <= last_place))) {
        const uint32_t at = atomicAdd(&s.listed, 1u);
        if (at < kList) s.list[at] = key_of(o, (uint32_t)(g * kVec + k - row.lead));
      }
    }
  }
  __syncthreads();
  const int listed = (int)s.listed;
  if (listed <= kList) {
    for (int i = tid; i < listed; i += kThreads) {
      const uint64_t k = s.list[i];
      int above = 0;
      for (int j = 0; j < listed; ++j) above += s.list[j] > k;
      if (above < keep) r.key[above] = k;
    }
  } else {
    // more than the list holds (many large tokens in few threads' granules): the next largest, K times
    uint64_t last = ~0ull;
    for (int n = 0; n < keep; ++n) {
      uint64_t best = 0;
      for (int g = g0 + tid; g < g1; g += kThreads) {
        float x[kVec];
        row.get(g, x);
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
          const uint32_t o = ordered(x[k]);
          const uint64_t key = o ? key_of(o, (uint32_t)(g * kVec + k - row.lead)) : 0;
          if (key < last && key > best) best = key;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint64_t u = __shfl_xor_sync(0xffffffffu, best, o);
        best = u > best ? u : best;
      }
      __syncthreads();
      if (lane == 0) s.warp_key[warp] = best;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) best = s.warp_key[w] > best ? s.warp_key[w] : best;
      if (tid == 0) r.key[n] = best;
      last = best;
    }
  }
  if (tid == 0) {
    double sum = 0.0;
    uint32_t inf = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      sum += s.warp_d[w];
      inf += s.warp_u[w];
    }
    r.sum = sum;
    r.ref = ref;
    r.infinite = inf;
    r.n = (uint32_t)min(listed, keep);
  }
}

struct JoinShared {
  double base[kMaxBeams];      // c_w - ln of the sum of exp(x - ref); beams with tokens at +inf: c_w - ln of their count
  float ref[kMaxBeams];
  bool infinite[kMaxBeams];
  float2 table[64];
  unsigned long long sum[kMaxBeams];
  uint32_t unsure;             // beams whose neighbours in the order lie too close, and whose sum is not exact yet
  uint32_t exact;              // beams whose sum is
  uint64_t head[kMaxBeams * kMaxParts];       // each list's best score, and its index
  uint32_t head_index[kMaxBeams * kMaxParts];
  int32_t count[kMaxBeams * kMaxParts];       // and its entries
  int32_t list[kMaxKeep];                     // the lists with the K best heads, in order
  uint64_t score[kMaxKeep][kMaxKeep];         // of the r-th of them the first K - r scores and indexes
  uint32_t place[kMaxKeep][kMaxKeep];
  uint64_t order[kMaxKeep];                   // the best scores in order, and their indexes
  uint32_t index[kMaxKeep];
};
static_assert(kMaxKeep <= 32, "a lane per list");

// Order of scores as whole numbers: 0 for none.
__device__ __forceinline__ uint64_t ordered64(double v) {
  if (!(v > -INFINITY)) return 0;
  const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
  return u >> 63 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ double ordered64_value(uint64_t k) {
  return __longlong_as_double((long long)(k >> 63 ? k & ~(1ull << 63) : ~k));
}
// Whether (score, index) a comes before b.
__device__ __forceinline__ bool before(uint64_t a, uint32_t ia, uint64_t b, uint32_t ib) {
  return a > b || (a == b && ia < ib);
}

// By how much a beam's score may be off, with u = 2^-24.  An exponent d puts its power of e off by 2.23 u |d| (the
// difference, log2 e as a float, their product).  A term x lies d <= kAbove above its thread's reference; from there the
// raises and the factors that join threads and parts lead up to the row's largest reference, by D + d together where
// the row's largest logit lies D above x, and the term has at most e^-D of the sum: (2 kAbove + D) e^-D 2.23 u is
// 2.12e-6 at the most, for D = 0.  Four powers (term, raise, thread, part) by ex2.approx, 2^-22 each, 9.6e-7; sums of
// 8 (one after the other where one is NaN) and of 4, and a raise's product, 12 u = 7.2e-7.
constexpr double kMargin = 4e-6;
static_assert(2 * kAbove * 2.23 / (1 << 24) + 4.0 / (1 << 22) + 12.0 / (1 << 24) < kMargin, "see above");

// Notes beams w and v whose scores a >= b lie closer than their sums are known to.
__device__ __forceinline__ void doubt(JoinShared& s, uint64_t a, int w, uint64_t b, int v) {
  if (w == v) return;
  const uint32_t open = (1u << w | 1u << v) & ~s.exact;
  if (open == 0) return;
  const double margin = kMargin * __popc(open);
  if (ordered64_value(a) - ordered64_value(b) <= margin) atomicOr(&s.unsure, open);
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
beam_join_kernel(const BeamArgs a, const RowPart* __restrict__ in, int parts, const __grid_constant__ ExpTable exp_table) {
  __shared__ JoinShared s;
  const int tid = threadIdx.x, lane = tid & 31, warp_id = tid >> 5;
  const int W = a.beams, K = a.keep, V = a.vocab, lists = W * parts;
  const int64_t request = blockIdx.x;
  if (tid < 64) s.table[tid] = exp_table.t[tid];
  if (tid == 0) s.exact = 0;
  grid_dependents_launch();
  grid_dependency_wait();
  const RowPart* rows = in + request * lists;
  // a thread per list (the parts of a beam, a power of two, stand side by side in a warp)
  const bool real = tid < lists;
  const int my_beam = real ? tid / parts : 0;
  int count = 0;       // entries
  uint64_t first = 0;  // the first one's key
  if (tid < (lists + 31) / 32 * 32) {
    const RowPart& r = rows[real ? tid : 0];
    const float c = a.score[request * W + my_beam];
    const bool done = a.finished && a.finished[request * W + my_beam];
    const float own = real ? r.ref : -INFINITY;
    double sum = real ? r.sum : 0.0;
    uint32_t infinite = real ? r.infinite : 0;
    if (real) {
      count = (int)r.n;
      first = r.key[0];
      if (done && c > -INFINITY) {
        // a finished beam goes on by the padding token alone, its score as it is
        count = tid % parts == 0;
        first = key_of(ordered(0.f), (uint32_t)a.pad_token);
      }
    }
    if (real) s.count[tid] = count;
    float ref = own;
    for (int o = parts >> 1; o > 0; o >>= 1) {
      ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
      infinite += __shfl_xor_sync(0xffffffffu, infinite, o);
    }
    sum = own > -INFINITY ? sum * (double)ex2_approx((own - ref) * kLog2e) : 0.0;
    for (int o = parts >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (real && tid % parts == 0) {
      const bool counts = c > -INFINITY && !done;
      s.sum[my_beam] = 0;
      s.ref[my_beam] = counts && ref > -INFINITY ? ref : 0.f;
      s.infinite[my_beam] = counts && infinite > 0;
      s.base[my_beam] = counts ? (double)c - log(infinite ? (double)infinite : sum) : (double)c;
    }
  }
  __syncthreads();
  auto score_of = [&](int w, uint64_t key) -> uint64_t {
    const float x = ordered_value((uint32_t)(key >> 32));
    if (s.infinite[w]) return x == INFINITY ? ordered64(s.base[w]) : 0;
    return ordered64(s.base[w] + ((double)x - (double)s.ref[w]));
  };
  for (int pass = 0; pass <= W; ++pass) {
    // The lists are sorted, so an entry has those before it in its list and the better lists' heads in front of it:
    // entry k of the list with the r-th best head is among the K best only if r + k < K.
    uint64_t head = 0;
    uint32_t head_index = 0;
    if (real) {
      if (count > 0) {
        head = score_of(my_beam, first);
        head_index = (uint32_t)(my_beam * V) + ~(uint32_t)first;
      }
      s.head[tid] = head;
      s.head_index[tid] = head_index;
    }
    if (tid < K) s.list[tid] = -1;
    if (tid == 0) s.unsure = 0;
    __syncthreads();
    int rank = K;
    if (head != 0) {
      rank = 0;
#pragma unroll 4
      for (int l = 0; l < lists; ++l) rank += before(s.head[l], s.head_index[l], head, head_index);
      if (rank < K) {
        s.list[rank] = tid;
        s.score[rank][0] = head;
        s.place[rank][0] = head_index;
      }
    }
    __syncthreads();
    constexpr int kEach = (kMaxKeep * kMaxKeep + kThreads - 1) / kThreads;
    uint64_t key[kEach];
    int from[kEach];
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int i = tid + u * kThreads, r = i / K, k = i - r * K;
      from[u] = r < K && k > 0 && r + k < K ? s.list[r] : -1;
      if (from[u] >= 0 && k < s.count[from[u]]) key[u] = rows[from[u]].key[k];
    }
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int i = tid + u * kThreads, r = i / K, k = i - r * K, l = from[u];
      if (l < 0) continue;
      const bool is = k < s.count[l];
      s.score[r][k] = is ? score_of(l / parts, key[u]) : 0;
      s.place[r][k] = is ? (uint32_t)(l / parts * V) + ~(uint32_t)key[u] : 0;
    }
    __syncthreads();
    if (warp_id == 0) {
      // a lane per list, its next entry in registers: K times the best of them
      const bool has = lane < K && s.list[lane < K ? lane : 0] >= 0;
      int at = 0;
      uint64_t v = has ? s.score[lane][0] : 0;
      uint32_t x = has ? s.place[lane][0] : 0;
      for (int n = 0; n < K; ++n) {
        const uint32_t hi = (uint32_t)(v >> 32), most = __reduce_max_sync(0xffffffffu, hi);
        unsigned who = __ballot_sync(0xffffffffu, hi == most);
        if (who & (who - 1)) {
          const uint32_t lo = hi == most ? (uint32_t)v : 0, more = __reduce_max_sync(0xffffffffu, lo);
          const bool tie = hi == most && lo == more;
          const uint32_t ix = tie ? x : 0xffffffffu, least = __reduce_min_sync(0xffffffffu, ix);
          who = __ballot_sync(0xffffffffu, tie && ix == least);
        }
        if (lane == __ffs(who) - 1) {
          s.order[n] = v;
          s.index[n] = x;
          ++at;
          const bool more = v != 0 && lane + at < K;
          v = more ? s.score[lane][at] : 0;
          x = more ? s.place[lane][at] : 0;
        }
      }
      __syncwarp();
      // what lies closest behind the last one kept: of each list the entry at which it stands
      const uint64_t last = s.order[K - 1];
      if (last != 0 && v != 0) doubt(s, last, (int)s.index[K - 1] / V, v, (int)x / V);
    }
    __syncthreads();
    if (tid < K) {
      const uint64_t v = s.order[tid];
      const int x = (int)s.index[tid], w = v ? x / V : -1;
      const int64_t o = request * K + tid;
      a.parent[o] = w;
      a.token[o] = v ? x - w * V : -1;
      a.new_score[o] = v ? (float)ordered64_value(v) : -INFINITY;
      if (tid > 0 && v != 0) doubt(s, s.order[tid - 1], (int)s.index[tid - 1] / V, v, w);
    }
    if (s.order[K - 1] != 0 && head != 0 && rank >= K) doubt(s, s.order[K - 1], (int)s.index[K - 1] / V, head, my_beam);
    __syncthreads();
    uint32_t unsure = s.unsure;
    if (unsure == 0) break;
    __syncthreads();
    if (tid == 0) s.exact |= unsure;
    // the sums of the beams concerned again, exactly
    for (; unsure != 0; unsure &= unsure - 1) {
      const int w = __ffs(unsure) - 1;
      if (s.infinite[w] || (a.finished && a.finished[request * W + w])) continue;  // exact already
      uint32_t top = 0;
      for (int p = 0; p < parts; ++p)
        if (rows[w * parts + p].n > 0) top = max(top, (uint32_t)(rows[w * parts + p].key[0] >> 32));
      const Exponent e = {ordered_value(top), 1.44269502162933349609f, 1.92596299112661746887e-8f};
      const Row<T> row(a.logits, a.stride, request * W + w, V);
      const int all = row.granules();
      unsigned long long sum = 0;
      for (int g = tid; g < all; g += kThreads) {
        float x[Row<T>::kVec];
        row.get(g, x);
#pragma unroll
        for (int k = 0; k < Row<T>::kVec; ++k) sum += x[k] > -INFINITY ? weight_units(x[k], e, s.table) : 0;
      }
      atomicAdd(&s.sum[w], sum);
      __syncthreads();
      if (tid == 0) {
        s.ref[w] = e.max;
        s.base[w] = (double)a.score[request * W + w] - (log((double)s.sum[w]) - kUnitBits * kLn2);
      }
    }
    __syncthreads();
  }
}

// Rows of 32-bit words, `length` of each (or all), from the parents' to the children's places.
__global__ void __launch_bounds__(kThreads)
beam_reorder_kernel(const ReorderArgs a, int64_t rows) {
  grid_dependency_wait();
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    const int64_t request = r / a.keep;
    const int p = a.parent[r];
    const bool real = p >= 0 && p < a.beams;
    const int64_t source = request * a.beams + (real ? p : 0);
    int64_t n = a.row_words;
    if (a.length) {
      const int32_t len = real ? a.length[source] : 0;
      if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (len < 0 || (int64_t)len > a.row_words) record_status(a.status, VMLA_ERR_INDEX, (uint32_t)r);
        if (a.new_length) a.new_length[r] = len;
      }
      n = len < 0 ? 0 : (int64_t)len < n ? (int64_t)len : n;
    }
    if (!real) {
      if (blockIdx.x == 0 && threadIdx.x == 0 && p != -1) record_status(a.status, VMLA_ERR_INDEX, (uint32_t)r);
      continue;
    }
    const uint32_t* src = a.src + source * a.src_stride;
    uint32_t* dst = a.dst + r * a.dst_stride;
    const int64_t me = (int64_t)blockIdx.x * kThreads + threadIdx.x, step = (int64_t)gridDim.x * kThreads;
    int64_t from = 0;
    if (((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 15) == 0) {
      const int64_t whole = n / 4;
#pragma unroll 2
      for (int64_t i = me; i < whole; i += step)
        reinterpret_cast<uint4*>(dst)[i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
      from = whole * 4;
    }
    for (int64_t i = from + me; i < n; i += step) dst[i] = __ldg(src + i);
  }
}

// CTAs per row of logits: three for each SM, as far as each has 4096 tokens.  (64 x 8 rows of 131 072: one part each
// 45 us, two 47; 135 rows of 151 001: four parts 48 us, two 48, eight 56, as lists to merge grow with the parts.)
int parts_of(int64_t rows, int vocab, int sms) {
  int parts = 1;
  while (parts < kMaxParts && rows * parts < 3 * (int64_t)sms && vocab / (parts * 2) >= 4096) parts *= 2;
  return parts;
}

template <typename T>
int launch_select(const BeamArgs& a, int64_t requests, int parts, void* workspace, cudaStream_t stream) {
  RowPart* part = static_cast<RowPart*>(workspace);
  const int64_t rows = requests * a.beams;
  beam_rows_kernel<T><<<(unsigned)(rows * parts), kThreads, 0, stream>>>(a, part, parts);
  if (cudaGetLastError() != cudaSuccess) return VMLA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {early_start_attribute()};
  cfg.gridDim = dim3((unsigned)requests, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, beam_join_kernel<T>, a, (const RowPart*)part, parts, exp_table()) == cudaSuccess
             ? VMLA_OK
             : VMLA_ERR_CUDA;
}

}  // namespace

size_t beam_workspace_used(int64_t rows, int vocab, int sms) {
  return (size_t)rows * parts_of(rows, vocab, sms) * sizeof(RowPart);
}

// What every call of up to `rows` rows and `vocab` tokens uses at most (fewer rows may have more parts).
size_t beam_workspace(int64_t rows, int vocab, int sms) {
  int64_t most = rows;
  for (int parts = 2; parts <= kMaxParts && vocab / parts >= 4096; parts *= 2) {
    const int64_t last = (6 * (int64_t)sms - 1) / parts;  // the most rows that get so many (see parts_of)
    most = std::max(most, std::min(rows, last) * parts);
  }
  return (size_t)most * sizeof(RowPart);
}

int launch_beam_select(const BeamArgs& a, int64_t requests, bool fp32, int sms, void* workspace, void* stream) {
  if (requests == 0) return VMLA_OK;
  const int64_t rows = requests * a.beams;
  const int parts = parts_of(rows, a.vocab, sms);
  if (rows * parts > INT32_MAX) return VMLA_ERR_SHAPE;
  return fp32 ? launch_select<float>(a, requests, parts, workspace, (cudaStream_t)stream)
              : launch_select<uint16_t>(a, requests, parts, workspace, (cudaStream_t)stream);
}

int launch_beam_reorder(const ReorderArgs& a, int64_t requests, int sms, void* stream) {
  const int64_t rows = requests * a.keep;
  if (rows == 0) return VMLA_OK;
  const int64_t wide = (a.row_words + 4 * kThreads - 1) / (4 * kThreads);
  const unsigned y = (unsigned)(rows < 65535 ? rows : 65535);
  const int64_t most = (16 * (int64_t)sms + y - 1) / y;
  const unsigned x = (unsigned)(wide < 1 ? 1 : wide < most ? wide : most);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {early_start_attribute()};
  cfg.gridDim = dim3(x, y, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = (cudaStream_t)stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, beam_reorder_kernel, a, rows) == cudaSuccess ? VMLA_OK : VMLA_ERR_CUDA;
}

}  // namespace vmla
