// Append of new tokens' rows to a pool of 8-bit codes with one scale per block of slots.
//
// A row is [latent (512) | rotated part (64)] as in the append with one scale.  The rows that a call brings to one
// block (a run: tokens that stand together, slots ascending) get the block's scale
//   need  = the smallest power of two 2^k, k >= -100, with every finite |value| of the run <= 448 x 2^k
//   scale = need where the run begins the block, else max(the block's scale, need)
//   code  = e4m3(value / scale), nearest even,
// and where that raises the scale the block's rows in front of the run are coded again, e4m3(code x old / new).
// A power of two makes value / scale exact, so a code is off by its own rounding only (half of 2^-3), and lets the
// cache's readers scale in any order; against amax / 448 it gives away less than one bit at the bottom of the range.
//
// A token costs 1152 bytes in, 256 of table, 576 out and 256 per head.  With blocks of one slot a warp takes a token
// and has its row in registers while the largest value is found.  Otherwise a CTA takes a run: each of its 16 warps has
// four rows at a time, all their loads on their way together; the CTA agrees on the scale in shared memory, and the rows
// are coded from the registers (a run of more than 64 rows is read a second time, from L1 or L2).  A CTA looks for runs
// that begin in a window of tokens: one token where there are few (each run then has its own CTA; the others leave at
// once), else as many as a block has slots.
// Measured: 17 000 tokens of 16 heads in blocks of 64 24.9 us, 4.1 TB/s (a row at a time by eight warps, read twice: 32.1);
// a step of 144 tokens of 64 heads 6 to 8.2 us, which are launch and latencies.
#include <cuda_runtime.h>

#include "vmla_device.cuh"
#include "vmla_rope.cuh"

namespace vmla {
using namespace rope;
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBlock = VMLA_MAX_BLOCK_TOKENS;
constexpr int kHeadPasses = 2;  // 16 heads per warp
constexpr int kSide = 4;        // rows of a run that a warp has at a time
static_assert(kMaxBlock <= kThreads, "one thread per token of a window");

// Granules 2 lane, 2 lane + 1 of the latent and, in lanes 0 to 3, the turned granules lane and lane + 4 of the rest.
struct Row {
  float x0[8], x1[8], lo[8], hi[8];
};

__device__ __forceinline__ void load_row(const AppendArgs& a, int64_t t, int32_t pos, int lane, Row& r) {
  const uint4* lat = reinterpret_cast<const uint4*>(a.latent + t * a.latent_stride);
  const uint4* rope = reinterpret_cast<const uint4*>(a.k_rope + t * a.k_rope_stride);
  const uint4 v0 = __ldg(lat + 2 * lane), v1 = __ldg(lat + 2 * lane + 1);
  if (lane < 4) {
    const uint4 r0 = __ldg(rope + lane), r1 = __ldg(rope + lane + 4);
    const bool neighbours = a.neighbours != 0;
    rotate(r0, r1, load_angles(a.cos_sin + (int64_t)pos * kRopeDim, lane, neighbours), neighbours, r.lo, r.hi);
  }
  unpack8(v0, r.x0);
  unpack8(v1, r.x1);
}

// The row's largest magnitude (NaN left out), in every lane.
__device__ __forceinline__ float largest(const Row& r, int lane) {
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = fmaxf(m, fmaxf(fabsf(r.x0[k]), fabsf(r.x1[k])));
  if (lane < 4)
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, fmaxf(fabsf(r.lo[k]), fabsf(r.hi[k])));
  return warp_max(m);
}

// The smallest 2^k with amax <= 448 x 2^k = 1.75 x 2^(k + 8), -100 <= k <= 120 (beyond every finite float's need).
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  int k = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  k = k < -100 ? -100 : k > 120 ? 120 : k;
  return __uint_as_float((uint32_t)(k + 127) << 23);
}

// Eight values -> codes: by a product where the scale is a power of two (then exact) whose reciprocal is a normal number,
// else by a division.
__device__ __forceinline__ uint2 codes_of(const float (&x)[8], float scale) {
  if ((__float_as_uint(scale) & 0x7FFFFFu) != 0 || !(scale >= 0x1p-120f && scale <= 0x1p126f)) return codes8(x, scale);
  const float inv = __uint_as_float((254u << 23) - __float_as_uint(scale));
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(x[2 * k + 1] * inv), "f"(x[2 * k] * inv));
    w[k] = c;
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

__device__ __forceinline__ void store_row(const AppendArgs& a, int32_t slot, int lane, const Row& r, float scale) {
  uint8_t* dst = reinterpret_cast<uint8_t*>(a.pool) + (int64_t)slot * kDqk;
  const uint2 c0 = codes_of(r.x0, scale), c1 = codes_of(r.x1, scale);
  reinterpret_cast<uint4*>(dst)[lane] = make_uint4(c0.x, c0.y, c1.x, c1.y);
  if (lane < 4) {
    *reinterpret_cast<uint2*>(dst + kDv + 8 * lane) = codes_of(r.lo, scale);
    *reinterpret_cast<uint2*>(dst + kDv + 8 * (lane + 4)) = codes_of(r.hi, scale);
  }
}

// Four codes, each times `ratio` (below 1) and coded again.
__device__ __forceinline__ uint32_t recode4(uint32_t w, float ratio) {
  uint32_t out = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t pair;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(pair) : "h"((uint16_t)(w >> (16 * h))));
    float lo, hi;
    asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;}"
        : "=f"(lo), "=f"(hi)
        : "r"(pair));
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi * ratio), "f"(lo * ratio));
    out |= (uint32_t)c << (16 * h);
  }
  return out;
}

__device__ __forceinline__ bool slot_ok(const AppendArgs& a, int32_t slot) {
  return slot >= 0 && (int64_t)slot < a.pool_slots;
}

// Four rows of a run by one warp.  Of each lane's: granules 2 lane, 2 lane + 1 of every latent as they came, and of
// row lane / 8 the eight turned elements 4 h .. 4 h + 3 and 32 + 4 h .. 32 + 4 h + 3, h = lane mod 8, and the slot
// (-1: nothing to write).
struct Four {
  uint4 v0[kSide], v1[kSide];
  float x[8];
  int32_t slot;
};

// Tokens t0 + k .. t0 + k + 3 below t0 + n.
__device__ __forceinline__ void fetch_four(const AppendArgs& a, int64_t t0, int k, int n, int lane, Four& f) {
  const int mine = k + (lane >> 3), h = lane & 7;
  const int64_t t = t0 + mine;
  int32_t slot = -1, pos = -1;
  uint2 lo = make_uint2(0, 0), hi = lo;
  if (mine < n) {
    const uint2* rope = reinterpret_cast<const uint2*>(a.k_rope + t * a.k_rope_stride);
    slot = __ldg(a.slots + t);
    pos = __ldg(a.positions + t);
    lo = __ldg(rope + h);
    hi = __ldg(rope + h + 8);
  }
#pragma unroll
  for (int i = 0; i < kSide; ++i) {
    f.v0[i] = f.v1[i] = make_uint4(0, 0, 0, 0);
    if (k + i < n) {
      const uint4* lat = reinterpret_cast<const uint4*>(a.latent + (t0 + k + i) * a.latent_stride);
      f.v0[i] = __ldg(lat + 2 * lane);
      f.v1[i] = __ldg(lat + 2 * lane + 1);
    }
  }
  f.slot = slot_ok(a, slot) && pos >= 0 && (int64_t)pos < a.table_rows ? slot : -1;
  if (f.slot >= 0) {
    const float* row = a.cos_sin + (int64_t)pos * kRopeDim;
    float c[4], sn[4];
    auto load4 = [&](const float* from, float (&to)[4]) {
      if (a.neighbours != 0) {
        const float2 u = __ldg(reinterpret_cast<const float2*>(from) + h), v = __ldg(reinterpret_cast<const float2*>(from) + 8 + h);
        to[0] = u.x; to[1] = u.y; to[2] = v.x; to[3] = v.y;
      } else {
        const float4 u = __ldg(reinterpret_cast<const float4*>(from) + h);
        to[0] = u.x; to[1] = u.y; to[2] = u.z; to[3] = u.w;
      }
    };
    load4(row, c);
    load4(row + kRopeDim / 2, sn);
    unpack8(make_uint4(lo.x, lo.y, hi.x, hi.y), f.x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (a.neighbours != 0) turn(f.x[2 * i], f.x[2 * i + 1], c[i], sn[i]);
      else turn(f.x[i], f.x[4 + i], c[i], sn[i]);
    }
  }
}

// Their largest finite magnitude, in every lane: a scale that an infinity set would leave nothing of the block's other rows.
// (Magnitudes' bits order as whole numbers do, and with one more in the exponent infinities and NaN are negative.)
__device__ __forceinline__ float largest(const Four& f) {
  constexpr uint32_t kOne = 0x00800080u;
  uint32_t m2 = kOne;  // of two columns
  auto take = [&](uint32_t w) { m2 = __viaddmax_s16x2(w & 0x7FFF7FFFu, kOne, m2); };
#pragma unroll
  for (int i = 0; i < kSide; ++i)
    if (__shfl_sync(0xffffffffu, f.slot, 8 * i) >= 0) {
      take(f.v0[i].x); take(f.v0[i].y); take(f.v0[i].z); take(f.v0[i].w);
      take(f.v1[i].x); take(f.v1[i].y); take(f.v1[i].z); take(f.v1[i].w);
    }
  int m = (int)max(m2 << 16, m2 & 0xFFFF0000u);
  if (f.slot >= 0)
#pragma unroll
    for (int k = 0; k < 8; ++k) m = __viaddmax_s32((int)(__float_as_uint(f.x[k]) & 0x7FFFFFFFu), (int)(kOne & 0xFFFF0000u), m);
  return __uint_as_float((uint32_t)__reduce_max_sync(0xffffffffu, m) - (kOne & 0xFFFF0000u));
}

__device__ __forceinline__ void store_four(const AppendArgs& a, int lane, const Four& f, float scale) {
  uint8_t* pool = reinterpret_cast<uint8_t*>(a.pool);
#pragma unroll
  for (int i = 0; i < kSide; ++i) {
    const int32_t slot = __shfl_sync(0xffffffffu, f.slot, 8 * i);
    if (slot < 0) continue;
    float x0[8], x1[8];
    unpack8(f.v0[i], x0);
    unpack8(f.v1[i], x1);
    const uint2 c0 = codes_of(x0, scale), c1 = codes_of(x1, scale);
    reinterpret_cast<uint4*>(pool + (int64_t)slot * kDqk)[lane] = make_uint4(c0.x, c0.y, c1.x, c1.y);
  }
  if (f.slot >= 0) {
    uint32_t* dst = reinterpret_cast<uint32_t*>(pool + (int64_t)f.slot * kDqk + kDv) + (lane & 7);
    const uint2 c = codes_of(f.x, scale);
    dst[0] = c.x;
    dst[8] = c.y;
  }
}

struct RunShared {
  int32_t start[kThreads];
  int32_t starts;
  int32_t warp_len[kWarps];
  int32_t first[kWarps], last[kWarps];
  float amax[kWarps];
};

// All runs whose first token lies in [w0, w0 + window), by the whole CTA.
__device__ void append_runs(const AppendArgs& a, int64_t w0, int window, RunShared& s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int shift = a.block_shift, mask = a.block - 1;
  if (tid == 0) s.starts = 0;
  __syncthreads();
  if (tid < window && w0 + tid < a.tokens) {
    const int64_t t = w0 + tid;
    const int32_t slot = __ldg(a.slots + t);
    if (slot_ok(a, slot)) {
      // (tokens without a slot may stand between those of a block)
      int64_t before = t - 1;
      while (before >= 0 && !slot_ok(a, __ldg(a.slots + before))) --before;
      if (before < 0 || (__ldg(a.slots + before) >> shift) != (slot >> shift)) s.start[atomicAdd(&s.starts, 1)] = tid;
      const int32_t pos = __ldg(a.positions + t);
      if (!(pos >= 0 && (int64_t)pos < a.table_rows)) record_status(a.status, VMLA_ERR_INDEX, (uint32_t)t);
    } else if (slot != -1) {
      record_status(a.status, VMLA_ERR_INDEX, (uint32_t)t);
    }
  }
  __syncthreads();
  const int starts = s.starts;
  for (int i = 0; i < starts; ++i) {
    const int64_t t0 = w0 + s.start[i];
    const int32_t block = __ldg(a.slots + t0) >> shift;
    // its length: up to the first token of another block, and the first row that it brings
    int n = 0, used_n = 0, first = -1;
    for (bool more = true; more;) {
      const int64_t t = t0 + n + tid;
      const int32_t slot = t < a.tokens ? __ldg(a.slots + t) : -1, pos = t < a.tokens ? __ldg(a.positions + t) : -1;
      const bool in = slot_ok(a, slot) && (slot >> shift) == block, ends = t >= a.tokens || (slot_ok(a, slot) && !in);
      const unsigned end = __ballot_sync(0xffffffffu, ends);
      const int len = end ? __ffs(end) - 1 : 32;
      const unsigned used = __ballot_sync(0xffffffffu, in && lane < len && pos >= 0 && (int64_t)pos < a.table_rows);
      const int32_t at = __shfl_sync(0xffffffffu, slot & mask, used ? __ffs(used) - 1 : 0);
      if (lane == 0) {
        s.warp_len[warp] = len;
        s.first[warp] = used ? at : -1;
        s.last[warp] = used ? 32 - __clz(used) : 0;
      }
      __syncthreads();
      const int n0 = n;
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        if (n == n0 + 32 * w) {
          n += s.warp_len[w];
          if (first < 0) first = s.first[w];
          if (s.last[w] > 0) used_n = n0 + 32 * w + s.last[w];
        }
      more = n == n0 + kThreads;
      __syncthreads();
    }
    n = used_n;  // (padding behind the last row of the block costs nothing more)
    const float old = first < 0 ? 0.f : a.kv_scales[block];
    float m = 0.f;
    Four f;
    for (int k = kSide * warp; k < n; k += kSide * kWarps) {
      fetch_four(a, t0, k, n, lane, f);
      m = fmaxf(m, largest(f));
    }
    if (lane == 0) s.amax[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s.amax[w]);
    const float need = scale_for(m), scale = first == 0 ? need : fmaxf(old, need);
    if (first > 0 && scale > old) {
      const float ratio = old / scale;
      for (int row = warp; row < first; row += kWarps) {
        uint4* codes = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(a.pool) +
                                                (((int64_t)block << shift) + row) * kDqk);
        for (int g = lane; g < kDqk / 16; g += 32) {
          uint4 v = codes[g];
          v.x = recode4(v.x, ratio);
          v.y = recode4(v.y, ratio);
          v.z = recode4(v.z, ratio);
          v.w = recode4(v.w, ratio);
          codes[g] = v;
        }
      }
    }
    if (tid == 0 && first >= 0) a.kv_scales[block] = scale;
    for (int k = kSide * warp; k < n; k += kSide * kWarps) {
      if (n > kSide * kWarps) fetch_four(a, t0, k, n, lane, f);  // (else it has them still)
      store_four(a, lane, f, scale);
    }
    __syncthreads();
  }
}

template <bool kRuns>
__global__ void __launch_bounds__(kThreads, 2)
append_scaled_kernel(const AppendArgs a, int64_t row_ctas, int window, int parts) {
  __shared__ RunShared s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if ((int64_t)blockIdx.x < row_ctas) {
    if (kRuns) {
      append_runs(a, (int64_t)blockIdx.x * window, window, s);
      return;
    }
    const int64_t t = (int64_t)blockIdx.x * kWarps + warp;
    if (t >= a.tokens) return;
    const int32_t slot = __ldg(a.slots + t), pos = __ldg(a.positions + t);
    if (!slot_ok(a, slot) || !(pos >= 0 && (int64_t)pos < a.table_rows)) {
      if (lane == 0 && slot != -1) record_status(a.status, VMLA_ERR_INDEX, (uint32_t)t);
      return;
    }
    Row r;
    load_row(a, t, pos, lane, r);
    const float scale = scale_for(largest(r, lane));
    store_row(a, slot, lane, r, scale);
    if (lane == 0) a.kv_scales[slot] = scale;
    return;
  }
  const int64_t unit = ((int64_t)blockIdx.x - row_ctas) * kWarps + warp;
  const int64_t t = unit / parts;
  if (t >= a.tokens) return;
  const int32_t slot = __ldg(a.slots + t), pos = __ldg(a.positions + t);
  const bool use = slot_ok(a, slot) && pos >= 0 && (int64_t)pos < a.table_rows;
  turn_heads<kHeadPasses>(a, t, (int)(unit - t * parts), lane, use, a.cos_sin + (int64_t)(use ? pos : 0) * kRopeDim);
}

}  // namespace

int launch_append_scaled(const AppendArgs& a, void* stream) {
  if (a.tokens == 0) return VMLA_OK;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) !=
                                                cudaSuccess)
    return VMLA_ERR_CUDA;
  const int heads = kHeadPasses * kHeadsPerPass;
  const int parts = (a.num_heads + heads - 1) / heads;
  const bool runs = a.block > 1;
  const int window = a.tokens > 8 * (int64_t)sms ? a.block : 1;
  const int64_t row_ctas = runs ? (a.tokens + window - 1) / window : (a.tokens + kWarps - 1) / kWarps;
  const int64_t ctas = row_ctas + (a.tokens * parts + kWarps - 1) / kWarps;
  if (ctas > INT32_MAX) return VMLA_ERR_SHAPE;
  const auto kernel = runs ? append_scaled_kernel<true> : append_scaled_kernel<false>;
  kernel<<<(unsigned)ctas, kThreads, 0, (cudaStream_t)stream>>>(a, row_ctas, window, parts);
  return cudaGetLastError() == cudaSuccess ? VMLA_OK : VMLA_ERR_CUDA;
}

}  // namespace vmla
