// Attention over a pool of 8-bit codes with one scale per block of slots, in 8 bits on the tensor cores.
//
// For a query row r (a draft's head) and key j with slot s, codes k_j (e4m3) and scale a_j = scales[s / block]:
//   s_rj = sm_scale a_j <q_r, k_j>,  p_rj = 2^(s_rj log2 e - m_r),  out_r = sum_j p_rj a_j k_j[:512] / sum_j p_rj.
// The codes are operands as they are: nothing is converted to bf16, staged, or written back.  What is not 8 bits wide
// is split into parts that are, exactly or nearly so:
//   queries  q a = hi + lo / 16, both e4m3, a the power of two that brings the largest of the 32 rows to (224, 448]:
//            off by at most 2^-14 of what is 448 at the largest (2^-22.8), less than an fp32 dot product's rounding
//   weights  p a_j 2^11, in fp16 rounded to 9 bits, cut into three parts of three bits, e5m2: the upper byte of an fp16
//            number is an e5m2 number, so a part is an AND and the rest an exact difference.  Its range (2^-16 to 2^15
//            here) is why it is not two e4m3 parts: beside a key of much weight, 10^5 keys of weight 10^-5 each still count.
//
// Keys are the matrix products' M (tiles of 128), query rows their N (units of 32), so that few rows waste nothing:
//   S^T [128 keys x 64]  = K [128 x 576] (Q hi | Q lo)^T               18 products, M128 N64 K32
//   O^T [512 x 96]      += V^T [512 x 128 keys] (P hi | P mid | P lo)^T  16 products, M128 N96 K32, V being K's first columns
// O^T takes 384 of the 512 columns of tensor memory, two S^T the rest.  One read of a tile's rows serves both products.
// A softmax thread has one key and 16 rows: a_j is its own number, the reference m_r is raised only when a weight passes
// 2^15 (told by one barrier with a vote per tile), and row sums stay in registers until the unit ends.
//
// Rows are fetched by tile::gather4 (four slots x 128 bytes, swizzled as the products read them) straight from the pool;
// a slot that is none, or a place behind the last key, is a coordinate outside the tensor and reads zeros.
//
// Work: CTAs (one per SM) form lanes of G; row blocks of a sequence form streams of G over its key tiles, laid end to end
// (a stream costs its tiles and kFixed more); lane l takes the l-th share of the whole length.  The G CTAs of a lane read
// the same rows at about the same time, from L2 but for the first.  Streams cut by a lane's end leave fp32 partials
// (at most two per CTA), and a second launch joins them.  Every CTA works the plan out from the device's lengths.
#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

#include "vmla_device.cuh"
#include "vmla_sm100.cuh"

namespace vmla {
using namespace sm100;
namespace {

constexpr int kTile = 128;          // keys
constexpr int kRows = 32;           // query rows of a unit
constexpr int kChunks = kDv / 128;  // 4 column chunks of 128 bytes, and one of 64
constexpr int kParts = 3;           // of a weight
constexpr int kStages = 2;
constexpr int kSoftWarps = 8;       // two per quarter of the tile's keys, 16 rows each
constexpr int kSoftThreads = kSoftWarps * 32;
constexpr int kHalf = kRows / 2;
constexpr int kLoadWarps = 3;
constexpr int kMmaWarp = kSoftWarps, kLoadWarp = kMmaWarp + 1;
constexpr int kThreads = 32 * (kSoftWarps + 1 + kLoadWarps);
constexpr uint32_t kOCols = kParts * kRows;      // 96 columns of tensor memory per 128 value columns
constexpr uint32_t kSCol = kChunks * kOCols;     // 384
constexpr uint32_t kStageBytes = kTile * kDqk;
constexpr int kFixed = 2;           // what a unit costs beside its tiles, in tiles
constexpr float kNone = -3e38f;     // reference of a row that has seen no key
constexpr float kUnit = 2048.f;     // weights are held times 2^11
constexpr float kMost = 32768.f;    // largest weight held
constexpr float kTiny = 0x1p-100f;  // smaller scales count as zero
static_assert(kSCol + 2 * 2 * kRows == 512, "tensor memory");

struct Stage {
  uint8_t latent[kChunks][kTile * 128];  // [key][128 bytes], 128-byte swizzle
  uint8_t rope[kTile * 64];              // [key][64 bytes], 64-byte swizzle
};
static_assert(sizeof(Stage) == kStageBytes, "stage");

struct Shared {
  Stage stage[kStages];
  uint8_t q_latent[kChunks][2 * kRows * 128];  // [hi rows, lo rows][128 bytes], 128-byte swizzle
  uint8_t q_rope[2 * kRows * 64];              // 64-byte swizzle
  uint8_t p[2][kTile * 128];                   // [key][hi 32 | mid 32 | lo 32 | -], 128-byte swizzle
  int64_t cost[VMLA_MAX_BATCH + 1];            // cost position of each sequence's first stream
  int32_t kv[VMLA_MAX_BATCH + 1], qo[VMLA_MAX_BATCH + 1];
  uint64_t mask[kRows];                        // the unit's rows: visible drafts
  int32_t parent[VMLA_MAX_DRAFT];
  float part[4][kRows];                        // per quarter of the keys: row maxima, or row sums
  float q_max[kSoftWarps];
  int64_t sums[4][kThreads / 32];
  uint64_t kfull[kStages], kfree[kStages], sfull[2], sfree[2], pfull[2], pfree[2], qfull, ofree, done;
  uint32_t tmem;
  volatile int32_t abort_flag;
  int32_t stop;
  uint32_t fault[2];                           // first fault of this CTA: code, info
};
constexpr size_t kSharedBytes = sizeof(Shared) + 1024;
static_assert(kSharedBytes <= 232448, "shared memory");

// What a CTA tells the joining launch: the stream that starts in its lane and is cut by the lane's end, and its fault.
struct alignas(32) CtaInfo {
  int64_t row;      // first row of out
  int32_t pieces;   // 0: no such stream
  int32_t rows;
  int32_t group;    // G
  uint32_t fault, fault_info;
  int32_t pad;
};

struct Partials {
  float* o;        // [2 x CTAs][kRows][512], weights times kUnit
  float2* ml;      // [2 x CTAs][kRows]: reference (log2), sum
};

__device__ __forceinline__ void fault(Shared& sm, int code, uint32_t info) {
  if (atomicCAS(&sm.fault[0], 0u, (uint32_t)code) == 0u) sm.fault[1] = info;
}

// ------------------------------------------------------------------ plan
struct Plan {
  int64_t length;  // of all streams
  int64_t share;   // of a lane
  int32_t group;   // CTAs of a lane
  int32_t lanes;
};

__device__ __forceinline__ int row_blocks(const Shared& sm, const ScaledArgs& a, int b) {
  return ((sm.qo[b + 1] - sm.qo[b]) * a.num_heads + kRows - 1) / kRows;
}
__device__ __forceinline__ int tiles_of(const Shared& sm, int b) { return (sm.kv[b + 1] - sm.kv[b] + kTile - 1) / kTile; }

// Reads the lengths and shares the work out (whole CTA); false where the lengths are out of order or past a bound.
__device__ bool make_plan(Shared& sm, const ScaledArgs& a, Plan& plan) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int b = tid; b <= a.batch; b += kThreads) {
    sm.kv[b] = a.kv_indptr[b];
    sm.qo[b] = a.qo_indptr[b];
  }
  __syncthreads();
  bool ok = sm.kv[0] == 0 && sm.qo[0] == 0 && sm.kv[a.batch] <= a.max_kv && sm.qo[a.batch] <= a.max_q;
  int64_t sum[4] = {0, 0, 0, 0};
  for (int b = tid; b < a.batch; b += kThreads) {
    const int64_t nk = (int64_t)sm.kv[b + 1] - sm.kv[b], nq = (int64_t)sm.qo[b + 1] - sm.qo[b];
    ok = ok && nq >= 0 && nq <= VMLA_MAX_DRAFT && nk >= nq;
    if (ok) {
      const int64_t n = row_blocks(sm, a, b), span = tiles_of(sm, b) + kFixed;
#pragma unroll
      for (int k = 0; k < 4; ++k) sum[k] += ((n + (1 << k) - 1) >> k) * span;
    }
  }
  if (!__syncthreads_and(ok)) return false;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], o);
    if (lane == 0) sm.sums[k][warp] = sum[k];
  }
  __syncthreads();
  // the largest G whose shares are within 1/32 of the smallest ones
  int64_t least = INT64_MAX, length[4], share[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    length[k] = 0;
    for (int w = 0; w < kThreads / 32; ++w) length[k] += sm.sums[k][w];
    const int lanes = (int)gridDim.x >> k;
    share[k] = lanes > 0 ? (length[k] + lanes - 1) / lanes : INT64_MAX / 2;
    least = share[k] < least ? share[k] : least;
  }
  int pick = 0;
#pragma unroll
  for (int k = 1; k < 4; ++k)
    if (share[k] <= least + least / 32) pick = k;
  plan.group = 1 << pick;
  plan.lanes = (int)gridDim.x >> pick;
  plan.length = length[pick];
  plan.share = share[pick] > 0 ? share[pick] : 1;
  if (warp == 0) {  // running sums of the sequences' costs
    constexpr int kEach = VMLA_MAX_BATCH / 32;
    int64_t each[kEach], all = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int b = lane * kEach + i;
      each[i] = b < a.batch ? ((row_blocks(sm, a, b) + plan.group - 1) >> pick) * (int64_t)(tiles_of(sm, b) + kFixed) : 0;
      all += each[i];
    }
    int64_t before = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += v;
    }
    before -= all;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int b = lane * kEach + i;
      if (b <= a.batch) sm.cost[b] = before;
      before += each[i];
    }
    if (lane == 31 && a.batch == VMLA_MAX_BATCH) sm.cost[a.batch] = before;
  }
  __syncthreads();
  return true;
}

// One row block of a sequence over some of its tiles.
struct Unit {
  int b, row_block, rows;   // rows of the block that are the sequence's
  int tile0, tiles;         // its tiles
  int64_t out_row;          // first row in q and out
  int kv0, keys, prefix;    // first entry of kv_indices; keys and prefix of the sequence
  bool whole, head;         // every tile of the stream; its first tile is among these
  int pieces;
};

// The units of CTA j of lane l, in order.
struct Units {
  int64_t at, end, from;  // cost position of the current stream; of the lane's end and start
  int b, g, streams, tiles, n;
  __device__ __forceinline__ void enter(const Shared& sm, const ScaledArgs& a, const Plan& p, int sequence) {
    b = sequence;
    while (b < a.batch && (n = row_blocks(sm, a, b)) == 0) ++b;
    if (b >= a.batch) {
      at = INT64_MAX;
      return;
    }
    streams = (n + p.group - 1) / p.group;
    tiles = tiles_of(sm, b);
    g = 0;
    at = sm.cost[b];
  }
  __device__ __forceinline__ Units(const Shared& sm, const ScaledArgs& a, const Plan& p) {
    const int lane = blockIdx.x / p.group;
    from = (int64_t)lane * p.share;
    end = from + p.share < p.length ? from + p.share : p.length;
    at = INT64_MAX;
    if (lane >= p.lanes || from >= end) return;
    int lo = 0, hi = a.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sm.cost[mid] <= from) lo = mid; else hi = mid;
    }
    enter(sm, a, p, lo);
    if (at <= from) {
      g = (int)((from - at) / (tiles + kFixed));
      at += (int64_t)g * (tiles + kFixed);
    }
  }
  __device__ __forceinline__ bool next(const Shared& sm, const ScaledArgs& a, const Plan& p, Unit& u) {
    while (at < end) {
      const int64_t lo = at > from ? at : from, stop = at + tiles, hi = stop < end ? stop : end;
      const int block = g * p.group + (int)blockIdx.x % p.group;
      const bool use = lo < hi && block < n;
      if (use) {
        u.b = b;
        u.row_block = block;
        const int R = (sm.qo[b + 1] - sm.qo[b]) * a.num_heads;
        u.rows = min(kRows, R - block * kRows);
        u.out_row = (int64_t)sm.qo[b] * a.num_heads + (int64_t)block * kRows;
        u.tile0 = (int)(lo - at);
        u.tiles = (int)(hi - lo);
        u.kv0 = sm.kv[b];
        u.keys = sm.kv[b + 1] - u.kv0;
        u.prefix = u.keys - (sm.qo[b + 1] - sm.qo[b]);
        u.head = lo == at;
        u.whole = u.tiles == tiles;
        u.pieces = (int)((stop - 1) / p.share - at / p.share) + 1;
      }
      if (++g < streams) at += tiles + kFixed;
      else enter(sm, a, p, b + 1);
      if (use) return true;
    }
    return false;
  }
};

// ------------------------------------------------------------------ waits
__device__ __noinline__ bool wait_slow(Shared& sm, uint64_t* bar, uint32_t parity, long long budget, uint32_t where) {
  const long long t0 = clock64();
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (sm.abort_flag) return false;
    if (clock64() - t0 > budget) {
      fault(sm, VMLA_ERR_TIMEOUT, where);
      sm.abort_flag = 1;
      return false;
    }
  }
}
// Bounded wait; false once it ran out, here or in another warp.
__device__ __forceinline__ bool wait(Shared& sm, uint64_t* bar, uint32_t parity, const ScaledArgs& a, uint32_t where) {
  return mbar_try_wait(bar, parity) || wait_slow(sm, bar, parity, a.wait_cycles, where);
}

// A barrier of the softmax warps that tells each whether `any` held in one of them.
__device__ __forceinline__ bool soft_vote(bool any) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)any), "n"(kSoftThreads)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void soft_sync() { named_bar_sync(1, kSoftThreads); }

// ------------------------------------------------------------------ loads (every lane of three warps)
__device__ void load_role(Shared& sm, const CUtensorMap* latent, const CUtensorMap* rope, const ScaledArgs& a,
                          const Plan& plan) {
  const int warp = (threadIdx.x >> 5) - kLoadWarp, lane = threadIdx.x & 31;
  const int none = (int)a.pool_slots;  // outside the tensor: zeros
  Units units(sm, a, plan);
  Unit u;
  int it = 0;
  while (units.next(sm, a, plan, u)) {
    const int32_t* index = a.kv_indices + u.kv0;
    int32_t next[4];
    auto fetch = [&](int tile) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int key = tile * kTile + 4 * lane + k;
        next[k] = key < u.keys && tile < u.tile0 + u.tiles ? __ldg(index + key) : -1;
      }
    };
    fetch(u.tile0);
    for (int t = 0; t < u.tiles; ++t, ++it) {
      int32_t y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        y[k] = next[k];
        if (y[k] < 0 || y[k] >= none) {
          const int key = (u.tile0 + t) * kTile + 4 * lane + k;
          if (warp == 0 && key < u.keys) fault(sm, VMLA_ERR_INDEX, (uint32_t)(u.kv0 + key));
          y[k] = none;
        }
      }
      fetch(u.tile0 + t + 1);
      const int s = it % kStages;
      if (!wait(sm, &sm.kfree[s], ((it / kStages) & 1) ^ 1, a, 100)) return;
      if (warp == 0 && lane == 0) mbar_arrive_expect_tx(&sm.kfull[s], kStageBytes);
      const uint32_t bar = smem_u32(&sm.kfull[s]);
      Stage& st = sm.stage[s];
#pragma unroll
      for (int c = 0; c <= kChunks; ++c) {
        if (c % kLoadWarps != warp) continue;
        if (c < kChunks) tma_gather4(smem_u32(st.latent[c]) + lane * 512, latent, c * 128, y[0], y[1], y[2], y[3], bar);
        else tma_gather4(smem_u32(st.rope) + lane * 256, rope, kDv, y[0], y[1], y[2], y[3], bar);
      }
    }
  }
  // the last releases of the stages have arrived before the CTA leaves
  for (int k = 1; k <= kStages && it - k >= 0; ++k)
    wait(sm, &sm.kfree[(it - k) % kStages], ((it - k) / kStages) & 1, a, 101);
}

// ------------------------------------------------------------------ matrix products (one thread)
__device__ void mma_role(Shared& sm, const ScaledArgs& a, const Plan& plan, uint32_t tmem) {
  constexpr uint32_t kScores = idesc_f8_f32(kTile, 2 * kRows, 0, 0, 0, 0);
  constexpr uint32_t kValues = idesc_f8_f32(128, kParts * kRows, 0, 1, 1, 1);
  Units units(sm, a, plan);
  Unit u;
  int units_begun = 0;
  auto scores = [&](int it) -> bool {
    const int s = it % kStages, sb = it & 1;
    if (!wait(sm, &sm.kfull[s], (it / kStages) & 1, a, 200)) return false;
    if (!wait(sm, &sm.sfree[sb], ((it >> 1) & 1) ^ 1, a, 201)) return false;
    tc_fence_after();
    const uint32_t d = tmem + kSCol + (uint32_t)sb * 2 * kRows;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const uint32_t k = smem_u32(sm.stage[s].latent[c]), q = smem_u32(sm.q_latent[c]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        mma_ss_f8(d, smem_desc(k + 32 * i, 16, 1024), smem_desc(q + 32 * i, 16, 1024), kScores, (c | i) != 0);
    }
    const uint32_t k = smem_u32(sm.stage[s].rope), q = smem_u32(sm.q_rope);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      mma_ss_f8(d, smem_desc(k + 32 * i, 16, 512, 4), smem_desc(q + 32 * i, 16, 512, 4), kScores, 1u);
    mma_commit(&sm.sfull[sb]);
    return true;
  };
  auto values = [&](int it, bool first) -> bool {
    const int s = it % kStages, pb = it & 1;
    if (!wait(sm, &sm.pfull[pb], (it >> 1) & 1, a, 202)) return false;
    tc_fence_after();
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int i = 0; i < kTile / 32; ++i)
        mma_ss_f8(tmem + c * kOCols, smem_desc(smem_u32(sm.stage[s].latent[c]) + 4096 * i, 16, 1024),
                  smem_desc(smem_u32(sm.p[pb]) + 4096 * i, 16, 1024), kValues, !first || i > 0);
    mma_commit(&sm.pfree[pb]);
    mma_commit(&sm.kfree[s]);
    return true;
  };
  // scores of a tile go ahead of the values of the one before, but for a unit's first tile, whose queries come later
  int it = 0;
  bool ok = true;
  while (ok && units.next(sm, a, plan, u)) {
    ok = wait(sm, &sm.qfull, units_begun & 1, a, 203) && scores(it);
    for (int t = 0; ok && t < u.tiles; ++t, ++it) {
      if (t + 1 < u.tiles) ok = scores(it + 1);
      // (the first product into O: the unit before has been read out)
      if (ok && t == 0) ok = wait(sm, &sm.ofree, (units_begun & 1) ^ 1, a, 204);
      if (ok) ok = values(it, t == 0);
    }
    ++units_begun;
  }
  mma_commit(&sm.done);
  const long long t0 = clock64();
  while (!mbar_try_wait(&sm.done, 0) && clock64() - t0 < a.wait_cycles) {
  }
}

// ------------------------------------------------------------------ queries (softmax warps)
// The unit's rows into shared memory in two e4m3 parts, their masks; the factor that makes a score of a product.
__device__ float load_queries(Shared& sm, const ScaledArgs& a, const Unit& u) {
  constexpr int kGranules = kDqk / 8;                           // of 8 bf16
  constexpr int kEach = kRows * kGranules / kSoftThreads;      // 9 per thread
  static_assert(kRows * kGranules % kSoftThreads == 0, "granules per thread");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint4* src = reinterpret_cast<const uint4*>(a.q + u.out_row * kDqk);
  uint4 v[kEach];
  const int valid = u.rows * kGranules;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int i = tid + k * kSoftThreads;
    v[k] = i < valid ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
  }
  const int q0 = sm.qo[u.b], nq = sm.qo[u.b + 1] - q0;
  if (a.parent && tid < nq) sm.parent[tid] = a.parent[q0 + tid];
  uint32_t m = 0;  // largest magnitude, as bits of a bf16
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max(m, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if (lane == 0) sm.q_max[warp] = __uint_as_float(m << 16);
  soft_sync();
  float top = 0.f;
#pragma unroll
  for (int w = 0; w < kSoftWarps; ++w) top = fmaxf(top, sm.q_max[w]);
  // a: 448 = 1.75 x 2^8; queries below 2^-100 are zero to any score
  const uint32_t bits = __float_as_uint(top);
  int e = 8 - ((int)(bits >> 23) - 127) - ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e > 108 ? 108 : e < -119 ? -119 : e;
  const float scale = __uint_as_float((uint32_t)(e + 127) << 23), back = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int i = tid + k * kSoftThreads, row = i / kGranules, col = (i - row * kGranules) * 8;
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
    uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x0 = bf16_lo(w[j]) * scale, x1 = bf16_hi(w[j]) * scale;
      uint16_t h, l;
      uint32_t back2;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(x1), "f"(x0));
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back2) : "h"(h));
      float y0, y1;
      asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;}"
          : "=f"(y0), "=f"(y1)
          : "r"(back2));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(l) : "f"((x1 - y1) * 16.f), "f"((x0 - y0) * 16.f));
      hi[j >> 1] |= (uint32_t)h << (16 * (j & 1));
      lo[j >> 1] |= (uint32_t)l << (16 * (j & 1));
    }
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const int r = row + part * kRows;
      const uint2 out = part ? make_uint2(lo[0], lo[1]) : make_uint2(hi[0], hi[1]);
      uint8_t* dst = col < kDv ? sm.q_latent[col >> 7] + r * 128 + ((((col & 127) >> 4) ^ (r & 7)) << 4)
                               : sm.q_rope + r * 64 + ((((col - kDv) >> 4) ^ ((r >> 1) & 3)) << 4);
      *reinterpret_cast<uint2*>(dst + (col & 8)) = out;
    }
  }
  if (tid < kRows) {
    uint64_t word = 0;
    if (tid < u.rows) {
      const int i = (u.row_block * kRows + tid) / a.num_heads;
      if (a.masks) {
        word = a.masks[q0 + i];
      } else if (a.parent) {
        int k = i;
        while (k >= 0) {
          word |= 1ull << k;
          const int p = sm.parent[k];
          if (p >= k || p < -1) {
            fault(sm, VMLA_ERR_PARENT, (uint32_t)(q0 + i));
            word = 0;
            break;
          }
          k = p;
        }
      } else {
        word = causal_bits(i);
      }
    }
    sm.mask[tid] = word;
  }
  fence_proxy_async_smem();
  soft_sync();
  if (lane == 0 && a.test_fault != kFaultNoQReady) mbar_arrive(&sm.qfull);
  return a.sm_scale * 1.4426950408889634f * back;
}

// ------------------------------------------------------------------ softmax (eight warps)
// Order of floats as whole numbers, for the maximum over a warp.
__device__ __forceinline__ float warp_top(float v) {
  const int i = __float_as_int(v);
  const int m = __reduce_max_sync(0xffffffffu, i ^ ((i >> 31) & 0x7FFFFFFF));
  return __int_as_float(m ^ ((m >> 31) & 0x7FFFFFFF));
}

__device__ void softmax_role(Shared& sm, const ScaledArgs& a, const Plan& plan, uint32_t tmem, const Partials& part) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int quarter = warp & 3, half = warp >> 2;      // its 32 keys of a tile; its 16 rows
  const int my_key = quarter * 32 + lane;
  const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
  Units units(sm, a, plan);
  Unit u;
  int it = 0, units_done = 0;
  bool more = units.next(sm, a, plan, u);
  float factor = more ? load_queries(sm, a, u) : 0.f;
  while (more) {
    float m[kHalf], l[kHalf];
#pragma unroll
    for (int r = 0; r < kHalf; ++r) {
      m[r] = kNone;
      l[r] = 0.f;
    }
    // the scales of this thread's keys, fetched a tile ahead, their slots two
    const int32_t* index = a.kv_indices + u.kv0;
    auto slot_of = [&](int t) {
      const int key = (u.tile0 + t) * kTile + my_key;
      return t < u.tiles && key < u.keys ? __ldg(index + key) : -1;
    };
    auto scale_of = [&](int32_t slot) {
      return slot >= 0 && (int64_t)slot < a.pool_slots ? __ldg(a.kv_scales + (slot >> a.block_shift)) : 1.f;
    };
    float scale = scale_of(slot_of(0));
    int32_t slot = slot_of(1);
    for (int t = 0; t < u.tiles; ++t, ++it) {
      const float next_scale = scale_of(slot);
      slot = slot_of(t + 2);
      const int sb = it & 1;
      wait(sm, &sm.sfull[sb], (it >> 1) & 1, a, 300);  // (should it run out, the vote below ends the work)
      __syncwarp();
      tc_fence_after();
      uint32_t hi[kHalf], lo[kHalf];
      const uint32_t col = tmem + lanes + kSCol + (uint32_t)(sb * 2 * kRows + half * kHalf);
      tmem_ld16(col, hi);
      tmem_ld16(col + kRows, lo);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.sfree[sb]);
      float y[kHalf];
#pragma unroll
      for (int r = 0; r < kHalf; ++r) y[r] = fmaf(__uint_as_float(lo[r]), 0.0625f, __uint_as_float(hi[r]));
      const int key = (u.tile0 + t) * kTile + my_key;
      uint32_t seen = key < u.keys ? 0xFFFFu : 0u;  // rows that see the key
      if (key >= u.prefix && key < u.keys) {
        seen = 0;
#pragma unroll
        for (int r = 0; r < kHalf; ++r) seen |= (uint32_t)((sm.mask[half * kHalf + r] >> (key - u.prefix)) & 1) << r;
      }
      const bool all_seen = __all_sync(0xffffffffu, seen == 0xFFFFu);
      const float c = scale * factor, held = fmaxf(scale, kTiny) * kUnit;
      const uint32_t counts = scale >= kTiny ? 0xFFFFFFFFu : 0u;
      float p[kHalf], w[kHalf];
      auto weigh = [&]() -> float {
        float most = 0.f;
#pragma unroll
        for (int r = 0; r < kHalf; ++r) {
          p[r] = ex2_approx(fmaf(y[r], c, -m[r]));
          if (!all_seen) p[r] = (seen >> r) & 1 ? p[r] : 0.f;
          w[r] = p[r] * held;
          most = fmaxf(most, w[r]);
        }
        return most;
      };
      const float most = weigh();
      if (soft_vote(most > kMost || sm.abort_flag != 0)) {
        // some weight is too large for its row's reference: raise the references to the tile's largest
        if (tid == 0) sm.stop = sm.abort_flag;
        const float height = __log2f(fmaxf(scale, kTiny));
#pragma unroll
        for (int r = 0; r < kHalf; ++r) {
          const float top = warp_top((seen >> r) & 1 ? fmaf(y[r], c, height) : -INFINITY);
          if (lane == 0) sm.part[quarter][half * kHalf + r] = top;
        }
        soft_sync();
        if (sm.stop) return;
        float f[kHalf];
#pragma unroll
        for (int r = 0; r < kHalf; ++r) {
          float top = m[r];
#pragma unroll
          for (int k = 0; k < 4; ++k) top = fmaxf(top, sm.part[k][half * kHalf + r]);
          f[r] = ex2_approx(m[r] - top);
          m[r] = top;
          l[r] *= f[r];
        }
        if (t > 0) {
          // what has been summed so far, once the products before are complete
          wait(sm, &sm.pfree[(it - 1) & 1], ((it - 1) >> 1) & 1, a, 301);
          __syncwarp();
          tc_fence_after();
#pragma unroll 1
          for (int k = 0; k < kChunks * kParts; ++k) {
            const uint32_t at = tmem + lanes + (uint32_t)(k * kRows + half * kHalf);
            uint32_t o[kHalf];
            tmem_ld16(at, o);
            tmem_wait_ld();
#pragma unroll
            for (int r = 0; r < kHalf; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * f[r]);
            tmem_st16(at, o);
          }
          tmem_wait_st();
          tc_fence_before();
        }
        soft_sync();  // (part is written again only past this)
        weigh();
      }
#pragma unroll
      for (int r = 0; r < kHalf; ++r) l[r] += p[r];
      // three parts of each weight, four rows to a word
      uint32_t parts[kParts][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t h[2][kParts];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t x, r1, r2;
          asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(x) : "f"(w[4 * k + 2 * j + 1]), "f"(w[4 * k + 2 * j]));
          x = ((x + 0x00020002u) & 0xFFFCFFFCu) & counts;
          h[j][0] = x & 0xFF00FF00u;
          asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r1) : "r"(x), "r"(h[j][0]));
          h[j][1] = r1 & 0xFF00FF00u;
          asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r2) : "r"(r1), "r"(h[j][1]));
          h[j][2] = r2;
        }
#pragma unroll
        for (int q = 0; q < kParts; ++q) parts[q][k] = __byte_perm(h[0][q], h[1][q], 0x7531);
      }
      const int pb = it & 1;
      if (wait(sm, &sm.pfree[pb], ((it >> 1) & 1) ^ 1, a, 302)) {
        uint8_t* row = sm.p[pb] + my_key * 128;
#pragma unroll
        for (int q = 0; q < kParts; ++q)
          *reinterpret_cast<uint4*>(row + (((2 * q + half) ^ (my_key & 7)) << 4)) =
              make_uint4(parts[q][0], parts[q][1], parts[q][2], parts[q][3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.pfull[pb]);
      scale = next_scale;
    }
    // row sums over the keys
#pragma unroll
    for (int r = 0; r < kHalf; ++r) {
      l[r] = warp_sum(l[r]);
      if (lane == 0) sm.part[quarter][half * kHalf + r] = l[r];
    }
    soft_sync();
#pragma unroll
    for (int r = 0; r < kHalf; ++r) {
      const int row = half * kHalf + r;
      l[r] = (sm.part[0][row] + sm.part[1][row]) + (sm.part[2][row] + sm.part[3][row]);
    }
    const Unit done = u;
    // the next unit's queries while this one's last products run
    more = units.next(sm, a, plan, u);
    if (more) factor = load_queries(sm, a, u);
    wait(sm, &sm.pfree[(it - 1) & 1], ((it - 1) >> 1) & 1, a, 303);
    __syncwarp();
    tc_fence_after();
    const int64_t piece = (int64_t)blockIdx.x * 2 + (done.head ? 1 : 0);
    float* po = part.o + piece * kRows * kDv;
#pragma unroll 1
    for (int c = 0; c < kChunks; ++c) {
      const int dim = 128 * c + my_key;  // this thread's lane of O^T
      uint32_t o[kHalf], x[kHalf];
      const uint32_t at = tmem + lanes + (uint32_t)(c * kOCols + half * kHalf);
      tmem_ld16(at, o);
      tmem_ld16(at + kRows, x);
      tmem_wait_ld();
#pragma unroll
      for (int r = 0; r < kHalf; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) + __uint_as_float(x[r]));
      tmem_ld16(at + 2 * kRows, x);
      tmem_wait_ld();
#pragma unroll
      for (int r = 0; r < kHalf; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) + __uint_as_float(x[r]));
      if (done.whole) {
        // pairs of lanes exchange a value each, so that a lane stores two columns of one row
#pragma unroll
        for (int r = 0; r < kHalf; r += 2) {
          const float s0 = l[r] > 0.f ? __fdividef(1.f, l[r] * kUnit) : 0.f, s1 = l[r + 1] > 0.f ? __fdividef(1.f, l[r + 1] * kUnit) : 0.f;
          const float a0 = __uint_as_float(o[r]) * s0, a1 = __uint_as_float(o[r + 1]) * s1;
          const float other = __shfl_xor_sync(0xffffffffu, lane & 1 ? a0 : a1, 1);
          const uint32_t pair = lane & 1 ? pack_bf16x2(other, a1) : pack_bf16x2(a0, other);
          const int row = half * kHalf + r + (lane & 1);
          if (row < done.rows)
            *reinterpret_cast<uint32_t*>(a.out + (done.out_row + row) * kDv + (dim & ~1)) = pair;
        }
      } else {
#pragma unroll
        for (int r = 0; r < kHalf; ++r) po[(half * kHalf + r) * kDv + dim] = __uint_as_float(o[r]);
      }
    }
    if (quarter == 0) {
#pragma unroll
      for (int r = 0; r < kHalf; ++r) {
        const int row = half * kHalf + r;
        if (lane == r) {
          if (!done.whole) part.ml[piece * kRows + row] = make_float2(m[r], l[r]);
          else if (row < done.rows)
            a.lse[done.out_row + row] = l[r] > 0.f ? (m[r] + log2f(l[r])) * 0.6931471805599453f : -INFINITY;
        }
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.ofree);
    ++units_done;
  }
}

__global__ void __launch_bounds__(kThreads, 1)
scaled_kernel(const __grid_constant__ CUtensorMap latent, const __grid_constant__ CUtensorMap rope,
              const __grid_constant__ ScaledArgs a, CtaInfo* __restrict__ info, const Partials part) {
  extern __shared__ uint8_t raw[];
  Shared& sm = *reinterpret_cast<Shared*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.kfull[s], 1);
      mbar_init(&sm.kfree[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.sfull[s], 1);
      mbar_init(&sm.sfree[s], kSoftWarps);
      mbar_init(&sm.pfull[s], kSoftWarps);
      mbar_init(&sm.pfree[s], 1);
    }
    mbar_init(&sm.qfull, kSoftWarps);
    mbar_init(&sm.ofree, kSoftWarps);
    mbar_init(&sm.done, 1);
    sm.abort_flag = 0;
    sm.fault[0] = sm.fault[1] = 0;
    fence_mbar_init();
    prefetch_tensormap(&latent);
    prefetch_tensormap(&rope);
  }
  Plan plan;
  const bool ok = make_plan(sm, a, plan);
  CtaInfo mine = {};
  if (ok) {
    if (tid == 0) {
      Units units(sm, a, plan);
      Unit u;
      while (units.next(sm, a, plan, u))
        if (u.head && !u.whole) {
          mine.row = u.out_row;
          mine.pieces = u.pieces;
          mine.rows = u.rows;
          mine.group = plan.group;
        }
    }
    __syncwarp();
    if (warp == kMmaWarp) {
      tmem_alloc(&sm.tmem, 512);
      tmem_relinquish();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    if (warp < kSoftWarps) {
      softmax_role(sm, a, plan, tmem, part);
    } else if (warp == kMmaWarp) {
      if ((tid & 31) == 0) mma_role(sm, a, plan, tmem);
    } else {
      load_role(sm, &latent, &rope, a, plan);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    grid_dependents_launch();
    if (sm.abort_flag) {
      // a wait ran out: loads, commits and products issued before may still be on their way into this CTA's memories,
      // each for microseconds; half a millisecond of the global timer (at most 2^26 reads of it)
      if (tid == 0) {
        uint64_t t0, t;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
        for (int k = 0; k < (1 << 26); ++k) {
          asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
          if (t - t0 > 500000ull) break;
        }
      }
      __syncthreads();
    }
    __syncwarp();
    if (warp == kMmaWarp) {
      tc_fence_after();
      tmem_dealloc(tmem, 512);
    }
  }
  if (tid == 0) {
    mine.fault = ok ? sm.fault[0] : (uint32_t)VMLA_ERR_SHAPE;
    mine.fault_info = ok ? sm.fault[1] : 0;
    if (sm.abort_flag) mine.pieces = 0;
    info[blockIdx.x] = mine;
  }
}

// Joins the partials of one row of a cut stream: one block per (CTA that begins the stream, row).
constexpr int kJoinThreads = kDv / 4;
constexpr int kMaxCtas = 512;
__global__ void __launch_bounds__(kJoinThreads)
scaled_join_kernel(const CtaInfo* __restrict__ info, int ctas, const Partials part, uint16_t* __restrict__ out,
                   float* __restrict__ lse, uint32_t* __restrict__ status) {
  __shared__ float2 ml[kMaxCtas];
  const int tid = threadIdx.x, cta = blockIdx.x, row = blockIdx.y;
  grid_dependency_wait();
  if (cta == 0 && row == 0 && tid < 32) {
    // the call's status: the first CTA's fault
    uint32_t first = 0xffffffffu;
    for (int k = tid; k < ctas; k += 32)
      if (info[k].fault != 0) first = min(first, (uint32_t)k);
    first = __reduce_min_sync(0xffffffffu, first);
    if (tid == 0) {
      status[0] = first == 0xffffffffu ? 0u : info[first].fault;
      status[1] = first == 0xffffffffu ? 0u : info[first].fault_info;
    }
  }
  const CtaInfo i = info[cta];
  if (row >= i.rows || i.pieces == 0) return;
  // piece 0 lies in this CTA's second slot, piece k in the first slot of the CTA k lanes on
  auto slot = [&](int k) { return k == 0 ? (int64_t)cta * 2 + 1 : ((int64_t)cta + (int64_t)k * i.group) * 2; };
  for (int k = tid; k < i.pieces; k += kJoinThreads) ml[k] = part.ml[slot(k) * kRows + row];
  __syncthreads();
  float top = kNone;
  for (int k = 0; k < i.pieces; ++k) top = fmaxf(top, ml[k].x);
  float sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < i.pieces; ++k) {
    const float w = ex2_approx(ml[k].x - top);
    const float4 v = reinterpret_cast<const float4*>(part.o + (slot(k) * kRows + row) * kDv)[tid];
    sum = fmaf(ml[k].y, w, sum);
    o.x = fmaf(v.x, w, o.x);
    o.y = fmaf(v.y, w, o.y);
    o.z = fmaf(v.z, w, o.z);
    o.w = fmaf(v.w, w, o.w);
  }
  const float f = sum > 0.f ? 1.f / (sum * kUnit) : 0.f;
  reinterpret_cast<uint2*>(out + (i.row + row) * kDv)[tid] =
      make_uint2(pack_bf16x2(o.x * f, o.y * f), pack_bf16x2(o.z * f, o.w * f));
  if (tid == 0) lse[i.row + row] = sum > 0.f ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

// Workspace: status words, the CTAs' infos, the partials.
constexpr size_t kInfoOff = 256;
size_t ml_off(int sms) { return kInfoOff + (((size_t)sms * sizeof(CtaInfo) + 255) & ~(size_t)255); }
size_t o_off(int sms) { return ml_off(sms) + (size_t)sms * 2 * kRows * sizeof(float2); }

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// The pool as rows of bytes, boxes one row high and `width` bytes wide for gathers of four rows.
bool encode_pool(EncodeTiledFn enc, CUtensorMap* map, const uint8_t* pool, int64_t slots, uint32_t width,
                 CUtensorMapSwizzle swizzle) {
  cuuint64_t gdim[2] = {(cuuint64_t)kDqk, (cuuint64_t)(slots > 0 ? slots : 1)};
  cuuint64_t gstride[1] = {(cuuint64_t)kDqk};
  cuuint32_t box[2] = {width, 1};
  cuuint32_t estride[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(pool), gdim, gstride, box, estride,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t scaled_workspace(int sms) { return o_off(sms) + (size_t)sms * 2 * kRows * kDv * sizeof(float); }

int launch_scaled(const ScaledArgs& a, int sms, void* stream) {
  if (sms > kMaxCtas) return VMLA_ERR_DEVICE;
  EncodeTiledFn enc = encode_fn();
  if (!enc) return VMLA_ERR_DEVICE;
  CUtensorMap latent, rope;
  // (without keys nothing is fetched: any address does)
  const uint8_t* pool = a.pool ? a.pool : reinterpret_cast<const uint8_t*>(a.workspace);
  if (!encode_pool(enc, &latent, pool, a.pool_slots, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_pool(enc, &rope, pool, a.pool_slots, 64, CU_TENSOR_MAP_SWIZZLE_64B))
    return VMLA_ERR_CUDA;
  static std::mutex mu;
  static bool ready[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return VMLA_ERR_CUDA;
  {
    std::lock_guard<std::mutex> g(mu);
    if (dev >= 64 || !ready[dev]) {
      if (cudaFuncSetAttribute(scaled_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSharedBytes) !=
          cudaSuccess)
        return VMLA_ERR_CUDA;
      if (dev < 64) ready[dev] = true;
    }
  }
  CtaInfo* info = reinterpret_cast<CtaInfo*>(a.workspace + kInfoOff);
  Partials part;
  part.ml = reinterpret_cast<float2*>(a.workspace + ml_off(sms));
  part.o = reinterpret_cast<float*>(a.workspace + o_off(sms));
  scaled_kernel<<<sms, kThreads, kSharedBytes, (cudaStream_t)stream>>>(latent, rope, a, info, part);
  if (cudaGetLastError() != cudaSuccess) return VMLA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {early_start_attribute()};
  cfg.gridDim = dim3((unsigned)sms, kRows, 1);
  cfg.blockDim = dim3(kJoinThreads, 1, 1);
  cfg.stream = (cudaStream_t)stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, scaled_join_kernel, (const CtaInfo*)info, sms, part, a.out, a.lse, a.status) ==
                 cudaSuccess
             ? VMLA_OK
             : VMLA_ERR_CUDA;
}

}  // namespace vmla
