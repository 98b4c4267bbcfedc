// Attention over a pool of 8-bit codes with one scale per block of slots, in 8 bits on the tensor cores.
//
// For a query row r (a draft's head) and key j with slot s, codes k_j (e4m3) and scale a_j = scales[s / block]:
//   s_rj = sm_scale a_j <q_r, k_j>,  p_rj = 2^(s_rj log2 e - m_r),  out_r = sum_j p_rj a_j k_j[:512] / sum_j p_rj.
// The codes are operands as they are: nothing is converted to bf16, staged, or written back.  What is not 8 bits wide
// is split into parts that are, exactly or nearly so:
//   queries  q a_r = hi + lo / 16, both e4m3, a_r the power of two that brings the row's largest to (224, 448]:
//            off by at most 2^-14 of what is 448 at the largest (2^-22.8), less than an fp32 dot product's rounding
//   weights  p a_j 2^9, in fp16 rounded to 9 bits, cut into three parts of three bits, e5m2: the upper byte of an fp16
//            number is an e5m2 number, so a part is an AND and the rest an exact difference.  The last part is held times
//            2^6 (it has sums of its own) and rounded: its range ends at 2^-22 instead of 2^-16, where small weights would
//            all be cut, a loss that grows with their number.  The range (2^-22 to 2^15) is why it is not two e4m3 parts:
//            beside a key of much weight, 10^5 keys of weight 10^-8 each still count.
//
// Keys are the matrix products' M (tiles of 128), query rows their N (units of 32), so that few rows waste nothing:
//   S^T [128 keys x 64]  = K [128 x 576] (Q hi | Q lo)^T               18 products, M128 N64 K32
//   O^T [512 x 96]      += V^T [512 x 128 keys] (P hi | P mid | P lo)^T  16 products, M128 N96 K32, V being K's first columns
// O^T takes 384 of the 512 columns of tensor memory, two S^T the rest.  One read of a tile's rows serves both products.
// A softmax thread has one key and 16 rows: a_j is its own number, the reference m_r is raised only when a weight passes
// 2^15 (told by one barrier with a vote per tile), and row sums stay in registers until the unit ends.
//
// Rows are fetched straight from the pool, 128 columns at a time into a ring of ten such chunks (two and a half tiles): by
// boxes of 16 slots where the slots of a tile are consecutive in 16s, else by gathers of four slots; a slot that is none,
// or a place behind the last key, is a coordinate outside the tensor and reads zeros.
//
// Work: the row blocks (32 rows) of a sequence form streams over its key tiles, laid end to end (a stream costs its tiles
// and kFixed more); the l-th of the CTAs, one per SM, takes the l-th share of the whole length.  Streams cut by the end of a
// share leave fp32 partials (at most two per CTA), and a second launch joins them.  Every CTA works the plan out from the
// device's lengths.
//
// What bounds it: shared memory.  Of its 128 bytes a clock a tile takes 1755 wavefronts as operands of the products, 540
// as it arrives, and some 900 for weights, references, indices and shuffles; with eight trees of 40 to 64 drafts over
// 9 000 to 16 000 keys the pipe is busy 83 % of the whole launch, the tensor pipe 37 %, DRAM 4 %.  A tile takes 1.5 us
// there, of which its products are 0.9; 1.65 us where the rows come from DRAM (32 requests of 64 heads).  About 16 us of
// a call are launches, plan, queries, the first tile's loads, results and the join (one request of 1024 keys: 18.4 us, of
// which 1.2 the barriers, 0.8 the plan, 3.9 the queries and 3.1 the first tile's scores and weights).
// Measured (us): 32 requests of 64 heads, up to 60 000 keys 114; 64 requests of 8 heads and 4 drafts, up to 32 768 keys 80;
// eight trees 264 to 272; 185 000 keys, 64 heads, 4 drafts 136.  Tried, without gain: clusters of two and four CTAs that share
// each tile's loads by multicast (faster than one issuing thread that also loaded, slower than this form: 142 us against
// 121); units of 64 rows (as fast; the accumulators of three parts would not fit, so the parts took turns); 16 softmax
// warps of 8 rows; a vote by word and barrier or cast early and counted late; longer sleeps of the waiting warps;
// references in registers; rows fetched into L2 ahead (all within 2 %).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <mutex>

#include "vmla_device.cuh"
#include "vmla_sm100.cuh"
#include "vmla_weights.cuh"

namespace vmla {
using namespace sm100;
using weights::both;
using weights::fma2;
using weights::mul2;
namespace {

constexpr int kTile = 128;          // keys
constexpr int kRows = 32;           // query rows of a unit
constexpr int kChunks = kDv / 128;  // 4 column chunks of 128 bytes, and one of 64
constexpr int kPieces = kChunks + 1;
constexpr int kRopePiece = 3;       // place of the rotated columns among a tile's pieces
constexpr int kParts = 3;           // of a weight
constexpr int kPerThread = 16;      // rows of a softmax thread
constexpr int kSoftWarps = 4 * kRows / kPerThread;  // per quarter of the tile's keys, 16 rows each
constexpr int kSoftThreads = kSoftWarps * 32;
constexpr int kScoreWarp = kSoftWarps, kValueWarp = kScoreWarp + 1, kLoadWarp = kValueWarp + 1;
constexpr int kLoadWarps = 6;
constexpr int kThreads = 32 * (kLoadWarp + kLoadWarps);
constexpr int kRun = 16;            // consecutive slots that one box fetches
constexpr uint32_t kOCols = kParts * kRows;       // 96 columns of tensor memory per 128 value columns
constexpr uint32_t kSCol = kChunks * kOCols;      // 384
constexpr int kSlots = 10;          // chunks in shared memory: two and a half tiles
constexpr int kFixed = 8;           // what a unit costs beside its tiles, in tiles
constexpr float kNone = -3e38f;     // reference of a row that has seen no key
constexpr float kUnitBits = 9.f;    // weights are held times 2^9
constexpr float kMost = 32768.f;    // largest weight held
constexpr float kLow = 64.f;        // what the last part of a weight is held times: it is below 2^9
constexpr float kTiny = 0x1p-100f;  // smaller scales count as zero
static_assert(kSCol + 2 * 2 * kRows == 512, "tensor memory");
static_assert(kThreads % 128 == 0, "whole register banks");
static_assert(kLoadWarps == kChunks + 2 && kTile / kRun == 8, "see load_role");

// A sequence's lengths.
struct Seq {
  int32_t q0, nq, kv0, nk;
};

// Barriers.
struct Bars {
  uint64_t full[kSlots], free[kSlots], rope_full, rope_free;
  uint64_t sfull[2], sfree[2], pfull, pfree, qfull, ofree;
};

struct Shared {
  uint8_t latent[kSlots][kTile * 128];        // a tile's chunk: [key][128 bytes], 128-byte swizzle
  uint8_t q_latent[kChunks][2 * kRows * 128]; // [hi rows, lo rows][128 bytes], 128-byte swizzle
  uint8_t p[kTile * 128];                     // [key][hi 32 | mid 32 | lo 32 | -], 128-byte swizzle
  uint8_t rope[kTile * 64];                   // [key][64 bytes], 64-byte swizzle
  uint8_t q_rope[2 * kRows * 64];             // 64-byte swizzle
  float back[kRows];                          // of each row: what its products are times as a score (log2)
  float minus[kRows], f[kRows];               // kUnitBits less each row's reference (log2), factor of its last change
  float part[4][kRows];                       // per quarter of the keys: row maxima, or row sums
  uint64_t mask[kRows];                       // the unit's rows: visible drafts
  uint32_t cost[VMLA_MAX_BATCH + 1];          // cost position of each sequence's first stream
  Seq first_seq;                              // where this CTA's share begins: sequence, row block, cost position
  int32_t first_b, first_g;
  uint32_t first_at;
  int32_t parent[VMLA_MAX_DRAFT];
  uint32_t sums[2][kThreads / 32];
  Bars bars;
  uint32_t tmem;
  volatile int32_t abort_flag;
  int32_t stop;
  uint32_t fault[2];                          // first fault of this CTA: code, info
  int32_t cut_pieces, cut_rows;               // the stream that starts in this CTA's share and goes on in the next
  int64_t cut_row;
};
constexpr size_t kSharedBytes = sizeof(Shared) + 1024;
static_assert(kSharedBytes <= 232448, "shared memory");

// What a CTA tells the joining launch: the stream that starts in its share and is cut by the share's end, and its fault.
struct alignas(32) CtaInfo {
  int64_t row;      // first row of out
  int32_t pieces;   // 0: no such stream
  int32_t rows;
  uint32_t fault, fault_info;
  int32_t pad[2];
};

struct Partials {
  float* o;        // [2 x CTAs][kRows][512]
  float2* ml;      // [2 x CTAs][kRows]: reference less kUnitBits (log2), sum
};

__device__ __forceinline__ void fault(Shared& sm, int code, uint32_t info) {
  if (atomicCAS(&sm.fault[0], 0u, (uint32_t)code) == 0u) sm.fault[1] = info;
}

struct Maps {
  CUtensorMap latent, rope;          // gathers of four rows
  CUtensorMap latent_run, rope_run;  // boxes of kRun rows
};

// ------------------------------------------------------------------ plan
// Costs are counted in tiles; a call whose cost does not fit 31 bits (2^27 for a warp's 32 sequences) is refused.
// Keys are looked up to two tiles ahead of the last one, in 32 bits.
static_assert(VMLA_MAX_SCALED_KV <= INT32_MAX - 3 * kTile, "positions of keys fit 32 bits");
struct Plan {
  uint32_t length;  // of all streams
  uint32_t share;   // of a CTA
};

__device__ __forceinline__ Seq seq_of(const ScaledArgs& a, int b) {
  Seq s;
  s.q0 = __ldg(a.qo_indptr + b);
  s.nq = __ldg(a.qo_indptr + b + 1) - s.q0;
  s.kv0 = __ldg(a.kv_indptr + b);
  s.nk = __ldg(a.kv_indptr + b + 1) - s.kv0;
  return s;
}
__device__ __forceinline__ int row_blocks(const ScaledArgs& a, int nq) {
  return (nq * a.num_heads + kRows - 1) / kRows;
}
__device__ __forceinline__ int tiles_of(int nk) { return nk / kTile + (nk % kTile != 0); }

// Ends of a thread's sequence in the lengths' arrays.
struct Ends {
  int32_t k0 = 0, k1 = 0, q0 = 0, q1 = 0;
  __device__ __forceinline__ explicit Ends(const ScaledArgs& a) {
    const int b = threadIdx.x;
    if (b < a.batch) {
      k0 = __ldg(a.kv_indptr + b);
      k1 = __ldg(a.kv_indptr + b + 1);
      q0 = __ldg(a.qo_indptr + b);
      q1 = __ldg(a.qo_indptr + b + 1);
    }
  }
};

// Shares the work out (whole CTA); false where the lengths are out of order or past a bound.
__device__ bool make_plan(Shared& sm, const ScaledArgs& a, const Ends& mine, Plan& plan) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  static_assert(kThreads >= VMLA_MAX_BATCH, "a thread per sequence");
  bool ok = true;
  uint64_t cost = 0;
  if (tid < a.batch) {
    const int64_t k0 = mine.k0, k1 = mine.k1, q0 = mine.q0, q1 = mine.q1;
    ok = q1 >= q0 && q1 - q0 <= VMLA_MAX_DRAFT && k1 - k0 >= q1 - q0;
    if (tid == 0) ok = ok && k0 == 0 && q0 == 0;
    if (tid == a.batch - 1) ok = ok && k1 <= a.max_kv && q1 <= a.max_q;
    if (ok) cost = (uint64_t)row_blocks(a, (int)(q1 - q0)) * (uint64_t)(tiles_of((int)(k1 - k0)) + kFixed);
  }
  uint64_t upto = cost;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += u;
  }
  if (upto > 0x08000000u) ok = false;  // (so that sixteen warps' sums fit 32 bits)
  if (lane == 31) sm.sums[0][warp] = (uint32_t)upto;
  if (!__syncthreads_and(ok)) return false;
  uint32_t all = lane < kThreads / 32 ? sm.sums[0][lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, all, o);
    if (lane >= o) all += u;
  }
  plan.length = __shfl_sync(0xffffffffu, all, 31);
  const uint32_t before = warp > 0 ? __shfl_sync(0xffffffffu, all, warp - 1) : 0;
  if (tid <= a.batch) sm.cost[tid] = before + (uint32_t)(upto - cost);
  if (tid == 0 && a.batch == kThreads) sm.cost[a.batch] = plan.length;
  plan.share = (plan.length + gridDim.x - 1) / gridDim.x;
  if (plan.share == 0) plan.share = 1;
  // the sequence that this CTA's share begins in
  const uint32_t from = blockIdx.x * plan.share, at = before + (uint32_t)(upto - cost);  // (from: below length + share)
  if (from >= at && from - at < (uint32_t)cost) {
    const Seq s = {mine.q0, mine.q1 - mine.q0, mine.k0, mine.k1 - mine.k0};
    const uint32_t span = tiles_of(s.nk) + kFixed, g = (from - at) / span;
    sm.first_seq = s;
    sm.first_b = tid;
    sm.first_g = (int)g;
    sm.first_at = at + g * span;
  }
  __syncthreads();
  return true;
}

// One row block of a sequence over some of its tiles.
struct Unit {
  int row_block, rows;      // rows of the block that are the sequence's
  int tile0, tiles;         // its tiles
  int q0, nq;               // the sequence's drafts
  int kv0, keys, prefix;    // first entry of kv_indices; keys and prefix of the sequence
  bool whole, head;         // every tile of the stream; its first tile is among these
  uint32_t stop;            // cost position behind the stream's tiles
};

// The units of a CTA, in order.
struct Units {
  uint32_t at, end, from;  // cost position of the current stream; of the share's end and start
  int b, g, n;
  Seq s;
  __device__ __forceinline__ void enter(const Shared& sm, const ScaledArgs& a, int sequence) {
    for (b = sequence; b < a.batch; ++b) {
      s = seq_of(a, b);
      n = row_blocks(a, s.nq);
      if (n > 0) break;
    }
    g = 0;
    at = b < a.batch ? sm.cost[b] : 0xFFFFFFFFu;
  }
  __device__ __forceinline__ Units(const Shared& sm, const ScaledArgs& a, const Plan& p) {
    from = blockIdx.x * p.share;
    end = from + p.share < p.length ? from + p.share : p.length;
    if (from >= end) {
      end = 0;
      at = 0xFFFFFFFFu;
      return;
    }
    b = sm.first_b;
    g = sm.first_g;
    at = sm.first_at;
    s = sm.first_seq;
    n = row_blocks(a, s.nq);
  }
  // The current stream's tiles that lie in the share; whether there are any.
  __device__ __forceinline__ bool current(const ScaledArgs& a, Unit& u) const {
    const int tiles = tiles_of(s.nk);
    const uint32_t lo = at > from ? at : from, stop = at + tiles, hi = stop < end ? stop : end;
    if (lo >= hi) return false;
    u.row_block = g;
    u.rows = min(kRows, s.nq * a.num_heads - g * kRows);
    u.tile0 = (int)(lo - at);
    u.tiles = (int)(hi - lo);
    u.q0 = s.q0;
    u.nq = s.nq;
    u.kv0 = s.kv0;
    u.keys = s.nk;
    u.prefix = s.nk - s.nq;
    u.head = lo == at;
    u.whole = u.tiles == tiles;
    u.stop = stop;
    return true;
  }
  __device__ __noinline__ bool next(const Shared& sm, const ScaledArgs& a, Unit& u) {
    do {
      if (++g < n) at += tiles_of(s.nk) + kFixed;
      else enter(sm, a, b + 1);
      if (at >= end) return false;
    } while (!current(a, u));
    return true;
  }
  __device__ __forceinline__ bool first(const Shared& sm, const ScaledArgs& a, Unit& u) {
    return at < end && (current(a, u) || next(sm, a, u));
  }
};
__device__ __forceinline__ int64_t out_row(const ScaledArgs& a, const Unit& u) {
  return (int64_t)u.q0 * a.num_heads + (int64_t)u.row_block * kRows;
}

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

// A position in the ring of chunks, and the parity of its round.
struct Ring {
  uint32_t slot = 0, parity = 0;
  __device__ __forceinline__ Ring plus(uint32_t n) const {  // n < kSlots
    Ring r;
    const bool wrap = slot + n >= kSlots;
    r.slot = wrap ? slot + n - kSlots : slot + n;
    r.parity = parity ^ wrap;
    return r;
  }
};

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

// ------------------------------------------------------------------ loads (six warps)
// A tile's pieces are its four chunks and the rotated columns, each with a barrier of its own per place.  Where all of the
// tile's slots are consecutive in groups of kRun, a piece is eight boxes and one or two warps'; otherwise it is 32 gathers
// of four rows, dealt out to all six: starting a copy takes its thread some 80 clocks.  The slots are brought to all lanes
// of a warp, and one lane starts the copies, with operands that the whole warp has (see elect_one).
// A barrier's parity tells apart two rounds of its stage, no more.  Every warp has a part in a chunk of every tile and waits
// for it, so it is never two rounds ahead of any piece (its chunk's release three tiles ago follows all of the tile before
// that), and no round that it waits for can pass unseen, since the piece lacks its part.
__device__ void load_role(Shared& sm, const Maps& maps, const ScaledArgs& a, Units& units, Unit& u, bool more) {
  const int warp = (threadIdx.x >> 5) - kLoadWarp, lane = threadIdx.x & 31;
  const int none = (int)a.pool_slots;       // outside the tensor: zeros
  constexpr int kGroups = (kTile / 4 + kLoadWarps - 1) / kLoadWarps;  // of four keys, the warp's: warp, warp + 6 ..
  constexpr int kBoxes = kTile / kRun;
  const bool last_group = warp + kLoadWarps * (kGroups - 1) < kTile / 4;
  const uint32_t full0 = smem_u32(&sm.bars.full[0]), latent0 = smem_u32(sm.latent[0]), rope0 = smem_u32(sm.rope),
                 rope_bar = smem_u32(&sm.bars.rope_full);
  Ring ring;  // of the tile's first chunk
  uint32_t it = 0;
  for (; more; more = units.next(sm, a, u)) {
    const int32_t* index = a.kv_indices + u.kv0;
    const int last = min(u.keys, (u.tile0 + u.tiles) * kTile);  // behind this unit's keys
    const int tiles = u.tiles;
    int key = u.tile0 * kTile + 4 * lane;
    int32_t ahead[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) ahead[k] = key + k < last ? __ldg(index + key + k) : -1;
#pragma unroll 1
    for (int t = 0; t < tiles; ++t, ++it, ring = ring.plus(kChunks)) {
      int32_t y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        y[k] = ahead[k];
        if ((uint32_t)y[k] >= (uint32_t)none) {
          if (warp == 0 && key + k < last) fault(sm, VMLA_ERR_INDEX, (uint32_t)(u.kv0 + key + k));
          y[k] = none;
        }
      }
      key += kTile;
#pragma unroll
      for (int k = 0; k < 4; ++k) ahead[k] = key + k < last ? __ldg(index + key + k) : -1;
      const int first = __shfl_sync(0xffffffffu, y[0], lane & ~3);
      const bool runs = __all_sync(0xffffffffu, y[0] == first + 4 * (lane & 3) && y[1] == y[0] + 1 && y[2] == y[0] + 2 &&
                                                    y[3] == y[0] + 3 && y[3] < none);
      if (runs) {
        // warps 0 to 3 have a chunk each, 4 and 5 half of chunks 0 and 1, and the rotated columns
        const int chunk = warp & 3;
        const Ring at = ring.plus(chunk);
        const bool upper = warp >= kChunks, whole = chunk >= kLoadWarps - kChunks;
        int32_t r[kBoxes];
#pragma unroll
        for (int k = 0; k < kBoxes; ++k) r[k] = __shfl_sync(0xffffffffu, y[0], (upper ? k ^ (kBoxes / 2) : k) * (kRun / 4));
        const uint32_t at0 = upper ? kBoxes / 2 : 0;  // r[k]: box k ^ at0
        if (!__all_sync(0xffffffffu, wait(sm, &sm.bars.free[at.slot], at.parity ^ 1, a, 100))) return;
        if (elect_one()) {
          const uint32_t bar = full0 + at.slot * 8, dst = latent0 + at.slot * (kTile * 128);
          if (!upper) mbar_arrive_expect_tx(bar, kTile * 128);
#pragma unroll
          for (int k = 0; k < kBoxes; ++k)
            if (k < kBoxes / 2 || whole) tma_load_2d(dst + (k ^ at0) * kRun * 128, &maps.latent_run, chunk * 128, r[k], bar);
        }
        __syncwarp();
        if (upper) {
          if (!__all_sync(0xffffffffu, wait(sm, &sm.bars.rope_free, (it & 1) ^ 1, a, 101))) return;
          if (elect_one()) {
            if (warp == kChunks) mbar_arrive_expect_tx(rope_bar, kTile * 64);
            // (boxes 4 to 7 by warp 4, which has them first, 0 to 3 by warp 5)
#pragma unroll
            for (int k = 0; k < kBoxes / 2; ++k) {
              const int q = warp == kChunks ? k : k + kBoxes / 2;
              tma_load_2d(rope0 + (q ^ at0) * kRun * 64, &maps.rope_run, kDv, warp == kChunks ? r[k] : r[k + kBoxes / 2],
                          rope_bar);
            }
          }
          __syncwarp();
        }
        continue;
      }
      int32_t g[kGroups][4];
#pragma unroll
      for (int k = 0; k < kGroups; ++k)
#pragma unroll
        for (int q = 0; q < 4; ++q) g[k][q] = __shfl_sync(0xffffffffu, y[q], (warp + kLoadWarps * k) & 31);
#pragma unroll
      for (int piece = 0; piece < kPieces; ++piece) {
        const int chunk = piece < kRopePiece ? piece : piece - 1, row = piece == kRopePiece ? 64 : 128;
        const Ring at = ring.plus(chunk);
        if (!__all_sync(0xffffffffu, piece == kRopePiece ? wait(sm, &sm.bars.rope_free, (it & 1) ^ 1, a, 102)
                                                         : wait(sm, &sm.bars.free[at.slot], at.parity ^ 1, a, 102)))
          return;
        if (elect_one()) {
          const uint32_t bar = piece == kRopePiece ? rope_bar : full0 + at.slot * 8,
                         dst = piece == kRopePiece ? rope0 : latent0 + at.slot * (kTile * 128);
          if (warp == 0) mbar_arrive_expect_tx(bar, kTile * row);
#pragma unroll
          for (int k = 0; k < kGroups; ++k)
            if (k < kGroups - 1 || last_group)
              tma_gather4(dst + (warp + kLoadWarps * k) * 4 * row, piece == kRopePiece ? &maps.rope : &maps.latent,
                          piece == kRopePiece ? kDv : chunk * 128, g[k][0], g[k][1], g[k][2], g[k][3], bar);
        }
        __syncwarp();
      }
    }
  }
  // the pieces' last releases have arrived before the CTA may leave
  // (each is waited for by a warp that filled its slot last: the first warp fills part of every tile's first chunk, and
  // the later ones follow it)
  if (warp == 0) {
    for (uint32_t k = 0; k < kSlots; ++k) {
      const Ring at = ring.plus(k);
      wait(sm, &sm.bars.free[at.slot], at.parity ^ 1, a, 103);
    }
    wait(sm, &sm.bars.rope_free, (it & 1) ^ 1, a, 104);
  }
  __syncwarp();
}

// ------------------------------------------------------------------ matrix products (a warp each for scores and values)
// Lower words of the operands' descriptors; the upper words depend on the layout alone.
constexpr uint32_t kHi128 = (uint32_t)(smem_desc_fixed(16, 1024, 2) >> 32), kHi64 = (uint32_t)(smem_desc_fixed(16, 512, 4) >> 32);
__device__ __forceinline__ uint32_t desc_low(const void* at) { return smem_u32(at) >> 4 | (uint32_t)smem_desc_fixed(16, 0, 0); }

// Piece by piece as a tile's columns arrive.
__device__ void score_role(Shared& sm, const ScaledArgs& a, uint32_t tmem, Units& units, Unit& u, bool more) {
  constexpr uint32_t kDesc = idesc_f8_f32(kTile, 2 * kRows, 0, 0, 0, 0);
  const uint32_t latent_lo = desc_low(sm.latent[0]), rope_lo = desc_low(sm.rope), q_latent_lo = desc_low(sm.q_latent[0]),
                 q_rope_lo = desc_low(sm.q_rope);
  Ring ring;
  uint32_t it = 0, unit = 0;
  for (; more; more = units.next(sm, a, u), ++unit) {
    const int tiles = u.tiles;
    if (!__all_sync(0xffffffffu, wait(sm, &sm.bars.qfull, unit & 1, a, 200))) return;
#pragma unroll 1
    for (int t = 0; t < tiles; ++t, ++it, ring = ring.plus(kChunks)) {
      const uint32_t sb = it & 1, d = tmem + kSCol + sb * 2 * kRows;
      if (!__all_sync(0xffffffffu, wait(sm, &sm.bars.sfree[sb], ((it >> 1) & 1) ^ 1, a, 201))) return;
#pragma unroll
      for (int piece = 0; piece < kPieces; ++piece) {
        const int chunk = piece < kRopePiece ? piece : piece - 1;
        const Ring at = ring.plus(chunk);
        if (!__all_sync(0xffffffffu, piece == kRopePiece ? wait(sm, &sm.bars.rope_full, it & 1, a, 202)
                                                         : wait(sm, &sm.bars.full[at.slot], at.parity, a, 202)))
          return;
        tc_fence_after();
        if (elect_one()) {
          if (piece == kRopePiece) {
#pragma unroll
            for (int i = 0; i < 2; ++i) mma_ss_f8(d, rope_lo + 2 * i, kHi64, q_rope_lo + 2 * i, kHi64, kDesc, 1u);
            mma_commit(&sm.bars.rope_free);
          } else {
            const uint32_t key = latent_lo + at.slot * (kTile * 128 / 16), q = q_latent_lo + chunk * (2 * kRows * 128 / 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) mma_ss_f8(d, key + 2 * i, kHi128, q + 2 * i, kHi128, kDesc, piece > 0 || i > 0);
          }
          if (piece == kPieces - 1) mma_commit(&sm.bars.sfull[sb]);
        }
        __syncwarp();
      }
    }
  }
}

// A tile at a time; each chunk makes room for a later tile's.
__device__ void value_role(Shared& sm, const ScaledArgs& a, uint32_t tmem, Units& units, Unit& u, bool more) {
  constexpr uint32_t kDesc = idesc_f8_f32(128, kOCols, 0, 1, 1, 1);
  const uint32_t latent_lo = desc_low(sm.latent[0]), p_lo = desc_low(sm.p);
  Ring ring;
  uint32_t it = 0, unit = 0;
  for (; more; more = units.next(sm, a, u), ++unit) {
    const int tiles = u.tiles;
    // (the first product into O: the unit before has been read out)
    if (!__all_sync(0xffffffffu, wait(sm, &sm.bars.ofree, (unit & 1) ^ 1, a, 210))) return;
#pragma unroll 1
    for (int t = 0; t < tiles; ++t, ++it, ring = ring.plus(kChunks)) {
      if (!__all_sync(0xffffffffu, wait(sm, &sm.bars.pfull, it & 1, a, 211))) return;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t go_on = t > 0;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          const Ring at = ring.plus(c);
          const uint32_t v = latent_lo + at.slot * (kTile * 128 / 16);
#pragma unroll
          for (int i = 0; i < kTile / 32; ++i)
            mma_ss_f8(tmem + c * kOCols, v + 256 * i, kHi128, p_lo + 256 * i, kHi128, kDesc, i > 0 ? 1u : go_on);
          mma_commit(&sm.bars.free[at.slot]);
        }
        mma_commit(&sm.bars.pfree);
      }
      __syncwarp();
    }
  }
}

// ------------------------------------------------------------------ queries (softmax warps)
// The unit's rows into shared memory in two e4m3 parts, what makes a score of each row's products, their masks.
// (What runs once per unit is kept in loops: straight-line code that is run once costs more in fetching it.)
__device__ __noinline__ void load_queries(Shared& sm, const ScaledArgs& a, const Unit& u) {
  constexpr int kGranules = kDqk / 8;              // of 8 bf16
  constexpr int kWarpRows = kRows / kSoftWarps;    // a warp has four whole rows
  constexpr int kEach = kWarpRows * kGranules / 32;  // 9 granules per thread
  static_assert(kWarpRows * kGranules % 32 == 0, "granules per thread");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, first = warp * kWarpRows;
  const uint4* src = reinterpret_cast<const uint4*>(a.q + (out_row(a, u) + first) * kDqk);
  uint4 v[kEach];
  const int valid = (u.rows - first) * kGranules;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int i = lane + k * 32;
    v[k] = i < valid ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
  }
  if (a.parent && tid < u.nq) sm.parent[tid] = a.parent[u.q0 + tid];
  // each row's largest magnitude, as bits of bf16
  uint32_t most[kWarpRows];
#pragma unroll
  for (int r = 0; r < kWarpRows; ++r) most[r] = 0;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x = w[j] & 0x7FFF7FFFu;
      asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(x));
    }
    m = max(m >> 16, m & 0xFFFFu);
#pragma unroll
    for (int r = 0; r < kWarpRows; ++r)
      if (k * 32 < (r + 1) * kGranules && (k + 1) * 32 > r * kGranules) {  // (known when compiling)
        const int i = lane + k * 32;
        if (i >= r * kGranules && i < (r + 1) * kGranules) most[r] = max(most[r], m);
      }
  }
  float mine = 0.f;  // lane r < 4: the power of two that brings row r's largest to (224, 448], 448 = 1.75 x 2^8
#pragma unroll
  for (int r = 0; r < kWarpRows; ++r) {
    const uint32_t bits = __reduce_max_sync(0xffffffffu, most[r]) << 16;
    int e = 8 - ((int)(bits >> 23) - 127) - ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    e = e > 108 ? 108 : e < -119 ? -119 : e;  // (queries below 2^-100 are zero to any score)
    const float scale = __uint_as_float((uint32_t)(e + 127) << 23), back = __uint_as_float((uint32_t)(127 - e) << 23);
    if (lane == r) {
      mine = scale;
      // a row with an infinity or NaN has scores of NaN
      sm.back[first + r] = bits >= 0x7F800000u ? __uint_as_float(0x7FFFFFFFu) : a.sm_scale * 1.4426950408889634f * back;
    }
  }
  constexpr int kSide = 3;  // granules worked on side by side
  static_assert(kEach % kSide == 0, "granules per thread");
#pragma unroll 1
  for (int k = 0; k < kEach; k += kSide) {
#pragma unroll
    for (int side = 0; side < kSide; ++side) {
      const int i = lane + (k + side) * 32, at = i / kGranules, row = first + at, col = (i - at * kGranules) * 8;
      const float scale = __shfl_sync(0xffffffffu, mine, at);
      const uint32_t w[4] = {v[side].x, v[side].y, v[side].z, v[side].w};
      uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // (as fp16 exact wherever a part shows it: a bf16 number from 2^-14 to 448)
        const float x0 = bf16_lo(w[j]) * scale, x1 = bf16_hi(w[j]) * scale;
        uint16_t h, l;
        uint32_t x, y;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(x) : "f"(x1), "f"(x0));
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h) : "r"(x));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"(h));
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(x) : "r"(y));
        asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(x) : "r"(0x4C004C00u));  // 16
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(l) : "r"(x));
        hi[j >> 1] |= (uint32_t)h << (16 * (j & 1));
        lo[j >> 1] |= (uint32_t)l << (16 * (j & 1));
      }
      // (rows r and kRows + r have the same swizzle)
      uint8_t* dst = col < kDv ? sm.q_latent[col >> 7] + row * 128 + ((((col & 127) >> 4) ^ (row & 7)) << 4)
                               : sm.q_rope + row * 64 + ((((col - kDv) >> 4) ^ ((row >> 1) & 3)) << 4);
      dst += col & 8;
      *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(dst + kRows * (col < kDv ? 128 : 64)) = make_uint2(lo[0], lo[1]);
    }
#pragma unroll
    for (int j = 0; j + kSide < kEach; ++j) v[j] = v[j + kSide];
  }
  named_bar_sync(1, kSoftThreads);  // (the parents)
  if (tid < kRows) {
    uint64_t word = 0;
    if (tid < u.rows) {
      const int i = (u.row_block * kRows + tid) / a.num_heads;
      if (a.masks) {
        word = a.masks[u.q0 + i];
      } else if (a.parent) {
        int k = i;
        while (k >= 0) {
          word |= 1ull << k;
          const int p = sm.parent[k];
          if (p >= k || p < -1) {
            fault(sm, VMLA_ERR_PARENT, (uint32_t)(u.q0 + i));
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
    sm.minus[tid] = -kNone;
  }
  fence_proxy_async_smem();
  named_bar_sync(1, kSoftThreads);
  if (lane == 0 && a.test_fault != kFaultNoQReady) mbar_arrive(&sm.bars.qfull);
}

// ------------------------------------------------------------------ softmax
// 16 values per lane, each reduced over the warp: lane l ends up with value l >> 1.
template <typename Op>
__device__ __forceinline__ float reduce16(const float (&v)[16], int lane, Op op) {
  float a[8], b[4], c[2];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float keep = lane & 16 ? v[i + 8] : v[i], send = lane & 16 ? v[i] : v[i + 8];
    a[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, 16));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float keep = lane & 8 ? a[i + 4] : a[i], send = lane & 8 ? a[i] : a[i + 4];
    b[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, 8));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float keep = lane & 4 ? b[i + 2] : b[i], send = lane & 4 ? b[i] : b[i + 2];
    c[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, 4));
  }
  const float keep = lane & 2 ? c[1] : c[0], send = lane & 2 ? c[0] : c[1];
  const float d = op(keep, __shfl_xor_sync(0xffffffffu, send, 2));
  return op(d, __shfl_xor_sync(0xffffffffu, d, 1));
}

// Puts zeros in place of a key's NaN codes, once its scores are there (rows that see it have sums of NaN, so their
// results are NaN all the same; the others' weights of zero would make NaN of them).
__device__ __noinline__ void clear_nan(Shared& sm, const ScaledArgs& a, uint32_t tile, int key, bool mine) {
  for (uint32_t c = 0; c < kChunks; ++c) {
    const uint32_t at = (tile * kChunks + c) % kSlots;
    wait(sm, &sm.bars.full[at], ((tile * kChunks + c) / kSlots) & 1, a, 304);  // (long ago: the scores came of it)
    if (!mine) continue;
    uint4* row = reinterpret_cast<uint4*>(sm.latent[at] + key * 128);
    for (int g = 0; g < 8; ++g) {
      uint32_t w[4] = {row[g].x, row[g].y, row[g].z, row[g].w};
      for (int j = 0; j < 4; ++j)
        for (int k = 0; k < 4; ++k)
          if ((w[j] >> (8 * k) & 0x7F) == 0x7F) w[j] &= ~(0xFFu << (8 * k));
      row[g] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

__device__ void softmax_role(Shared& sm, const ScaledArgs& a, const Plan& plan, uint32_t tmem, const Partials& part,
                             Units& units, Unit& u, bool more) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int quarter = warp & 3, row0 = (warp >> 2) * kPerThread;  // its 32 keys of a tile; its first of 16 rows
  const int my_key = quarter * 32 + lane;
  const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
  auto sync = [] { named_bar_sync(1, kSoftThreads); };
  int it = 0;
  if (more) load_queries(sm, a, u);
  while (more) {
    float l[kPerThread];
#pragma unroll
    for (int r = 0; r < kPerThread; ++r) l[r] = 0.f;
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
      const int sb = it & 1, key = (u.tile0 + t) * kTile + my_key;
      uint32_t seen = key < u.keys ? 0xFFFFu : 0u;  // rows that see the key
      if (key >= u.prefix && key < u.keys) {
        seen = 0;
#pragma unroll 1
        for (int r = 0; r < kPerThread; ++r) seen |= (uint32_t)((sm.mask[row0 + r] >> (key - u.prefix)) & 1) << r;
      }
      const bool all_seen = __all_sync(0xffffffffu, seen == 0xFFFFu);
      const float held = fmaxf(scale, kTiny);
      wait(sm, &sm.bars.sfull[sb], (it >> 1) & 1, a, 300);  // (should it run out, the vote below ends the work)
      __syncwarp();
      const uint32_t col = tmem + lanes + kSCol + (uint32_t)(sb * 2 * kRows + row0);
      float w[kPerThread];
      // (a unit's first tile sets the references before anything else)
      for (bool raised = false, look = t > 0;; raised = look = true) {
        tc_fence_after();
        if (look) {
          float most = 0.f;
          {
            uint32_t hi[kPerThread], lo[kPerThread];
            tmem_ld16(col, hi);
            tmem_ld16(col + kRows, lo);
            tmem_wait_ld();
#pragma unroll
            for (int r = 0; r < kPerThread; r += 2) {
              const float2 c = mul2(*reinterpret_cast<const float2*>(&sm.back[row0 + r]), both(scale));
              const float2 y = fma2(make_float2(__uint_as_float(lo[r]), __uint_as_float(lo[r + 1])), both(0.0625f),
                                    make_float2(__uint_as_float(hi[r]), __uint_as_float(hi[r + 1])));
              const float2 z = fma2(y, c, *reinterpret_cast<const float2*>(&sm.minus[row0 + r]));
              const float2 e = mul2(make_float2(ex2_approx(z.x), ex2_approx(z.y)), both(held));
              w[r] = e.x;
              w[r + 1] = e.y;
            }
          }
          if (!all_seen) {
            bool broken = false;  // NaN in a place that is not seen: the key's codes may be NaN, and must not reach the sums
#pragma unroll
            for (int r = 0; r < kPerThread; ++r) {
              const bool is = (seen >> r) & 1;
              broken |= !is && w[r] != w[r];
              w[r] = is ? w[r] : 0.f;
            }
            if (__any_sync(0xffffffffu, broken)) clear_nan(sm, a, (uint32_t)it, my_key, broken);
          }
#pragma unroll
          for (int r = 0; r < kPerThread; ++r) most = fmaxf(most, w[r]);
          if (raised) {
            // 2^9 at the most now, but for scores so large that a unit in their last place is several powers of two: there the
            // reference is rounded down, so that the largest weight is not lost, and what passes 2^15 is cut
            if (most > kMost) {
#pragma unroll
              for (int r = 0; r < kPerThread; ++r) w[r] = w[r] > kMost ? kMost : w[r];  // (NaN stays)
            }
            break;
          }
          if (!soft_vote(most > kMost || sm.abort_flag != 0)) break;
        }
        // some weight is too large for its row's reference: raise the references to the tile's largest
        if (tid == 0) sm.stop = sm.abort_flag;
        {
          uint32_t hi[kPerThread], lo[kPerThread];
          tmem_ld16(col, hi);
          tmem_ld16(col + kRows, lo);
          tmem_wait_ld();
          const float height = __log2f(fmaxf(scale, kTiny));
          float top[kPerThread];
#pragma unroll
          for (int r = 0; r < kPerThread; ++r) {
            const float y = fmaf(__uint_as_float(lo[r]), 0.0625f, __uint_as_float(hi[r]));
            top[r] = (seen >> r) & 1 ? __fmaf_rd(y, sm.back[row0 + r] * scale, height) : -INFINITY;
          }
          const float v = reduce16(top, lane, [](float x, float y) { return fmaxf(x, y); });
          sm.part[quarter][row0 + (lane >> 1)] = v;
        }
        sync();
        if (sm.stop) return;
        if (tid < kRows) {
          const float old = sm.minus[tid];
          const float top = fmaxf(fmaxf(sm.part[0][tid], sm.part[1][tid]), fmaxf(sm.part[2][tid], sm.part[3][tid]));
          const float now = fminf(__fsub_ru(kUnitBits, top), old);
          sm.f[tid] = ex2_approx(now - old);
          sm.minus[tid] = now;
        }
        sync();
        float f[kPerThread];
#pragma unroll
        for (int r = 0; r < kPerThread; ++r) {
          f[r] = sm.f[row0 + r];
          l[r] *= f[r];
        }
        if (t > 0) {
          // what has been summed so far, once the products before are complete
          wait(sm, &sm.bars.pfree, (it - 1) & 1, a, 301);
          __syncwarp();
          tc_fence_after();
#pragma unroll 1
          for (int k = 0; k < (int)kSCol / kRows; k += 2) {
            const uint32_t at = tmem + lanes + (uint32_t)(k * kRows + row0);
            uint32_t o[kPerThread], o2[kPerThread];
            tmem_ld16(at, o);
            tmem_ld16(at + kRows, o2);
            tmem_wait_ld();
#pragma unroll
            for (int r = 0; r < kPerThread; ++r) {
              o[r] = __float_as_uint(__uint_as_float(o[r]) * f[r]);
              o2[r] = __float_as_uint(__uint_as_float(o2[r]) * f[r]);
            }
            tmem_st16(at, o);
            tmem_st16(at + kRows, o2);
          }
          tmem_wait_st();
        }
        tc_fence_before();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.bars.sfree[sb]);
      const float back = __frcp_rn(held);
#pragma unroll
      for (int r = 0; r < kPerThread; r += 2) {
        const float2 sum = fma2(make_float2(w[r], w[r + 1]), both(back), make_float2(l[r], l[r + 1]));
        l[r] = sum.x;
        l[r + 1] = sum.y;
      }
      // three parts of each weight, four rows to a word
      const uint32_t counts = scale >= kTiny ? 0xFFFCFFFCu : 0u;
      uint32_t parts[kParts][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t h[2][kParts];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t x, r1, r2;
          // (cut to 11 bits, then rounded to 9: one rounding, not two)
          asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(x) : "f"(w[4 * k + 2 * j + 1]), "f"(w[4 * k + 2 * j]));
          x = (x + 0x00020002u) & counts;
          h[j][0] = x & 0xFF00FF00u;
          asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r1) : "r"(x), "r"(h[j][0]));
          h[j][1] = r1 & 0xFF00FF00u;
          asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r2) : "r"(r1), "r"(h[j][1]));
          // (three bits at the most for weights from 2^-10 on, whose rounding changes nothing; up to six below that)
          asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(r2) : "r"(0x54005400u));  // kLow
          h[j][2] = r2 + 0x00800080u;
        }
#pragma unroll
        for (int q = 0; q < kParts; ++q) parts[q][k] = __byte_perm(h[0][q], h[1][q], 0x7531);
      }
      if (wait(sm, &sm.bars.pfree, (it & 1) ^ 1, a, 302)) {
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
          uint8_t* dst = sm.p + my_key * 128 + (((2 * q + (row0 >> 4)) ^ (my_key & 7)) << 4);
          *reinterpret_cast<uint4*>(dst) = make_uint4(parts[q][0], parts[q][1], parts[q][2], parts[q][3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.bars.pfull);
      scale = next_scale;
    }
    // row sums over the keys; what the rows' results are scaled by
    const float sum = reduce16(l, lane, [](float x, float y) { return x + y; });
    sm.part[quarter][row0 + (lane >> 1)] = sum;
    sync();
    const int64_t piece = (int64_t)blockIdx.x * 2 + (u.head ? 1 : 0), first_row = out_row(a, u);
    if (tid < kRows) {
      const float total = (sm.part[0][tid] + sm.part[1][tid]) + (sm.part[2][tid] + sm.part[3][tid]), m = -sm.minus[tid];
      sm.f[tid] = !u.whole ? 1.f : total != 0.f ? 1.f / total : 0.f;
      if (!u.whole) part.ml[piece * kRows + tid] = make_float2(m, total);
      else if (tid < u.rows) a.lse[first_row + tid] = total != 0.f ? (m + log2f(total)) * 0.6931471805599453f : -INFINITY;
    }
    if (tid == 0 && u.head && !u.whole) {
      sm.cut_pieces = (int)((u.stop - 1) / plan.share) - (int)blockIdx.x + 1;
      sm.cut_rows = u.rows;
      sm.cut_row = first_row;
    }
    sync();
    float* po = part.o + piece * kRows * kDv;
    uint16_t* out = u.whole ? a.out + first_row * kDv : nullptr;
    const int rows = u.rows;
    // the next unit's queries while this one's last products run
    more = units.next(sm, a, u);
    if (more) load_queries(sm, a, u);
    wait(sm, &sm.bars.pfree, (it - 1) & 1, a, 303);
    __syncwarp();
    tc_fence_after();
#pragma unroll 1
    for (int k = 0; k < kChunks * kPerThread / 8; ++k) {
      const int chunk = k >> 1, r0 = row0 + 8 * (k & 1);
      const int dim = 128 * chunk + my_key;  // this thread's lane of O^T
      const uint32_t at = tmem + lanes + (uint32_t)(chunk * kOCols + r0);
      float o[8];
      {
        uint32_t x[8];
        tmem_ld8(at, x);
        uint32_t y[8], z[8];
        tmem_ld8(at + kRows, y);
        tmem_ld8(at + 2 * kRows, z);
        tmem_wait_ld();
#pragma unroll
        for (int r = 0; r < 8; ++r) o[r] = fmaf(__uint_as_float(z[r]), 1.f / kLow, __uint_as_float(x[r]) + __uint_as_float(y[r]));
      }
      if (out) {
        // pairs of lanes exchange a value each, so that a lane stores two columns of one row
#pragma unroll
        for (int r = 0; r < 8; r += 2) {
          const float a0 = o[r] * sm.f[r0 + r], a1 = o[r + 1] * sm.f[r0 + r + 1];
          const float other = __shfl_xor_sync(0xffffffffu, lane & 1 ? a0 : a1, 1);
          const uint32_t pair = lane & 1 ? pack_bf16x2(other, a1) : pack_bf16x2(a0, other);
          const int row = r0 + r + (lane & 1);
          if (row < rows) *reinterpret_cast<uint32_t*>(out + row * kDv + (dim & ~1)) = pair;
        }
      } else {
#pragma unroll
        for (int r = 0; r < 8; ++r) po[(r0 + r) * kDv + dim] = o[r];
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.bars.ofree);
  }
}

__global__ void __launch_bounds__(kThreads, 1)
scaled_kernel(const __grid_constant__ Maps maps, const __grid_constant__ ScaledArgs a, CtaInfo* __restrict__ info,
              const Partials part) {
  extern __shared__ uint8_t raw[];
  Shared& sm = *reinterpret_cast<Shared*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5;
  const Ends ends(a);  // (on their way while the barriers are made)
  if (warp == kValueWarp) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  static_assert(sizeof(Bars) == 8 * 30, "every barrier is counted here");
  if (tid < (int)(sizeof(Bars) / 8)) {
    constexpr int first = offsetof(Bars, sfree) / 8;
    const bool soft = tid == first || tid == first + 1 || tid == (int)offsetof(Bars, pfull) / 8 ||
                      tid == (int)offsetof(Bars, qfull) / 8 || tid == (int)offsetof(Bars, ofree) / 8;
    mbar_init(reinterpret_cast<uint64_t*>(&sm.bars) + tid, soft ? kSoftWarps : 1);
    fence_mbar_init();
  } else if (tid == 32) {
    sm.abort_flag = 0;
    sm.fault[0] = sm.fault[1] = 0;
    sm.cut_pieces = 0;
  } else if (tid == kLoadWarp * 32) {
    prefetch_tensormap(&maps.latent);
    prefetch_tensormap(&maps.rope);
    prefetch_tensormap(&maps.latent_run);
    prefetch_tensormap(&maps.rope_run);
  }
  __syncwarp();
  Plan plan;
  const bool ok = make_plan(sm, a, ends, plan);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  if (ok) {
    // the CTA's first unit, which every role begins with
    Units units(sm, a, plan);
    Unit u;
    const bool more = units.first(sm, a, u);
    if (warp < kSoftWarps) {
      softmax_role(sm, a, plan, tmem, part, units, u, more);
    } else if (warp == kScoreWarp) {
      score_role(sm, a, tmem, units, u, more);
    } else if (warp == kValueWarp) {
      value_role(sm, a, tmem, units, u, more);
    } else {
      load_role(sm, maps, a, units, u, more);
    }
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
  if (warp == kValueWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (tid == 0) {
    CtaInfo mine = {};
    mine.fault = ok ? sm.fault[0] : (uint32_t)VMLA_ERR_SHAPE;
    mine.fault_info = ok ? sm.fault[1] : 0;
    if (ok && !sm.abort_flag && sm.cut_pieces > 0) {
      mine.pieces = sm.cut_pieces;
      mine.rows = sm.cut_rows;
      mine.row = sm.cut_row;
    }
    info[blockIdx.x] = mine;
  }
}

// Joins the partials of a cut stream: a warp per 128 columns of a row, in CTAs of kJoinRows rows of the stream that begins
// in a CTA's share.  (A CTA per row: 4864 of them, most with nothing to do, cost 1 us more; a warp for a whole row has too
// few loads on their way: 185 000 keys in 19 pieces 5 us more.)
constexpr int kJoinRows = 2, kJoinWarps = 4 * kJoinRows;
constexpr int kMaxCtas = 512;
__global__ void __launch_bounds__(kJoinWarps * 32)
scaled_join_kernel(const CtaInfo* __restrict__ info, int ctas, const Partials part, uint16_t* __restrict__ out,
                   float* __restrict__ lse, uint32_t* __restrict__ status) {
  __shared__ float weight[kJoinWarps][kMaxCtas + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cta = blockIdx.x, row = blockIdx.y * kJoinRows + (warp >> 2), at = (warp & 3) * 32 + lane;
  grid_dependency_wait();
  const CtaInfo i = info[cta];
  if (cta == 0 && blockIdx.y == 0 && warp == 0) {
    // the call's status: the first CTA's fault
    uint32_t first = 0xffffffffu;
    for (int k = lane; k < ctas; k += 32)
      if (info[k].fault != 0) first = min(first, (uint32_t)k);
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) {
      status[0] = first == 0xffffffffu ? 0u : info[first].fault;
      status[1] = first == 0xffffffffu ? 0u : info[first].fault_info;
    }
  }
  if (row >= i.rows || i.pieces == 0) return;
  // piece 0 lies in this CTA's second slot, piece k in the first slot of the k-th CTA after it
  auto slot = [&](int k) { return k == 0 ? (int64_t)cta * 2 + 1 : ((int64_t)cta + k) * 2; };
  float top = kNone;
  for (int k = lane; k < i.pieces; k += 32) {
    const float m = part.ml[slot(k) * kRows + row].x;
    weight[warp][k] = m;
    top = fmaxf(top, m);
  }
  top = warp_max(top);
  float sum = 0.f;
  for (int k = lane; k < i.pieces; k += 32) {
    const float w = ex2_approx(weight[warp][k] - top);
    weight[warp][k] = w;
    sum = fmaf(part.ml[slot(k) * kRows + row].y, w, sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  __syncwarp();
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int k = 0; k < i.pieces; ++k) {
    const float w = weight[warp][k];
    const float4 x = reinterpret_cast<const float4*>(part.o + (slot(k) * kRows + row) * kDv)[at];
    o.x = fmaf(x.x, w, o.x);
    o.y = fmaf(x.y, w, o.y);
    o.z = fmaf(x.z, w, o.z);
    o.w = fmaf(x.w, w, o.w);
  }
  const float f = sum != 0.f ? 1.f / sum : 0.f;
  reinterpret_cast<uint2*>(out + (i.row + row) * kDv)[at] = make_uint2(pack_bf16x2(o.x * f, o.y * f), pack_bf16x2(o.z * f, o.w * f));
  if (at == 0) lse[i.row + row] = sum != 0.f ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}
static_assert(kRows % kJoinRows == 0 && kDv == 4 * 32 * 4, "four warps per row, four columns a lane");

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

// The pool as rows of bytes: boxes `width` bytes wide, one row high for gathers of four rows, or kRun.
bool encode_pool(EncodeTiledFn enc, CUtensorMap* map, const uint8_t* pool, int64_t slots, uint32_t width, uint32_t rows,
                 CUtensorMapSwizzle swizzle) {
  cuuint64_t gdim[2] = {(cuuint64_t)kDqk, (cuuint64_t)(slots > 0 ? slots : 1)};
  cuuint64_t gstride[1] = {(cuuint64_t)kDqk};
  cuuint32_t box[2] = {width, rows};
  cuuint32_t estride[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(pool), gdim, gstride, box, estride,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int launch(const ScaledArgs& a, int sms, const Maps& maps, cudaStream_t stream) {
  static std::mutex mu;
  static bool ready[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return VMLA_ERR_CUDA;
  {
    std::lock_guard<std::mutex> g(mu);
    if (dev >= 64 || !ready[dev]) {
      if (cudaFuncSetAttribute(scaled_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSharedBytes) != cudaSuccess)
        return VMLA_ERR_CUDA;
      if (dev < 64) ready[dev] = true;
    }
  }
  CtaInfo* info = reinterpret_cast<CtaInfo*>(a.workspace + kInfoOff);
  Partials part;
  part.ml = reinterpret_cast<float2*>(a.workspace + ml_off(sms));
  part.o = reinterpret_cast<float*>(a.workspace + o_off(sms));
  scaled_kernel<<<sms, kThreads, kSharedBytes, stream>>>(maps, a, info, part);
  if (cudaGetLastError() != cudaSuccess) return VMLA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1] = {early_start_attribute()};
  cfg.gridDim = dim3((unsigned)sms, kRows / kJoinRows, 1);
  cfg.blockDim = dim3(kJoinWarps * 32, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, scaled_join_kernel, (const CtaInfo*)info, sms, part, a.out, a.lse, a.status) ==
                 cudaSuccess
             ? VMLA_OK
             : VMLA_ERR_CUDA;
}

}  // namespace

size_t scaled_workspace(int sms) { return o_off(sms) + (size_t)sms * 2 * kRows * kDv * sizeof(float); }

int launch_scaled(const ScaledArgs& a, int sms, void* stream) {
  if (sms > kMaxCtas) return VMLA_ERR_DEVICE;
  EncodeTiledFn enc = encode_fn();
  if (!enc) return VMLA_ERR_DEVICE;
  Maps maps;
  // (without keys nothing is fetched: any address does)
  const uint8_t* pool = a.pool ? a.pool : reinterpret_cast<const uint8_t*>(a.workspace);
  if (!encode_pool(enc, &maps.latent, pool, a.pool_slots, 128, 1, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_pool(enc, &maps.rope, pool, a.pool_slots, 64, 1, CU_TENSOR_MAP_SWIZZLE_64B) ||
      !encode_pool(enc, &maps.latent_run, pool, a.pool_slots, 128, kRun, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_pool(enc, &maps.rope_run, pool, a.pool_slots, 64, kRun, CU_TENSOR_MAP_SWIZZLE_64B))
    return VMLA_ERR_CUDA;
  return launch(a, sms, maps, (cudaStream_t)stream);
}

}  // namespace vmla
