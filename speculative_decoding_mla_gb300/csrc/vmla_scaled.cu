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
constexpr int kPieces = kChunks + 1;
constexpr int kRopePiece = 3;       // place of the rotated columns among a tile's pieces
constexpr int kParts = 3;           // of a weight
constexpr int kPerThread = 16;      // rows of a softmax thread
constexpr int kSoftWarps = 4 * kRows / kPerThread;  // per quarter of the tile's keys, 16 rows each
constexpr int kSoftThreads = kSoftWarps * 32;
constexpr int kLoadWarps = 7;
constexpr int kMmaWarp = kSoftWarps, kLoadWarp = kMmaWarp + 1;
constexpr int kThreads = 32 * (kLoadWarp + kLoadWarps);
constexpr int kRun = 16;            // consecutive slots that one box fetches
constexpr uint32_t kOCols = kParts * kRows;       // 96 columns of tensor memory per 128 value columns
constexpr uint32_t kSCol = kChunks * kOCols;      // 384
constexpr int kLatentSlots = 8, kRopeSlots = 2, kPSlots = 2;
constexpr int kFixed = 2;           // what a unit costs beside its tiles, in tiles
constexpr float kNone = -3e38f;     // reference of a row that has seen no key
constexpr float kUnit = 2048.f;     // weights are held times 2^11
constexpr float kMost = 32768.f;    // largest weight held
constexpr float kTiny = 0x1p-100f;  // smaller scales count as zero
static_assert(kSCol + 2 * 2 * kRows == 512, "tensor memory");
static_assert(kThreads % 128 == 0, "whole register banks");
static_assert(kLoadWarps <= kLatentSlots && kLatentSlots <= 2 * kLoadWarps && kLatentSlots % 4 == 0 && kRopeSlots == 2,
              "see load_role");

struct Shared {
  uint8_t latent[kLatentSlots][kTile * 128];  // a tile's chunk: [key][128 bytes], 128-byte swizzle
  uint8_t q_latent[kChunks][2 * kRows * 128]; // [hi rows, lo rows][128 bytes], 128-byte swizzle
  uint8_t p[kPSlots][kTile * 128];            // [key][hi 32 | mid 32 | lo 32 | -], 128-byte swizzle
  uint8_t rope[kRopeSlots][kTile * 64];       // [key][64 bytes], 64-byte swizzle
  uint8_t q_rope[2 * kRows * 64];             // 64-byte swizzle
  float m[kRows], f[kRows];                   // reference of each row (log2), factor of its last change
  float part[4][kRows];                       // per quarter of the keys: row maxima, or row sums
  uint64_t mask[kRows];                       // the unit's rows: visible drafts
  uint32_t cost[VMLA_MAX_BATCH + 1];          // cost position of each sequence's first stream
  int32_t parent[VMLA_MAX_DRAFT];
  float q_max[kSoftWarps];
  uint32_t sums[2][kThreads / 32];
  uint64_t lfull[kLatentSlots], lfree[kLatentSlots], rfull[kRopeSlots], rfree[kRopeSlots];
  uint64_t sfull[2], sfree[2], pfull[kPSlots], pfree[kPSlots], qfull, ofree, done;
  uint32_t tmem;
  volatile int32_t abort_flag;
  int32_t stop;
  uint32_t fault[2];                          // first fault of this CTA: code, info
  int32_t cut_pieces, cut_rows;               // the stream that starts in this CTA's lane and goes on in the next
  int64_t cut_row;
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

struct Maps {
  CUtensorMap latent, rope;          // gathers of four rows
  CUtensorMap latent_run, rope_run;  // boxes of kRun rows
};

// Ends the work of every CTA of the lane: their waits give up.
template <int C>
__device__ __noinline__ void give_up(Shared& sm) {
  sm.abort_flag = 1;
  if (C > 1) {
    const uint32_t flag = smem_u32(const_cast<const int32_t*>(&sm.abort_flag));
    for (uint32_t r = 0; r < C; ++r) st_cluster_u32(mapa(flag, r), 1u);
  }
}

// One arrival at the barrier, in every CTA of the lane, once this thread's products so far are complete.
template <int C>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if (C == 1) mma_commit(bar);
  else mma_commit_multicast(bar, (uint16_t)((1 << C) - 1));
}

// Copies into the same place of every CTA of the lane.
template <int C>
__device__ __forceinline__ void load_gather(uint32_t dst, const CUtensorMap* map, int x, int y0, int y1, int y2, int y3,
                                            uint32_t bar) {
  if (C == 1) tma_gather4(dst, map, x, y0, y1, y2, y3, bar);
  else tma_gather4_multicast(dst, map, x, y0, y1, y2, y3, bar, (uint16_t)((1 << C) - 1));
}
template <int C>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if (C == 1) tma_load_2d(dst, map, x, y, bar);
  else tma_load_2d_multicast(dst, map, x, y, bar, (uint16_t)((1 << C) - 1));
}

// ------------------------------------------------------------------ plan
// Costs are counted in tiles of whole lanes: at most 2^24 tiles (2^31 keys) x 256 row blocks / C, and kFixed a stream,
// which fit 32 bits but for C = 1, where a sequence has few row blocks on the average of the call's bounds; a plan whose
// cost does not fit is refused.
struct Plan {
  uint32_t length;  // of all streams
  uint32_t share;   // of a lane
  int32_t lanes;
};

// A sequence's lengths.
struct Seq {
  int32_t q0, nq, kv0, nk;
};
__device__ __forceinline__ Seq seq_of(const ScaledArgs& a, int b) {
  Seq s;
  s.q0 = __ldg(a.qo_indptr + b);
  s.nq = __ldg(a.qo_indptr + b + 1) - s.q0;
  s.kv0 = __ldg(a.kv_indptr + b);
  s.nk = __ldg(a.kv_indptr + b + 1) - s.kv0;
  return s;
}
// Streams of C row blocks.
template <int C>
__device__ __forceinline__ int streams_of(const ScaledArgs& a, int nq) {
  return (nq * a.num_heads + C * kRows - 1) / (C * kRows);
}
__device__ __forceinline__ int tiles_of(int nk) { return nk / kTile + (nk % kTile != 0); }

// Reads the lengths and shares the work out (whole CTA); false where the lengths are out of order or past a bound.
template <int C>
__device__ bool make_plan(Shared& sm, const ScaledArgs& a, Plan& plan) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  static_assert(kThreads >= VMLA_MAX_BATCH, "a thread per sequence");
  bool ok = true;
  uint64_t cost = 0;
  if (tid < a.batch) {
    const int64_t k0 = __ldg(a.kv_indptr + tid), k1 = __ldg(a.kv_indptr + tid + 1), q0 = __ldg(a.qo_indptr + tid),
                  q1 = __ldg(a.qo_indptr + tid + 1);
    ok = q1 >= q0 && q1 - q0 <= VMLA_MAX_DRAFT && k1 - k0 >= q1 - q0;
    if (tid == 0) ok = ok && k0 == 0 && q0 == 0;
    if (tid == a.batch - 1) ok = ok && k1 <= a.max_kv && q1 <= a.max_q;
    if (ok) cost = (uint64_t)streams_of<C>(a, (int)(q1 - q0)) * (uint64_t)(tiles_of((int)(k1 - k0)) + kFixed);
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
  plan.lanes = (int)gridDim.x / C;
  plan.share = (plan.length + plan.lanes - 1) / plan.lanes;
  if (plan.share == 0) plan.share = 1;
  __syncthreads();
  return true;
}

// One row block of a sequence over some of its tiles.
struct Unit {
  int row_block, rows;      // rows of the block that are the sequence's (0: none; the CTA goes along for its lane's loads)
  int tile0, tiles;         // its tiles
  int q0, nq;               // the sequence's drafts
  int kv0, keys, prefix;    // first entry of kv_indices; keys and prefix of the sequence
  bool whole, head;         // every tile of the stream; its first tile is among these
  uint32_t stop;            // cost position behind the stream's tiles
};

// The units of a CTA in its lane, in order; the CTAs of a lane have the same tiles.
template <int C>
struct Units {
  uint32_t at, end, from;  // cost position of the current stream; of the lane's end and start
  int b, g, n;
  Seq s;
  __device__ __forceinline__ void enter(const Shared& sm, const ScaledArgs& a, int sequence) {
    for (b = sequence; b < a.batch; ++b) {
      s = seq_of(a, b);
      n = streams_of<C>(a, s.nq);
      if (n > 0) break;
    }
    g = 0;
    at = b < a.batch ? sm.cost[b] : 0xFFFFFFFFu;
  }
  __device__ __forceinline__ Units(const Shared& sm, const ScaledArgs& a, const Plan& p) {
    const uint32_t lane = blockIdx.x / C;
    from = lane * p.share;  // (below the length plus one share: fits)
    end = from + p.share < p.length ? from + p.share : p.length;
    at = 0xFFFFFFFFu;
    if ((int)lane >= p.lanes || from >= end) {
      end = 0;
      return;
    }
    int lo = 0, hi = a.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sm.cost[mid] <= from) lo = mid; else hi = mid;
    }
    enter(sm, a, lo);
    if (at <= from) {
      const uint32_t span = tiles_of(s.nk) + kFixed;
      g = (int)((from - at) / span);
      at += (uint32_t)g * span;
    }
  }
  __device__ __noinline__ bool next(const Shared& sm, const ScaledArgs& a, Unit& u) {
    while (at < end) {
      const int tiles = tiles_of(s.nk);
      const uint32_t lo = at > from ? at : from, stop = at + tiles, hi = stop < end ? stop : end;
      const bool use = lo < hi;
      if (use) {
        u.row_block = g * C + (int)(blockIdx.x % C);
        u.rows = max(0, min(kRows, s.nq * a.num_heads - u.row_block * kRows));
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
      }
      if (++g < n) at += tiles + kFixed;
      else enter(sm, a, b + 1);
      if (use) return true;
    }
    return false;
  }
};
__device__ __forceinline__ int64_t out_row(const ScaledArgs& a, const Unit& u) {
  return (int64_t)u.q0 * a.num_heads + (int64_t)u.row_block * kRows;
}

// ------------------------------------------------------------------ waits
template <int C>
__device__ __noinline__ bool wait_slow(Shared& sm, uint64_t* bar, uint32_t parity, long long budget, uint32_t where) {
  const long long t0 = clock64();
  for (;;) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if (sm.abort_flag) return false;
    if (clock64() - t0 > budget) {
      fault(sm, VMLA_ERR_TIMEOUT, where);
      give_up<C>(sm);
      return false;
    }
  }
}
// Bounded wait; false once it ran out, here or in another warp.
template <int C>
__device__ __forceinline__ bool wait(Shared& sm, uint64_t* bar, uint32_t parity, const ScaledArgs& a, uint32_t where) {
  return mbar_try_wait_cluster(bar, parity) || wait_slow<C>(sm, bar, parity, a.wait_cycles, where);
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

// A position in a ring of slots, and the parity of its round.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void step() {
    if (++slot == N) {
      slot = 0;
      parity ^= 1;
    }
  }
};

// ------------------------------------------------------------------ loads (every lane of seven warps)
// A tile's pieces in the order of their use by the score product: chunks 0, 1, 2, the rotated columns, chunk 3.  The CTAs
// of a lane fetch them in turn, each for all; in a CTA its warps, a lane the four keys 4 lane .. 4 lane + 3.  (An
// instruction that starts a copy takes its thread some 50 clocks, and the lanes' go one by one: seven warps keep the copy
// engine busy, three do not.)  Where all of a tile's slots are consecutive in groups of kRun, a box fetches each group.
template <int C>
__device__ void load_role(Shared& sm, const Maps& maps, const ScaledArgs& a, Units<C>& units, Unit& u, bool more) {
  const int warp = (threadIdx.x >> 5) - kLoadWarp, lane = threadIdx.x & 31;
  const uint32_t me = C > 1 ? cluster_ctarank() : 0;
  const int none = (int)a.pool_slots;  // outside the tensor: zeros
  Ring<kLatentSlots> lr;
  Ring<kRopeSlots> rr;
  // the warp that sees to the next chunk, in every CTA.  A barrier's parity tells apart two rounds of its slot, no more, so
  // a warp's chunks lie no further apart than there are slots (when it comes to one, the slot's round before the last is
  // over, since that of its own chunk before was), and nothing waits for a slot but who fills it next (the round that it
  // waits for cannot pass unseen); the rotated columns' slots have a warp each for the same reason
  int turn = 0;
  for (; more; more = units.next(sm, a, u)) {
    const int32_t* index = a.kv_indices + u.kv0;
    const int last = min(u.keys, (u.tile0 + u.tiles) * kTile);  // behind this unit's keys
    int32_t ahead[4];
    auto fetch = [&](int t) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int key = (u.tile0 + t) * kTile + 4 * lane + k;
        ahead[k] = key < last ? __ldg(index + key) : -1;
      }
    };
    fetch(0);
    for (int t = 0; t < u.tiles; ++t) {
      int32_t y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        y[k] = ahead[k];
        if (y[k] < 0 || y[k] >= none) {
          const int key = (u.tile0 + t) * kTile + 4 * lane + k;
          if (warp == 0 && key < last) fault(sm, VMLA_ERR_INDEX, (uint32_t)(u.kv0 + key));
          y[k] = none;
        }
      }
      fetch(t + 1);
      const int first = __shfl_sync(0xffffffffu, y[0], lane & ~3);
      const bool runs = __all_sync(0xffffffffu, y[0] == first + 4 * (lane & 3) && y[1] == y[0] + 1 && y[2] == y[0] + 2 &&
                                                    y[3] == y[0] + 3 && y[3] < none);
#pragma unroll 1
      for (int piece = 0; piece < kPieces; ++piece) {
        const bool is_rope = piece == kRopePiece;
        const bool mine = is_rope ? warp == kLoadWarps - 1 - rr.slot : turn == warp;
        // (pieces by turns, also where a tile has fewer of a kind than there are CTAs)
        const bool here = C == 1 || (is_rope ? (uint32_t)rr.slot + 2 * rr.parity : (uint32_t)lr.slot) % C == me;
        if (mine) {
          uint64_t* full = is_rope ? &sm.rfull[rr.slot] : &sm.lfull[lr.slot];
          uint64_t* free = is_rope ? &sm.rfree[rr.slot] : &sm.lfree[lr.slot];
          if (!__all_sync(0xffffffffu, wait<C>(sm, free, (is_rope ? rr.parity : lr.parity) ^ 1, a, 100))) return;
          if (lane == 0) mbar_arrive_expect_tx(full, is_rope ? kTile * 64 : kTile * 128);
          __syncwarp();
          if (here) {
            const uint32_t bar = smem_u32(full), dst = is_rope ? smem_u32(sm.rope[rr.slot]) : smem_u32(sm.latent[lr.slot]);
            const int x = is_rope ? kDv : (piece < kRopePiece ? piece : piece - 1) * 128, row = is_rope ? 64 : 128;
            if (runs) {
              if ((lane & 3) == 0)
                load_box<C>(dst + lane * 4 * row, is_rope ? &maps.rope_run : &maps.latent_run, x, y[0], bar);
            } else {
              load_gather<C>(dst + lane * 4 * row, is_rope ? &maps.rope : &maps.latent, x, y[0], y[1], y[2], y[3], bar);
            }
          }
        }
        if (is_rope) {
          rr.step();
        } else {
          lr.step();
          turn = turn == kLoadWarps - 1 ? 0 : turn + 1;
        }
      }
    }
  }
  // the slots' last releases, which come from every CTA of the lane, have arrived before this CTA may leave: each is
  // waited for by who filled the slot last
  for (int k = 0; k < kLatentSlots; ++k) {
    if ((turn + k + kLoadWarps * 2 - kLatentSlots) % kLoadWarps == warp) wait<C>(sm, &sm.lfree[lr.slot], lr.parity ^ 1, a, 101);
    lr.step();
  }
  for (int k = 0; k < kRopeSlots; ++k) {
    if (warp == kLoadWarps - 1 - rr.slot) wait<C>(sm, &sm.rfree[rr.slot], rr.parity ^ 1, a, 102);
    rr.step();
  }
  __syncwarp();
}

// ------------------------------------------------------------------ matrix products (one warp)
// Two sequences of products: scores, piece by piece as a tile's columns arrive, and values, a tile at a time.  Whatever
// is ready goes next, scores first: they keep the softmax busy, and only values make room for further loads.  What lies
// between two products is short: a look at a barrier and the bookkeeping take as long as ten of them.
template <int C>
__device__ void mma_role(Shared& sm, const ScaledArgs& a, uint32_t tmem, const Units<C>& units, const Unit& first,
                         bool more) {
  constexpr uint32_t kScores = idesc_f8_f32(kTile, 2 * kRows, 0, 0, 0, 0);
  constexpr uint32_t kValues = idesc_f8_f32(128, kOCols, 0, 1, 1, 1);
  Units<C> q_units = units, v_units = units;
  Unit u = first;
  bool q_more = more, v_more = more;
  int q_tiles = u.tiles, v_tiles = u.tiles;  // left of the unit
  bool q_first = true, v_first = true;       // no tile of the unit yet
  Ring<kLatentSlots> ql, vl;
  Ring<kRopeSlots> qr;
  // lower words of the descriptors at the first slot, and the upper words, which depend on the layout alone
  constexpr uint32_t kHi128 = (uint32_t)(smem_desc_fixed(16, 1024, 2) >> 32), kHi64 = (uint32_t)(smem_desc_fixed(16, 512, 4) >> 32);
  constexpr uint32_t kLo = (uint32_t)smem_desc_fixed(16, 0, 0);
  auto low = [&](const void* at) { return smem_u32(at) >> 4 | kLo; };
  const uint32_t latent_lo = low(sm.latent[0]), rope_lo = low(sm.rope[0]), q_latent_lo = low(sm.q_latent[0]),
                 q_rope_lo = low(sm.q_rope), p_lo = low(sm.p[0]);
  uint32_t q_it = 0, v_it = 0, q_unit = 0, v_unit = 0;
  int piece = 0;
  auto ready = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_test_wait_cluster(bar, parity)) != 0; };
  auto scores = [&]() -> bool {
    const uint32_t sb = q_it & 1;
    if (piece == 0 && ((q_first && !ready(&sm.qfull, q_unit & 1)) || !ready(&sm.sfree[sb], ((q_it >> 1) & 1) ^ 1)))
      return false;
    const uint32_t d = tmem + kSCol + sb * 2 * kRows;
    const int begun = piece;
#pragma unroll
    for (int k = 0; k <= kChunks; ++k) {
      if (k != piece) continue;
      if (k == kRopePiece) {
        if (!ready(&sm.rfull[qr.slot], qr.parity)) break;
        tc_fence_after();
        const uint32_t key = rope_lo + qr.slot * (kTile * 64 / 16);
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < 2; ++i) mma_ss_f8(d, key + 2 * i, kHi64, q_rope_lo + 2 * i, kHi64, kScores, 1u);
          commit<C>(&sm.rfree[qr.slot]);
        }
        qr.step();
      } else {
        if (!ready(&sm.lfull[ql.slot], ql.parity)) break;
        tc_fence_after();
        const uint32_t key = latent_lo + ql.slot * (kTile * 128 / 16),
                       q = q_latent_lo + (k < kRopePiece ? k : k - 1) * (2 * kRows * 128 / 16);
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma_ss_f8(d, key + 2 * i, kHi128, q + 2 * i, kHi128, kScores, k > 0 || i > 0);
          if (k == kChunks) mma_commit(&sm.sfull[sb]);
        }
        ql.step();
      }
      __syncwarp();
      piece = k + 1;
    }
    if (piece == begun) return false;
    if (piece > kChunks) {
      piece = 0;
      ++q_it;
      q_first = false;
      if (--q_tiles == 0) {
        ++q_unit;
        q_first = true;
        q_more = q_units.next(sm, a, u);
        q_tiles = u.tiles;
      }
    }
    return true;
  };
  auto values = [&]() -> bool {
    // (the first product into O: the unit before has been read out)
    const uint32_t pb = v_it % kPSlots;
    if (!ready(&sm.pfull[pb], (v_it / kPSlots) & 1) || (v_first && !ready(&sm.ofree, (v_unit & 1) ^ 1))) return false;
    tc_fence_after();
    const uint32_t go_on = v_first ? 0u : 1u, p = p_lo + pb * (kTile * 128 / 16);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const uint32_t v = latent_lo + vl.slot * (kTile * 128 / 16), d = tmem + c * kOCols;
      if (elect_one()) {
#pragma unroll
        for (int i = 0; i < kTile / 32; ++i)
          mma_ss_f8(d, v + 256 * i, kHi128, p + 256 * i, kHi128, kValues, i > 0 ? 1u : go_on);
        commit<C>(&sm.lfree[vl.slot]);
        if (c == kChunks - 1) mma_commit(&sm.pfree[pb]);
      }
      __syncwarp();
      vl.step();
    }
    ++v_it;
    v_first = false;
    if (--v_tiles == 0) {
      ++v_unit;
      v_first = true;
      v_more = v_units.next(sm, a, u);
      v_tiles = u.tiles;
    }
    return true;
  };
  int idle = 0;
  long long t0 = 0;
  while (q_more || v_more) {
    if (q_more && scores()) idle = 0;
    if (v_more && values()) idle = 0;
    if (++idle < 256) continue;
    if (idle == 256) t0 = clock64();
    if (__any_sync(0xffffffffu, sm.abort_flag != 0)) break;
    if (__any_sync(0xffffffffu, clock64() - t0 > a.wait_cycles)) {
      if (elect_one()) fault(sm, VMLA_ERR_TIMEOUT, 200);
      give_up<C>(sm);
      __syncwarp();
    }
  }
  // everything issued is complete, and its signals have arrived, before the CTA leaves
  if (elect_one()) mma_commit(&sm.done);
  __syncwarp();
  t0 = clock64();
  while (!mbar_try_wait(&sm.done, 0) && clock64() - t0 < a.wait_cycles) {
  }
}

// ------------------------------------------------------------------ queries (softmax warps)
// The unit's rows into shared memory in two e4m3 parts, their masks; the factor that makes a score of a product.
// (What runs once per unit is kept in loops: straight-line code that is run once costs more in fetching it.)
__device__ __noinline__ float load_queries(Shared& sm, const ScaledArgs& a, const Unit& u) {
  constexpr int kGranules = kDqk / 8;                      // of 8 bf16
  constexpr int kEach = kRows * kGranules / kSoftThreads;   // 9 per thread
  static_assert(kRows * kGranules % kSoftThreads == 0, "granules per thread");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint4* src = reinterpret_cast<const uint4*>(a.q + out_row(a, u) * kDqk);
  uint4 v[kEach];
  const int valid = u.rows * kGranules;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int i = tid + k * kSoftThreads;
    v[k] = i < valid ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
  }
  if (a.parent && tid < u.nq) sm.parent[tid] = a.parent[u.q0 + tid];
  uint32_t m = 0;  // largest magnitude of either half, as bits of bf16
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x = w[j] & 0x7FFF7FFFu;
      asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(x));
    }
  }
  m = __reduce_max_sync(0xffffffffu, max(m >> 16, m & 0xFFFFu));
  if (lane == 0) sm.q_max[warp] = __uint_as_float(m << 16);
  named_bar_sync(1, kSoftThreads);
  float top = lane < kSoftWarps ? sm.q_max[lane] : 0.f;
  top = warp_max(top);
  // a: 448 = 1.75 x 2^8; queries below 2^-100 are zero to any score
  const uint32_t bits = __float_as_uint(top);
  int e = 8 - ((int)(bits >> 23) - 127) - ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e > 108 ? 108 : e < -119 ? -119 : e;
  const float scale = __uint_as_float((uint32_t)(e + 127) << 23), back = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll 1
  for (int k = 0; k < kEach; ++k) {
    const int i = tid + k * kSoftThreads, row = i / kGranules, col = (i - row * kGranules) * 8;
    const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
    for (int j = 0; j + 1 < kEach; ++j) v[j] = v[j + 1];
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
    // (rows r and kRows + r have the same swizzle)
    uint8_t* dst = col < kDv ? sm.q_latent[col >> 7] + row * 128 + ((((col & 127) >> 4) ^ (row & 7)) << 4)
                             : sm.q_rope + row * 64 + ((((col - kDv) >> 4) ^ ((row >> 1) & 3)) << 4);
    dst += col & 8;
    *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0], hi[1]);
    *reinterpret_cast<uint2*>(dst + kRows * (col < kDv ? 128 : 64)) = make_uint2(lo[0], lo[1]);
  }
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
    sm.m[tid] = kNone;
  }
  fence_proxy_async_smem();
  named_bar_sync(1, kSoftThreads);
  if (lane == 0 && a.test_fault != kFaultNoQReady) mbar_arrive(&sm.qfull);
  return a.sm_scale * 1.4426950408889634f * back;
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

template <int C>
__device__ void softmax_role(Shared& sm, const ScaledArgs& a, const Plan& plan, uint32_t tmem, const Partials& part,
                             Units<C>& units, Unit& u, bool more) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int quarter = warp & 3, row0 = (warp >> 2) * kPerThread;  // its 32 keys of a tile; its first of 16 rows
  const int my_key = quarter * 32 + lane;
  const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
  auto sync = [] { named_bar_sync(1, kSoftThreads); };
  int it = 0;
  float factor = more ? load_queries(sm, a, u) : 0.f;
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
      const float c = scale * factor, held = fmaxf(scale, kTiny) * kUnit;
      wait<C>(sm, &sm.sfull[sb], (it >> 1) & 1, a, 300);  // (should it run out, the vote below ends the work)
      __syncwarp();
      const uint32_t col = tmem + lanes + kSCol + (uint32_t)(sb * 2 * kRows + row0);
      float w[kPerThread];
      for (;;) {
        tc_fence_after();
        float most = 0.f;
        {
          uint32_t hi[kPerThread], lo[kPerThread];
          tmem_ld16(col, hi);
          tmem_ld16(col + kRows, lo);
          tmem_wait_ld();
#pragma unroll
          for (int r = 0; r < kPerThread; r += 4) {
            const float4 m = *reinterpret_cast<const float4*>(&sm.m[row0 + r]);
            const float mr[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float y = fmaf(__uint_as_float(lo[r + j]), 0.0625f, __uint_as_float(hi[r + j]));
              w[r + j] = ex2_approx(fmaf(y, c, -mr[j])) * held;
            }
          }
        }
        if (!all_seen) {
#pragma unroll
          for (int r = 0; r < kPerThread; ++r) w[r] = (seen >> r) & 1 ? w[r] : 0.f;
        }
#pragma unroll
        for (int r = 0; r < kPerThread; ++r) most = fmaxf(most, w[r]);
        if (!soft_vote(most > kMost || sm.abort_flag != 0)) break;
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
            top[r] = (seen >> r) & 1 ? fmaf(y, c, height) : -INFINITY;
          }
          const float v = reduce16(top, lane, [](float x, float y) { return fmaxf(x, y); });
          sm.part[quarter][row0 + (lane >> 1)] = v;
        }
        sync();
        if (sm.stop) return;
        if (tid < kRows) {
          const float old = sm.m[tid];
          const float top = fmaxf(fmaxf(fmaxf(sm.part[0][tid], sm.part[1][tid]), fmaxf(sm.part[2][tid], sm.part[3][tid])), old);
          sm.f[tid] = ex2_approx(old - top);
          sm.m[tid] = top;
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
          wait<C>(sm, &sm.pfree[(it - 1) % kPSlots], ((it - 1) / kPSlots) & 1, a, 301);
          __syncwarp();
          tc_fence_after();
#pragma unroll 1
          for (int k = 0; k < (int)kSCol / kRows; ++k) {
            const uint32_t at = tmem + lanes + (uint32_t)(k * kRows + row0);
            uint32_t o[kPerThread];
            tmem_ld16(at, o);
            tmem_wait_ld();
#pragma unroll
            for (int r = 0; r < kPerThread; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * f[r]);
            tmem_st16(at, o);
          }
          tmem_wait_st();
        }
        tc_fence_before();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.sfree[sb]);
      const float back = __frcp_rn(held);
#pragma unroll
      for (int r = 0; r < kPerThread; ++r) l[r] = fmaf(w[r], back, l[r]);
      // three parts of each weight, four rows to a word
      const uint32_t counts = scale >= kTiny ? 0xFFFCFFFCu : 0u;
      uint32_t parts[kParts][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t h[2][kParts];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t x, r1, r2;
          asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(x) : "f"(w[4 * k + 2 * j + 1]), "f"(w[4 * k + 2 * j]));
          x = (x + 0x00020002u) & counts;
          h[j][0] = x & 0xFF00FF00u;
          asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r1) : "r"(x), "r"(h[j][0]));
          h[j][1] = r1 & 0xFF00FF00u;
          asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r2) : "r"(r1), "r"(h[j][1]));
          h[j][2] = r2;
        }
#pragma unroll
        for (int q = 0; q < kParts; ++q) parts[q][k] = __byte_perm(h[0][q], h[1][q], 0x7531);
      }
      const int pb = it % kPSlots;
      if (wait<C>(sm, &sm.pfree[pb], ((it / kPSlots) & 1) ^ 1, a, 302)) {
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
          uint8_t* dst = sm.p[pb] + my_key * 128 + (((2 * q + (row0 >> 4)) ^ (my_key & 7)) << 4);
          *reinterpret_cast<uint4*>(dst) = make_uint4(parts[q][0], parts[q][1], parts[q][2], parts[q][3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.pfull[pb]);
      scale = next_scale;
    }
    // row sums over the keys; what the rows' results are scaled by
    const float sum = reduce16(l, lane, [](float x, float y) { return x + y; });
    sm.part[quarter][row0 + (lane >> 1)] = sum;
    sync();
    const int64_t piece = (int64_t)blockIdx.x * 2 + (u.head ? 1 : 0), first_row = out_row(a, u);
    if (tid < kRows) {
      const float total = (sm.part[0][tid] + sm.part[1][tid]) + (sm.part[2][tid] + sm.part[3][tid]), m = sm.m[tid];
      sm.f[tid] = !u.whole ? 1.f : total > 0.f ? 1.f / (total * kUnit) : 0.f;
      if (!u.whole) part.ml[piece * kRows + tid] = make_float2(m, total);
      else if (tid < u.rows) a.lse[first_row + tid] = total > 0.f ? (m + log2f(total)) * 0.6931471805599453f : -INFINITY;
    }
    if (tid == 0 && u.head && !u.whole) {
      sm.cut_pieces = (int)((u.stop - 1) / plan.share) - (int)(blockIdx.x / C) + 1;
      sm.cut_rows = u.rows;
      sm.cut_row = first_row;
    }
    sync();
    float* po = part.o + piece * kRows * kDv;
    uint16_t* out = u.whole ? a.out + first_row * kDv : nullptr;
    const int rows = u.rows;
    // the next unit's queries while this one's last products run
    more = units.next(sm, a, u);
    if (more) factor = load_queries(sm, a, u);
    wait<C>(sm, &sm.pfree[(it - 1) % kPSlots], ((it - 1) / kPSlots) & 1, a, 303);
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
        for (int r = 0; r < 8; ++r) o[r] = (__uint_as_float(x[r]) + __uint_as_float(y[r])) + __uint_as_float(z[r]);
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
    if (lane == 0) mbar_arrive(&sm.ofree);
  }
}

template <int C>
__global__ void __launch_bounds__(kThreads, 1)
scaled_kernel(const __grid_constant__ Maps maps, const __grid_constant__ ScaledArgs a, CtaInfo* __restrict__ info,
              const Partials part) {
  extern __shared__ uint8_t raw[];
  Shared& sm = *reinterpret_cast<Shared*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5;
  if (warp == kMmaWarp) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int s = 0; s < kLatentSlots; ++s) {
      mbar_init(&sm.lfull[s], 1);
      mbar_init(&sm.lfree[s], C);  // every CTA of the lane has used it
    }
    for (int s = 0; s < kRopeSlots; ++s) {
      mbar_init(&sm.rfull[s], 1);
      mbar_init(&sm.rfree[s], C);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.sfull[s], 1);
      mbar_init(&sm.sfree[s], kSoftWarps);
    }
    for (int s = 0; s < kPSlots; ++s) {
      mbar_init(&sm.pfull[s], kSoftWarps);
      mbar_init(&sm.pfree[s], 1);
    }
    mbar_init(&sm.qfull, kSoftWarps);
    mbar_init(&sm.ofree, kSoftWarps);
    mbar_init(&sm.done, 1);
    sm.abort_flag = 0;
    sm.fault[0] = sm.fault[1] = 0;
    sm.cut_pieces = 0;
    fence_mbar_init();
    prefetch_tensormap(&maps.latent);
    prefetch_tensormap(&maps.rope);
    prefetch_tensormap(&maps.latent_run);
    prefetch_tensormap(&maps.rope_run);
  }
  __syncwarp();
  Plan plan;
  const bool ok = make_plan<C>(sm, a, plan);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (C > 1) {  // no copy or signal goes to a CTA whose barriers are not ready
    cluster_arrive();
    cluster_wait();
  }
  const uint32_t tmem = sm.tmem;
  if (ok) {
    // the CTA's first unit, which every role begins with
    Units<C> units(sm, a, plan);
    Unit u;
    const bool more = units.next(sm, a, u);
    if (warp < kSoftWarps) {
      softmax_role<C>(sm, a, plan, tmem, part, units, u, more);
    } else if (warp == kMmaWarp) {
      mma_role<C>(sm, a, tmem, units, u, more);
    } else {
      load_role<C>(sm, maps, a, units, u, more);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  grid_dependents_launch();
  if (C > 1) {  // nor leaves a CTA while another may still signal to it
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }
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
  if (tid == 0) {
    CtaInfo mine = {};
    mine.fault = ok ? sm.fault[0] : (uint32_t)VMLA_ERR_SHAPE;
    mine.fault_info = ok ? sm.fault[1] : 0;
    if (ok && !sm.abort_flag && sm.cut_pieces > 0) {
      mine.pieces = sm.cut_pieces;
      mine.rows = sm.cut_rows;
      mine.row = sm.cut_row;
      mine.group = C;
    }
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

template <int C>
cudaLaunchConfig_t kernel_config(int ctas, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)ctas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSharedBytes;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// Lanes that are resident together on the current device (a GPC's last SMs may not fill one).
template <int C>
int max_lanes(int sms, int* lanes) {
  static std::mutex mu;
  static int known[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return VMLA_ERR_CUDA;
  std::lock_guard<std::mutex> g(mu);
  if (dev >= 64 || known[dev] == 0) {
    if (cudaFuncSetAttribute(scaled_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSharedBytes) !=
        cudaSuccess)
      return VMLA_ERR_CUDA;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = kernel_config<C>(C, attr);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, scaled_kernel<C>, &cfg) != cudaSuccess || n < 1) return VMLA_ERR_CUDA;
    n = n < sms / C ? n : sms / C;
    if (dev >= 64) {
      *lanes = n;
      return VMLA_OK;
    }
    known[dev] = n;
  }
  *lanes = known[dev];
  return VMLA_OK;
}

template <int C>
int launch(const ScaledArgs& a, int sms, const Maps& maps, cudaStream_t stream) {
  int lanes = 0;
  const int rc = max_lanes<C>(sms, &lanes);
  if (rc != VMLA_OK) return rc;
  CtaInfo* info = reinterpret_cast<CtaInfo*>(a.workspace + kInfoOff);
  Partials part;
  part.ml = reinterpret_cast<float2*>(a.workspace + ml_off(sms));
  part.o = reinterpret_cast<float*>(a.workspace + o_off(sms));
  const int ctas = lanes * C;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = kernel_config<C>(ctas, attr);
  cfg.stream = stream;
  if (cudaLaunchKernelEx(&cfg, scaled_kernel<C>, maps, a, info, part) != cudaSuccess) return VMLA_ERR_CUDA;
  attr[0] = early_start_attribute();
  cfg.gridDim = dim3((unsigned)ctas, kRows, 1);
  cfg.blockDim = dim3(kJoinThreads, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, scaled_join_kernel, (const CtaInfo*)info, ctas, part, a.out, a.lse, a.status) ==
                 cudaSuccess
             ? VMLA_OK
             : VMLA_ERR_CUDA;
}

}  // namespace

size_t scaled_workspace(int sms) { return o_off(sms) + (size_t)sms * 2 * kRows * kDv * sizeof(float); }

int launch_scaled(const ScaledArgs& a, int sms, void* stream) {
  if (sms > kMaxCtas || sms < 4) return VMLA_ERR_DEVICE;
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
  // lanes of as many CTAs as a sequence has row blocks on the average of the bounds, up to four
  const int64_t rows = a.max_q * a.num_heads, blocks = (int64_t)a.batch * kRows;
  cudaStream_t st = (cudaStream_t)stream;
  return rows > 2 * blocks ? launch<4>(a, sms, maps, st) : rows > blocks ? launch<2>(a, sms, maps, st) : launch<1>(a, sms, maps, st);
}

}  // namespace vmla
