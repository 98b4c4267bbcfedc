// The tables of a decode step from its requests' lengths.
//
// Request b holds cached[b] tokens and gets new[b] more, so with n_b = cached[b] + new[b] and blocks of bt slots
//   kv_indptr, qo_indptr = running sums of n_b and of new[b]
//   its blocks           = the table's first ceil(cached[b] / bt), then fresh ones from the free list's end,
//                          dealt out in the order of the requests
//   slot(b, p)           = block(b, p / bt) bt + p mod bt
//   kv_indices[kv_indptr[b] + p] = slot(b, p);  slots, positions: the same of the new tokens
//
// A call writes 4 bytes a key and reads 4 a block, so large ones are bound by the writes and small ones by a chain of
// loads.  One launch: every CTA takes the running sums of all requests itself (at most 512, two a thread: one chain
// of loads and three barriers, instead of a second launch behind a first), checks them, and then writes its part of
// each array.  A warp takes 256 keys at a time: one bisection in shared memory, and where they lie in one request's
// old blocks, which is mostly so, eight keys a lane looked up side by side; else key by key.
// Measured: 256 requests of up to 65 536 tokens in blocks of 64 (5.7 M keys, 23 MB) 14.3 us, 1.6 TB/s, of which some 5 us
// are the launch and the sums (a bisection and a block's test per four keys: 22.5 us, bound by instructions); 32
// requests slot by slot (0.3 M keys) 6.6 us.
// Entries that the call adds to the block table are never read back from it (they follow from the free list), so
// CTAs need no order among them; the count of free blocks, which may be updated in place, is written by the CTA that
// finishes last.
#include <cuda_runtime.h>

#include "vmla_device.cuh"

namespace vmla {
namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = VMLA_MAX_BATCH / kThreads;
constexpr int kVec = 4;                    // keys of a lane together, one 16-byte store where the array is aligned
constexpr int kSide = 2;                   // such quads that a lane looks up side by side
constexpr int kRound = 32 * kVec * kSide;  // keys of a warp at a time
static_assert(VMLA_MAX_BATCH % kThreads == 0, "requests per thread");

struct Sums {
  int32_t kv[VMLA_MAX_BATCH + 1], qo[VMLA_MAX_BATCH + 1], grown[VMLA_MAX_BATCH + 1];
  int32_t have[VMLA_MAX_BATCH];  // blocks in the table
  int32_t cached[VMLA_MAX_BATCH];
  int64_t warp[3][kThreads / 32];
  int32_t bad;  // first request whose lengths are out of range, or INT32_MAX
};

// Last b with off[b] <= x among off[0 .. n].
__device__ __forceinline__ int owner(const int32_t* off, int n, int32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads)
tables_kernel(const TablesArgs a) {
  __shared__ Sums s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int count = *a.free_count;
  if (tid == 0) s.bad = INT32_MAX;
  __syncthreads();
  // a thread's requests: n, new tokens, new blocks; then running sums over the block
  int64_t sum[3] = {0, 0, 0}, mine[kPerThread][3];
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const int b = tid * kPerThread + k;
    int64_t n = 0, q = 0, grown = 0;
    if (b < a.batch) {
      const int64_t c = a.cached[b], m = a.added[b];
      n = c + m;
      q = m;
      const int64_t have = (c + a.block - 1) >> a.block_shift, need = (n + a.block - 1) >> a.block_shift;
      grown = need - have;
      if (c < 0 || m < 0 || need > a.table_width) {
        atomicMin(&s.bad, b);
        n = q = grown = 0;
      }
      s.have[b] = (int32_t)have;
      s.cached[b] = (int32_t)c;
    }
    mine[k][0] = n;
    mine[k][1] = q;
    mine[k][2] = grown;
#pragma unroll
    for (int j = 0; j < 3; ++j) sum[j] += mine[k][j];
  }
  int64_t before[3];
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    int64_t v = sum[j];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    before[j] = v - sum[j];
    if (lane == 31) s.warp[j][warp] = v;
  }
  __syncthreads();
  int64_t total[3] = {0, 0, 0};
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w)
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      if (w < warp) before[j] += s.warp[j][w];
      total[j] += s.warp[j][w];
    }
  const bool lengths = s.bad == INT32_MAX;
  const bool fits = lengths && total[0] <= a.max_kv && total[1] <= a.max_q && total[2] <= count && count <= a.free_size;
  if (fits) {
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      const int b = tid * kPerThread + k;
      if (b < a.batch) {
        s.kv[b] = (int32_t)before[0];
        s.qo[b] = (int32_t)before[1];
        s.grown[b] = (int32_t)before[2];
#pragma unroll
        for (int j = 0; j < 3; ++j) before[j] += mine[k][j];
      }
    }
    if (tid == 0) {
      s.kv[a.batch] = (int32_t)total[0];
      s.qo[a.batch] = (int32_t)total[1];
      s.grown[a.batch] = (int32_t)total[2];
    }
  } else if (blockIdx.x == 0 && tid == 0) {
    // lengths out of range, or more keys, tokens or blocks than there is room for: an empty step
    record_status(a.status, lengths ? VMLA_ERR_FULL : VMLA_ERR_SHAPE, lengths ? 0u : (uint32_t)s.bad);
  }
  __syncthreads();
  const int32_t n_kv = fits ? s.kv[a.batch] : 0, n_q = fits ? s.qo[a.batch] : 0, n_new = fits ? s.grown[a.batch] : 0;
  // block k of request b, and the slot of position p in it (-1: no block, or its slots pass 2^31)
  const int32_t mask = a.block - 1;
  const uint32_t last_block = (uint32_t)INT32_MAX >> a.block_shift;
  auto block_of = [&](int b, int k) -> int32_t {
    const int h = s.have[b];
    return k < h ? a.table[(int64_t)b * a.table_stride + k] : a.free_blocks[count - 1 - (s.grown[b] + (k - h))];
  };
  auto slot_in = [&](int32_t block, int p) -> int32_t {
    return (uint32_t)block > last_block ? -1 : (block << a.block_shift) + (p & mask);
  };
  const int64_t threads = (int64_t)gridDim.x * kThreads, me = (int64_t)blockIdx.x * kThreads + tid;
  const bool wide = (reinterpret_cast<uintptr_t>(a.kv_indices) & 15) == 0;
  auto put = [&](int64_t j, const int32_t (&out)[kVec]) {
    if (wide && j + kVec <= n_kv) {
      *reinterpret_cast<int4*>(a.kv_indices + j) = make_int4(out[0], out[1], out[2], out[3]);
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (j + i < n_kv) a.kv_indices[j + i] = out[i];
    }
  };
  for (int64_t base = (me >> 5) * kRound; base < n_kv; base += (threads >> 5) * kRound) {
    // the whole warp's keys: one bisection, and mostly all in blocks that one request had before
    int b = owner(s.kv, a.batch, (int32_t)base);
    while (s.kv[b + 1] <= (int32_t)base) ++b;
    const int p0 = (int32_t)base - s.kv[b];
    if (s.kv[b + 1] - (int32_t)base >= kRound && (p0 + kRound - 1) >> a.block_shift < s.have[b]) {
      const int32_t* __restrict__ row = a.table + (int64_t)b * a.table_stride;
      int32_t out[kSide][kVec];
#pragma unroll
      for (int u = 0; u < kSide; ++u)
#pragma unroll
        for (int i = 0; i < kVec; ++i) out[u][i] = row[(p0 + (u * 32 + lane) * kVec + i) >> a.block_shift];
#pragma unroll
      for (int u = 0; u < kSide; ++u) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) out[u][i] = slot_in(out[u][i], p0 + (u * 32 + lane) * kVec + i);
        put(base + (u * 32 + lane) * kVec, out[u]);
      }
      continue;
    }
    for (int u = 0; u < kSide; ++u) {
      const int64_t j0 = base + (u * 32 + lane) * kVec;
      int32_t out[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int64_t j = j0 + i;
        out[i] = -1;
        if (j < n_kv) {
          while (s.kv[b + 1] <= (int32_t)j) ++b;
          const int p = (int32_t)j - s.kv[b];
          out[i] = slot_in(block_of(b, p >> a.block_shift), p);
        }
      }
      put(j0, out);
    }
  }
  for (int64_t t = me; t < a.max_q; t += threads) {
    int32_t slot = -1, p = 0;
    if (t < n_q) {
      int b = owner(s.qo, a.batch, (int32_t)t);
      while (s.qo[b + 1] <= (int32_t)t) ++b;
      p = s.cached[b] + ((int32_t)t - s.qo[b]);
      slot = slot_in(block_of(b, p >> a.block_shift), p);
    }
    a.positions[t] = p;
    a.slots[t] = slot;
  }
  for (int64_t g = me; g < n_new; g += threads) {
    int b = owner(s.grown, a.batch, (int32_t)g);
    while (s.grown[b + 1] <= (int32_t)g) ++b;
    a.table[(int64_t)b * a.table_stride + s.have[b] + ((int32_t)g - s.grown[b])] = a.free_blocks[count - 1 - (int32_t)g];
  }
  if (blockIdx.x == 0)
    for (int b = tid; b <= a.batch; b += kThreads) {
      a.kv_indptr[b] = fits ? s.kv[b] : 0;
      a.qo_indptr[b] = fits ? s.qo[b] : 0;
    }
  __syncthreads();
  if (tid == 0) {
    // every thread of this CTA has read the count; the last CTA writes it
    __threadfence();
    if (atomicAdd(a.scratch, 1u) == gridDim.x - 1) {
      *a.free_left = count - n_new;
      *a.scratch = 0;
    }
  }
}

}  // namespace

int launch_tables(const TablesArgs& a, void* stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) !=
                                                cudaSuccess)
    return VMLA_ERR_CUDA;
  const int64_t lanes = (a.max_kv + kVec * kSide - 1) / (kVec * kSide), items = lanes > a.max_q ? lanes : a.max_q;
  const int64_t want = (items + kThreads - 1) / kThreads, most = (int64_t)sms * 4;
  const int64_t blocks = want < 1 ? 1 : want < most ? want : most;
  tables_kernel<<<(unsigned)blocks, kThreads, 0, (cudaStream_t)stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? VMLA_OK : VMLA_ERR_CUDA;
}

}  // namespace vmla
