// Attention over a pool of 8-bit codes with one scale per block of slots.
#include <cuda_runtime.h>

#include "vmla_device.cuh"

namespace vmla {
namespace {

constexpr int kWarps = 8;

// Whether the lengths are in order and inside the call's bounds (by the whole block).
__device__ bool lengths_ok(const ScaledArgs& a) {
  bool ok = true;
  for (int b = threadIdx.x; b < a.batch; b += blockDim.x) {
    const int64_t nq = (int64_t)a.qo_indptr[b + 1] - a.qo_indptr[b], nk = (int64_t)a.kv_indptr[b + 1] - a.kv_indptr[b];
    ok = ok && nq >= 0 && nq <= VMLA_MAX_DRAFT && nk >= nq && a.qo_indptr[b] >= 0 && a.kv_indptr[b] >= 0;
  }
  ok = ok && a.qo_indptr[0] == 0 && a.kv_indptr[0] == 0 && a.qo_indptr[a.batch] <= a.max_q &&
       a.kv_indptr[a.batch] <= a.max_kv;
  return __syncthreads_and(ok);
}

// One block per (query, head) row, its warps taking every kWarps-th key.
__global__ void __launch_bounds__(kWarps * 32)
scaled_row_kernel(const ScaledArgs a) {
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][kDv];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (!lengths_ok(a)) {
    if (threadIdx.x == 0) record_status(a.status, VMLA_ERR_SHAPE, 0);
    return;
  }
  const int64_t r = blockIdx.x;
  const int t = (int)(r / a.num_heads);
  if (t >= a.qo_indptr[a.batch]) return;
  int b = 0;
  while (a.qo_indptr[b + 1] <= t) ++b;
  const int i = t - a.qo_indptr[b], nq = a.qo_indptr[b + 1] - a.qo_indptr[b];
  const int k0 = a.kv_indptr[b], n = a.kv_indptr[b + 1] - k0, prefix = n - nq;
  uint64_t vis = a.masks ? a.masks[t] : causal_bits(i);
  if (a.parent) {
    vis = 0;
    int k = i;
    for (; k >= 0;) {
      vis |= 1ull << k;
      const int p = a.parent[a.qo_indptr[b] + k];
      if (p >= k || p < -1) break;
      k = p;
    }
    if (k >= 0) {
      vis = 0;
      if (threadIdx.x == 0) record_status(a.status, VMLA_ERR_PARENT, (uint32_t)t);
    }
  }
  float q[18];
  for (int k = 0; k < 18; ++k) q[k] = __uint_as_float((uint32_t)a.q[r * kDqk + lane + 32 * k] << 16);
  float m = -INFINITY, l = 0.f, o[16] = {};
  for (int j = warp; j < n; j += kWarps) {
    if (j >= prefix && !((vis >> (j - prefix)) & 1)) continue;
    const int32_t slot = a.kv_indices[k0 + j];
    const bool ok = slot >= 0 && (int64_t)slot < a.pool_slots;
    if (!ok && lane == 0) record_status(a.status, VMLA_ERR_INDEX, (uint32_t)(k0 + j));
    float c[18], s = 0.f;
    const float scale = ok ? a.kv_scales[slot >> a.block_shift] : 0.f;
    for (int k = 0; k < 18; ++k) {
      uint32_t h = 0;
      if (ok) asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)a.pool[(int64_t)slot * kDqk + lane + 32 * k]));
      asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;}" : "=f"(c[k]) : "r"(h));
      s = fmaf(q[k], c[k], s);
    }
    s = warp_sum(s) * scale * a.sm_scale;
    const float m2 = fmaxf(m, s), f = __expf(m - m2), p = __expf(s - m2);
    l = l * f + p;
    for (int k = 0; k < 16; ++k) o[k] = o[k] * f + p * scale * c[k];
    m = m2;
  }
  for (int k = 0; k < 16; ++k) so[warp][lane + 32 * k] = o[k];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  float top = -INFINITY, total = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
  for (int w = 0; w < kWarps; ++w) total += sm[w] > -INFINITY ? sl[w] * __expf(sm[w] - top) : 0.f;
  for (int d = threadIdx.x; d < kDv; d += kWarps * 32) {
    float v = 0.f;
    for (int w = 0; w < kWarps; ++w) v += sm[w] > -INFINITY ? so[w][d] * __expf(sm[w] - top) : 0.f;
    a.out[r * kDv + d] = (uint16_t)pack_bf16x2(total > 0.f ? v / total : 0.f, 0.f);
  }
  if (threadIdx.x == 0) a.lse[r] = total > 0.f ? top + logf(total) : -INFINITY;
}

}  // namespace

size_t scaled_workspace(int) { return 256; }

int launch_scaled(const ScaledArgs& a, void* stream) {
  scaled_row_kernel<<<(unsigned)(a.max_q * a.num_heads), kWarps * 32, 0, (cudaStream_t)stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? VMLA_OK : VMLA_ERR_CUDA;
}

}  // namespace vmla
