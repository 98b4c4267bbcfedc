// Append of new tokens' rows to the latent pool, with the position rotation.
//
// A cache row is [latent (512) | rotated part (64)].  The model hands over the
// latent and the unrotated part of each new token; the 32 pairs (a, b) of the
// latter are turned by the token's position, with (c, s) = (cos, sin) of
// position x frequency from the caller's table:
//   (a, b) -> (a c - b s, a s + b c),
// pairs being (2i, 2i + 1) or (i, i + 32).  The query heads' rotated parts are
// turned by the same angles, so one launch serves both: the row goes to the
// token's slot (bf16, or e4m3 codes of value / scale), the queries into the
// last 64 columns of q.  Products and sums are fp32, rounded once at the store;
// quotients by the scale are correctly rounded, since a reciprocal's rounding
// would move values across code borders.
//
// A token costs 1152 bytes in, 256 of table, 1152 (or 576) out and 256 per
// head, and nothing is read twice, so the kernel is bound by memory for many
// tokens and by one chain of loads (slot and position, table, store) for few.
// One warp takes one token's row, or 16 or 32 of its heads: a lane holds the
// 16-byte granules g and g + 4 of a 64-wide part (g = lane & 3), which contain
// whole pairs in either pairing, and its 8 cosines and sines serve every head of
// the warp.  The data loads do not depend on the slot or the position and are
// issued with them.  32 heads (eight loads per lane in flight, 32 warps on an
// SM) pay off where there are many tokens of more than 16 heads: 16,384 x 64
// heads took 55.5 us against 57.5 with 16; 16,001 x 16 heads, e4m3, 28.9 against
// 26.0 us; 144 x 64 heads 4.2 against 3.8 us.  Blocks of four warps leave an SM
// in smaller steps than blocks of eight: 53.6 us (5.8 TB/s) against 55.4, and 5,000
// x 16 heads, e4m3, 8.7 against 10.2; of two warps, or 48 warps on an SM, gain
// nothing.  16,001 x 16 heads take 22.6 us in both types (4.7 and 4.3 TB/s), of which
// 10.4 to 12.4 are the cache rows'; rows two or four to a warp took longer.
#include <cuda_runtime.h>

#include "vmla_device.cuh"
#include "vmla_rope.cuh"

namespace vmla {
using namespace rope;
namespace {

constexpr int kAppendWarps = 4;                               // of a block

template <int kPasses>
__global__ void __launch_bounds__(kAppendWarps * 32, kPasses == 4 ? 8 : 10)
append_kernel(const AppendArgs a, int parts) {
  const int lane = threadIdx.x & 31, g = lane & 3;
  const int64_t unit = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);  // warp-uniform
  const int64_t t = a.tokens * parts <= UINT32_MAX ? (int64_t)((uint32_t)unit / (uint32_t)parts) : unit / parts;
  const int part = (int)(unit - t * parts);  // 0: the cache row; p > 0: the (p - 1)-th 8 kPasses heads
  if (t >= a.tokens) return;
  const int32_t slot = __ldg(a.slots + t), pos = __ldg(a.positions + t);
  const bool neighbours = a.neighbours != 0;
  const bool use = slot >= 0 && (int64_t)slot < a.pool_slots && pos >= 0 && (int64_t)pos < a.table_rows;
  const float* row = a.cos_sin + (int64_t)(use ? pos : 0) * kRopeDim;
  if (part == 0) {
    const bool fp8 = a.kv_scale > 0.f;
    const uint4* lat = reinterpret_cast<const uint4*>(a.latent + t * a.latent_stride);
    const uint4* rope = reinterpret_cast<const uint4*>(a.k_rope + t * a.k_rope_stride);
    // e4m3: granules 2 lane, 2 lane + 1, the sources of code granule `lane`
    const uint4 v0 = __ldg(lat + (fp8 ? 2 * lane : lane)), v1 = __ldg(lat + (fp8 ? 2 * lane + 1 : lane + 32));
    uint4 r0 = make_uint4(0, 0, 0, 0), r1 = r0;
    if (lane < 4) {
      r0 = __ldg(rope + g);
      r1 = __ldg(rope + g + 4);
    }
    if (!use) {
      // -1 is padding; anything else out of range is reported and left out
      if (lane == 0 && slot != -1) record_status(a.status, VMLA_ERR_INDEX, (uint32_t)t);
      return;
    }
    float lo[8], hi[8];
    if (lane < 4) rotate(r0, r1, load_angles(row, g, neighbours), neighbours, lo, hi);
    if (fp8) {
      uint8_t* dst = reinterpret_cast<uint8_t*>(a.pool) + (int64_t)slot * kDqk;
      float x0[8], x1[8];
      unpack8(v0, x0);
      unpack8(v1, x1);
      const uint2 c0 = codes8(x0, a.kv_scale), c1 = codes8(x1, a.kv_scale);
      reinterpret_cast<uint4*>(dst)[lane] = make_uint4(c0.x, c0.y, c1.x, c1.y);
      if (lane < 4) {
        *reinterpret_cast<uint2*>(dst + kDv + 8 * g) = codes8(lo, a.kv_scale);
        *reinterpret_cast<uint2*>(dst + kDv + 8 * (g + 4)) = codes8(hi, a.kv_scale);
      }
    } else {
      uint4* dst = reinterpret_cast<uint4*>(a.pool) + (int64_t)slot * (kDqk / 8);
      dst[lane] = v0;
      dst[lane + 32] = v1;
      if (lane < 4) {
        dst[kLatentU4 + g] = pack8(lo);
        dst[kLatentU4 + g + 4] = pack8(hi);
      }
    }
    return;
  }
  turn_heads<kPasses>(a, t, part - 1, lane, use, row);
}

}  // namespace

int launch_append(const AppendArgs& a, void* stream) {
  if (a.tokens == 0) return VMLA_OK;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) !=
                                                cudaSuccess)
    return VMLA_ERR_CUDA;
  // 32 heads per warp once they fill the SMs' warps twice over
  const bool wide = a.num_heads > 2 * kHeadsPerPass && a.tokens * ((a.num_heads + 31) / 32) >= (int64_t)sms * 64;
  const int heads = (wide ? 4 : 2) * kHeadsPerPass;
  const int parts = 1 + (a.num_heads + heads - 1) / heads;
  const int64_t blocks = (a.tokens * parts + kAppendWarps - 1) / kAppendWarps;
  if (blocks > INT32_MAX) return VMLA_ERR_SHAPE;
  const auto kernel = wide ? append_kernel<4> : append_kernel<2>;
  kernel<<<(unsigned)blocks, kAppendWarps * 32, 0, (cudaStream_t)stream>>>(a, parts);
  return cudaGetLastError() == cudaSuccess ? VMLA_OK : VMLA_ERR_CUDA;
}

}  // namespace vmla
