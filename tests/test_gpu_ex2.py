"""The error of the approximate power of two that sampling's single-precision weights use, over every float it is given.

Their bound (3.6e-7 of a weight) has 3.1e-8 for the argument's roundings and 3 x 2^-24 = 1.79e-7 for the sums in a tree;
their bound for a sum made anew (5.4e-7) has that and 3.1e-8 again.  Both leave the instruction at least 1.49e-7.  Its
argument is at most 1/2 + 2^-4 in magnitude: the rest of a rounding to a whole number, and a correction of below 2^-4."""
import ctypes
import os
import subprocess

import pytest

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include "vmla_device.cuh"

// The largest |ex2(f) / 2^f - 1| over the floats of magnitude below 1/2 + 2^-4, as a float's bits (which order as
// numbers do, being positive), rounded up.
__global__ void sweep(unsigned* worst) {
  const unsigned last = __float_as_uint(0.5625f), step = gridDim.x * blockDim.x;
  float most = 0.f;
  for (unsigned b = blockIdx.x * blockDim.x + threadIdx.x; b <= last; b += step)
    for (int s = 0; s < 2; ++s) {
      const float f = __uint_as_float(b | (s ? 0x80000000u : 0u));
      most = fmaxf(most, __double2float_ru(fabs((double)vmla::ex2_approx(f) * exp2(-(double)f) - 1.0)));
    }
  atomicMax(worst, __float_as_uint(most));
}

extern "C" int run(unsigned* worst) {
  sweep<<<1216, 256>>>(worst);
  return (int)cudaDeviceSynchronize();
}
"""


def test_error_of_the_power_of_two(tmp_path):
    import torch
    from speculative_decoding_mla_gb300 import build as vbuild
    src, lib = tmp_path / "ex2.cu", tmp_path / "ex2.so"
    src.write_text(SOURCE)
    csrc = os.path.join(vbuild.HERE, "csrc")
    subprocess.run([vbuild.nvcc(), *vbuild.ARCH, "-O3", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", f"-I{csrc}",
                    f"-I{os.path.join(vbuild.ROOT, 'include')}", str(src), "-o", str(lib)], check=True)
    worst = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert ctypes.CDLL(str(lib)).run(ctypes.c_void_p(worst.data_ptr())) == 0
    error = float(worst.view(torch.float32))
    print(error)
    assert 1e-8 < error <= 1.49e-7
