"""Packed sums, roots and quotients (rounded.cuh) against CUDA's rounded operations:
every root of the range, every reciprocal, quotients of random numbers and of the
largest and smallest.  A small library is compiled with the header for this.
"""
import ctypes as C
import os
import shutil
import subprocess

import pytest
import torch

from gradient_sync_rcc_gb300 import build

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include "rounded.cuh"
using namespace rcc::lm;

__device__ uint32_t stir(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}
__device__ void count(unsigned long long* wrong, float got, float want) {
  if (__float_as_uint(got) != __float_as_uint(want)) atomicAdd(wrong, 1ull);
}

__global__ void roots(unsigned long long* wrong) {
  const uint64_t most = __float_as_uint(kMostSquare), step = 2ull * gridDim.x * blockDim.x;
  for (uint64_t i = 2ull * (blockIdx.x * blockDim.x + threadIdx.x); i <= most; i += step) {
    const float2 v = make_float2(__uint_as_float((uint32_t)i), __uint_as_float((uint32_t)min(i + 1, most)));
    const float2 s = root2(v);
    count(wrong, s.x, __fsqrt_rn(v.x));
    count(wrong, s.y, __fsqrt_rn(v.y));
  }
}
__global__ void reciprocals(unsigned long long* wrong) {
  const uint32_t fraction = blockIdx.x * blockDim.x + threadIdx.x;   // of 2^23
  for (int e = -50; e < 24; ++e) {
    const float b = __uint_as_float((uint32_t)(127 + e) << 23 | fraction);
    const float2 q = quotient2(both(1.f), both(b));
    count(wrong, q.x * 0x1p-64f, __frcp_rn(b));
    count(wrong, q.y * 0x1p-64f, __frcp_rn(b));
  }
}
__global__ void quotients(unsigned long long* wrong, uint32_t seed, int each, float one) {
  for (int k = 0; k < each; ++k) {
    const uint32_t i = (blockIdx.x * blockDim.x + threadIdx.x) * each + k;
    const uint32_t h = stir(i ^ seed), l = stir(h + 0x9E3779B9u), b0 = stir(l ^ seed);
    // |m| from 2^-76 to 2^10, every 16th zero; b from kLeastBelow = 2^-50 to 2^24: all
    // quotients are normal numbers
    const float m = __uint_as_float((l & 0x80000000u) | (l & 0x7FFFFFu) |
                                    (h % 16 ? (uint32_t)(51 + (h >> 4) % 86) << 23 : 0u));
    const float b = __uint_as_float((uint32_t)(77 + (h >> 16) % 74) << 23 | (b0 & 0x7FFFFFu));
    const float x = h % 16 ? m : copysignf(0.f, m);
    const float2 q = quotient2(make_float2(x, -x), both(b));
    count(wrong, q.x * 0x1p-64f, __fdiv_rn(x, b));
    count(wrong, q.y * 0x1p-64f, __fdiv_rn(-x, b));
    // a sum of two products, which a packed sum would take as one operation
    const float c = __uint_as_float(0x3F800000u | (h & 0x7FFFFFu));
    const float d = __uint_as_float(0xBF800000u | (l & 0x7FFFFFu));
    const float e = __uint_as_float(0x3F800000u | (b0 & 0x7FFFFFu));
    const float2 s = sum2(mul2(both(c), both(d)), mul2(both(d), both(e)), one);
    count(wrong + 1, s.x, __fadd_rn(__fmul_rn(c, d), __fmul_rn(d, e)));
  }
}

extern "C" int run(int what, unsigned long long* wrong, unsigned seed) {
  if (what == 0) roots<<<152 * 8, 256>>>(wrong);
  if (what == 1) reciprocals<<<1 << 15, 256>>>(wrong);
  if (what == 2) quotients<<<4096, 256>>>(wrong, seed, 512, 1.f);
  return (int)cudaDeviceSynchronize();
}
"""


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    if not shutil.which(build.NVCC):
        pytest.skip("no nvcc")
    where = tmp_path_factory.mktemp("rounded")
    source, lib = where / "rounded_test.cu", where / "rounded_test.so"
    source.write_text(SOURCE)
    subprocess.run([build.NVCC, *build.ARCH, "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-shared",
                    "-I", build.CSRC, "-I", build.INCLUDE, str(source), "-o", str(lib)], check=True)
    return C.CDLL(os.fspath(lib))


def wrong(library, what, seed=0):
    counts = torch.zeros(2, dtype=torch.int64, device="cuda:0")
    torch.cuda.synchronize()
    assert library.run(what, C.c_void_p(counts.data_ptr()), C.c_uint(seed)) == 0
    return counts.tolist()


def test_every_root(library):
    assert wrong(library, 0) == [0, 0]


def test_every_reciprocal(library):
    assert wrong(library, 1) == [0, 0]


@pytest.mark.parametrize("seed", range(8))
def test_quotients_and_sums(library, seed):
    assert wrong(library, 2, 0x1234567 * seed + 1) == [0, 0]
