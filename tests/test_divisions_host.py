"""CPU test of the divisions by constants that choose every unit, share and part border of the few-token layer and of the
integer linear: div_by_const of csrc/internal.h, compiled for the host, with the kernels' (umulhi(n, mul) + n) >> shift."""

import ctypes
import os
import subprocess

import numpy as np
import pytest

from nf3_moe_gb300 import build

SOURCE = r"""
#include "internal.h"
extern "C" long long wrong(const unsigned* ds, int nd, const unsigned* ns, int nn) {
  for (int i = 0; i < nd; ++i) {
    const hmoe::DivBy by = hmoe::div_by_const(ds[i]);
    for (int j = 0; j < nn; ++j) {
      const uint32_t n = ns[j], hi = (uint32_t)(((uint64_t)n * by.mul) >> 32);
      if (((hi + n) >> by.shift) != n / ds[i]) return ((long long)ds[i] << 32) | n;
    }
  }
  return -1;
}
"""


@pytest.fixture(scope="module")
def wrong(tmp_path_factory):
    at = tmp_path_factory.mktemp("div")
    src, lib = str(at / "div.cu"), str(at / "div.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-O2", "-shared", "-Xcompiler", "-fPIC", "-I", build.CSRC, "-I",
                    os.path.join(build.ROOT, "include"), "-o", lib, src], check=True, capture_output=True)
    fn = ctypes.CDLL(lib).wrong
    fn.restype = ctypes.c_longlong

    def first_wrong(ds, ns):
        ds, ns = (np.ascontiguousarray(v, dtype=np.uint32) for v in (ds, ns))
        return fn(ds.ctypes.data_as(ctypes.c_void_p), len(ds), ns.ctypes.data_as(ctypes.c_void_p), len(ns))
    return first_wrong


TOP = 2 ** 31 - 1


def test_every_small_divisor_and_small_number(wrong):
    assert wrong(np.arange(1, 2049), np.arange(0, 8192)) == -1


def test_every_divisor_at_its_multiples(wrong):
    """All the divisors that occur (SMs, blocks of K up to 8192, steps) and the neighbours of powers of two, at their
    multiples' ends and at the ends of the range."""
    r = np.random.default_rng(0)
    near = [d for e in range(31) for d in (2 ** e - 1, 2 ** e, 2 ** e + 1) if 1 <= d <= TOP]
    for d in sorted(set(range(1, 8194)) | {132, 148, 152, 160, 192} | set(near)):
        most = TOP // d
        k = np.unique(np.concatenate([np.arange(0, min(most, 4) + 1), most - np.arange(0, min(most, 4) + 1), r.integers(0, most + 1, 32)]))
        ns = np.concatenate([k * d, np.maximum(k * d - 1, 0), np.minimum(k * d + 1, TOP), np.minimum(k * d + d - 1, TOP), [0, 1, TOP - 1, TOP]])
        assert wrong([d], ns) == -1


def test_a_wrong_multiplier_would_show():
    """The formula without its + 1, on the CPU."""
    def divided(n, d):
        shift = (d - 1).bit_length()
        return (((n * (((2 ** shift - d) << 32) // d)) >> 32) + n) >> shift
    assert any(divided(k * d, d) != k for d in (3, 7, 152) for k in range(1, 200))
