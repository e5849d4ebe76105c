"""The sums of verification: residuals as whole numbers of a small unit, against fractions.  The
kernel's own source, compiled for the host with no contraction of products and additions."""
import ctypes
import os
import subprocess
from fractions import Fraction

import numpy as np
import pytest

ROOT = os.path.join(os.path.dirname(__file__), "..")
SHIM = r"""
#include "verify_sum.cuh"
extern "C" {
int unit_bits() { return pkv::kUnitBits; }
void sums(const float *p, const float *d, float mh, float ml, long long *out, int n) {
  for (int i = 0; i < n; ++i) {
    pkv::Sum sum;
    float s, t;
    pkv::residual(p[i], d[i], mh, ml, s, t);
    sum.add(s, t);
    out[i] = (long long)sum.value();
  }
}
long long total(const float *p, int n) {
  pkv::Sum sum;
  for (int i = 0; i < n; ++i) sum.add(p[i], 0.f);
  return (long long)sum.value();
}
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    at = tmp_path_factory.mktemp("sums")
    (at / "shim.cpp").write_text(SHIM)
    so = str(at / "shim.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "paged_kv_cache_272_gb300", "csrc"),
                    str(at / "shim.cpp"), "-o", so], check=True)
    l = ctypes.CDLL(so)
    F = np.ctypeslib.ndpointer(np.float32, flags="C")
    l.sums.argtypes = [F, F, ctypes.c_float, ctypes.c_float,
                       np.ctypeslib.ndpointer(np.int64, flags="C"), ctypes.c_int]
    l.total.argtypes, l.total.restype = [F, ctypes.c_int], ctypes.c_longlong
    return l


def check(lib, p, d, M):
    """Each value within half a unit, 2^-44, of p - M d, and of what its parts are rounded to: the
    remainder (2^-22 at most) and the low number (less) are added in fp32, whose half step below
    2^-21 is 2^-46; the low number is off by 2^-47 of the larger of p and M d (below 2^-22.4 of
    it, rounded twice at 2^-24 of itself; M to 2^-48)."""
    p, d = np.float32(p), np.float32(d)
    mh = np.float32(M)
    ml = np.float32(M - float(mh))
    out = np.zeros(len(p), np.int64)
    lib.sums(p, d, float(mh), float(ml), out, len(p))
    unit = Fraction(1, 2 ** lib.unit_bits())
    for x, y, got in zip(p, d, out):
        x, y = Fraction(float(x)), Fraction(float(y))
        r = max(x - Fraction(M) * y, Fraction(0))
        bound = Fraction(1, 2 ** 44) + Fraction(1, 2 ** 46) + max(x, Fraction(M) * y) / 2 ** 47
        assert abs(int(got) * unit - r) <= bound, (float(x), float(y), M, int(got), float(r))


@pytest.mark.parametrize("M", [0.0, 1.0, 1.0 + 2.0 ** -30, 1.37, 1.9, 2.5])
@pytest.mark.parametrize("top", [1.0, 0.07, 0.001])
def test_residuals(lib, M, top):
    rng = np.random.default_rng(int(1000 * M))
    p = (rng.random(4000) * top).astype(np.float32)
    check(lib, p, (p * rng.random(4000)).astype(np.float32), M)
    check(lib, p, (p * rng.random(4000) * 0.05).astype(np.float32), M)
    # p and M d alike but for the last places
    check(lib, p, (p.astype(np.float64) / max(M, 1.0) * (1 - rng.random(4000) * 2.0 ** -20)), M)


def test_dominant_tokens(lib):
    """Differences at odd multiples of 2^-22, half of the high part's unit, with what their rounding
    left out beyond: the low part's number is the largest then."""
    check(lib, [.99967974], [.04772803], 1.0)
    rng = np.random.default_rng(2)
    k = 2 * rng.integers(2 ** 19, 2 ** 21, 6000) + 1
    d = (rng.random(6000) * 0.05 + 0.001).astype(np.float32)
    p = k * 2.0 ** -22 + d
    near = rng.integers(-2, 3, 6000) * 2.0 ** -24
    check(lib, np.minimum(p + near, 1.9), d, 1.0)
    check(lib, [1.0 - 2.0 ** -24, 1.9999999, 1.9999999], [1e-7, 0.5, 1.0], 1.0)


def test_whole_values(lib):
    """As many values as are summed before the parts are joined."""
    rng = np.random.default_rng(3)
    for p in (rng.random(32), np.full(32, 1.9999999), np.full(32, 3 * 2.0 ** -22),
              2.0 ** -rng.integers(0, 44, 32).astype(float)):
        p = p.astype(np.float32)
        want = sum(Fraction(float(x)) for x in p)
        got = Fraction(lib.total(p, len(p)), 2 ** lib.unit_bits())
        assert abs(got - want) <= Fraction(len(p), 2 ** 44)
