"""The verification's sums of two floats, compiled from the kernel's source for the host."""
import os
import re
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_kv_attention_photon_gb300", "csrc")
HOST = r"""
#include <cmath>
#define __device__
#define __forceinline__ inline
static float __shfl_xor_sync(unsigned, float x, int) { return x; }
%s
extern "C" void add(float* a, const float* b, int n) {   // a[i] += b[i], pairs of floats
  for (int i = 0; i < n; ++i) {
    Sum2 s;
    s.hi = a[2 * i], s.lo = a[2 * i + 1];
    s.add(b[2 * i], b[2 * i + 1]);
    a[2 * i] = s.hi, a[2 * i + 1] = s.lo;
  }
}
"""


@pytest.fixture(scope="module")
def add(tmp_path_factory):
    import ctypes
    with open(os.path.join(CSRC, "verify_tree.cu")) as f:
        struct = re.search(r"^struct Sum2 \{.*?^\};$", f.read(), re.S | re.M).group(0)
    at = tmp_path_factory.mktemp("sums")
    (at / "sums.cpp").write_text(HOST % struct)
    subprocess.run(["g++", "-O1", "-ffp-contract=off", "-shared", "-fPIC", "-o", str(at / "sums.so"),
                    str(at / "sums.cpp")], check=True)
    lib = ctypes.CDLL(str(at / "sums.so"))

    def call(a, b):
        a, b = np.array(a, dtype=np.float32), np.ascontiguousarray(b, dtype=np.float32)
        lib.add(ctypes.c_void_p(a.ctypes.data), ctypes.c_void_p(b.ctypes.data), len(a))
        return a
    return call


def pairs(rng, n):
    hi = rng.random(n) * 2.0 ** rng.integers(-20, 1, n)
    lo = (rng.random(n) - 0.5) * hi * 2.0 ** rng.integers(-26, -20, n)
    return np.stack([hi, lo], -1).astype(np.float32)


def test_lanes_that_exchange_sums_hold_the_same_bits(add):
    """A warp's lanes add up by exchanges, each its own sum and another lane's.  What follows is
    decided by every lane for itself, and they have to go the same way."""
    rng = np.random.default_rng(0)
    lanes = pairs(rng, 32 * 4000).reshape(4000, 32, 2)
    for o in (1, 2, 4, 8, 16):
        other = lanes[:, np.arange(32) ^ o]
        lanes = add(lanes.reshape(-1, 2), other.reshape(-1, 2)).reshape(lanes.shape)
    assert (lanes.view(np.int32) == lanes.view(np.int32)[:, :1]).all()


def test_sums_keep_what_they_round_off(add):
    """64 additions.  Each leaves at most 2^-24 of the sum S to lo, and the terms' own lo are at
    most 2^-21 of them: |lo| <= (2^-18 + 2^-21) S < 2^-17 S.  Adding to lo rounds it twice each
    time, 2^-24 of it: off by at most 64 x 2 x 2^-24 x 2^-17 S = 2^-34 S."""
    rng = np.random.default_rng(1)
    terms = pairs(rng, 64 * 500).reshape(64, 500, 2)
    s = np.zeros((500, 2), dtype=np.float32)
    for t in terms:
        s = add(s, t)
    exact = terms.astype(np.longdouble).sum((0, 2))
    assert (np.abs(s.astype(np.longdouble).sum(-1) - exact) <= 2.0 ** -34 * exact).all()
