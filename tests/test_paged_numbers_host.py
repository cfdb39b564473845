"""Arithmetic of the paged cache's kernels at the ends of its numbers, without a GPU: what
csrc/paged.h says (compiled here as plain C++), and the error bounds that it rests on."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "attention_gqa_b200", "csrc")

SHIM = """
#include "paged.h"
using namespace gqa;
extern "C" {
int near_border(unsigned bits) { return paged_near_border(bits); }
unsigned scale_bits(unsigned bits) { return paged_scale_bits(bits); }
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    d = tmp_path_factory.mktemp("paged_numbers")
    src, so = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o",
                    str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.near_border.argtypes = lib.scale_bits.argtypes = [ctypes.c_uint]
    lib.scale_bits.restype = ctypes.c_uint
    return lib


def test_values_near_a_scales_border(host):
    for e in (-60, -50, -1, 0, 8, 100):
        at = int(np.float32(1.75 * 2.0 ** e).view(np.uint32))
        assert all(host.near_border(at + d) for d in (-16, -3, -1, 0, 1, 3, 16))
        assert not any(host.near_border(at + d) for d in (-17, -1000, 17, 1000, 2 ** 20, -2 ** 21))
        # the scale changes there and nowhere else of the binade
        scales = {d: host.scale_bits(at + d) for d in (-17, 0, 1, 17)}
        assert scales[-17] == scales[0] and scales[1] == scales[17]
        assert (scales[0] != scales[1]) == (e >= -56)  # below, 2^-64 holds the whole binade
    assert not host.near_border(0)


def test_the_rounded_rotation_stays_within_three_ulps_of_the_pairs_largest(host):
    """fma(a, c, -rn(h s)) in fp32 against the value: so 16 ulps are enough."""
    rng = np.random.default_rng(1)
    n = 400000
    a, h = (rng.integers(128, 256, n) * 2.0 ** rng.integers(-3, 4, n) * rng.choice([-1, 1], n)
            for _ in range(2))
    angle = rng.uniform(0, 2 * np.pi, n)
    c, s = (np.float32(1.3466 * f(angle)).astype(np.float64) for f in (np.cos, np.sin))

    def plain(x, u, y, v):  # (64 bits hold x u and its sum with an fp32 to far below an ulp)
        return np.float32(x * u + np.float32(y * v).astype(np.float64)).astype(np.float64)
    lo, hi = a * c - h * s, h * c + a * s
    ulp = np.exp2(np.floor(np.log2(np.maximum(np.abs(lo), np.abs(hi)))) - 23)
    assert np.all(np.abs(plain(a, c, -h, s) - lo) <= 3 * ulp)
    assert np.all(np.abs(plain(h, c, a, s) - hi) <= 3 * ulp)
