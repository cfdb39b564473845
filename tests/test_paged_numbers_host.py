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
int wave(int row_tokens, int num_sms) { return paged_wave(row_tokens, num_sms); }
long long max_parts(int row_tokens) { return paged_max_parts(paged_target(row_tokens)); }
float power(int e) { return paged_power(e); }
int unit(float scale) { return paged_unit(scale); }
int scale_far(float scale) { return paged_scale_far(scale); }
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
    lib.power.restype = ctypes.c_float
    lib.unit.argtypes = lib.scale_far.argtypes = [ctypes.c_float]
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


def test_units_of_value_scales(host):
    inf, nan = float("inf"), float("nan")
    assert all(host.power(e) == 2.0 ** e for e in range(-126, 128))
    for scale, unit in ((1.0, 0), (1.99, 0), (0.01, -7), (2.0 ** -16, -16), (2.0 ** -64, -16),
                        (2.0 ** -149, -16), (0.0, -16), (2.0 ** 120, 120), (3.4e38, 126), (inf, 126),
                        (-1.0, 0), (nan, 0)):
        assert host.unit(scale) == unit, scale
    # what an append writes for a page of zeros is near enough to ordinary scales
    assert not host.scale_far(2.0 ** -64 * host.power(-host.unit(0.01)))
    for v, far in ((1.0, 0), (2.0 ** -76, 0), (2.0 ** 20, 0), (2.0 ** -77, 1), (2.0 ** 21, 1), (0.0, 1),
                   (inf, 1), (nan, 1)):
        assert host.scale_far(v) == far, v
    # of two scales of which neither is far, the smaller's weights down to 2^-30 of the largest
    # stay above fp32's least normal number when the larger holds the running maximum
    assert 2.0 ** -30 * 2.0 ** -76 / 2.0 ** 20 >= 2.0 ** -126


def test_a_wave_follows_the_sms_and_fits_the_workspace(host):
    assert [host.wave(nt, 148) for nt in (1, 2, 16)] == [74, 55, 37]
    for nt in (1, 2, 16):
        waves = [host.wave(nt, sms) for sms in (1, 7, 74, 132, 148, 160, 10000)]
        assert waves == sorted(waves) and waves[0] >= 1 and waves[2] < waves[4] < waves[5]
        assert waves[-1] == host.max_parts(nt)
