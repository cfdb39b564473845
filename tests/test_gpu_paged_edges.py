"""The paged key/value cache on the GPU at the ends of its numbers: infinities, values at the
largest exponent, scales far apart, maxima that move, against plain fp64 implementations.

Tolerances are those of test_gpu_paged.py, where they are derived; what a test adds to them
stands beside it.
"""
import numpy as np
import pytest
import torch

import attention_gqa_b200 as gqa
from tests._util import dev_to_f64
from tests.test_gpu_paged import (E4M3, Cache, _attend, _check_attention, _f64, _int, _nearest_e4m3,
                                  _queries, _rotate, _scale_of)

pytestmark = pytest.mark.gpu

LARGEST = 3.3895313892515355e38  # the largest finite bf16


# ----------------------------------------------------------------------- append

def _check_codes(cache, b, length, x, xr, scales, codes, what):
    """Codes and scales of a sequence whose pages were all new: x [length, 8, 64] in fp64 with
    xr, the error of the rotation behind each value."""
    P = cache.page
    for i in range(-(-length // P)):
        rows = x[i * P:(i + 1) * P]
        p = int(cache.table_host[b, i])
        finite = np.where(np.isfinite(rows), np.abs(rows), 0.0)
        s = np.array([_scale_of(a) for a in finite.max(axis=(0, 2))])
        assert np.array_equal(_f64(scales[p]), s), what
        got = _f64(codes[p].float())[:len(rows)]
        nan, inf = np.isnan(rows), np.isinf(rows)
        assert np.array_equal(np.isnan(got), nan), what
        assert np.array_equal(got[inf], 448.0 * np.sign(rows[inf])), what
        ok = ~(nan | inf)
        want = np.where(ok, rows, 0.0) / s[None, :, None]
        slack = xr[i * P:(i + 1) * P] / s[None, :, None]
        # the code of some value within the rotation's error
        lo, hi = _nearest_e4m3(want - slack), _nearest_e4m3(want + slack)
        assert np.all((got >= lo) & (got <= hi) | ~ok), what


@pytest.mark.parametrize("rope", ["plain", "yarn"])
@pytest.mark.parametrize("n,page", [(1, 16), (16, 16), (150, 128)])
def test_infinite_and_huge_keys(cuda_device, rope, n, page):
    """Infinities in either half of a key saturate wherever the token stands, and decide no
    scale; keys whose rotation passes fp32's range are finite values like others."""
    g = torch.Generator().manual_seed(31)
    B, inf = 6, float("inf")
    pos = torch.tensor([1, 2, 77, 4095, 50001, 131072 - n])[:, None] + torch.arange(n)
    pos = pos.to(torch.int32)
    k = torch.randn(B, n, 8, 64, generator=g)
    t = n // 2
    k[:, t, 0, 3] = inf
    k[:, t, 1, 40] = -inf
    k[:, t, 2, 5], k[:, t, 2, 37] = LARGEST, -LARGEST
    k[:, t, 3, 7], k[:, t, 3, 39] = inf, -inf
    k[:, t, 4, 9] = float("nan")
    k[:, :, 5] = LARGEST * torch.sign(k[:, :, 5])
    k[:, t, 6, 63] = LARGEST
    k[:, 0, 7, 1], k[:, n - 1, 7, 33], k[:, t, 7, 20] = LARGEST, -LARGEST, inf
    k = k.to(torch.bfloat16)
    cache = Cache([n] * B, page, E4M3, stale=0.0)
    kd = k.cuda()
    gqa.paged_append(kd, kd, pos.cuda(), cache.k, cache.v, cache.table, _int([n] * B), rope=rope,
                     **cache.scales())
    gqa.check()
    kf = _f64(k.float())
    with np.errstate(invalid="ignore"):
        turned = np.stack([_rotate(kf[b], pos[b].numpy(), rope) for b in range(B)])
    mag = np.abs(kf) + np.abs(np.roll(kf, 32, axis=-1))
    mag = np.where(np.isfinite(mag), mag, 0.0)
    for b in range(B):
        _check_codes(cache, b, n, turned[b], 2.0 ** -21 * 1.4 * mag[b], cache.ks, cache.k, (b, "k"))
        _check_codes(cache, b, n, kf[b], 0.0 * mag[b], cache.vs, cache.v, (b, "v"))
