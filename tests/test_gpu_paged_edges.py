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


@pytest.mark.parametrize("n,page", [(1, 16), (9, 16), (128, 128)])
def test_a_scale_at_a_border_follows_the_value_itself(cuda_device, n, page):
    """Keys (position, pair, a, b) whose a cos - b sin lies within two fp32 steps of 448, where
    a rotation with a rounded product comes out on the other side: the scale is
    the least that holds the value, which 64 bits and fp32's table and nearest rounding agree on."""
    cases = [(42766, 29, -180.0, 434.0, True), (83011, 1, 576.0, 23.0, True),
             (6688, 29, 402.0, -366.0, True), (104611, 30, -238.0, 426.0, True),
             (127121, 13, -79.0, 458.0, True), (29667, 9, -234.0, -386.0, False),
             (122418, 17, -188.0, 410.0, False), (92642, 21, -229.0, -486.0, False)]
    B = 8
    g = torch.Generator().manual_seed(32)
    k = torch.randn(B, n, 8, 64, generator=g)
    pos = torch.zeros(B, n, dtype=torch.int32)
    for b in range(B):
        for h in range(8):
            p, pair, x, y, _ = cases[b]
            t = (5 * h) % n
            pos[b] = p
            e = 2.0 ** ((7 * h) % 11 - 5)
            k[b, t, h, pair], k[b, t, h, pair + 32] = e * x, e * y
    k = k.to(torch.bfloat16).cuda()
    cache = Cache([n] * B, page, E4M3, stale=0.0)
    gqa.paged_append(k, k, pos.cuda(), cache.k, cache.v, cache.table, _int([n] * B), **cache.scales())
    gqa.check()
    for b, (p, pair, x, y, above) in enumerate(cases):
        got = _f64(cache.ks[int(cache.table_host[b, 0])])
        e = np.array([2.0 ** ((7 * h) % 11 - 5) for h in range(8)])
        unit = np.eye(64)
        value = abs(_rotate((x * unit[pair] + y * unit[pair + 32])[None], p, "plain")[0, pair])
        assert (value > 448.0) == above and abs(value - 448.0) < 2.0 ** -14
        assert np.array_equal(got, e * (2.0 if above else 1.0)), (b, got / e)


@pytest.mark.parametrize("rope", ["plain", "yarn"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_scales_of_rotated_keys_and_of_pages_used_before(cuda_device, page, rope):
    """Every touched page's scale is the least that holds its new tokens, or the one that its
    earlier tokens had if that is larger; what an earlier owner left in a page counts for
    nothing once the page gets its first slot."""
    lengths = [1, page, page + 1, 2 * page + 5, 300, 301, 3 * page, 7]
    counts = [1, page, 1, page + 9, 150, 7, 3 * page, 0]
    B, n = len(lengths), max(counts)
    starts = [a - c for a, c in zip(lengths, counts)]
    g = torch.Generator().manual_seed(90 + page)
    cache = Cache(lengths, page, E4M3)
    cache.ks.fill_(2.0 ** 40)
    cache.vs.fill_(2.0 ** 40)
    cache.fill(starts, g)
    before = cache.ks.clone(), cache.vs.clone()
    size = torch.exp(2.0 * torch.randn(B, n, 8, 1, generator=g))
    k = (size * torch.randn(B, n, 8, 64, generator=g)).to(torch.bfloat16).cuda()
    v = (size * torch.randn(B, n, 8, 64, generator=g)).to(torch.bfloat16).cuda()
    pos = torch.tensor([[s + t for t in range(n)] for s in starts], dtype=torch.int32)
    gqa.paged_append(k, v, pos.cuda(), cache.k, cache.v, cache.table, _int(lengths),
                     counts=_int(counts), rope=rope, **cache.scales())
    gqa.check()
    seen = near = 0
    for b, (length, c) in enumerate(zip(lengths, counts)):
        kf, vf = _f64(k[b, :c].float()), _f64(v[b, :c].float())
        turned = _rotate(kf, pos[b, :c].numpy(), rope) if c else kf
        for i in range(starts[b] // page, -(-length // page)):
            lo, hi = max(starts[b], i * page), min(length, (i + 1) * page)
            if lo >= hi:
                continue
            p = int(cache.table_host[b, i])
            for x, scales, old in ((turned, cache.ks, before[0]), (vf, cache.vs, before[1])):
                top = np.abs(x[lo - starts[b]:hi - starts[b]]).max(axis=(0, 2))
                m, _ = np.frexp(top / 448.0)
                want = np.array([_scale_of(a) for a in top])
                if lo > i * page:
                    want = np.maximum(want, _f64(old[p]))
                got = _f64(scales[p])
                # within the rotation's error of a border either power may be right
                border = (np.abs(m - 0.5) < 2.0 ** -19) | (np.abs(m - 1.0) < 2.0 ** -19)
                border &= x is turned
                assert np.all((got == want) | border), (b, i, got, want)
                seen, near = seen + 8, near + int(border.sum())
    assert near <= seen // 100


# -------------------------------------------------------------------- attention

def _check_rows(got, cache, q, sinks, length, window, n):
    """Attention of one sequence with infinities among what it sees: where the definition gives
    an infinity or NaN so does the kernel; elsewhere test_gpu_paged's tolerance (of the keys
    without infinite scores, and the values without infinities)."""
    r = 2.0 ** -16 if cache.dtype == torch.bfloat16 else 2.0 ** -11
    rp = 2.0 ** -8 if cache.dtype == torch.bfloat16 and n > 2 else r
    k, v = cache.sequence(0, length)
    got = dev_to_f64(got).reshape(n, 64, 64)
    kz, vz = (np.where(np.isfinite(x), x, 0.0) for x in (k, v))
    for t in range(n):
        i = length - n + t
        turned = _rotate(_f64(q.float())[0, t], i, "plain")
        with np.errstate(invalid="ignore"):
            ref, _, _ = _attend(turned, k, v, _f64(sinks), i, window)
        _, S, V = _attend(turned, kz, vz, _f64(sinks), i, window)
        assert np.array_equal(np.isnan(got[t]), np.isnan(ref)), t
        inf = np.isinf(ref)
        assert np.array_equal(got[t][inf], ref[inf]), t
        ok = np.isfinite(ref)
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 * V * (2.0 * (r + 2.0 ** -19) * S + rp)
        assert np.all(np.abs(got[t] - np.where(ok, ref, 0.0))[ok] <= tol[ok]), t


@pytest.mark.parametrize("n", [1, 2, 3, 20])
@pytest.mark.parametrize("length,window", [(700, 0), (700, 300), (5000, 0)])
def test_infinities_that_a_token_sees(cuda_device, n, length, window):
    """bf16 pages. An infinite key element is a score of one sign or the other: -inf weighs
    nothing, +inf makes the row NaN. An infinite value makes its element infinite."""
    page, inf = 32, float("inf")
    for seed in (0, 1):
        g = torch.Generator().manual_seed(40 + seed)
        cache = Cache([length], page, torch.bfloat16)
        cache.fill([length], g)
        q, sinks = _queries(1, n, g)

        def put(pages, key, h, d, x):
            pages[int(cache.table_host[0, key // page]), key % page, h, d] = x
        if seed == 0:  # keys: in the last tile, inside, before a window
            put(cache.k, length - 1, 0, 5, inf)
            put(cache.k, length - n, 1, 33, -inf)
            put(cache.k, length - 150, 2, 63, inf)
            put(cache.k, length - 290, 3, 0, -inf)
            put(cache.k, 1, 4, 17, inf)
        else:  # values
            put(cache.v, length - 1, 0, 5, inf)
            put(cache.v, length - n, 1, 33, -inf)
            put(cache.v, length - 150, 2, 63, inf)
            put(cache.v, length - 260, 3, 0, -inf)
            put(cache.v, 1, 4, 17, inf)
            put(cache.v, length - 2, 5, 9, inf)
            put(cache.v, length - 100, 5, 9, -inf)
        got = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int([length]),
                                  window=window)
        gqa.check()
        _check_rows(got, cache, q, sinks, length, window, n)


SPREADS = {  # exponent of page i of m
    "one large": lambda i, m: 119 if i == m // 2 else -64,
    "one small": lambda i, m: -64 if i == m // 2 else 119,
    "first small": lambda i, m: -64 if i < 3 else 110,
    "halves": lambda i, m: -60 if i < m // 2 else 70,
    "ramp": lambda i, m: -105 + (224 * i) // m,
    "all small": lambda i, m: -110,
    "all large": lambda i, m: 119,
    "moderate": lambda i, m: (-56, 0, 10)[i % 3],
}


@pytest.mark.parametrize("n,lengths", [(1, [400]), (2, [400]), (5, [400, 33]), (20, [600]),
                                       (1, [5000]), (2, [5000]), (20, [3000])])
@pytest.mark.parametrize("spread", SPREADS)
def test_value_scales_far_apart(cuda_device, n, lengths, spread):
    """Pages whose value scales lie up to 2^224 apart share one softmax: what a small page weighs
    counts whole, whichever came first, inside a chunk and where chunks are joined."""
    page = 16
    g = torch.Generator().manual_seed(50 + n)
    cache = Cache(lengths, page, E4M3)
    cache.fill(lengths, g)
    q, sinks = _queries(len(lengths), n, g)
    sinks[3::8] = float("-inf")
    sinks[5::8] = 6.0
    # the pages of the largest scale hold zeros: the others' values are all there is to see
    for zeros in (False, True) if spread != "moderate" else (False,):
        for b, length in enumerate(lengths):
            m = -(-length // page)
            for i in range(m):
                e = SPREADS[spread](i, m)
                p = int(cache.table_host[b, i])
                # the largest value stays finite in bf16
                cache.vs[p] = cache.vs[p].clamp(2.0 ** -9, 2.0 ** -7) * 2.0 ** e
                if zeros and e == max(SPREADS[spread](j, m) for j in range(m)):
                    cache.v[p] = torch.zeros_like(cache.v[p].float()).to(E4M3)
        out = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int(lengths),
                                  **cache.scales())
        gqa.check()
        _check_attention(out, cache, q, sinks, lengths, 0)


@pytest.mark.parametrize("n", [1, 2, 5])
def test_huge_and_tiny_queries_of_e4m3_pages(cuda_device, n):
    """Queries up to 2^119 and down to 2^-118, against keys that make ordinary scores of them."""
    page, L = 16, 100
    g = torch.Generator().manual_seed(60)
    for e in (100, 110, 116, 118, -100, -110, -118):
        cache = Cache([L], page, E4M3)
        cache.fill([L], g)
        cache.ks.mul_(2.0 ** -e)
        q, sinks = _queries(1, n, g)
        q = (q.float().clamp(-1.9, 1.9) * 2.0 ** e).to(torch.bfloat16)
        out = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int([L]), **cache.scales())
        gqa.check()
        _check_attention(out, cache, q, sinks, [L], 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 2, 3, 5, 20])
@pytest.mark.parametrize("L", [640, 6400])
def test_maxima_that_move_in_every_tile(cuda_device, dtype, n, L):
    """Scores that rise by 12 to 25 in the exponent's units from tile to tile and fall back at
    the end, so that sums and outputs are rescaled again and again, in whole rows and in cut
    ones, and parts of very different maxima are joined. Scores are exact products (a power of
    two and a code), so the output's and the weights' roundings are all that is left."""
    page = 64
    g = torch.Generator().manual_seed(70)
    cache = Cache([L], page, dtype, stale=0.0)
    rise = torch.arange(L // 64, dtype=torch.float32)
    rise = torch.where(rise > L // 64 - 3, rise - 4, rise)  # the last tiles weigh less
    # steps of 16 of 256: whole numbers of bf16's and, up to 16 tiles, of e4m3's grid
    level = (rise % 15 + 1).repeat_interleave(64)
    k = torch.zeros(1, L, 8, 64)
    k[:, :, :, 31] = level[None, :, None]
    k[:, ::7, 1::2, 31] *= 0.5
    v = torch.randn(1, L, 8, 64, generator=g)
    zero = torch.zeros(1, L, dtype=torch.int32, device="cuda")
    gqa.paged_append(k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), zero, cache.k,
                     cache.v, cache.table, _int([L]), **cache.scales())
    q = torch.zeros(1, n, 64, 64, dtype=torch.bfloat16, device="cuda")
    q[:, :, :, 31] = 128.0
    q[:, :, 1::4, 31] = 64.0
    q[:, 1::2, 2::4, 31] = -64.0
    sinks = torch.zeros(64, device="cuda")
    sinks[::5] = float("-inf")
    sinks[1::5] = 200.0
    out = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int([L]),
                              pos=torch.zeros(1, n, dtype=torch.int32, device="cuda"),
                              **cache.scales())
    gqa.check()
    kf, vf = cache.sequence(0, L)
    rp = 2.0 ** -8 if dtype == torch.bfloat16 and n > 2 else 2.0 ** -11
    got = dev_to_f64(out)[0]
    for t in range(n):
        ref, S, V = _attend(_f64(q[0, t].float()), kf, vf, _f64(sinks), L - n + t, 0)
        # a score in the exponent is held to 2^-24 of itself, with 2^-22 for the exponential
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 * V * (rp + 2.0 ** -21 * (1.0 + S))
        err = np.abs(got[t] - ref)
        assert np.all(err <= tol), (t, (err - tol).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 2, 5, 20])
@pytest.mark.parametrize("lengths", [[300, 0, 3], [6000, 40, 0]])
def test_sinks_of_nothing_and_of_everything(cuda_device, dtype, n, lengths):
    """Sinks of -inf and far above the scores, in whole rows and in joined ones, with rows
    that see nothing."""
    g = torch.Generator().manual_seed(80)
    cache = Cache(lengths, 64, dtype)
    cache.fill(lengths, g, spread=0.5)
    q, sinks = _queries(3, n, g)
    sinks[::3] = float("-inf")
    sinks[1::6] = 90.0
    out = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int(lengths), **cache.scales())
    gqa.check()
    _check_attention(out, cache, q, sinks, lengths, 0)


# ------------------------------------------------------------------- error state

@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
def test_append_skips_work_while_a_timeout_is_pending(cuda_device, dtype):
    """What follows a kernel that gave up leaves the pages and their scales as they are."""
    lib = gqa._load()
    g = torch.Generator().manual_seed(95)
    cache = Cache([40, 7], 16, dtype, stale=0.0)
    cache.fill([30, 2], g)
    k = (100.0 * torch.randn(2, 10, 8, 64, generator=g)).to(torch.bfloat16).cuda()
    pos = torch.zeros(2, 10, dtype=torch.int32, device="cuda")
    args = (k, k, pos, cache.k, cache.v, cache.table, _int([40, 7]))
    counts = _int([10, 5])
    state = [x for x in (cache.k, cache.v, cache.ks, cache.vs) if x is not None]
    before = [x.clone() for x in state]

    def same():
        return [torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(state, before)]
    stream = torch.cuda.current_stream().cuda_stream
    gqa.check()
    assert lib.gptoss_attn_debug_wait_timeout(1000, stream) == 0
    gqa.paged_append(*args, counts=counts, **cache.scales())
    assert lib.gptoss_attn_check(stream) == -9
    assert all(same())
    gqa.paged_append(*args, counts=counts, **cache.scales())
    gqa.check()
    assert not any(same())


@pytest.mark.parametrize("n", [1, 2, 5, 20])
@pytest.mark.parametrize("layout,window", [("token", 0), ("head", 40), ("both", 1)])
def test_value_scales_far_apart_in_windows_and_odd_places(cuda_device, n, layout, window):
    """Scales that swing by 2^120 from page to page, with windows, other strides, given
    positions, rows that see nothing, and a page that is none (zeros, and reported)."""
    page, lengths = 16, [400, 3, 0, 17]
    g = torch.Generator().manual_seed(55 + n)
    cache = Cache(lengths, page, E4M3, layout)
    cache.fill(lengths, g)
    for b, length in enumerate(lengths):
        for i in range(-(-length // page)):
            cache.vs[int(cache.table_host[b, i])] *= 2.0 ** (60 if i % 2 else -60)
    q, sinks = _queries(len(lengths), n, g)
    pos = torch.randint(0, 131072, (len(lengths), n), generator=g, dtype=torch.int32)
    out = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int(lengths), window=window,
                              pos=pos.cuda(), rope="yarn", **cache.scales())
    gqa.check()
    _check_attention(out, cache, q, sinks, lengths, window, "yarn", pos)
    assert not out[2].any()
    # the last page's number of sequence 3 is out of range: its one key and value are zeros
    bad = cache.table_host.clone()
    bad[3, 1] = cache.num
    got = gqa.paged_attention(q, cache.k, cache.v, bad.cuda(), sinks, _int(lengths), window=window,
                              pos=pos.cuda(), rope="yarn", **cache.scales())
    with pytest.raises(gqa.GptossAttnError) as e:
        gqa.check()
    assert e.value.status == -12
    assert torch.equal(got[:3], out[:3])
    p = int(cache.table_host[3, 1])
    cache.k[p], cache.v[p] = (torch.zeros(page, 8, 64, device="cuda").to(E4M3) for _ in range(2))
    _check_attention(got, cache, q, sinks, lengths, window, "yarn", pos, only={3})


def test_a_captured_call_follows_scales_that_change(cuda_device):
    """Replays of one graph over scales near each other, far apart, and near again."""
    gqa.init()
    page, lengths = 32, [300, 2000]
    g = torch.Generator().manual_seed(57)
    cache = Cache(lengths, page, E4M3)
    cache.fill(lengths, g)
    near = cache.vs.clone()
    graphs = []
    ln = _int(lengths)
    for n in (1, 5):
        q, sinks = _queries(2, n, g)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, ln, **cache.scales())
        graphs.append((graph, q, sinks, out))
    torch.cuda.synchronize()
    for factor in (1.0, 2.0 ** 90, 1.0, 2.0 ** -90, 2.0 ** 3):
        cache.vs.copy_(near)
        cache.vs[::2] *= factor
        for graph, q, sinks, out in graphs:
            graph.replay()
            gqa.check()
            _check_attention(out, cache, q, sinks, lengths, 0)
    for graph, *_ in graphs:
        graph.reset()
