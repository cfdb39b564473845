"""The paged key/value cache on the GPU: appending and attending, against plain fp64
implementations.

Tolerances. A rounding to a type with eps is off by at most eps/2 of the value.
  append, bf16 pages: 2^-8 |x| for the one rounding, plus 2^-21 (|a| + |b|) for the
    fp32 rotation a c - b s (table entries 2^-24, three roundings).
  append, e4m3 pages: half a step of the code, 2^-4 of the value or half of the
    subnormal step 2^-9 of the scale, plus the rotation's 2^-21 (|a| + |b|).
  attention: |out| 2^-8 for the output's rounding, plus what the other roundings
    move the weighted mean: a score is off by at most r S, S = sum |q_d k_d| / 8 and r
    the rounding of q (bf16 pages: two bf16 terms, 2^-16; e4m3: f16 of a head scaled to
    its largest element, 2^-12 |q_d| + 2^-25 max|q|, together under 2^-11 S), so with the
    fp32 work (2^-19 S) every weight is off by a factor within 1 +- 2 r' S (for
    r' S < 0.4), and by its own rounding (bf16 pages: 2^-16 in two terms for up to two
    tokens, 2^-8 in one beyond; e4m3: 2^-11); the mean of values up to V moves by
    at most twice that times V. Over a whole output the output's rounding, and for one-term
    weights theirs too, add up as independent errors of at most 2^-8 each.
"""
import numpy as np
import pytest
import torch

import attention_gqa_b200 as gqa
import oracle
from tests._util import dev_to_f64

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
THETA = 150000.0


# ------------------------------------------------------------------ plain fp64

def _f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def _rotate(x, pos, rope):
    """x [..., heads, 64] at pos [...]."""
    return oracle.rope(x, np.asarray(pos, dtype=np.float64)[..., None], rope=rope)


def _nearest_e4m3(y):
    _, e = np.frexp(np.maximum(np.abs(y), 2.0 ** -6))
    step = np.ldexp(1.0, e - 4)
    return np.clip(np.round(y / step) * step, -448.0, 448.0)


def _scale_of(largest):
    if not largest > 0:
        return 2.0 ** -64
    m, e = np.frexp(largest / 448.0)
    return 2.0 ** float(np.clip(e - 1 if m == 0.5 else e, -64, 120))


class Cache:
    """A pool of pages with its plain fp64 twin (values by sequence)."""

    def __init__(self, lengths, page, dtype, layout="token", max_pages=None, spare=3, seed=0,
                 stale=float("nan"), hole=-1):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lengths]
        self.page, self.dtype = page, dtype
        self.num = sum(need) + spare
        B, width = len(lengths), max_pages or max(1, max(need))
        order = torch.randperm(self.num, generator=g)[:sum(need)].to(torch.int32)
        table = torch.full((B, width), hole, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.table_host, self.table = table, table.cuda()
        shape = {"token": (self.num, page, 8, 64), "head": (self.num, 8, page, 64),
                 "both": (self.num, page, 2, 8, 64)}[layout]

        def pool(which):
            if layout == "both":  # K and V of a token side by side
                if which == 0:
                    self.buf = torch.full(shape, stale, device="cuda").to(dtype)
                return self.buf[:, :, which]
            x = torch.full(shape, stale, device="cuda").to(dtype)
            return x.transpose(1, 2) if layout == "head" else x
        self.k, self.v = pool(0), pool(1)
        self.ks = self.vs = None
        if dtype == E4M3:
            self.ks = torch.zeros(self.num, 8, device="cuda")
            self.vs = torch.zeros(self.num, 8, device="cuda")

    def scales(self):
        return dict(kscales=self.ks, vscales=self.vs)

    def fill(self, lengths, g, spread=0.0):
        """Random earlier tokens in every sequence; the rest of the pages stays stale."""
        for b, n in enumerate(lengths):
            for i in range(-(-n // self.page)):
                m = min(self.page, n - i * self.page)
                p = int(self.table_host[b, i])
                for pages, scales in ((self.k, self.ks), (self.v, self.vs)):
                    x = torch.randn(m, 8, 64, generator=g)
                    if self.dtype == E4M3:
                        x *= torch.exp(spread * torch.randn(1, 8, 1, generator=g))
                        s = torch.tensor([_scale_of(float(a)) for a in x.abs().amax(dim=(0, 2))])
                        x = x / s[None, :, None]
                        scales[p] = s.cuda()
                    pages[p, :m] = x.to(self.dtype).cuda()

    def sequence(self, b, n):
        """Keys and values of sequence b's first n tokens, [n, 8, 64] in fp64."""
        out = []
        for pages, scales in ((self.k, self.ks), (self.v, self.vs)):
            rows = [np.zeros((0, 8, 64))]
            for i in range(-(-n // self.page)):
                p = int(self.table_host[b, i])
                x = _f64(pages[p].float())
                if scales is not None:
                    x = x * _f64(scales[p])[None, :, None]
                rows.append(x)
            out.append(np.concatenate(rows)[:n])
        return out


def _attend(q, k, v, sinks, index, window):
    """One rotated token q [64, 64] at `index` over k, v [n, 8, 64]; also S and V of the
    tolerance. All fp64."""
    out = np.zeros((64, 64))
    bound = np.zeros((64, 1))
    lo = max(0, index + 1 - window) if window > 0 else 0
    if index < 0:
        return out, bound, bound
    k, v = k[lo:index + 1], v[lo:index + 1]
    size, vmax = np.zeros((64, 1)), np.zeros((64, 1))
    for h in range(64):
        s = k[:, h // 8] @ q[h] / 8.0
        top = max(s.max(), sinks[h])
        p = np.exp(s - top)
        out[h] = (p @ v[:, h // 8]) / (p.sum() + np.exp(sinks[h] - top))
        size[h] = (np.abs(k[:, h // 8]) @ np.abs(q[h])).max() / 8.0
        vmax[h] = np.abs(v[:, h // 8]).max()
    return out, size, vmax


def _check_attention(got, cache, q, sinks, lengths, window, rope="plain", pos=None, what="",
                     only=None):
    B, n = q.shape[0], q.shape[1]
    got = dev_to_f64(got).reshape(B, n, 64, 64)
    qf, sk = _f64(q.float()), _f64(sinks)
    r = 2.0 ** -16 if cache.dtype == torch.bfloat16 else 2.0 ** -11
    rp = 2.0 ** -8 if cache.dtype == torch.bfloat16 and n > 2 else r
    assert np.all(np.isfinite(got)), what
    off = norm = 0.0
    for b, length in enumerate(lengths):
        if only is not None and b not in only:
            continue
        k, v = cache.sequence(b, length)
        for t in range(n):
            i = length - n + t
            p = i if pos is None else int(pos[b, t])
            ref, S, V = _attend(_rotate(qf[b, t], max(p, 0), rope), k, v, sk, i, window)
            move = (r + 2.0 ** -19) * S
            assert move.max(initial=0.0) < 0.4
            tol = 2.0 ** -8 * np.abs(ref) + 2.0 * V * (2.0 * move + rp)
            err = np.abs(got[b, t] - ref)
            assert np.all(err <= tol), "%s b=%d t=%d: err %.3e tol %.3e" % (
                what, b, t, (err - tol).max() + tol.max(), tol.max())
            off += float((err ** 2).sum())
            norm += float((ref ** 2).sum())
    whole = 2.0 ** -8 * (2.0 ** 0.5 if rp == 2.0 ** -8 else 1.0)
    assert off ** 0.5 <= (whole + 2.0 ** -10) * norm ** 0.5, what


def _queries(B, n, g):
    return (torch.randn(B, n, 64, 64, generator=g).to(torch.bfloat16).cuda(),
            torch.randn(64, generator=g).cuda())


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ----------------------------------------------------------------------- append

def _append_ref(cache, before, k, v, pos, lengths, counts, rope):
    """What the pages' sequences hold after an append: per sequence (keys, values), and
    the largest error allowed, all [len, 8, 64]; scales checked on the way."""
    out = []
    for b, (length, c) in enumerate(zip(lengths, counts)):
        start = length - c
        kf, vf = _f64(k[b, :c].float()), _f64(v[b, :c].float())
        mag = np.abs(kf) + np.abs(np.roll(kf, 32, axis=-1))
        new = (_rotate(kf, pos[b, :c], rope) if c else kf, vf)
        slack = (2.0 ** -21 * mag * 1.4, np.zeros_like(vf))
        res = []
        for x, add, old, scales in ((new[0], slack[0], before[b][0], cache.ks),
                                    (new[1], slack[1], before[b][1], cache.vs)):
            val = np.concatenate([old[:start], x])
            tol = np.zeros_like(val)
            if cache.dtype == torch.bfloat16:
                tol[start:] = 2.0 ** -8 * np.abs(x) + add if add.any() else 0.0
            else:
                for i in range(start // cache.page, -(-length // cache.page)):
                    a, z = i * cache.page, min(length, (i + 1) * cache.page)
                    s = _f64(scales[int(cache.table_host[b, i])])[None, :, None]
                    f = max(start, a)
                    w = np.maximum(np.abs(val[f:z]), 2.0 ** -6 * s)
                    # half a step of the value's binade
                    tol[f:z] = np.exp2(np.floor(np.log2(w * (1 + 2.0 ** -20)))) * 2.0 ** -4 \
                        + add[f - start:z - start]
                    tol[a:f] = 2.0 ** -10 * s  # moved codes: at most half a subnormal step
            res.append((val, tol))
        out.append(res)
    return out


def _run_append(page, dtype, lengths, counts, n, layout="token", rope="plain", fused=False, seed=1,
                scale=1.0, use_counts=True):
    g = torch.Generator().manual_seed(seed)
    cache = Cache(lengths, page, dtype, layout, seed=seed)
    starts = [a - c for a, c in zip(lengths, counts)]
    cache.fill(starts, g)
    B = len(lengths)
    before = [cache.sequence(b, starts[b]) for b in range(B)]
    if fused:
        qkv = (scale * torch.randn(B, n, 80, 64, generator=g)).to(torch.bfloat16).cuda()
        k, v = qkv[:, :, 64:72], qkv[:, :, 72:]
    else:
        k = (scale * torch.randn(B, n, 8, 64, generator=g)).to(torch.bfloat16).cuda()
        v = (scale * torch.randn(B, n, 8, 64, generator=g)).to(torch.bfloat16).cuda()
    pos = torch.tensor([[max(0, s) + t for t in range(n)] for s in starts], dtype=torch.int32)
    pages = [(p.clone(), None if s is None else s.clone())
             for p, s in ((cache.k, cache.ks), (cache.v, cache.vs))]
    gqa.paged_append(k, v, pos.cuda(), cache.k, cache.v, cache.table, _int(lengths),
                     counts=_int(counts) if use_counts else None, rope=rope, **cache.scales())
    gqa.check()
    ref = _append_ref(cache, before, k, v, pos.numpy(), lengths, counts, rope)
    for b, length in enumerate(lengths):
        for got, (val, tol) in zip(cache.sequence(b, length), ref[b]):
            err = np.abs(got - val)
            assert np.all(err <= tol), "sequence %d: %s" % (b, np.argwhere(err > tol)[:4])
    return cache, pages, k, v, pos


def _same_bits(a, b):
    if a.dtype == E4M3:
        return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("layout,fused,rope", [("token", False, "plain"), ("head", True, "yarn"),
                                               ("both", True, "plain")])
def test_append_ragged(cuda_device, page, dtype, layout, fused, rope):
    """Nothing, one token, whole pages, ends and starts at and beside page borders."""
    lengths = [0, 1, page, page + 1, 2 * page - 1, 5 * page, 300, 301, 299]
    counts = [0, 1, page, 1, page, 2 * page + 3, 0, 150, 7]
    n = max(counts)
    cache, pages, *_ = _run_append(page, dtype, lengths, counts, n, layout, rope, fused)
    # every slot that is no new token's keeps its bits, unless its page's scale grew
    new = torch.zeros(cache.num, page, dtype=torch.bool)
    touched = torch.zeros(cache.num, dtype=torch.bool)
    for b, (a, c) in enumerate(zip(lengths, counts)):
        for i in range(a - c, a):
            new[int(cache.table_host[b, i // page]), i % page] = True
            touched[int(cache.table_host[b, i // page])] = True
    for now, (was, was_s), s in ((cache.k, pages[0], cache.ks), (cache.v, pages[1], cache.vs)):
        assert _same_bits(now[~touched], was[~touched])
        if dtype == torch.bfloat16:
            assert _same_bits(now[~new], was[~new])
        else:
            assert torch.equal(s[~touched], was_s[~touched])
            same = (s == was_s).all(dim=1).cpu() & touched
            assert _same_bits(now[same][~new[same]], was[same][~new[same]])


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
def test_append_one_token_to_a_batch(cuda_device, dtype):
    lengths = [1 + (37 * b) % 250 for b in range(64)]
    _run_append(16, dtype, lengths, [1] * 64, 1, use_counts=False)


def test_append_bf16_writes_what_prefill_chunk_writes(cuda_device):
    B, S, page = 2, 333, 32
    g = torch.Generator().manual_seed(5)
    k = torch.randn(B, S, 8, 64, generator=g).to(torch.bfloat16).cuda()
    v = torch.randn(B, S, 8, 64, generator=g).to(torch.bfloat16).cuda()
    q, sinks = _queries(B, S, g)
    pos = _int([list(range(S))] * B)
    for rope in ("plain", "yarn"):
        kc = torch.zeros(B, S, 8, 64, dtype=torch.bfloat16, device="cuda")
        vc = torch.zeros_like(kc)
        gqa.prefill_chunk(q, k, v, sinks, pos, kc, vc, 0, rope=rope)
        cache = Cache([S] * B, page, torch.bfloat16)
        gqa.paged_append(k, v, pos, cache.k, cache.v, cache.table, _int([S] * B), rope=rope)
        gqa.check()
        table = cache.table.long()
        for got, want in ((cache.k, kc), (cache.v, vc)):
            assert torch.equal(got[table].reshape(B, -1, 8, 64)[:, :S], want)


def test_scales_are_the_least_that_hold_the_page(cuda_device):
    """Fresh pages of many sizes; an all-zero page; values at the very border."""
    page, B = 16, 40
    g = torch.Generator().manual_seed(7)
    v = torch.randn(B, page, 8, 64, generator=g) * torch.exp(8 * torch.randn(B, 1, 8, 1, generator=g))
    v[0] = 0
    v[1, 3, 0, 5], v[1, :, 1] = 448.0, 0.0
    v[1, :, 0] = v[1, :, 0].clamp(-448, 448)
    v[2] = 3e38
    v[3] = 1e-30
    v = v.to(torch.bfloat16).cuda()
    cache = Cache([page] * B, page, E4M3)
    pos = torch.zeros(B, page, dtype=torch.int32, device="cuda")  # position 0: no rotation
    gqa.paged_append(v, v, pos, cache.k, cache.v, cache.table, _int([page] * B), **cache.scales())
    gqa.check()
    for b in range(B):
        p = int(cache.table_host[b, 0])
        x = _f64(v[b].float())
        s = np.array([_scale_of(a) for a in np.abs(x).max(axis=(0, 2))])
        for got, codes in ((cache.ks, cache.k), (cache.vs, cache.v)):
            assert np.array_equal(_f64(got[p]), s)
            assert np.array_equal(_f64(codes[p].float()), _nearest_e4m3(x / s[None, :, None]))


def test_a_growing_scale_moves_the_codes_there(cuda_device):
    """One token after another into the same page, each larger than the last."""
    page, steps = 16, 16
    g = torch.Generator().manual_seed(8)
    rows = torch.randn(1, steps, 8, 64, generator=g) * 2.0 ** torch.arange(steps)[None, :, None, None]
    rows = rows.to(torch.bfloat16).cuda()
    cache = Cache([page], page, E4M3)
    p = int(cache.table_host[0, 0])
    pos = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    held, s = np.zeros((0, 8, 64)), np.full(8, 2.0 ** -64)
    for i in range(steps):
        x = rows[:, i:i + 1].contiguous()
        gqa.paged_append(x, x, pos, cache.k, cache.v, cache.table, _int([i + 1]), **cache.scales())
        gqa.check()
        xf = _f64(x[0].float())
        new = np.maximum(s if i else 0.0, [_scale_of(a) for a in np.abs(xf).max(axis=(0, 2))])
        held = np.concatenate([_nearest_e4m3(held * (s / new)[None, :, None]),
                               _nearest_e4m3(xf / new[None, :, None])])
        s = new
        for codes, scales in ((cache.k, cache.ks), (cache.v, cache.vs)):
            assert np.array_equal(_f64(scales[p]), s)
            assert np.array_equal(_f64(codes[p, :i + 1].float()), held)
    # a smaller token keeps the scale, and the same call again changes nothing
    # (a sequence cut back to 9 tokens goes on)
    x = rows[:, :1].contiguous()
    for _ in range(2):
        gqa.paged_append(x, x, pos, cache.k, cache.v, cache.table, _int([9]), **cache.scales())
        gqa.check()
        held[8] = _nearest_e4m3(_f64(x[0, 0].float()) / s[:, None])
        assert np.array_equal(_f64(cache.ks[p]), s)
        assert np.array_equal(_f64(cache.k[p].float()), held)


def test_infinities_saturate_and_nan_stays(cuda_device):
    page = 16
    x = torch.ones(1, page, 8, 64)
    x[0, 2, 0, 3], x[0, 3, 0, 4], x[0, 4, 1, 5] = float("inf"), float("-inf"), float("nan")
    x[0, :, 2] = float("nan")
    x = x.to(torch.bfloat16).cuda()
    pos = torch.zeros(1, page, dtype=torch.int32, device="cuda")
    cache = Cache([page], page, E4M3, stale=0.0)
    gqa.paged_append(x, x, pos, cache.k, cache.v, cache.table, _int([page]), **cache.scales())
    gqa.check()
    p = int(cache.table_host[0, 0])
    codes = cache.v[p].float().cpu()
    assert cache.vs[p, :2].tolist() == [2.0 ** -8] * 2 and float(cache.vs[p, 2]) == 2.0 ** -64
    assert float(codes[2, 0, 3]) == 448 and float(codes[3, 0, 4]) == -448
    assert bool(torch.isnan(codes[4, 1, 5])) and bool(torch.isnan(codes[:, 2]).all())
    assert int(torch.isnan(codes).sum()) == 1 + page * 64
    assert float(codes[0, 0, 0]) == 256
    bf = Cache([page], page, torch.bfloat16, stale=0.0)
    gqa.paged_append(x, x, pos, bf.k, bf.v, bf.table, _int([page]))
    gqa.check()
    assert torch.equal(bf.v[int(bf.table_host[0, 0])].view(torch.int16), x[0].view(torch.int16))


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
def test_append_reports_what_it_skips(cuda_device, dtype):
    """A page number or a length out of range is reported; nothing is written for it."""
    page = 16
    k = torch.ones(3, 4, 8, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    cases = [(dict(lengths=[4, 33, 4]), -11), (dict(lengths=[4, 3, 4]), -11),
             (dict(lengths=[4, -2 ** 31, 4]), -11), (dict(counts=[4, 5, 4]), -11),
             (dict(counts=[4, -1, 4]), -11), (dict(page=6), -12), (dict(page=-1), -12),
             (dict(page=2 ** 31 - 1), -12)]
    for change, status in cases:
        cache = Cache([32, 32, 32], page, dtype, spare=0, stale=0.0)
        table = cache.table_host.clone()
        if "page" in change:
            table[1, 0] = change["page"]
        counts = change.get("counts")
        gqa.paged_append(k, k, pos, cache.k, cache.v, table.cuda(),
                         _int(change.get("lengths", [4, 4, 4])),
                         counts=None if counts is None else _int(counts), **cache.scales())
        with pytest.raises(gqa.GptossAttnError) as e:
            gqa.check()
        assert e.value.status == status, change
        gqa.check()
        written = (cache.v.float() != 0).flatten(1).any(dim=1).cpu()
        assert sorted(torch.nonzero(written).flatten().tolist()) == sorted(
            [int(cache.table_host[0, 0]), int(cache.table_host[2, 0])]), change
    # a position out of the table is clamped and reported, as in the other entry points
    cache = Cache([4, 4, 4], page, dtype)
    bad = pos.clone()
    bad[1, 2] = 131072
    gqa.paged_append(k, k, bad, cache.k, cache.v, cache.table, _int([4, 4, 4]), **cache.scales())
    with pytest.raises(gqa.GptossAttnError) as e:
        gqa.check()
    assert e.value.status == -10


# -------------------------------------------------------------------- attention

@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("n,window,layout", [(1, 0, "token"), (1, 128, "head"), (2, 5, "both"),
                                             (3, 0, "head"), (4, 100, "token"), (9, 0, "both"),
                                             (6, 1, "token")])
def test_attention_ragged(cuda_device, page, dtype, n, window, layout):
    """Empty, shorter than n, one key, tile and page borders; stale slots hold NaN, and
    entries past a sequence's pages are unset."""
    lengths = [0, 1, 2, 63, 64, 65, 127, 128, 129, 300, 517]
    g = torch.Generator().manual_seed(10 * n + page)
    cache = Cache(lengths, page, dtype, layout, seed=page + n)
    cache.fill(lengths, g, spread=0.7)
    q, sinks = _queries(len(lengths), n, g)
    out = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int(lengths),
                              window=window, **cache.scales())
    gqa.check()
    _check_attention(out, cache, q, sinks, lengths, window)


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("n,lengths", [(1, [3000]), (1, [1] * 3 + [6000]), (5, [2500, 40]),
                                       (70, [700, 70, 69])])
def test_attention_split(cuda_device, dtype, n, lengths):
    """Sequences cut into many chunks, beside short ones; YaRN and given positions."""
    g = torch.Generator().manual_seed(n)
    cache = Cache(lengths, 64, dtype, seed=n, max_pages=max(lengths) // 64 + 40)
    cache.fill(lengths, g, spread=0.5)
    q, sinks = _queries(len(lengths), n, g)
    for window, rope in ((0, "plain"), (1000, "yarn")):
        out = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int(lengths),
                                  window=window, rope=rope, **cache.scales())
        gqa.check()
        _check_attention(out, cache, q, sinks, lengths, window, rope)
    pos = torch.randint(0, 131072, (len(lengths), n), generator=g, dtype=torch.int32)
    out = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int(lengths),
                              pos=pos.cuda(), **cache.scales())
    gqa.check()
    _check_attention(out, cache, q, sinks, lengths, 0, pos=pos)


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("B,n", [(96, 1), (97, 1), (250, 2), (40, 70), (1030, 1), (520, 17)])
def test_attention_of_many_rows(cuda_device, dtype, B, n):
    """Around the counts of rows at which the work is planned in another way, with a few long
    sequences among short ones; those, and some others, are looked at."""
    rng = np.random.default_rng(B + n)
    lengths = [int(x) for x in rng.integers(0, 30, B)]
    long = [0, B // 2, B - 1]
    for i, b in enumerate(long):
        lengths[b] = 2500 - 700 * i
    g = torch.Generator().manual_seed(B)
    cache = Cache(lengths, 64, dtype, seed=n)
    cache.fill(lengths, g)
    q, sinks = _queries(B, n, g)
    only = set(long) | {int(x) for x in rng.integers(0, B, 8)}
    for window in (0, 100):
        out = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int(lengths),
                                  window=window, **cache.scales())
        gqa.check()
        _check_attention(out, cache, q, sinks, lengths, window, only=only)
        assert all(not out[b].any() for b in range(B) if lengths[b] == 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 2, 16, 33])
@pytest.mark.parametrize("batch", [1, 7, 26, 30])
def test_attention_of_equal_and_unequal_rows_in_a_wave(cuda_device, dtype, n, batch):
    """Rows cut to one wave of chunks: every row alike, and one much longer than the others."""
    g = torch.Generator().manual_seed(batch)
    for lengths in ([1300] * batch, [3900] + [150] * (batch - 1)):
        cache = Cache(lengths, 128, dtype, seed=n)
        cache.fill(lengths, g)
        q, sinks = _queries(batch, n, g)
        out = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int(lengths),
                                  **cache.scales())
        gqa.check()
        _check_attention(out, cache, q, sinks, lengths, 0, only={0, batch - 1})


def test_attention_matches_contiguous_decode(cuda_device):
    """The same keys and values through decode(), single token."""
    B, L, page = 5, 1000, 64
    lengths = [1000, 999, 64, 1, 0]
    g = torch.Generator().manual_seed(4)
    cache = Cache([L] * B, page, torch.bfloat16, spare=0)
    cache.fill([L] * B, g)
    q, sinks = _queries(B, 1, g)
    table = cache.table.long()
    kc, vc = (x[table].reshape(B, -1, 8, 64)[:, :L].contiguous() for x in (cache.k, cache.v))
    for window in (0, 128):
        a = gqa.paged_attention(q[:, 0], cache.k, cache.v, cache.table, sinks, _int(lengths),
                                window=window)
        b = gqa.decode(q[:, 0].contiguous(), kc, vc, sinks, _int(lengths), window)
        gqa.check()
        assert a.shape == b.shape
        assert float((a.float() - b.float()).abs().max()) <= 2e-2
        _check_attention(a, cache, q, sinks, lengths, window)


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
def test_masked_values_never_reach_the_output(cuda_device, dtype):
    """Keys and values of later tokens, of keys before the window, and of stale slots may
    be NaN: tokens that do not see them are not touched."""
    lengths, n, window, page = [200, 77], 5, 20, 32
    g = torch.Generator().manual_seed(2)
    cache = Cache(lengths, page, dtype)
    cache.fill(lengths, g)
    q, sinks = _queries(2, n, g)
    ref = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int(lengths),
                              window=window, **cache.scales())
    for b, length in enumerate(lengths):
        for i in (length - 1, length - n + 1 - window):  # the last token; one that only t = 0 sees
            p = int(cache.table_host[b, i // page])
            cache.k[p, i % page] = float("nan")
            cache.v[p, i % page] = float("nan")
    got = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int(lengths),
                              window=window, **cache.scales())
    gqa.check()
    assert torch.equal(got[:, 1:4], ref[:, 1:4])
    assert torch.isnan(got[:, 0].float()).all() and torch.isnan(got[:, 4].float()).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("n", [2, 20])
def test_infinite_and_nan_values_reach_only_what_sees_them(cuda_device, dtype, n):
    """Single elements of values, some in tiles that all tokens see and some not: an output
    element is infinite or NaN exactly where a token sees one in it."""
    length, window, page = 700, 300, 32
    g = torch.Generator().manual_seed(21)
    cache = Cache([length], page, dtype)
    cache.fill([length], g)
    q, sinks = _queries(1, n, g)
    ref = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int([length]),
                              window=window, **cache.scales())
    hits = [(length - 1, 0, 5), (length - n // 2 - 1, 3, 40), (length - 150, 6, 63),
            (length - n - window + 2, 1, 7), (length - n - window, 2, 2), (0, 4, 4)]
    bad = float("inf") if dtype == torch.bfloat16 else float("nan")
    want = torch.zeros(n, 64, 64, dtype=torch.bool)
    for key, h, d in hits:
        cache.v[int(cache.table_host[0, key // page]), key % page, h, d] = bad
        for t in range(n):
            i = length - n + t
            if i - window < key <= i:
                want[t, 8 * h:8 * h + 8, d] = True
    got = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int([length]),
                              window=window, **cache.scales())
    gqa.check()
    assert torch.equal(~torch.isfinite(got[0].float().cpu()), want)
    keep = ~want.cuda()
    # a value row with such an element is added apart, with unrounded weights
    assert float((got[0].float() - ref[0].float())[keep].abs().max()) <= 2.0 ** -5


def test_pages_before_the_window_may_be_gone(cuda_device):
    lengths, page, window, n = [1000, 515], 16, 100, 3
    g = torch.Generator().manual_seed(3)
    for dtype in (torch.bfloat16, E4M3):
        cache = Cache(lengths, page, dtype)
        cache.fill(lengths, g)
        q, sinks = _queries(2, n, g)
        table = cache.table_host.clone()
        for b, length in enumerate(lengths):
            table[b, :(length - n + 1 - window) // page] = -7
        out = gqa.paged_attention(q, cache.k, cache.v, table.cuda(), sinks, _int(lengths),
                                  window=window, **cache.scales())
        gqa.check()
        _check_attention(out, cache, q, sinks, lengths, window)


def test_extreme_scales_and_sinks(cuda_device):
    """Value scales from 2^-60 to 2^60 across pages: what is large decides, whatever its
    page's scale; a sink of -inf and one far above the scores."""
    page, L = 16, 160
    g = torch.Generator().manual_seed(6)
    cache = Cache([L], page, E4M3)
    cache.fill([L], g)
    q, sinks = _queries(1, 2, g)
    sinks[:8] = float("-inf")
    sinks[8:16] = 60.0
    for exps in ([0] * 9 + [60], [60] + [0] * 9, [-60] * 10, list(range(-60, 60, 12))):
        for i, e in enumerate(exps):
            cache.vs[int(cache.table_host[0, i])] = 2.0 ** e
        out = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int([L]),
                                  **cache.scales())
        gqa.check()
        _check_attention(out, cache, q, sinks, [L], 0)
    # scales that are no powers of two (another program's)
    cache.vs.uniform_(0.01, 0.02)
    cache.ks.mul_(1.37)
    out = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int([L]), **cache.scales())
    gqa.check()
    _check_attention(out, cache, q, sinks, [L], 0)


def test_large_scores_keep_the_softmax(cuda_device):
    """Scores in the hundreds, rising along the sequence, so that the running maximum moves
    in every tile; the tolerance's S grows with them, so this checks the leading weight."""
    L, page = 640, 64
    for dtype in (torch.bfloat16, E4M3):
        cache = Cache([L], page, dtype, stale=0.0)
        k = torch.zeros(1, L, 8, 64)
        k[:, :, :, 31] = torch.arange(L)[None, :, None] * 0.5  # the slowest pair barely turns
        v = torch.randn(1, L, 8, 64, generator=torch.Generator().manual_seed(1))
        zero = torch.zeros(1, L, dtype=torch.int32, device="cuda")
        gqa.paged_append(k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), zero, cache.k,
                         cache.v, cache.table, _int([L]), **cache.scales())
        q = torch.zeros(1, 1, 64, 64, dtype=torch.bfloat16, device="cuda")
        q[:, :, :, 31] = 16.0
        sinks = torch.zeros(64, device="cuda")
        out = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int([L]),
                                  pos=torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                                  **cache.scales())
        gqa.check()
        kf, vf = cache.sequence(0, L)
        ref, _, _ = _attend(_f64(q[0, 0].float()), kf, vf, np.zeros(64), L - 1, 0)
        # scores here are exact products of 16 and a code (or bf16), so only the
        # output's rounding and the weights' (2^-11) are left
        assert np.all(np.abs(dev_to_f64(out)[0, 0] - ref) <= 2.0 ** -8 * np.abs(ref) + 4 * 2.0 ** -10)


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
def test_attention_reports_bad_lengths_and_pages(cuda_device, dtype):
    page, L = 16, 64
    g = torch.Generator().manual_seed(9)
    cache = Cache([L, L], page, dtype)
    cache.fill([L, L], g)
    q, sinks = _queries(2, 1, g)
    good = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int([L, L]), **cache.scales())
    gqa.check()
    for lengths, status, same in (([L, L + 1], -11, True), ([L, -1], -11, False)):
        out = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int(lengths),
                                  **cache.scales())
        with pytest.raises(gqa.GptossAttnError) as e:
            gqa.check()
        assert e.value.status == status
        assert torch.equal(out[0], good[0])
        assert torch.equal(out[1], good[1] if same else torch.zeros_like(out[1]))
    for bad in (-1, cache.num, 2 ** 31 - 1, -2 ** 31):
        table = cache.table_host.clone()
        table[1, 2] = bad
        out = gqa.paged_attention(q, cache.k, cache.v, table.cuda(), sinks, _int([L, L]),
                                  **cache.scales())
        with pytest.raises(gqa.GptossAttnError) as e:
            gqa.check()
        assert e.value.status == -12
        assert torch.equal(out[0], good[0]) and torch.isfinite(out[1].float()).all()
    gqa.check()


@pytest.mark.parametrize("n", [1, 4])
def test_attention_canaries_and_repeat(cuda_device, n):
    """Nothing outside workspace and output is written; the workspace needs no
    initialisation, and the same call gives the same bits."""
    lengths = [3000, 20, 700]
    g = torch.Generator().manual_seed(11)
    cache = Cache(lengths, 32, torch.bfloat16)
    cache.fill(lengths, g)
    q, sinks = _queries(3, n, g)
    need = gqa.paged_attention_workspace_bytes(3, n, cache.table.shape[1] * 32)
    assert need > 0
    ws = torch.full((need + 8192,), 0xFF, dtype=torch.uint8, device="cuda")
    buf = torch.full((3 * n * 4096 + 2048,), 2.5, dtype=torch.bfloat16, device="cuda")
    out = buf[1024:1024 + 3 * n * 4096].view(3, n, 64, 64)
    gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int(lengths), out=out,
                        workspace=ws[4096:4096 + need])
    gqa.check()
    assert torch.all(ws[:4096] == 0xFF) and torch.all(ws[4096 + need:] == 0xFF)
    assert torch.all(buf[:1024] == 2.5) and torch.all(buf[1024 + 3 * n * 4096:] == 2.5)
    _check_attention(out, cache, q, sinks, lengths, 0)
    again = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int(lengths),
                                workspace=ws[4096:4096 + need])
    assert torch.equal(again, out)


def test_queries_from_a_fused_projection(cuda_device):
    g = torch.Generator().manual_seed(12)
    lengths = [100, 3]
    cache = Cache(lengths, 16, E4M3)
    cache.fill(lengths, g)
    qkv = torch.randn(2, 3, 80, 64, generator=g).to(torch.bfloat16).cuda()
    sinks = torch.randn(64, generator=g).cuda()
    a = gqa.paged_attention(qkv[:, :, :64], cache.k, cache.v, cache.table, sinks, _int(lengths),
                            **cache.scales())
    b = gqa.paged_attention(qkv[:, :, :64].contiguous(), cache.k, cache.v, cache.table, sinks,
                            _int(lengths), **cache.scales())
    gqa.check()
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
def test_pages_past_32_bits(cuda_device, dtype):
    """Pages whose offsets in elements and bytes do not fit 32 bits."""
    page = 128
    num = (1 << 32) // (page * 512) + 40  # elements pass 2^32
    k = torch.empty(num, page, 8, 64, dtype=dtype, device="cuda")
    v = torch.empty(num, page, 8, 64, dtype=dtype, device="cuda")
    sc = {}
    if dtype == E4M3:
        sc = dict(kscales=torch.zeros(num, 8, device="cuda"), vscales=torch.zeros(num, 8, device="cuda"))
    L = 300
    ids = [num - 1, (1 << 31) // (page * 512), num - 7]
    table = _int([ids])
    g = torch.Generator().manual_seed(13)
    kk = torch.randn(1, L, 8, 64, generator=g).to(torch.bfloat16).cuda()
    vv = torch.randn(1, L, 8, 64, generator=g).to(torch.bfloat16).cuda()
    pos = _int([list(range(L))])
    gqa.paged_append(kk, vv, pos, k, v, table, _int([L]), **sc)
    q, sinks = _queries(1, 1, g)
    out = gqa.paged_attention(q, k, v, table, sinks, _int([L]), **sc)
    gqa.check()
    small = Cache([L], page, dtype)
    small.k = k[torch.tensor(ids)]
    small.v = v[torch.tensor(ids)]
    small.table_host = torch.arange(3, dtype=torch.int32)[None]
    if dtype == E4M3:
        small.ks, small.vs = sc["kscales"][torch.tensor(ids)], sc["vscales"][torch.tensor(ids)]
    else:
        assert torch.equal(small.v.reshape(-1, 8, 64)[:L], vv[0])
    _check_attention(out, small, q, sinks, [L], 0)
    del k, v
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ used together

@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("rope", ["plain", "yarn"])
def test_a_conversation(cuda_device, dtype, rope):
    """A prompt in pieces, decode steps, drafts that are cut back, and the window's layer:
    every output against attention over what the cache holds, and (bf16) against one
    prefill of the whole sequence."""
    B, S, page = 3, 300, 32
    g = torch.Generator().manual_seed(14)
    q, sinks = _queries(B, S, g)
    k = torch.randn(B, S, 8, 64, generator=g).to(torch.bfloat16).cuda()
    v = torch.randn(B, S, 8, 64, generator=g).to(torch.bfloat16).cuda()
    pos = _int([list(range(S))] * B)
    cache = Cache([S] * B, page, dtype)
    junk = torch.randn(B, 3, 8, 64, generator=g).to(torch.bfloat16).cuda()
    outs = {0: [], 128: []}
    cuts = [0, 101, 250, 251, 252, 256, 299, 300]
    for a, z in zip(cuts[:-1], cuts[1:]):
        args = (pos[:, a:z].contiguous(), cache.k, cache.v, cache.table)
        if z - a == 1 and z + 2 <= S:  # drafts behind the token, rejected
            three = torch.cat([k[:, a:z], junk[:, :2]], dim=1).contiguous()
            gqa.paged_append(three, three, pos[:, a:a + 3].contiguous(), *args[1:],
                             _int([a + 3] * B), rope=rope, **cache.scales())
        gqa.paged_append(k[:, a:z], v[:, a:z], *args, _int([z] * B), rope=rope, **cache.scales())
        for window, res in outs.items():
            res.append(gqa.paged_attention(q[:, a:z], cache.k, cache.v, cache.table, sinks,
                                           _int([z] * B), window=window, rope=rope,
                                           **cache.scales()))
    gqa.check()
    for window, res in outs.items():
        if dtype == torch.bfloat16:
            _check_attention(torch.cat(res, dim=1), cache, q, sinks, [S] * B, window, rope)
            whole = gqa.prefill(q, k, v, sinks, pos, window, rope=rope)
            gqa.check()
            assert float((torch.cat(res, dim=1).float() - whole.float()).abs().max()) <= 4e-2
        else:  # codes of a page may move when it grows, so the last piece is what the cache holds
            _check_attention(res[-1], cache, q[:, 299:], sinks, [S] * B, window, rope)


def test_a_captured_step_is_replayed(cuda_device):
    """Append and attention of one decode step in a CUDA graph, replayed while the
    lengths on the device grow; a second graph over the same pages has its own workspace."""
    gqa.init()
    B, page, L0, steps = 4, 16, 60, 9
    g = torch.Generator().manual_seed(15)
    for dtype in (torch.bfloat16, E4M3):
        cache = Cache([L0 + steps] * B, page, dtype, seed=2)
        eager = Cache([L0 + steps] * B, page, dtype, seed=2)
        state = g.get_state()
        cache.fill([L0] * B, g)
        g.set_state(state)
        eager.fill([L0] * B, g)
        q, sinks = _queries(B, steps, g)
        k = torch.randn(B, steps, 8, 64, generator=g).to(torch.bfloat16).cuda()
        v = torch.randn(B, steps, 8, 64, generator=g).to(torch.bfloat16).cuda()
        sq, sk, sv = (torch.zeros(B, 1, h, 64, dtype=torch.bfloat16, device="cuda")
                      for h in (64, 8, 8))
        ln, sp = _int([L0] * B), torch.zeros(B, 1, dtype=torch.int32, device="cuda")
        side = torch.cuda.Stream()

        def step(c, window):
            gqa.paged_append(sk, sv, sp, c.k, c.v, c.table, ln, **c.scales())
            return gqa.paged_attention(sq, c.k, c.v, c.table, sinks, ln, window=window, **c.scales())
        graphs = []
        with torch.cuda.stream(side):
            for window in (0, 30):
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    ln_out = step(cache, window)
                graphs.append((graph, ln_out, window))
        torch.cuda.synchronize()
        for t in range(steps):
            sq.copy_(q[:, t:t + 1])
            sk.copy_(k[:, t:t + 1])
            sv.copy_(v[:, t:t + 1])
            ln.fill_(L0 + t + 1)
            sp.fill_(L0 + t)
            for graph, out, window in graphs:
                graph.replay()
                want = step(eager, window)
                assert torch.equal(out, want)
        gqa.check()
        assert _same_bits(cache.k[cache.table.long()], eager.k[eager.table.long()])
        for graph, _, _ in graphs:
            graph.reset()


def test_two_streams_at_once(cuda_device):
    """Calls on two streams, each with its own pages and workspace, interleaved."""
    g = torch.Generator().manual_seed(16)
    streams = [torch.cuda.Stream() for _ in range(2)]
    runs = []
    for i, s in enumerate(streams):
        lengths = [900 + 100 * i, 10]
        cache = Cache(lengths, 32, E4M3 if i else torch.bfloat16, seed=i)
        cache.fill(lengths, g)
        runs.append((cache, lengths, _int(lengths), *_queries(2, 1, g)))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            cache, _, ln, q, sinks = runs[i]
            outs[i].append(gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, ln,
                                               stream=s, **cache.scales()))
    for i, s in enumerate(streams):
        gqa.check(s)
        cache, lengths, _, q, sinks = runs[i]
        _check_attention(outs[i][0], cache, q, sinks, lengths, 0)
        assert all(torch.equal(o, outs[i][0]) for o in outs[i][1:])


def test_another_stream_takes_no_memory_that_the_current_one_still_writes(cuda_device):
    g = torch.Generator().manual_seed(19)
    lengths = [2000] * 8
    cache = Cache(lengths, 64, torch.bfloat16)
    cache.fill(lengths, g)
    q, sinks = _queries(8, 1, g)
    ln, other = _int(lengths), torch.cuda.Stream()
    want = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, ln)
    need = gqa.paged_attention_workspace_bytes(8, 1, cache.table.shape[1] * 64)
    a = torch.zeros(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for _ in range(40):  # tens of milliseconds of the current stream
        a = a @ a
    given_back = [torch.empty(x, dtype=torch.bfloat16, device="cuda")
                  for x in (q.shape, (need // 2,))]
    for x in given_back:
        x.fill_(float("nan"))
    del x, given_back
    out = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, ln, stream=other)
    torch.cuda.synchronize()
    gqa.check(other)
    assert torch.equal(out, want)


def test_paged_attention_skips_work_while_a_timeout_is_pending(cuda_device):
    lib = gqa._load()
    g = torch.Generator().manual_seed(17)
    cache = Cache([700], 16, torch.bfloat16)
    cache.fill([700], g)
    q, sinks = _queries(1, 1, g)
    stream = torch.cuda.current_stream().cuda_stream
    gqa.check()
    assert lib.gptoss_attn_debug_wait_timeout(1000, stream) == 0
    out = torch.full((1, 1, 64, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int([700]), out=out)
    assert lib.gptoss_attn_check(stream) == -9
    assert torch.isnan(out.float()).all()
    gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int([700]), out=out)
    gqa.check()
    _check_attention(out, cache, q, sinks, [700], 0)


def test_shared_prefix_pages(cuda_device):
    """Two sequences whose first pages are the same ones."""
    page, g = 16, torch.Generator().manual_seed(18)
    cache = Cache([80, 70], page, torch.bfloat16)
    cache.table_host[1, :3] = cache.table_host[0, :3]
    cache.table = cache.table_host.cuda()
    cache.fill([80, 70], g)
    cache.fill([80, 0], g)
    q, sinks = _queries(2, 2, g)
    out = gqa.paged_attention(q, cache.k, cache.v, cache.table, sinks, _int([80, 70]))
    gqa.check()
    _check_attention(out, cache, q, sinks, [80, 70], 0)
