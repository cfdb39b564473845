"""The paged cache's host side, without a GPU: the arithmetic that host and kernels
share (csrc/paged.h, compiled here as plain C++), and the refusals of the C entry
points and of the Python binding."""
import ctypes
import os
import random
import subprocess
from fractions import Fraction

import numpy as np
import pytest
import torch

import attention_gqa_b200 as gqa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "attention_gqa_b200", "csrc")

SHIM = """
#include "paged.h"
using namespace gqa;
extern "C" {
void row_range(int len, int n, int t0, int nt, int w, int* out) {
  paged_row_range(len, n, t0, nt, w, out, out + 1);
}
int row_tiles(int lo, int hi, int tile) { return paged_row_tiles(lo, hi, tile); }
int chunk_tiles(long long total, int target) { return paged_chunk_tiles(total, target); }
int row_chunks(int tiles, int chunk) { return paged_row_chunks(tiles, chunk); }
long long max_chunks(long long rows, int most, int target) { return paged_max_chunks(rows, most, target); }
long long max_parts(int target) { return paged_max_parts(target); }
int longer_chunk(int chunk, int count, int wave) { return paged_longer_chunk(chunk, count, wave); }
long long estimate(long long total, int count, int longest, int wave, int cut) {
  return paged_estimate(total, count, longest, wave, cut);
}
int none_cut(long long rows, int most) { return paged_none_cut(rows, most); }
void chunk_range(int tiles, int chunks, int i, int* out) {
  paged_chunk_range(tiles, chunks, i, out, out + 1);
}
int page_ok(int page, int num) { return paged_page_ok(page, num); }
int append_ok(int len, int count, int n, int max_len) { return paged_append_ok(len, count, n, max_len); }
unsigned scale_bits(unsigned bits) { return paged_scale_bits(bits); }
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    d = tmp_path_factory.mktemp("paged")
    src, so = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o",
                    str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.max_chunks.restype = lib.max_parts.restype = lib.estimate.restype = ctypes.c_longlong
    lib.estimate.argtypes = [ctypes.c_longlong] + 4 * [ctypes.c_int]
    lib.none_cut.argtypes = [ctypes.c_longlong, ctypes.c_int]
    lib.max_chunks.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_int]
    lib.chunk_tiles.argtypes = [ctypes.c_longlong, ctypes.c_int]
    lib.scale_bits.restype = ctypes.c_uint
    lib.scale_bits.argtypes = [ctypes.c_uint]
    return lib


def _pair(fn, *args):
    out = (ctypes.c_int * 2)()
    fn(*args, out)
    return out[0], out[1]


def test_row_range_is_the_union_of_its_tokens_keys(host):
    rng = random.Random(1)
    for _ in range(3000):
        n, nt = rng.randint(1, 40), rng.choice((1, 2, 4, 16))
        length, w = rng.randint(0, 60), rng.choice((0, 0, 1, 2, 5, 39))
        t0 = rng.randrange(0, n, nt)
        seen = set()
        for t in range(t0, min(t0 + nt, n)):
            i = length - n + t
            seen |= {j for j in range(0, i + 1) if w == 0 or j > i - w}
        lo, hi = _pair(host.row_range, length, n, t0, nt, w)
        assert 0 <= lo and hi <= length
        if seen:
            assert (lo, hi) == (min(seen), max(seen) + 1)
        else:
            assert hi <= lo
    # the largest sizes do not overflow
    assert _pair(host.row_range, 131072, 1, 0, 1, 131071) == (1, 131072)
    assert _pair(host.row_range, 0, 131072, 131068, 4, 131071) == (0, 0)


def test_tiles_cover_a_range(host):
    for lo in (0, 1, 63, 64, 65, 200):
        for hi in range(lo - 2, lo + 200, 7):
            for tile in (64, 128):
                tiles = {j // tile for j in range(lo, hi)}
                assert host.row_tiles(lo, hi, tile) == len(tiles)


@pytest.mark.parametrize("target", [37, 222])
def test_chunks_cover_every_tile_once_within_the_grid_and_the_workspace(host, target):
    rng = random.Random(target)
    batches = [[0], [1], [8], [8, 9], [9] * 64, [0, 0, 0], [2048], [2048] * 64, [1] * 4000, [128] * 64, [129] * 64,
               [4, 5] * 30]
    for _ in range(400):
        rows = rng.choice((1, 2, 7, 64, 300))
        batches.append([int(2 ** rng.uniform(0, 11)) - 1 for _ in range(rows)])
    for tiles in batches:
        c = host.chunk_tiles(sum(tiles), target)
        assert c >= 1
        chunks = parts = 0
        for t in tiles:
            n = host.row_chunks(t, c)
            chunks += n
            parts += n if n > 1 else 0
            at = 0
            for i in range(n):
                a, b = _pair(host.chunk_range, t, n, i)
                assert a == at and b >= a and (b - a <= c or n == 1)
                at = b
            assert at == t
        for most in (max(tiles), max(tiles) + 1, 2048):
            assert chunks <= host.max_chunks(len(tiles), most, target)
        assert parts <= host.max_parts(target)


@pytest.mark.parametrize("wave", [37, 55, 74])
def test_few_rows_are_cut_to_one_wave(host, wave):
    """Chunks grow until they fit, in a few steps, and are no longer than they have to be but
    for the rounding of the rows' own divisions."""
    rng = random.Random(wave)
    for _ in range(500):
        rows = rng.randint(1, 3 * wave // 4)
        tiles = [int(2 ** rng.uniform(0, 11)) for _ in range(rows)]
        if rng.random() < 0.3:
            tiles = [tiles[0]] * rows
        c = first = host.chunk_tiles(sum(tiles), wave)
        count = sum(host.row_chunks(t, c) for t in tiles)
        steps = 0
        while count > wave:
            longer = host.longer_chunk(c, count, wave)
            assert longer > c
            c, steps = longer, steps + 1
            count = sum(host.row_chunks(t, c) for t in tiles)
        assert steps < 40 and c <= max(first, 2 * max(tiles))
        assert count <= host.max_chunks(rows, max(tiles), wave)
        assert sum(n for t in tiles if (n := host.row_chunks(t, c)) > 1) <= wave


def test_estimates_order_the_cuts_as_they_were_measured(host):
    def time(tiles, chunk):
        n = [host.row_chunks(t, chunk) for t in tiles]
        longest = max(-(-t // k) for t, k in zip(tiles, n))
        return host.estimate(sum(tiles), sum(n), longest, 37, max(n) > 1)
    whole = 2 ** 31 - 1
    for tiles in ([64] * 36, [36] * 32, [64] * 64):
        assert time(tiles, whole) <= time(tiles, host.chunk_tiles(sum(tiles), 55))  # ties: whole
    ragged = [64 * i // 36 for i in range(1, 37)]
    for tiles in (ragged, [256] * 24, [32] * 3 + [5] * 40):
        assert time(tiles, whole) > time(tiles, host.chunk_tiles(sum(tiles), 55))


def test_none_is_cut_of_short_or_very_many_rows(host):
    assert host.none_cut(1, 8) and not host.none_cut(1, 9)
    assert not host.none_cut(1023, 9) and host.none_cut(1024, 2048)
    assert host.max_chunks(1024, 2048, 111) == 1024


def test_scale_is_the_least_power_of_two_that_holds_the_value(host):
    rng = np.random.default_rng(3)
    values = [0.0, 2.0 ** -149, 2.0 ** -126, 448.0, np.nextafter(np.float32(448), np.float32(500)),
              1.75, 1.7500001, 2.0, 3.3895314e38, np.finfo(np.float32).max, 448 * 2.0 ** -64,
              448 * 2.0 ** -65, 1.0]
    values += list(np.exp(rng.uniform(-80, 80, 3000)))
    for v in np.array(values, dtype=np.float32):
        bits = int(v.view(np.uint32))
        s = np.uint32(host.scale_bits(bits)).view(np.float32)
        mantissa, e = np.frexp(s)
        assert mantissa == 0.5 and -64 <= e - 1 <= 120
        e = int(e) - 1
        x = Fraction(float(v))
        assert x <= 448 * Fraction(2) ** e or e == 120
        assert e == -64 or x > 448 * Fraction(2) ** (e - 1)


def test_page_and_append_bounds(host):
    assert [host.page_ok(p, 5) for p in (-2 ** 31, -1, 0, 4, 5, 2 ** 31 - 1)] == [0, 0, 1, 1, 0, 0]
    ok = [(0, 0, 1), (1, 1, 1), (100, 1, 1), (100, 100, 100), (100, 0, 7)]
    bad = [(-1, 0, 1), (0, 1, 1), (101, 1, 1), (50, -1, 3), (50, 4, 3), (-2 ** 31, -2 ** 31, 1)]
    assert all(host.append_ok(length, c, n, 100) for length, c, n in ok)
    assert not any(host.append_ok(length, c, n, 100) for length, c, n in bad)


# ------------------------------------------------------------------- C refusals

OK, NULL_PTR, BAD_SHAPE, BAD_ALIGN, SMALL = 0, -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    from attention_gqa_b200 import build
    build.build()
    return gqa._load()


def _cache(**kw):
    a = dict(k=16, v=32, k_scale=None, v_scale=None, page_stride=16 * 512, token_stride=512,
             head_stride=64, num_pages=4, page_size=16, type=0)
    a.update(kw)
    return gqa._PagedCache(**a)


BAD_CACHES = [
    (dict(k=None), NULL_PTR), (dict(v=None), NULL_PTR),
    (dict(type=1), NULL_PTR), (dict(type=1, k_scale=64), NULL_PTR),
    (dict(page_size=8), BAD_SHAPE), (dict(page_size=48), BAD_SHAPE), (dict(page_size=0), BAD_SHAPE),
    (dict(page_size=256), BAD_SHAPE), (dict(page_size=-16), BAD_SHAPE),
    (dict(num_pages=0), BAD_SHAPE), (dict(num_pages=-3), BAD_SHAPE), (dict(type=2), BAD_SHAPE),
    (dict(k_scale=64), BAD_SHAPE), (dict(page_stride=0), BAD_SHAPE),
    (dict(token_stride=-512), BAD_SHAPE), (dict(head_stride=8), BAD_SHAPE),
    (dict(page_stride=1 << 40), BAD_SHAPE), (dict(head_stride=68), BAD_ALIGN),
    (dict(type=1, k_scale=64, v_scale=64, token_stride=520), BAD_ALIGN),
    (dict(k=24), BAD_ALIGN), (dict(v=40), BAD_ALIGN),
    (dict(type=1, k_scale=66, v_scale=64), BAD_ALIGN),
]


@pytest.mark.parametrize("change,want", BAD_CACHES)
def test_both_entry_points_refuse_a_bad_cache(lib, change, want):
    assert _append(lib, cache=_cache(**change)) == want
    assert _attention(lib, cache=_cache(**change)) == want


def _append(lib, cache=None, fn="gptoss_attn_paged_append", **kw):
    a = dict(k=16, v=32, kb=512, kt=512, vb=512, vt=512, pos=64, table=80, len=96, count=None,
             batch=2, n=3, max_pages=4)
    a.update(kw)
    return getattr(lib, fn)(cache if cache is not None else _cache(), a["k"], a["v"], a["kb"],
                            a["kt"], a["vb"], a["vt"], a["pos"], a["table"], a["len"], a["count"],
                            a["batch"], a["n"], a["max_pages"], None)


def _attention(lib, cache=None, fn="gptoss_attn_paged_attention", **kw):
    a = dict(q=16, qb=4096, qt=4096, pos=None, table=80, sinks=64, len=96, window=0, out=112,
             batch=2, n=3, max_pages=80, ws=128, bytes=None)
    a.update(kw)
    if a["bytes"] is None:
        a["bytes"] = lib.gptoss_attn_paged_attention_workspace_bytes(
            a["batch"], a["n"], max(1, min(131072, a["max_pages"] * 16)), a["window"])
    return getattr(lib, fn)(cache if cache is not None else _cache(), a["q"], a["qb"], a["qt"],
                            a["pos"], a["table"], a["sinks"], a["len"], a["window"], a["out"],
                            a["batch"], a["n"], a["max_pages"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("fn", ["gptoss_attn_paged_append", "gptoss_attn_paged_append_yarn"])
def test_append_argument_errors(lib, fn):
    for name in ("k", "v", "pos", "table", "len"):
        assert _append(lib, fn=fn, **{name: None}) == NULL_PTR, name
    for change in (dict(batch=0), dict(batch=65536), dict(n=0), dict(n=131073), dict(max_pages=0),
                   dict(max_pages=8193), dict(max_pages=-1)):
        assert _append(lib, fn=fn, **change) == BAD_SHAPE, change
    for change in (dict(k=24), dict(v=24), dict(kt=516), dict(vb=4), dict(pos=66), dict(table=82),
                   dict(len=97), dict(count=98)):
        assert _append(lib, fn=fn, **change) == BAD_ALIGN, change


@pytest.mark.parametrize("fn", ["gptoss_attn_paged_attention", "gptoss_attn_paged_attention_yarn"])
def test_attention_argument_errors(lib, fn):
    for name in ("q", "table", "sinks", "len", "out", "ws"):
        assert _attention(lib, fn=fn, **{name: None}) == NULL_PTR, name
    for change in (dict(batch=0), dict(n=0), dict(batch=131073), dict(batch=2, n=65537),
                   dict(max_pages=0), dict(max_pages=8193)):
        assert _attention(lib, fn=fn, bytes=1 << 40, **change) == BAD_SHAPE, change
    for change in (dict(q=24), dict(out=120), dict(ws=136), dict(qt=4100), dict(pos=66),
                   dict(table=82), dict(sinks=65), dict(len=98)):
        assert _attention(lib, fn=fn, **change) == BAD_ALIGN, change
    need = lib.gptoss_attn_paged_attention_workspace_bytes(2, 3, 1280, 0)
    assert need > 0 and _attention(lib, fn=fn, bytes=need - 1) == SMALL


def test_attention_workspace_query(lib):
    ws = lib.gptoss_attn_paged_attention_workspace_bytes
    for batch, n in ((0, 1), (1, 0), (-1, 1), (1, -1), (131073, 1), (1, 131073), (512, 257)):
        assert ws(batch, n, 8192, 0) == 0
    for length in (0, -1, 131073):
        assert ws(1, 1, length, 0) == 0
    assert 0 < ws(1, 1, 8192, 0) <= ws(64, 1, 8192, 0) <= ws(131072, 1, 8192, 0)
    assert ws(64, 1, 8192, 0) == ws(64, 1, 131072, 0) < 16 << 20  # the chunks', not the cache's
    # none where no row of queries is cut: up to 8 tiles (of 64 keys; of 128 beyond two tokens)
    assert ws(64, 1, 512, 0) == 0 < ws(64, 1, 528, 0)
    assert ws(64, 1, 131072, 128) == 0 < ws(64, 1, 131072, 1000)
    assert ws(64, 3, 1024, 0) == 0 < ws(64, 3, 1040, 0)
    assert ws(64, 3, 131072, 128) == 0


# -------------------------------------------------------------- Python refusals

def _pages(dtype=torch.bfloat16, num=4, page=16):
    return torch.zeros(num, page, 8, 64, dtype=torch.uint8).to(dtype)


HOST = -1  # device index of host tensors


def test_binding_refuses_bad_pages():
    e4 = torch.float8_e4m3fn
    p, s = _pages(), torch.ones(4, 8)
    for args, kind in [
        ((_pages(torch.float32), p, None, None), TypeError),
        ((p, _pages(e4), None, None), TypeError),
        ((_pages(page=24), _pages(page=24), None, None), ValueError),
        ((p[0], p[0], None, None), ValueError),
        ((p[:, :, :4], p[:, :, :4], None, None), ValueError),
        ((p, _pages(num=5), None, None), ValueError),
        ((p, torch.zeros(4, 8, 16, 64, dtype=torch.bfloat16).transpose(1, 2), None, None), ValueError),
        ((p[..., ::2], p[..., ::2], None, None), ValueError),
        ((p, p, s, s), ValueError),
        ((_pages(e4), _pages(e4), None, s), ValueError),
        ((_pages(e4), _pages(e4), s, s[:3]), ValueError),
        ((_pages(e4), _pages(e4), s, s.double()), TypeError),
        ((_pages(e4), _pages(e4), s, torch.ones(8, 4).t()), ValueError),
    ]:
        with pytest.raises(kind):
            gqa._paged_cache(*args, HOST)
    with pytest.raises(ValueError, match="device"):
        gqa._paged_cache(p, p, None, None, 0)
    view = torch.zeros(4, 8, 16, 64, dtype=torch.bfloat16).transpose(1, 2)  # laid out by head
    c = gqa._paged_cache(view, view, None, None, HOST)
    assert (c.page_stride, c.token_stride, c.head_stride, c.page_size) == (8192, 64, 1024, 16)
    assert (c.num_pages, c.type, c.k_scale) == (4, 0, None)
    c = gqa._paged_cache(_pages(e4), _pages(e4), s, s, HOST)
    assert (c.type, c.k_scale, c.v_scale) == (1, s.data_ptr(), s.data_ptr())


def test_binding_refuses_bad_tokens():
    qkv = torch.zeros(2, 3, 80, 64, dtype=torch.bfloat16)
    assert gqa._heads_at(qkv[:, :, 64:72], 8, "k", HOST) == (2, 3, 3 * 80 * 64, 80 * 64)
    assert gqa._heads_at(qkv[:1, 1:2, :64], 64, "q", HOST) == (1, 1, 0, 0)
    for t, kind in ((qkv.float()[:, :, :8], TypeError), (qkv, ValueError), (qkv[0, :, :8], ValueError),
                    (qkv[:, :, :16:2], ValueError), (qkv[:, :, :8, :32], ValueError),
                    (torch.zeros(2, 3, 64, 8, dtype=torch.bfloat16).transpose(2, 3), ValueError)):
        with pytest.raises(kind):
            gqa._heads_at(t, 8, "k", HOST)
    with pytest.raises(ValueError, match="device"):
        gqa._heads_at(qkv[:, :, :8], 8, "k", 0)
    x = torch.zeros(2, dtype=torch.int32)
    assert gqa._array(x, torch.int32, (2,), "lengths", HOST) == x.data_ptr()
    for t, kind in ((x.long(), TypeError), (x[:1], ValueError), (x[:, None], ValueError),
                    (torch.zeros(4, dtype=torch.int32)[::2], ValueError)):
        with pytest.raises(kind):
            gqa._array(t, torch.int32, (2,), "lengths", HOST)
    with pytest.raises(ValueError, match="device"):
        gqa._array(x, torch.int32, (2,), "lengths", 0)


def test_binding_takes_device_tensors_only(monkeypatch):
    def no_library():
        raise AssertionError("the library was called")
    monkeypatch.setattr(gqa, "_load", no_library)
    k, p = torch.zeros(2, 3, 8, 64, dtype=torch.bfloat16), _pages()
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensors"):
        gqa.paged_append(k, k, i, p, p, i, i)
    with pytest.raises(ValueError, match="device tensors"):
        gqa.paged_attention(torch.zeros(2, 64, 64, dtype=torch.bfloat16), p, p, i, i, i)
