"""The paged key/value cache: appending to it and attending over it.

The cache is a pool of pages, each holding `page` tokens of one sequence (8 kv
heads of 64), found through a table of page numbers per sequence. Pages hold
bf16, or e4m3 with one fp32 power-of-two scale for each page and head.

`append`     rotates the new keys and writes keys and values to their pages
             (in 8 bits: choosing each page's scales, and moving the codes that
             a growing scale finds there);
`attention`  the n newest tokens of every sequence over its pages, with the
             sliding window and the per-head sink of the other entry points.

`lengths` counts a sequence's tokens with the new ones; token t of the n new
ones sits at index lengths - n + t, which is its rotary position too.
"""
import math

import torch

own = False

HEADS, KV, DIM = 64, 8, 64
GROUP = HEADS // KV
THETA = 150000.0
FACTOR, CONTEXT = 32.0, 4096.0  # YaRN
PAGES = (16, 32, 64, 128)
E4M3_MAX = 448.0
LOW, HIGH = -64, 120  # exponents that a scale may have


def listed():
    def append(name, kv, batch, n, length, page, ragged, rope, fused):
        return dict(name=name, op="append", kv=kv, batch=batch, n=n, length=length, page=page,
                    ragged=ragged, rope=rope, fused=fused, window=0)

    def attention(name, kv, batch, n, length, page, ragged, rope, window):
        return dict(name=name, op="attention", kv=kv, batch=batch, n=n, length=length, page=page,
                    ragged=ragged, rope=rope, fused=False, window=window)

    return [
        # one decode step of a batch: a token each, at any place of its page; latency
        append("append_step_bf16", "bf16", 64, 1, 1024, 16, True, "plain", False),
        # the prompts of a batch at once, read out of a fused qkv projection
        append("append_prompts_bf16", "bf16", 4, 16384, 16384, 64, False, "yarn", True),
        append("append_step_e4m3", "e4m3", 64, 1, 1024, 16, True, "plain", True),
        # the next pieces of prompts, of different lengths, starting inside pages
        append("append_pieces_e4m3", "e4m3", 7, 333, 1500, 32, True, "yarn", False),
        append("append_prompts_e4m3", "e4m3", 4, 16384, 16384, 64, False, "plain", False),
        # a single short conversation: latency
        attention("attention_one_bf16", "bf16", 1, 1, 257, 16, False, "plain", 0),
        # the decode step of a full batch
        attention("attention_batch_bf16", "bf16", 64, 1, 8192, 64, False, "plain", 0),
        # its sliding-window layers
        attention("attention_window_bf16", "bf16", 64, 1, 8192, 16, True, "plain", 128),
        # a question of 512 tokens asked on a prefix that is already cached
        attention("attention_piece_bf16", "bf16", 1, 512, 4608, 128, False, "yarn", 0),
        # one sequence at the model's longest context
        attention("attention_long_e4m3", "e4m3", 1, 1, 131072, 64, False, "yarn", 0),
        # a batch in which every conversation has its own length
        attention("attention_batch_e4m3", "e4m3", 64, 1, 8192, 32, True, "plain", 0),
        # drafted tokens looked at together with the last accepted one
        attention("attention_drafts_e4m3", "e4m3", 16, 5, 4001, 64, True, "yarn", 0),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("append", "attention", "attention"))
    batch = _log_uniform(rng, 1, 64)
    if op == "append":
        n = 1 if rng.random() < 0.3 else _log_uniform(rng, 1, min(16384, 65536 // batch))
        length = _log_uniform(rng, n, max(n, min(16384, 65536 // batch)))
    else:
        u = rng.random()
        n = 1 if u < 0.5 else rng.randint(2, 9) if u < 0.8 else _log_uniform(rng, 10, 512)
        length = _log_uniform(rng, n, max(n, min(131072, 524288 // batch, 2359296 // (batch * n))))
    window = rng.choice((0, 0, 128, _log_uniform(rng, 1, 4096))) if op == "attention" else 0
    return dict(op=op, kv=rng.choice(("bf16", "e4m3")), batch=batch, n=n, length=length,
                page=rng.choice(PAGES), ragged=rng.random() < 0.6,
                rope=rng.choice(("plain", "yarn")), fused=op == "append" and rng.random() < 0.5,
                window=window)


def _lengths(case):
    """(lengths, counts) of the case's sequences: the same for every seed."""
    B, n, L = case["batch"], case["n"], case["length"]
    if not case["ragged"]:
        return [L] * B, [n] * B
    part = [((b + 1) * 0.6180339887498949) % 1.0 for b in range(B)]
    part[0] = 1.0
    if case["op"] == "attention":
        return [n + int((L - n) * f) for f in part], [n] * B
    counts = [max(1, int(math.ceil(n * f))) for f in part]
    return [c + int((L - n) * f) for c, f in zip(counts, part)], counts


def _frequencies(rope):
    """(turns per token of the 32 pairs, factor on cos and sin), in 64 bits."""
    freq = [THETA ** (-2.0 * k / DIM) for k in range(DIM // 2)]
    if rope == "plain":
        return freq, 1.0

    def pair(turns):
        return DIM * math.log(CONTEXT / (turns * 2.0 * math.pi)) / (2.0 * math.log(THETA))
    lo, hi = max(pair(32.0), 0.0), min(pair(1.0), DIM - 1.0)
    ramp = [min(max((k - lo) / (hi - lo), 0.0), 1.0) for k in range(DIM // 2)]
    return ([w * f / FACTOR + (1.0 - w) * f for w, f in zip(ramp, freq)],
            0.1 * math.log(FACTOR) + 1.0)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    B, n, P = case["batch"], case["n"], case["page"]
    lengths, counts = _lengths(case)
    need = [-(-x // P) for x in lengths]
    width = max(need)
    pool = sum(need) + 3
    # pages in no order, each held by one sequence; entries past a sequence's pages are unset
    order = torch.randperm(pool, generator=gen, device=dev)[:sum(need)].to(torch.int32)
    held = torch.tensor([b * width + i for b in range(B) for i in range(need[b])], device=dev)
    table = torch.full((B * width,), -1, dtype=torch.int32, device=dev)
    table[held] = order
    freq, factor = _frequencies(case["rope"])
    s = dict(case=case, table=table.view(B, width),
             lengths=torch.tensor(lengths, dtype=torch.int32, device=dev),
             freq=torch.tensor(freq, dtype=torch.float64, device=dev), factor=factor)

    def pages():
        """A pool with what earlier tokens, or earlier owners, left there."""
        x = torch.randn(pool, P, KV, DIM, generator=gen, device=dev)
        if case["kv"] == "bf16":
            return x.to(torch.bfloat16), None
        # heads and pages differ in size; the largest value decides the scale
        x *= torch.exp(0.7 * torch.randn(pool, 1, KV, 1, generator=gen, device=dev))
        e = _exponent(x.abs().amax(dim=(1, 3)))
        return _to_e4m3(x, e[:, None, :, None]), _power(e)

    s["kpages"], s["kscales"] = pages()
    s["vpages"], s["vscales"] = pages()
    if case["op"] == "append":
        if case["fused"]:
            qkv = torch.randn(B, n, HEADS + 2 * KV, DIM, generator=gen, device=dev).to(torch.bfloat16)
            s["k"], s["v"] = qkv[:, :, HEADS:HEADS + KV], qkv[:, :, HEADS + KV:]
        else:
            s["k"] = torch.randn(B, n, KV, DIM, generator=gen, device=dev).to(torch.bfloat16)
            s["v"] = torch.randn(B, n, KV, DIM, generator=gen, device=dev).to(torch.bfloat16)
        s["counts"] = torch.tensor(counts, dtype=torch.int32, device=dev)
        first = s["lengths"] - s["counts"]
        s["pos"] = (first[:, None] + torch.arange(n, dtype=torch.int32, device=dev)).clamp_(max=131071)
        # what the host knows of the step: the new tokens, and the pages that they touch
        s["tokens"] = torch.tensor([b * n + t for b in range(B) for t in range(counts[b])], device=dev)
        starts = [x - c for x, c in zip(lengths, counts)]
        touched = [(b, i) for b in range(B) for i in range(starts[b] // P, need[b])]
        s["touched"] = torch.tensor(touched, device=dev)
    else:
        s["q"] = torch.randn(B, n, HEADS, DIM, generator=gen, device=dev).to(torch.bfloat16)
        s["sinks"] = torch.randn(HEADS, generator=gen, device=dev)
    return s


# ---------------------------------------------------------------- plain forms

def _exponent(largest):
    """The least e with largest <= 448 * 2^e, between LOW and HIGH."""
    m, x = torch.frexp(largest)  # largest = m * 2^x, 0.5 <= m < 1; 448 = 0.875 * 2^9
    return torch.where(largest > 0, x - 9 + (m > 0.875).to(x.dtype), torch.full_like(x, LOW)).clamp(LOW, HIGH)


def _power(e):
    """2^e in fp32, for whole e."""
    return ((e.clamp(min=-126).to(torch.int32) + 127) << 23).view(torch.float32)


def _to_e4m3(x, e):
    return (x * _power(-e)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _of_pages(pages, index):
    """pages[index] (through bytes, where the pages hold 8 bits)."""
    if pages.dtype == torch.float8_e4m3fn:
        return pages.view(torch.uint8)[index].view(pages.dtype)
    return pages[index]


def _rotated(x, angle, factor):
    """Half-split rotation in 64 bits; `angle` has x's shape without its heads, and 32 pairs."""
    c, s = torch.cos(angle)[..., None, :] * factor, torch.sin(angle)[..., None, :] * factor
    a, b = x[..., :DIM // 2].double(), x[..., DIM // 2:].double()
    return torch.cat((a * c - b * s, b * c + a * s), dim=-1)


def _plain_append(s):
    case, P, n = s["case"], s["case"]["page"], s["case"]["n"]
    k = _rotated(s["k"], s["pos"][..., None].double() * s["freq"], s["factor"])
    v = s["v"]
    at = (s["lengths"] - s["counts"])[:, None].long() + torch.arange(n, device=k.device)  # [B, n]
    if case["kv"] == "bf16":
        b, at = s["tokens"] // n, at.flatten()[s["tokens"]]
        row = s["table"][b, at // P].long() * P + at % P
        s["kpages"].view(-1, KV, DIM)[row] = k.flatten(0, 1)[s["tokens"]].to(torch.bfloat16)
        s["vpages"].view(-1, KV, DIM)[row] = v.flatten(0, 1)[s["tokens"]]
        return dict(k=s["kpages"], v=s["vpages"])
    # 8 bits: every touched page as a whole, [pages, P]
    b, i = s["touched"][:, 0], s["touched"][:, 1]
    page = s["table"][b, i].long()
    index = i[:, None] * P + torch.arange(P, device=k.device)
    start, end = (s["lengths"] - s["counts"]).long()[b][:, None], s["lengths"].long()[b][:, None]
    new, old = (index >= start) & (index < end), index < start
    token = (b[:, None] * n + (index - start).clamp(0, n - 1))
    for x, pages, scales in ((k, "kpages", "kscales"), (v, "vpages", "vscales")):
        rows = torch.where(new[..., None, None], x.reshape(-1, KV, DIM)[token].float(), 0.0)
        finite = torch.where(rows.isfinite(), rows.abs(), 0.0)
        e = _exponent(finite.amax(dim=(1, 3)))  # [pages, KV]
        _, before = torch.frexp(s[scales][page])
        before = torch.where(old.any(dim=1)[:, None], before - 1, torch.full_like(before, LOW))
        e = torch.maximum(e, before)
        there = _of_pages(s[pages], page).float()
        moved = _to_e4m3(there, (e - before)[:, None, :, None])
        made = torch.where(new[..., None, None], _to_e4m3(rows, e[:, None, :, None]).float(),
                           torch.where(old[..., None, None], moved.float(), there))
        s[pages].view(torch.uint8)[page] = made.to(torch.float8_e4m3fn).view(torch.uint8)
        s[scales][page] = _power(e)
    return dict(k=s["kpages"], v=s["vpages"], kscales=s["kscales"], vscales=s["vscales"])


def _plain_attention(s):
    case = s["case"]
    B, n, W = case["batch"], case["n"], case["window"]
    table = s["table"].clamp(min=0).long()
    L = table.shape[1] * case["page"]

    def gathered(pages, scales):
        x = _of_pages(pages, table).float()
        if scales is not None:
            x = x * scales[table][:, :, None, :, None]
        return x.reshape(B, L, KV, DIM).transpose(1, 2)  # [B, KV, L, DIM]

    at = s["lengths"][:, None].long() - n + torch.arange(n, device=table.device)  # [B, n]
    q = _rotated(s["q"], at[..., None].double() * s["freq"], s["factor"]).float()
    q = q.view(B, n, KV, GROUP, DIM).permute(0, 2, 1, 3, 4).reshape(B, KV, n * GROUP, DIM)
    x = torch.matmul(q, gathered(s["kpages"], s["kscales"]).transpose(2, 3)) * DIM ** -0.5
    x = x.view(B, KV, n, GROUP, L)
    key = torch.arange(L, device=table.device)
    seen = key <= at[..., None]
    if W > 0:
        seen &= key > at[..., None] - W
    x = x.masked_fill(~seen[:, None, :, None, :], float("-inf"))
    sink = s["sinks"].view(1, KV, 1, GROUP, 1)
    top = torch.maximum(x.amax(dim=-1, keepdim=True), sink)
    p = torch.exp(x - top)
    total = p.sum(dim=-1, keepdim=True) + torch.exp(sink - top)
    v = gathered(s["vpages"], s["vscales"])
    v = torch.where((key < s["lengths"][:, None])[:, None, :, None], v, 0.0)
    o = torch.matmul(p.view(B, KV, n * GROUP, L), v).view(B, KV, n, GROUP, DIM) / total
    return o.permute(0, 2, 1, 3, 4).reshape(B, n, HEADS, DIM).to(torch.bfloat16)


def run(s):
    case = s["case"]
    if own:
        import attention_gqa_b200 as gqa
        if case["op"] == "append":
            gqa.paged_append(s["k"], s["v"], s["pos"], s["kpages"], s["vpages"], s["table"],
                             s["lengths"], counts=s["counts"], kscales=s["kscales"],
                             vscales=s["vscales"], rope=case["rope"])
            if case["kv"] == "bf16":
                return dict(k=s["kpages"], v=s["vpages"])
            return dict(k=s["kpages"], v=s["vpages"], kscales=s["kscales"], vscales=s["vscales"])
        return gqa.paged_attention(s["q"], s["kpages"], s["vpages"], s["table"], s["sinks"],
                                   s["lengths"], window=case["window"], kscales=s["kscales"],
                                   vscales=s["vscales"], rope=case["rope"])
    return _plain_append(s) if case["op"] == "append" else _plain_attention(s)


# ------------------------------------------------------- by definition, 64 bits

def _turned(x, pos, freq, factor):
    """One token's heads [heads, 64] in 64 bits, each pair as a complex number."""
    z = torch.complex(x[:, :DIM // 2], x[:, DIM // 2:])
    z = z * torch.polar(torch.full_like(freq, factor), freq * float(pos))
    return torch.cat((z.real, z.imag), dim=1)


def _power64(e):
    """2^e in 64 bits, for whole e."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _nearest_e4m3(y):
    """64-bit values rounded to the nearest e4m3 value, ties to even, at most 448."""
    _, x = torch.frexp(y.abs().clamp(min=2.0 ** -6))  # 2^(x-1) <= |y| < 2^x
    step = _power64(x - 4)
    return (torch.round(y / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    lengths, counts = _lengths(case)
    P, n, W = case["page"], case["n"], case["window"]
    table = s["table"].tolist()
    if case["op"] == "append":
        out = {x: s[x + "pages"].double() for x in "kv"}
        scale = {x: None if case["kv"] == "bf16" else s[x + "scales"].double() for x in "kv"}
        for b, (length, count) in enumerate(zip(lengths, counts)):
            start = length - count
            rows = {"k": torch.stack([_turned(s["k"][b, t].double(), start + t, s["freq"], s["factor"])
                                      for t in range(count)]),
                    "v": s["v"][b, :count].double()}
            for x in "kv":
                for i in range(start // P, -(-length // P)):
                    lo, hi = max(start, i * P), min(length, (i + 1) * P)
                    page, new = table[b][i], rows[x][lo - start:hi - start]
                    a, z = lo - i * P, hi - i * P
                    if case["kv"] == "bf16":
                        out[x][page, a:z] = new
                        continue
                    top = new.abs().amax(dim=(0, 2))
                    size = _power64(torch.ceil(torch.log2(top / E4M3_MAX)).clamp(LOW, HIGH))
                    if a > 0:
                        size = torch.maximum(size, scale[x][page])
                        out[x][page, :a] = _nearest_e4m3(out[x][page, :a] * (scale[x][page] / size)[:, None])
                    out[x][page, a:z] = _nearest_e4m3(new / size[:, None])
                    scale[x][page] = size
        if case["kv"] == "bf16":
            return out
        return dict(k=out["k"], v=out["v"], kscales=scale["k"], vscales=scale["v"])
    if case["batch"] * n > 1200:
        return None
    out = torch.zeros(case["batch"], n, HEADS, DIM, dtype=torch.float64, device=s["q"].device)
    for b, length in enumerate(lengths):
        held = table[b][:-(-length // P)]
        kv = {}
        for x in "kv":
            y = s[x + "pages"][held].double()
            if case["kv"] == "e4m3":
                y = y * s[x + "scales"][held].double()[:, None, :, None]
            kv[x] = y.reshape(-1, KV, DIM).repeat_interleave(GROUP, dim=1)  # [tokens, 64, 64]
        for t in range(n):
            i = length - n + t
            lo = max(0, i + 1 - W) if W > 0 else 0
            q = _turned(s["q"][b, t].double(), i, s["freq"], s["factor"]) / math.sqrt(DIM)
            x = torch.einsum("hd,lhd->hl", q, kv["k"][lo:i + 1])
            x = torch.cat((x, s["sinks"].double()[:, None]), dim=1)
            weight = torch.exp(x - torch.logsumexp(x, dim=1, keepdim=True))[:, :-1]
            out[b, t] = torch.einsum("hl,lhd->hd", weight, kv["v"][lo:i + 1])
    return out


def work(case):
    lengths, counts = _lengths(case)
    n, W, P = case["n"], case["window"], case["page"]
    size = 2 if case["kv"] == "bf16" else 1
    if case["op"] == "append":
        new = sum(counts)
        read = new * KV * DIM * 2 * 2 + new * 4
        pages = sum(-(-x // P) - (x - c) // P for x, c in zip(lengths, counts))
        wrote = new * KV * DIM * 2 * size + (pages * KV * 2 * 4 if size == 1 else 0)
        return {"bytes": read + wrote + pages * 4, "flops": new * KV * DIM * 3}
    pairs = keys = pages = 0
    for x in lengths:
        first = max(0, x - n + 1 - W) if W > 0 else 0
        keys += x - first
        pages += -(-x // P) - first // P
        pairs += sum(min(i + 1, W) if W > 0 else i + 1 for i in range(x - n, x))
    rows = case["batch"] * n * HEADS
    return {"bytes": keys * KV * DIM * 2 * size + pages * (4 + (KV * 8 if size == 1 else 0))
            + rows * DIM * 2 * 2 + HEADS * 4, "flops": pairs * HEADS * DIM * 4}
