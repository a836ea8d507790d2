"""The operators of token-by-token serving, as measured cases: matrix-vector products with NVFP4 weights, the paged
NVFP4 cache written and read back, and attention of new tokens over it.

Format of everything held in 4 bits: E2M1 codes (two a byte, element 2i in bits 3:0), one E4M3 scale per 16 elements,
one binary32 tensor scale; value = e2m1 * s * a32.  A cache page holds [kv_heads][page_size][head_dim] of one tensor.
"""
import math
import random

import torch

own = False

DEV = "cuda"
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------
def _gemv(name, m, n, k, act=False, bias=False):
    return {"name": name, "kind": "gemv", "m": m, "n": n, "k": k, "act": act, "bias": bias}


def _cache(name, seqs, rows_min, rows_max, len_max, kv_heads, d, page, write, rope, ragged):
    return {"name": name, "kind": "cache", "seqs": seqs, "rows_min": rows_min, "rows_max": rows_max, "len_min": rows_max,
            "len_max": len_max, "heads": kv_heads, "kv_heads": kv_heads, "d": d, "page": page, "write": write,
            "rope": rope, "ragged": ragged}


def _attend(name, seqs, rows_min, rows_max, len_min, len_max, heads, kv_heads, d, page, window, sinks, ragged):
    return {"name": name, "kind": "attend", "seqs": seqs, "rows_min": rows_min, "rows_max": rows_max, "len_min": len_min,
            "len_max": len_max, "heads": heads, "kv_heads": kv_heads, "d": d, "page": page, "window": window,
            "sinks": sinks, "ragged": ragged}


def listed():
    return [
        # one token through an attention projection: the smallest product, all latency
        _gemv("gemv_1x4096x4096", 1, 4096, 4096),
        # three frames' conditioning vectors through a modulation layer of an odd width
        _gemv("gemv_3x10250x2624", 3, 10250, 2624, bias=True),
        # sixteen sequences' tokens through a wide FFN layer with its GELU
        _gemv("gemv_16x28672x8192", 16, 28672, 8192, act=True, bias=True),
        # one decode step: each of 64 sequences writes its token (keys turned), and it is read back
        _cache("cache_64x1", 64, 1, 1, 4000, 8, 128, 64, True, True, 1),
        # one video frame-chunk of 2640 tokens x 24 heads written and read back
        _cache("cache_1x2640", 1, 2640, 2640, 2640, 24, 128, 64, True, True, 2),
        # five sequences of unequal length read back whole (moved to another cache or another attention)
        _cache("read_5x20000", 5, 3000, 20000, 20000, 8, 64, 16, False, False, 3),
        # one sequence's next token over a short cache: latency
        _attend("decode_1x700", 1, 1, 1, 700, 700, 32, 8, 128, 16, 0, 0, 4),
        # a serving batch: 64 sequences of unequal length, one token each, four query heads a K/V head
        _attend("decode_64x12000", 64, 1, 1, 100, 12000, 32, 8, 128, 64, 0, 0, 5),
        # long contexts with two rows each (a token and a drafted one), five query heads a K/V head
        _attend("decode_4x131072", 4, 2, 2, 90000, 131072, 40, 8, 128, 128, 0, 0, 6),
        # long contexts seen through a window of 4096 with 4 sinks, heads of 64, eight query heads a K/V head
        _attend("window_32x60000", 32, 1, 1, 3000, 60000, 64, 8, 64, 32, 4096, 4, 7),
        # chunked prefill: six sequences with 1 .. 700 new tokens over caches of up to 6000
        _attend("chunk_6x700", 6, 1, 700, 1200, 6000, 32, 8, 128, 16, 0, 0, 8),
        # a frame-chunk of 2640 tokens over 13 chunks, seen through a sink chunk and a window of seven
        _attend("chunk_1x2640", 1, 2640, 2640, 34320, 34320, 24, 24, 128, 64, 18480, 2640, 9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("gemv", "cache", "attend", "attend"))
    if kind == "gemv":
        c = _gemv("", rng.randint(1, 16), _log(rng, 256, 28672), 64 * _log(rng, 4, 128), rng.random() < 0.4,
                  rng.random() < 0.5)
    elif kind == "cache":
        seqs = _log(rng, 1, 64)
        most = max(1, 100000 // seqs)
        rows = _log(rng, 1, min(4000, most))
        c = _cache("", seqs, max(1, rows // rng.randint(1, 4)), rows, rows + _log(rng, 1, min(4000, most)),
                   rng.choice((1, 2, 4, 5, 8)), rng.choice((64, 128)), rng.choice((16, 32, 64, 128)), True,
                   rng.random() < 0.5, rng.randrange(1 << 20))
    else:
        kv = rng.choice((1, 2, 4, 8))
        heads = kv * rng.choice((1, 2, 4, 5, 8, 16))
        seqs = _log(rng, 1, 32)
        if rng.random() < 0.5:  # single tokens and drafted ones
            rows, longest = rng.randint(1, 4), _log(rng, 64, max(64, 400000 // (seqs * kv)))
        else:  # chunks
            rows = _log(rng, 5, max(6, 3000 // seqs))
            longest = rows + _log(rng, 1, max(2, min(20000, 800000000 // (seqs * rows * heads))))
        window = rng.choice((0, 0, _log(rng, 16, max(17, longest))))
        c = _attend("", seqs, max(1, rows // rng.randint(1, 4)), rows, max(rows, longest // rng.randint(1, 5)),
                    max(rows, longest), heads, kv, rng.choice((64, 128)), rng.choice((16, 32, 64, 128)), window,
                    rng.choice((0, 1, 4, 100)) if window else 0, rng.randrange(1 << 20))
    del c["name"]
    return c


def _shape(case):
    """Rows and lengths of the case's sequences, whatever the seed of its values."""
    r = random.Random(case["ragged"])
    rows = [r.randint(case["rows_min"], case["rows_max"]) for _ in range(case["seqs"])]
    rows[0] = case["rows_max"]
    rows[-1] = case["rows_min"] if case["seqs"] > 1 else rows[-1]
    lens = [max(n, _log(r, max(1, case["len_min"]), case["len_max"])) for n in rows]
    lens[0] = max(rows[0], case["len_max"])
    if not case.get("write", True):  # read back whole
        lens = list(rows)
    return rows, lens


def _pairs(rows, length, window, sinks):
    """Visible (row, key) pairs and visible keys of one sequence."""
    if not window:
        return rows * length - rows * (rows - 1) // 2, length
    pairs = 0
    for p in range(length - rows, length):
        seen = min(p + 1, window)
        pairs += seen + min(sinks, p + 1 - seen)
    first = max(0, length - rows - window + 1)
    return pairs, length - first + min(sinks, first)


def work(case):
    if case["kind"] == "gemv":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": n * k * 9 / 16 + 2 * m * k + 2 * m * n + (2 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    rows, lens = _shape(case)
    if case["kind"] == "cache":
        e = 2 * sum(rows) * case["kv_heads"] * case["d"]
        rope = 4 * sum(rows) * case["d"] if case["rope"] else 0
        b = e * (2 + 9 / 16) * (2 if case["write"] else 1) + rope
        return {"bytes": b, "flops": e}
    pairs = keys = 0
    for n, length in zip(rows, lens):
        p, k = _pairs(n, length, case["window"], case["sinks"])
        pairs, keys = pairs + p, keys + k
    return {"bytes": keys * case["kv_heads"] * case["d"] * 2 * 9 / 16 + 4 * sum(rows) * case["heads"] * case["d"],
            "flops": 4 * pairs * case["heads"] * case["d"]}


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------
def _encode(x, a32):
    """binary32 [..., 16 b] -> (E2M1 codes, one a byte, [..., 16 b]; E4M3 scales [..., b]), every step in binary32."""
    blocks = x.unflatten(-1, (-1, 16))
    scales = (blocks.abs().amax(-1) / (6.0 * a32)).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = scales.float() * a32
    y = blocks * torch.where(d == 0, d, 1.0 / d).unsqueeze(-1)
    a = y.abs()
    codes = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    codes = codes + 8 * torch.signbit(y).to(torch.uint8)
    codes = torch.where((scales.float() == 0).unsqueeze(-1), torch.zeros_like(codes), codes)
    return codes.flatten(-2), scales.view(torch.uint8)


def _pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _decode(packed, scales):
    """Packed codes [..., d / 2] and E4M3 bytes [..., d / 16] -> e2m1 * s in binary32 [..., d] (exact)."""
    codes = torch.stack((packed & 15, packed >> 4), -1).flatten(-2).long()
    table = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float32, device=packed.device)
    s = scales.view(torch.float8_e4m3fn).float()
    return (table[codes].unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)


def _tiled(scales):
    """Row-major scales [n, k / 16] -> the 128 x 4 tiles of a weight operand, padding zero."""
    n, c = scales.shape
    full = torch.zeros((-(-n // 128) * 128, -(-c // 4) * 4), dtype=torch.uint8, device=scales.device)
    full[:n, :c] = scales
    return full.view(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untiled(tiles, n, c):
    rows, cols = -(-n // 128) * 128, -(-c // 4) * 4
    return tiles.view(rows // 128, cols // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rows, cols)[:n, :c]


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _values(g, heads, tokens, d):
    """Keys or values [heads][tokens][d]: normal, with a louder channel a head, as keys have."""
    x = _normal(g, heads, tokens, d)
    x[..., 5] *= 4.0
    return x


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if case["kind"] == "gemv":
        m, n, k = case["m"], case["n"], case["k"]
        w = _normal(g, n, k) * 0.02
        a32 = (w.abs().max() / 2688.0).reshape(1)
        codes, scales = _encode(w, a32)
        s = {"kind": "gemv", "x": _normal(g, m, k).bfloat16(), "codes": _pack(codes), "scales": _tiled(scales), "a32": a32,
             "bias": (_normal(g, n) * 0.02).bfloat16() if case["bias"] else None, "act": case["act"], "n": n, "k": k}
        if own:
            from bit_video_dit_b200 import nvfp4 as nv

            s["w"] = nv.NVFP4Tensor(s["codes"], s["scales"], a32, n, k)
            s["out"] = torch.empty((m, n), dtype=torch.bfloat16, device=DEV)
        return s
    rows, lens = _shape(case)
    page, kv, d = case["page"], case["kv_heads"], case["d"]
    held = [-(-n // page) for n in lens]
    n_pages = sum(held) + 3
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(held)), -1, dtype=torch.int32)
    ends = torch.tensor(held).cumsum(0)
    spot = torch.arange(max(held))[None].expand(len(held), -1)
    table[spot < torch.tensor(held)[:, None]] = order.cpu()[: int(ends[-1])]
    start = torch.tensor([0] + rows).cumsum(0).to(torch.int32)
    s = {"kind": case["kind"], "page": page, "rows_max": max(rows), "len_max": max(lens), "write": case.get("write", False),
         "start": start.to(DEV), "lens": torch.tensor(lens, dtype=torch.int32).to(DEV), "table": table.to(DEV),
         "n_rows": sum(rows), "kv_heads": kv, "heads": case["heads"], "d": d, "window": case.get("window", 0),
         "sinks": case.get("sinks", 0),  # a calibrated scale: the loudest value is about 11.7
         "a32": torch.tensor([0.00435713], device=DEV)}
    for t in ("k", "v"):
        codes, scales = [], []
        step = max(1, (1 << 27) // (kv * page * d))  # pages made at a time
        for i in range(0, n_pages, step):
            c, e = _encode(_values(g, min(step, n_pages - i) * kv, page, d), s["a32"])
            codes.append(_pack(c))
            scales.append(e)
        s[t + "_codes"] = torch.cat(codes).view(n_pages, kv, page, d // 2)
        s[t + "_scales"] = torch.cat(scales).view(n_pages, kv, page, d // 16)
    n = s["n_rows"]
    if case["kind"] == "attend":
        s["q"] = _normal(g, n, case["heads"], d).bfloat16()
    elif case["write"]:
        # the new rows as a fused projection leaves them: keys and values side by side
        s["kv"] = _values(g, n * 2, kv, d).view(n, 2, kv, d).bfloat16()
        if case["rope"]:
            angle = _normal(g, n, d // 2).mul(100.0).double()
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    if own:
        from bit_video_dit_b200 import nvfp4 as nv

        cache = nv.PagedKVCache(n_pages, page, kv, d, k_scale=s["a32"], v_scale=s["a32"])
        for t in ("k_codes", "k_scales", "v_codes", "v_scales"):
            getattr(cache, t).copy_(s[t])
            del s[t]
        s["cache"] = cache
        s["rows"] = nv.PagedRows(s["start"], s["lens"], s["table"], n_rows=n, max_rows=max(rows), max_len=max(lens))
        if case["kind"] == "attend":
            s["out"] = torch.empty_like(s["q"])
            s["ws"] = cache.attention_workspace(s["rows"], case["heads"], window=s["window"], sinks=s["sinks"])
        else:
            s["k_out"] = torch.empty((n, kv, d), dtype=torch.bfloat16, device=DEV)
            s["v_out"] = torch.empty((n, kv, d), dtype=torch.bfloat16, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------
def run(s):
    if own:
        return _own(s)
    if s["kind"] == "gemv":
        return _plain_gemv(s)
    return _plain_cache(s) if s["kind"] == "cache" else _plain_attention(s)


def _own(s):
    from bit_video_dit_b200 import nvfp4 as nv

    if s["kind"] == "gemv":
        return nv.gemv(s["x"], s["w"], out=s["out"], bias=s["bias"], act=nv.ACT_GELU_TANH if s["act"] else nv.ACT_NONE)
    cache, rows = s["cache"], s["rows"]
    if s["kind"] == "attend":
        return cache.attention(rows, s["q"], window=s["window"], sinks=s["sinks"], out=s["out"], ws=s["ws"])
    if s["write"]:
        cache.append(rows, s["kv"][:, 0], s["kv"][:, 1], rope=(s["cos"], s["sin"]) if "cos" in s else None)
    return cache.gather(rows, k_out=s["k_out"], v_out=s["v_out"])


def _plain_gemv(s):
    w = _decode(s["codes"], _untiled(s["scales"], s["n"], s["k"] // 16))
    y = (s["x"].float() @ w.T) * s["a32"]
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if s["act"]:
        y = 0.5 * y * (1.0 + torch.tanh(0.7978845608028654 * (y + 0.044715 * y * y * y)))
    return y.bfloat16()


def _places(s):
    """Page and offset of every row's own position."""
    row = torch.arange(s["n_rows"], device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(s["start"][1:], row, right=True)
    at = (s["lens"][seq] - s["start"][seq + 1] + row).long()
    return s["table"][seq, at // s["page"]].long(), at % s["page"]


def _plain_cache(s):
    page, offset = _places(s)
    if s["write"]:
        k, v = s["kv"][:, 0].float(), s["kv"][:, 1].float()
        if "cos" in s:
            c, n = s["cos"][:, None], s["sin"][:, None]
            a, b = k[..., 0::2], k[..., 1::2]
            k = torch.stack((a * c - b * n, a * n + b * c), -1).flatten(-2)
        codes, s["k_scales"][page, :, offset] = _encode(k, s["a32"])
        s["k_codes"][page, :, offset] = _pack(codes)
        codes, s["v_scales"][page, :, offset] = _encode(v, s["a32"])
        s["v_codes"][page, :, offset] = _pack(codes)
    k = _decode(s["k_codes"][page, :, offset], s["k_scales"][page, :, offset]) * s["a32"]
    v = _decode(s["v_codes"][page, :, offset], s["v_scales"][page, :, offset]) * s["a32"]
    return k.bfloat16(), v.bfloat16()


def _sequences(s, t):
    """One tensor's cached sequences, padded: binary32 [seqs][kv_heads][positions][d]."""
    pages = s["table"].clamp(min=0).long()
    x = _decode(s[t + "_codes"][pages], s[t + "_scales"][pages]) * s["a32"]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attention(s):
    most, kv, heads, d = s["rows_max"], s["kv_heads"], s["heads"], s["d"]
    n = s["start"][1:] - s["start"][:-1]
    row = torch.arange(most, device=DEV)
    real = row[None] < n[:, None]
    source = (s["start"][:-1, None] + row).long().clamp(max=s["n_rows"] - 1)
    q = s["q"][source].float().view(len(n), most, kv, heads // kv, d)
    q = q.permute(0, 2, 3, 1, 4).flatten(2, 3)  # [seqs][kv_heads][group * rows][d]
    scores = q @ _sequences(s, "k").transpose(2, 3)
    scores *= 1.0 / math.sqrt(d)
    at = (s["lens"] - n)[:, None] + row
    key = torch.arange(scores.shape[-1], device=DEV)
    seen = key <= at[..., None]
    if s["window"]:
        seen &= (key > at[..., None] - s["window"]) | (key < s["sinks"])
    scores = scores.view(len(n), kv, heads // kv, most, -1)
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    scores -= scores.amax(-1, keepdim=True)
    scores.exp_()
    total = scores.sum(-1, keepdim=True)
    o = (scores.flatten(2, 3) @ _sequences(s, "v")).view(*scores.shape[:-1], d) / total
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)  # [seqs][rows][heads][d]
    return o[real].bfloat16()


# ---------------------------------------------------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------------
def _nibbles(packed):
    low, high = (packed % 16).double(), torch.div(packed, 16, rounding_mode="floor").double()
    c = torch.stack((low, high), dim=-1).reshape(*packed.shape[:-1], -1)
    mag = c % 8
    val = torch.where(mag < 4, mag / 2, torch.where(mag < 6, mag - 2, 2 * mag - 8))
    return torch.where(c >= 8, -val, val)


def _scale_values(e4m3):
    e, m = torch.div(e4m3, 8, rounding_mode="floor").double(), (e4m3 % 8).double()
    return torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e - 10))


def _numbers(packed, e4m3, a32):
    return _nibbles(packed) * _scale_values(e4m3).repeat_interleave(16, dim=-1) * a32.double()


def _nearest(x, a32):
    """64-bit values -> the values that their encoding stands for."""
    b = x.reshape(*x.shape[:-1], -1, 16)
    want = (b.abs().amax(-1) / (6 * a32.double())).clamp(max=448.0)
    low = torch.exp2(torch.floor(torch.log2(want.clamp(min=2.0 ** -6)))) / 8
    s = torch.round(want / low) * low
    s = s.unsqueeze(-1) * a32.double()
    y = torch.where(s > 0, b / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(b))
    a = y.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.sign(y) * torch.round(a / step) * step * s).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "gemv":
        n, k = case["n"], case["k"]
        r = torch.arange(n, device=DEV)[:, None]
        c = torch.arange(k // 16, device=DEV)[None]
        place = (r // 128 * -(-k // 64) + c // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + c % 4
        y = torch.einsum("mk,nk->mn", s["x"].double(), _numbers(s["codes"], s["scales"][place], s["a32"]))
        if case["bias"]:
            y = y + s["bias"].double()
        return torch.nn.functional.gelu(y, approximate="tanh") if case["act"] else y
    rows, lens = _shape(case)
    start = [sum(rows[:i]) for i in range(len(rows) + 1)]
    table, page = s["table"].long(), case["page"]
    if case["kind"] == "cache":
        if case["write"]:
            k, v = s["kv"].double().unbind(1)
            if case["rope"]:
                turn = torch.complex(s["cos"].double(), s["sin"].double())[:, None]
                k = torch.view_as_real(torch.view_as_complex(k.reshape(*k.shape[:-1], -1, 2)) * turn).flatten(-2)
            return _nearest(k, s["a32"]), _nearest(v, s["a32"])
        got = {"k": [], "v": []}
        for b, n in enumerate(lens):
            used = table[b, : -(-n // page)]
            for t in got:
                x = _numbers(s[t + "_codes"][used], s[t + "_scales"][used], s["a32"])
                got[t].append(x.permute(0, 2, 1, 3).reshape(-1, case["kv_heads"], case["d"])[:n])
        return torch.cat(got["k"]), torch.cat(got["v"])
    group = case["heads"] // case["kv_heads"]
    o = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    for b, (n, length) in enumerate(zip(rows, lens)):
        used = table[b, : -(-length // page)]
        at = torch.arange(length - n, length, device=DEV)[:, None]
        key = torch.arange(length, device=DEV)[None]
        hidden = key > at
        if case["window"]:
            hidden = hidden | ((key <= at - case["window"]) & (key >= case["sinks"]))
        for h in range(case["kv_heads"]):
            k = _numbers(s["k_codes"][used, h], s["k_scales"][used, h], s["a32"]).reshape(-1, case["d"])[:length]
            v = _numbers(s["v_codes"][used, h], s["v_scales"][used, h], s["a32"]).reshape(-1, case["d"])[:length]
            for i in range(h * group, (h + 1) * group):
                w = s["q"][start[b] : start[b + 1], i].double() @ k.T / case["d"] ** 0.5
                o[start[b] : start[b + 1], i] = torch.softmax(w.masked_fill(hidden, float("-inf")), -1) @ v
    return o
