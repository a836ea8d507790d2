"""The paged NVFP4 cache on the GPU: append and gather bit for bit against the oracle's quantize and decode, attention
against a 64-bit softmax attention over the values the cache holds."""
import numpy as np
import pytest
import torch

import oracle
from bit_video_dit_b200 import nvfp4 as nv
from bit_video_dit_b200 import synthetic as syn

from .gpu_util import bf16_to_f64, dev_bf16, host_bits, require_gpu

pytestmark = pytest.mark.gpu

K_SCALE, V_SCALE = 11.0 / 2688.0, 9.0 / 2688.0


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Setup:
    """A cache whose sequences have the lengths `lens`, filled with seeded values under shuffled pages; everything that
    no sequence holds is 0xFF (codes -6, scales NaN).  counts[b] rows of sequence b are the step's."""

    def __init__(self, lens, counts, heads, d, page, seed, extra_rows=0, spare_pages=2, std=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.counts, self.heads, self.d, self.page = lens, counts, heads, d, page
        held = [-(-n // page) for n in lens]
        n_pages = max(1, sum(held) + spare_pages)
        order = rng.permutation(n_pages)
        self.table = np.full((len(lens), max([1, *held])), -1, np.int32)
        at = 0
        for b, h in enumerate(held):
            self.table[b, :h] = order[at:at + h]
            at += h
        self.spare = order[at:]
        start = np.concatenate([[0], np.cumsum(counts)])
        self.n_rows = int(start[-1]) + extra_rows
        self.start = start
        self.cache = nv.PagedKVCache(n_pages, page, heads, d, k_scale=K_SCALE, v_scale=V_SCALE)
        for t in (self.cache.k_codes, self.cache.k_scales, self.cache.v_codes, self.cache.v_scales):
            t.fill_(0xFF)
        self.k = [syn.f32_to_bf16_bits(std * rng.standard_normal((n, heads, d)).astype(np.float32)) for n in lens]
        self.v = [syn.f32_to_bf16_bits(std * rng.standard_normal((n, heads, d)).astype(np.float32)) for n in lens]

    def rows(self, counts=None, lens=None, n_rows=None, table=None, max_rows=None, max_len=None):
        counts = self.counts if counts is None else counts
        lens = self.lens if lens is None else lens
        start = np.concatenate([[0], np.cumsum(counts)])
        return nv.PagedRows(_i32(start), _i32(lens), _i32(self.table if table is None else table),
                            n_rows=int(start[-1]) if n_rows is None else n_rows,
                            max_rows=max([0, *counts]) if max_rows is None else max_rows,
                            max_len=max([0, *lens]) if max_len is None else max_len)

    def fill(self):
        """Append every sequence whole."""
        cat = lambda xs: dev_bf16(np.concatenate(xs, 0))  # noqa: E731
        self.cache.append(self.rows(counts=self.lens), cat(self.k), cat(self.v))
        self.check()
        return self

    def values(self, x, scale):
        flat = x.reshape(-1, self.d)
        return oracle.dequant_f32(*oracle.quantize(flat, alpha=scale)).reshape(x.shape).astype(np.float64)

    def check(self, ws=None):
        assert nv.read_device_error(self.cache.ws_rows if ws is None else ws) == (nv.OK, 0)


def _reference(q, k, v, window, sinks, scale):
    """64-bit attention of one sequence (q [n][heads][d], its last n positions) and the bound of the kernels' result:
    the weights in binary16 (2^-11 of each, 2^-25 below 2^-14 of a reference that is at most the row's largest), scores
    of binary32 sums (each product through at most d / 16 + 16 additions of 2^-23), the bf16 store (2^-8)."""
    n, heads, d = q.shape
    length, group = k.shape[0], heads // k.shape[1]
    o, e = np.zeros(q.shape), np.zeros(q.shape)
    pos = length - n + np.arange(n)[:, None]
    key = np.arange(length)[None]
    seen = (key <= pos) & ((key > pos - window) | (key < sinks) | (window == 0))
    some = seen.any(1)
    for h in range(heads):
        kk, vv = k[:, h // group], v[:, h // group]
        s = np.where(seen, q[:, h] @ kk.T * scale, -np.inf)
        p = np.where(seen, np.exp(s - np.where(some, s.max(1, initial=-np.inf), 0.0)[:, None]), 0.0)
        l = np.where(some, p.sum(1), 1.0)[:, None]
        o[:, h] = p @ vv / l
        weighted = p @ np.abs(vv) / l
        ds = (d / 16 * 18 + 16) * 2.0 ** -23 * (np.abs(q[:, h]) @ np.abs(kk).T * scale).max(1, initial=0.0)[:, None] + 2.0 ** -19
        low = (seen & (p < 2.0 ** -14)).sum(1)[:, None]
        e[:, h] = (2.0 ** -8 * np.abs(o[:, h]) + (2.0 ** -11 + 2 * ds) * weighted +
                   2.0 ** -25 * np.abs(vv).max(initial=0.0) * low / l)
    return o, 1.01 * e


def _attend(s, heads, window=0, sinks=0, scale=0.0, seed=0, lens=None, rows=None, strided=False):
    lens = s.lens if lens is None else lens
    rows = s.rows(n_rows=s.n_rows) if rows is None else rows
    qb = syn.f32_to_bf16_bits(np.random.default_rng(seed).standard_normal((s.n_rows, heads, s.d)).astype(np.float32))
    q = dev_bf16(qb)
    if strided:
        wide = torch.zeros((s.n_rows, 2 * heads, s.d), dtype=torch.bfloat16, device="cuda")
        wide[:, heads:] = q
        q = wide[:, heads:]
    out = torch.full((s.n_rows, heads, s.d), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = s.cache.attention_workspace(rows, heads, window=window, sinks=sinks)
    ws[256:] = 0xFF  # results do not depend on it
    s.cache.attention(rows, q, window=window, sinks=sinks, scale=scale, out=out, ws=ws)
    s.check(ws)
    got = bf16_to_f64(host_bits(out))
    real = 1.0 / np.sqrt(s.d) if scale == 0.0 else scale
    for b, n in enumerate(s.counts):
        r0 = s.start[b]
        k, v = s.values(s.k[b][:lens[b]], K_SCALE), s.values(s.v[b][:lens[b]], V_SCALE)
        ref, bound = _reference(bf16_to_f64(qb[r0:r0 + n]), k, v, window, sinks, real)
        bad = np.abs(got[r0:r0 + n] - ref) - bound
        assert not np.any(~(bad <= 0)), (b, np.unravel_index(np.argmax(bad), bad.shape), bad.max())
    assert np.all(got[s.start[-1]:] == 5.0)
    return out


# ---- append and gather -----------------------------------------------------------------------------------------------
@pytest.mark.parametrize("d,page,heads", [(128, 16, 3), (64, 48, 2), (128, 64, 1), (64, 16, 5)])
@pytest.mark.parametrize("rope", [False, True])
def test_append_and_gather(d, page, heads, rope):
    """Rows of several steps: none, one, many, across pages; the pages' bytes and what is read back, bit for bit."""
    require_gpu()
    s = Setup([1, 37, 0, 130, 16, 65], [1, 5, 0, 130, 2, 1], heads, d, page, seed=d + page, extra_rows=3)
    n = s.n_rows
    kb = syn.activations_bf16(n, heads * d, seed=1).reshape(n, heads, d)
    vb = syn.normal_bf16((n, heads, d), seed=2)
    kb[3, 0, :16] = 0  # a zero block; one beyond the scale's range; one far below it
    vb[4, 0, :16] = syn.f32_to_bf16_bits(np.linspace(-90.0, 90.0, 16, dtype=np.float32))
    vb[5, 0, :16] = syn.f32_to_bf16_bits(np.linspace(-1e-6, 1e-6, 16, dtype=np.float32))
    table = None
    if rope:
        ang = np.random.default_rng(3).uniform(-50, 50, (n, d // 2))
        cs, sn = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
        table = (torch.from_numpy(cs).cuda(), torch.from_numpy(sn).cuda())
    before = [t.clone() for t in (s.cache.k_codes, s.cache.k_scales, s.cache.v_codes, s.cache.v_scales)]
    # keys and values as slices of one projection
    both = torch.stack((dev_bf16(kb), dev_bf16(vb)), 1)
    rows = s.rows(n_rows=n)
    s.cache.append(rows, both[:, 0], both[:, 1], rope=table)
    s.check()
    kx = oracle.rope(kb, cs, sn) if rope else syn.bf16_bits_to_f32(kb)
    expect = [t.cpu().numpy().copy() for t in before]
    back = {}
    for i, (x, a) in enumerate(((kx, K_SCALE), (syn.bf16_bits_to_f32(vb), V_SCALE))):
        c, e, _ = oracle.quantize(np.ascontiguousarray(x.reshape(-1, d), np.float32), alpha=a)
        back[i] = oracle.dequant_bf16(c, e, a).reshape(n, heads, d)
        for b, cnt in enumerate(s.counts):
            for j in range(cnt):
                row, pos = s.start[b] + j, s.lens[b] - cnt + j
                p = s.table[b, pos // page]
                expect[2 * i][p, :, pos % page] = c.reshape(n, heads, -1)[row]
                expect[2 * i + 1][p, :, pos % page] = e.reshape(n, heads, -1)[row]
    for t, w in zip((s.cache.k_codes, s.cache.k_scales, s.cache.v_codes, s.cache.v_scales), expect):
        assert np.array_equal(t.cpu().numpy(), w)
    wide = torch.full((n, 2, heads, d), 3.0, dtype=torch.bfloat16, device="cuda")
    s.cache.gather(rows, k_out=wide[:, 0], v_out=wide[:, 1])
    s.check()
    owned = s.start[-1]
    for i in range(2):
        assert np.array_equal(host_bits(wide[:, i])[:owned], back[i][:owned])
    assert torch.all(wide[owned:] == 3.0)


def test_rows_aligned_to_16_bytes_only():
    """Rows 8 elements apart from a 32-byte boundary, as slices of an oddly padded projection may be."""
    require_gpu()
    s = Setup([40, 9], [40, 3], 2, 64, 16, seed=31)
    wide = torch.full((43, 3 * 128 + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    kb, vb = syn.normal_bf16((43, 2, 64), seed=1), syn.normal_bf16((43, 2, 64), seed=2)
    k, v = wide[:, 8:136].unflatten(1, (2, 64)), wide[:, 136:264].unflatten(1, (2, 64))
    k.copy_(dev_bf16(kb)), v.copy_(dev_bf16(vb))
    s.cache.append(s.rows(), k, v)
    k.fill_(0), v.fill_(0)
    s.cache.gather(s.rows(), k_out=k, v_out=v)
    s.check()
    for got, bits, a in ((k, kb, K_SCALE), (v, vb, V_SCALE)):
        want = oracle.dequant_bf16(*oracle.quantize(bits.reshape(-1, 64), alpha=a)).reshape(bits.shape)
        assert np.array_equal(host_bits(got), want)
    assert torch.all(wide[:, :8] == 3.0) and torch.all(wide[:, 264:] == 3.0)


def test_rows_before_the_first_position_and_many_sequences():
    """More rows than positions: nothing is written for the rows before the first, and they read as zeros.  Hundreds of
    sequences, most without rows, find their rows."""
    require_gpu()
    s = Setup([3], [8], 2, 64, 16, seed=1)
    k = dev_bf16(syn.normal_bf16((8, 2, 64), seed=1))
    s.cache.append(s.rows(), k, k)
    s.check()
    assert torch.all(s.cache.k_codes[int(s.table[0, 0]), :, 3:] == 0xFF)
    ko, vo = s.cache.gather(s.rows())
    s.check()
    assert not torch.any(ko[:5]) and not torch.any(vo[:5])
    want = oracle.dequant_bf16(*oracle.quantize(host_bits(k[5:]).reshape(-1, 64), alpha=K_SCALE))
    assert np.array_equal(host_bits(ko[5:]).reshape(-1, 64), want)
    rng = np.random.default_rng(2)
    counts = [int(c) if rng.random() < 0.3 else 0 for c in rng.integers(1, 5, 700)]
    s = Setup([c + int(x) for c, x in zip(counts, rng.integers(0, 20, 700))], counts, 1, 128, 16, seed=3)
    k = dev_bf16(syn.normal_bf16((s.n_rows, 1, 128), seed=4))
    s.cache.append(s.rows(), k, k)
    s.check()
    ko, _ = s.cache.gather(s.rows())
    want = oracle.dequant_bf16(*oracle.quantize(host_bits(k).reshape(-1, 128), alpha=K_SCALE))
    assert np.array_equal(host_bits(ko).reshape(-1, 128), want)


def test_bad_pages_and_rows_are_reported_and_skipped():
    require_gpu()
    for spoil, info in (("page", 1), ("behind", 1), ("order", 0), ("length", 1)):
        s = Setup([20, 40, 20], [2, 3, 2], 1, 64, 16, seed=5).fill()
        table, lens, counts = s.table.copy(), list(s.lens), list(s.counts)
        start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        if spoil == "page":
            table[1, 2] = s.cache.n_pages
        elif spoil == "behind":
            lens[1] = 16 * table.shape[1] + 3
        elif spoil == "order":
            start[1] = 9
            info = None  # sequence 0 has too many rows, sequence 1 a negative number: either may come first
        else:
            lens[1] = -1
        rows = nv.PagedRows(_i32(start), _i32(lens), _i32(table), n_rows=7, max_rows=3, max_len=60)
        x = torch.zeros((7, 1, 64), dtype=torch.bfloat16, device="cuda")
        for call in ("append", "gather", "attention"):
            ws = s.cache.attention_workspace(rows, 1)
            if call == "append":
                s.cache.append(rows, x, x, ws=ws)
            elif call == "gather":
                s.cache.gather(rows, ws=ws)
            else:
                s.cache.attention(rows, x, ws=ws)
            code, got = nv.read_device_error(ws)
            if spoil == "order" and call != "attention" and code == nv.OK:
                continue  # a row may find no sequence at all
            assert code == nv.ERR_DEVICE and info in (None, got), (spoil, call)
    # more rows than max_rows
    s = Setup([20, 40], [2, 3], 1, 64, 16, seed=5).fill()
    rows = s.rows(max_rows=2)
    ws = s.cache.attention_workspace(rows, 1)
    q = dev_bf16(syn.normal_bf16((5, 1, 64), seed=1))
    out = torch.full_like(q, 5.0)
    s.cache.attention(rows, q, out=out, ws=ws)
    assert nv.read_device_error(ws) == (nv.ERR_DEVICE, 1)
    assert torch.all(out[2:] == 5.0) and not torch.any(out[:2] == 5.0)


# ---- attention -------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv,heads", [(1, 1), (2, 6), (2, 16), (1, 16)])
def test_single_tokens(d, kv, heads):
    require_gpu()
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 100, 129, 700]
    s = Setup(lens, [1] * len(lens), kv, d, 16, seed=d + heads, extra_rows=2).fill()
    _attend(s, heads, seed=heads)


@pytest.mark.parametrize("d,page", [(64, 48), (128, 32)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (20, 0), (64, 4), (33, 17), (500, 40), (5, 300)])
def test_windows_and_sinks(d, page, window, sinks):
    require_gpu()
    s = Setup([1, 70, 333, 40, 256], [1, 3, 2, 4, 1], 2, d, page, seed=window + d).fill()
    _attend(s, 8, window=window, sinks=sinks, seed=1, strided=True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("counts", [[5, 1, 40], [130, 128, 129], [300, 1, 0]])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
def test_chunks(d, counts, window, sinks):
    require_gpu()
    s = Setup([300, 200, 129], counts[:1] + [min(counts[1], 200)] + [min(counts[2], 129)], 2, d, 16,
              seed=sum(counts) + d, extra_rows=1).fill()
    _attend(s, 6, window=window, sinks=sinks, seed=2)


def test_whole_prompts_from_an_empty_cache():
    require_gpu()
    s = Setup([257, 64, 1], [257, 64, 1], 1, 128, 64, seed=8).fill()
    _attend(s, 4)


@pytest.mark.parametrize("counts", [[1, 1], [3, 1], [20, 1], [200, 2]])
def test_long_sequences_split(counts):
    """Long enough to be split over CTAs, beside a short one; and with a length that the host's bound did not say."""
    require_gpu()
    s = Setup([9001, 40], counts, 1, 128, 64, seed=11).fill()
    a = _attend(s, 8, seed=3)
    b = _attend(s, 8, seed=3, rows=s.rows(max_len=4000))
    assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=1e-3)
    _attend(s, 8, window=5000, sinks=100, seed=3)


def test_rows_that_see_nothing():
    """More rows than positions: the rows before the first give zeros; a sequence of length 0 too."""
    require_gpu()
    for n in (6, 200):
        s = Setup([4, 0, 30], [n, 2, 1], 1, 64, 16, seed=4)
        cat = lambda xs: dev_bf16(np.concatenate(xs, 0))  # noqa: E731
        s.cache.append(s.rows(counts=s.lens), cat(s.k), cat(s.v))
        q = dev_bf16(syn.normal_bf16((s.n_rows, 2, 64), seed=5))
        out = torch.full_like(q, 5.0)
        ws = s.cache.attention_workspace(s.rows(), 2)
        s.cache.attention(s.rows(), q, out=out, ws=ws)
        s.check(ws)
        got = bf16_to_f64(host_bits(out))
        assert not np.any(got[:n - 4]) and not np.any(got[n:n + 2])
        qf = bf16_to_f64(host_bits(q))
        for r0, r1, b in ((n - 4, n, 0), (n + 2, n + 3, 2)):
            ref, bound = _reference(qf[r0:r1], s.values(s.k[b], K_SCALE), s.values(s.v[b], V_SCALE), 0, 0, 0.125)
            assert np.all(np.abs(got[r0:r1] - ref) <= bound)


@pytest.mark.parametrize("counts", [[1, 1, 2], [90, 40, 2]])
def test_pages_behind_the_window_may_be_gone(counts):
    """Entries of pages that hold no visible key are -1, and the pages' bytes are spoilt."""
    require_gpu()
    window, sinks, page = 40, 5, 16
    s = Setup([500, 130, 3], counts, 2, 128, page, seed=6).fill()
    want = _attend(s, 4, window=window, sinks=sinks, seed=7)
    for b, n in enumerate(s.counts):
        first = max(0, s.lens[b] - n - window + 1)
        for i in range(-(-sinks // page), first // page):
            p = int(s.table[b, i])
            for t in (s.cache.k_codes, s.cache.k_scales, s.cache.v_codes, s.cache.v_scales):
                t[p].fill_(0xFF)
            s.table[b, i] = -1
    assert (s.table == -1).sum() > 8
    assert torch.equal(_attend(s, 4, window=window, sinks=sinks, seed=7), want)


@pytest.mark.parametrize("counts", [[1, 1], [70, 3]])
@pytest.mark.parametrize("scale", [0.02, 1.0])
def test_scales_and_moving_maxima(counts, scale):
    """Scores spread over tens of binary exponents, keys in rising order, so the reference maximum moves often."""
    require_gpu()
    s = Setup([600, 90], counts, 1, 128, 16, seed=12, std=0.7)
    for b in range(2):
        x = syn.bf16_bits_to_f32(s.k[b])
        s.k[b] = syn.f32_to_bf16_bits((x * np.linspace(0.1, 2.5, s.lens[b])[:, None, None]).astype(np.float32))
    s.fill()
    _attend(s, 8, scale=scale, seed=9)


@pytest.mark.parametrize("counts", [[1], [150]])
def test_zero_tensor_scales_and_zero_queries(counts):
    require_gpu()
    s = Setup([200], counts, 1, 64, 16, seed=13).fill()
    s.cache.k_global.zero_()
    q = dev_bf16(syn.normal_bf16((s.n_rows, 2, 64), seed=1))
    got = bf16_to_f64(host_bits(s.cache.attention(s.rows(), q)))
    v = s.values(s.v[0], V_SCALE)
    for i in range(counts[0]):  # every score 0: the mean of the visible values
        seen = np.abs(v[:200 - counts[0] + i + 1, 0])
        mean = v[:200 - counts[0] + i + 1, 0].mean(0)
        assert np.all(np.abs(got[i] - mean) <= 2.0 ** -8 * np.abs(mean) + 2.0 ** -11 * seen.mean(0))
    s.cache.v_global.zero_()
    assert not torch.any(s.cache.attention(s.rows(), q))


@pytest.mark.parametrize("counts", [[1, 1], [100, 30]])
def test_captured_step_follows_the_sequences(counts):
    """A captured append and attention, replayed after lengths, pages and inputs changed; two graphs share a workspace."""
    require_gpu()
    s = Setup([180, 60], counts, 2, 128, 16, seed=14).fill()
    lens, table = _i32(s.lens), _i32(s.table)
    start = _i32(s.start)
    rows = nv.PagedRows(start, lens, table, n_rows=s.n_rows, max_rows=max(counts), max_len=190)
    q = torch.zeros((s.n_rows, 4, 128), dtype=torch.bfloat16, device="cuda")
    out, out2 = torch.empty_like(q), torch.empty_like(q)
    k = torch.zeros((s.n_rows, 2, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    ws = s.cache.attention_workspace(rows, 4)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    torch.cuda.synchronize()
    with torch.cuda.graph(graphs[0]):
        s.cache.append(rows, k, v)
        s.cache.attention(rows, q, out=out, ws=ws)
    with torch.cuda.graph(graphs[1]):
        s.cache.attention(rows, q, window=30, out=out2, ws=ws)
    for step, new in enumerate(([180, 60], [177, 45], [150, 33])):
        if min(n - c for n, c in zip(new, counts)) < 0:
            continue
        lens.copy_(_i32(new))
        kb, vb, qb = (syn.normal_bf16(tuple(t.shape), seed=50 + 3 * step + i) for i, t in enumerate((k, v, q)))
        for t, bits in ((k, kb), (v, vb), (q, qb)):
            t.copy_(dev_bf16(bits))
        graphs[0].replay()
        graphs[1].replay()
        s.check(ws)
        for b, n in enumerate(counts):
            r0, first = s.start[b], new[b] - n
            s.k[b][first:new[b]], s.v[b][first:new[b]] = kb[r0:r0 + n], vb[r0:r0 + n]
            vals = s.values(s.k[b][:new[b]], K_SCALE), s.values(s.v[b][:new[b]], V_SCALE)
            for o, window in ((out, 0), (out2, 30)):
                ref, bound = _reference(bf16_to_f64(qb[r0:r0 + n]), *vals, window, 0, 1 / np.sqrt(128))
                assert np.all(np.abs(bf16_to_f64(host_bits(o))[r0:r0 + n] - ref) <= bound)


def test_same_bits_every_time_and_on_another_stream():
    require_gpu()
    s = Setup([5000, 333], [2, 2], 2, 128, 32, seed=15).fill()
    q = dev_bf16(syn.normal_bf16((4, 8, 128), seed=1))
    want = s.cache.attention(s.rows(), q)
    side = torch.cuda.Stream()
    rows = s.rows()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        others = [s.cache.attention(rows, q) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    for o in others:
        assert torch.equal(o, want)


def test_python_refusals():
    require_gpu()
    s = Setup([20], [2], 2, 64, 16, seed=1).fill()
    r = s.rows()
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (k.float(), k[:1], k.transpose(0, 1), k.cpu(), torch.zeros((2, 64, 2), dtype=torch.bfloat16, device="cuda")):
        for call in (lambda t: s.cache.append(r, t, k), lambda t: s.cache.append(r, k, t),
                     lambda t: s.cache.gather(r, k_out=t)):
            if bad.shape == k.shape and bad.dtype == k.dtype and bad.is_cuda and bad.is_contiguous():
                continue
            with pytest.raises(ValueError):
                call(bad)
    with pytest.raises(ValueError):
        s.cache.append(r, k, k, rope=(torch.zeros((2, 32), device="cuda"), torch.zeros((2, 31), device="cuda")))
    with pytest.raises(ValueError):
        s.cache.attention(r, torch.zeros((2, 3, 64), dtype=torch.bfloat16, device="cuda"))  # 3 heads over 2
    with pytest.raises(ValueError):
        nv.PagedRows(r.row_start.long(), r.lens, r.pages, n_rows=2, max_rows=2, max_len=20)
    with pytest.raises(ValueError):
        nv.PagedRows(r.row_start[:-1], r.lens, r.pages, n_rows=2, max_rows=2, max_len=20)
    with pytest.raises(nv.NVFP4Error):
        s.cache.attention(r, torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda"), ws=s.cache.ws_rows[:128])


@pytest.mark.parametrize("d,page", [(64, 16), (64, 48), (128, 4112), (128, 64)])
@pytest.mark.parametrize("counts,heads", [([1, 1, 1, 1], 8), ([2, 1, 2, 0], 8), ([1, 1, 1, 1], 12), ([3, 1, 3, 3], 5)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (2500, 40)])
def test_long_decode_steps(d, page, counts, heads, window, sinks):
    """Spans of 2048 keys and more, with up to 8 and up to 16 (row, head) pairs; short sequences among them."""
    require_gpu()
    s = Setup([2100, 37, 5003, 3], counts, 1, d, page, seed=page + heads).fill()
    _attend(s, heads, window=window, sinks=sinks, seed=heads)


@pytest.mark.parametrize("heads,n", [(4, 230), (4, 296), (4, 297), (12, 120), (12, 149)])
def test_windows_of_many_sequences(heads, n):
    """Numbers of sequences around those at which long windows change their way of being shared out."""
    require_gpu()
    rng = np.random.default_rng(n)
    lens = [int(x) for x in rng.integers(1, 30, n)]
    lens[3], lens[n - 1] = 2300, 2111
    s = Setup(lens, [1] * n, 1, 64, 32, seed=n).fill()
    _attend(s, heads, window=2100, sinks=5, seed=heads)


@pytest.mark.parametrize("count", [1, 2])
@pytest.mark.parametrize("max_len", [0, 40])
def test_lengths_beyond_the_hosts_bound(count, max_len):
    """max_len says only how the work is dealt out."""
    require_gpu()
    s = Setup([3001, 40, 200], [count] * 3, 2, 64, 16, seed=41).fill()
    _attend(s, 16, rows=s.rows(max_len=max_len), seed=4)
    _attend(s, 16, rows=s.rows(max_len=max_len), window=77, sinks=9, seed=4)


@pytest.mark.parametrize("counts", [[1, 1], [9, 1]])
def test_many_heads_of_one_key(counts):
    """A group of 71 heads: a unit's rows begin and end inside a token."""
    require_gpu()
    s = Setup([500, 33], counts, 1, 64, 16, seed=42).fill()
    _attend(s, 71, seed=5)
    _attend(s, 71, window=20, sinks=2, seed=5)


@pytest.mark.parametrize("length,window,sinks,count", [(100, 10, 0, 1), (100, 13, 3, 2), (333, 50, 19, 3),
                                                       (5000, 3000, 7, 1), (5001, 2999, 33, 2), (300, 37, 5, 70)])
@pytest.mark.parametrize("d", [64, 128])
def test_places_that_no_row_sees_may_hold_anything(length, window, sinks, count, d):
    """Also those that share a page, or 16 keys, with visible ones: NaN scales there change nothing."""
    require_gpu()
    page = 64
    s = Setup([length], [count], 2, d, page, seed=43).fill()
    want = _attend(s, 4, window=window, sinks=sinks, seed=7)
    first = length - count - window + 1
    assert first > sinks
    for pos in range(sinks, first):
        p, o = int(s.table[0, pos // page]), pos % page
        for t in (s.cache.k_codes, s.cache.k_scales, s.cache.v_codes, s.cache.v_scales):
            t[p, :, o] = 0xFF
    assert torch.equal(_attend(s, 4, window=window, sinks=sinks, seed=7), want)


@pytest.mark.parametrize("length,count", [(60, 1), (3000, 2), (3000, 60)])
def test_entries_below_zero_are_reported(length, count):
    """-1, which also stands for a page given back, is no page where one is needed; lengths that the table does not
    reach are refused before they make work."""
    require_gpu()
    s = Setup([40, length], [1, count], 1, 64, 16, seed=44).fill()
    q = dev_bf16(syn.normal_bf16((s.n_rows, 2, 64), seed=1))
    for entry in (-1, -7, s.cache.n_pages, 2 ** 31 - 1):
        table = s.table.copy()
        table[1, 1] = entry
        rows = s.rows(table=table)
        ws = s.cache.attention_workspace(rows, 2)
        s.cache.attention(rows, q, ws=ws)
        assert nv.read_device_error(ws) == (nv.ERR_DEVICE, 1)
    for n in (16 * s.table.shape[1] + 1, 2 ** 31 - 1):
        rows = s.rows(lens=[40, n], max_len=length)
        out = torch.full_like(q, 5.0)
        ws = s.cache.attention_workspace(rows, 2)
        s.cache.attention(rows, q, ws=ws, out=out)
        assert nv.read_device_error(ws) == (nv.ERR_DEVICE, 1)
        assert torch.all(out[1:] == 5.0) and not torch.any(out[0] == 5.0)


@pytest.mark.parametrize("length,count", [(60, 2), (3000, 2), (9000, 60)])
def test_a_nan_query_stays_in_its_row(length, count):
    require_gpu()
    s = Setup([length], [count], 2, 128, 16, seed=45).fill()
    q = dev_bf16(syn.normal_bf16((count, 8, 128), seed=2))
    want = s.cache.attention(s.rows(), q).clone()
    q[count - 1, 3, 77] = float("nan")
    got = s.cache.attention(s.rows(), q)
    assert torch.all(torch.isnan(got[count - 1, 3]))
    want[count - 1, 3] = got[count - 1, 3] = 0
    assert torch.equal(got, want)


def test_calls_at_the_same_time_and_given_streams():
    """Two streams, each with workspaces of its own, given and made by the calls."""
    require_gpu()
    s = Setup([5000, 700], [1, 1], 2, 128, 32, seed=46).fill()
    c = Setup([900, 64], [300, 64], 2, 128, 32, seed=47).fill()
    q = dev_bf16(syn.normal_bf16((s.n_rows, 8, 128), seed=1))
    qc = dev_bf16(syn.normal_bf16((c.n_rows, 8, 128), seed=2))
    rows, rows_c = s.rows(), c.rows()
    want, want_c = s.cache.attention(rows, q), c.cache.attention(rows_c, qc)
    kv, kv_c = s.cache.gather(rows), c.cache.gather(rows_c)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        got += [(s.cache.attention(rows, q, stream=a), want), (c.cache.attention(rows_c, qc, stream=b), want_c)]
        got += list(zip(s.cache.gather(rows, stream=b), kv)) + list(zip(c.cache.gather(rows_c, stream=a), kv_c))
    torch.cuda.synchronize()
    for x, w in got:
        assert torch.equal(x, w)


def test_offsets_beyond_32_bits():
    """Pages behind the first 4 GiB of codes."""
    require_gpu()
    kv, d, page = 8, 128, 64
    n_pages = (1 << 32) // (kv * page * d // 2) + 40
    cache = nv.PagedKVCache(n_pages, page, kv, d, k_scale=K_SCALE, v_scale=V_SCALE)
    assert cache.k_codes.numel() > 1 << 32
    n = 20 * page + 5
    s = Setup([n], [n], kv, d, page, seed=48)
    table = _i32(n_pages - 1 - np.arange(21)[None])
    s.table = table.cpu().numpy()
    s.cache = cache
    s.fill()
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        assert not torch.any(t[:n_pages - 21]) and torch.any(t[n_pages - 21])
    _attend(s, 8, seed=1)
    s.counts, s.start, s.n_rows = [1], np.array([0, 1]), 1
    _attend(s, 16, seed=2)
    k, v = cache.gather(s.rows(counts=[n]))
    for got, x, a in ((k, s.k, K_SCALE), (v, s.v, V_SCALE)):
        assert np.array_equal(host_bits(got).reshape(-1, d), oracle.dequant_bf16(*oracle.quantize(x[0].reshape(-1, d), alpha=a)))


# ---- the operators together ------------------------------------------------------------------------------------------
def test_decoding_a_sequence_token_by_token():
    """A one-layer causal decoder on the operators: a prompt of 21 tokens as one chunk, then 12 single tokens, two
    sequences: fused projection (nvfp4_gemv, or a given bf16 product for the prompt), RoPE and append, attention with
    a window and sinks, output projection with a residual.  Every step against the same in 64 bits on what the step
    was given (bf16 q, cached values)."""
    require_gpu()
    kv, heads, d, width, page, window, sinks = 2, 4, 64, 256, 16, 24, 2
    rng = np.random.default_rng(20)
    prompt, steps, B = 21, 12, 2
    qkv_w = nv.quantize(dev_bf16(syn.normal_bf16(((heads + 2 * kv) * d, width), seed=1, std=0.06)))
    out_w = nv.quantize(dev_bf16(syn.normal_bf16((width, heads * d), seed=2, std=0.06)))
    wf = oracle.dequant_f32(*oracle.quantize(syn.normal_bf16((width, heads * d), seed=2, std=0.06))).astype(np.float64)
    s = Setup([prompt + steps] * B, [0] * B, kv, d, page, seed=21)
    held = [[np.zeros((0, kv, d))] * 2 for _ in range(B)]
    for step in range(steps + 1):
        n = prompt if step == 0 else 1
        length = prompt + step
        x = dev_bf16(syn.f32_to_bf16_bits(rng.standard_normal((B * n, width)).astype(np.float32)))
        qkv = torch.cat([nv.gemv(c, qkv_w) for c in x.split(16)]).view(B * n, heads + 2 * kv, d)
        pos = np.tile(np.arange(length - n, length), B)
        ang = pos[:, None] / 1000.0 ** (np.arange(d // 2) / (d // 2))
        cs, sn = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
        rows = s.rows(counts=[n] * B, lens=[length] * B)
        s.cache.append(rows, qkv[:, heads:heads + kv], qkv[:, heads + kv:],
                       rope=(torch.from_numpy(cs).cuda(), torch.from_numpy(sn).cuda()))
        o = s.cache.attention(rows, qkv[:, :heads], window=window, sinks=sinks)
        y = torch.cat([nv.gemv(c, out_w, residual=r) for c, r in zip(o.reshape(B * n, -1).split(16), x.split(16))])
        s.check()
        bits = host_bits(qkv)
        turned = oracle.rope(np.ascontiguousarray(bits[:, heads:heads + kv]), cs, sn)
        k = oracle.dequant_f32(*oracle.quantize(turned.reshape(-1, d), alpha=K_SCALE)).reshape(B * n, kv, d)
        v = s.values(np.ascontiguousarray(bits[:, heads + kv:]), V_SCALE)
        got, qf = bf16_to_f64(host_bits(o)), bf16_to_f64(bits[:, :heads])
        for b in range(B):
            at = slice(b * n, (b + 1) * n)
            held[b] = [np.concatenate((h, new[at])) for h, new in zip(held[b], (k, v))]
            ref, bound = _reference(qf[at], *held[b], window, sinks, 1 / np.sqrt(d))
            assert np.all(np.abs(got[at] - ref) <= bound), step
        of = got.reshape(B * n, -1)
        want = bf16_to_f64(host_bits(x)) + of @ wf.T
        tol = 2.0 ** -8 * np.abs(want) + (8 * 18 + 20) * 2.0 ** -23 * (np.abs(of) @ np.abs(wf).T) + 2.0 ** -22 * np.abs(want)
        assert np.all(np.abs(bf16_to_f64(host_bits(y)) - want) <= tol), step
