"""Attention over the paged cache where one key outweighs the others by tens of binary orders, as an attention sink does,
and has nothing in its value: the result is what the small weights carry.

Bound, relative to that result.  A weight goes to the second product in binary16 under a reference at least 7 binary
orders below the row's largest: 2^-11 of it, and 2^-25 of the reference, so 2^-32 of the largest weight, below 2^-21 of
that; scores are binary32 sums (each product through at most d / 16 + 16 additions of 2^-23, 2^-19 for the exponent's
own), the store is bf16 (2^-8 at most)."""
import numpy as np
import pytest
import torch

from bit_video_dit_b200 import synthetic as syn

from .gpu_util import bf16_to_f64, dev_bf16, host_bits, require_gpu
from .test_gpu_paged import K_SCALE, V_SCALE, Setup

pytestmark = pytest.mark.gpu


CASES = [(lens, counts, d, orders)
         for lens, counts in (([2000], [1]), ([2000], [2]), ([2100, 2500], [1, 1]), ([2100], [2]), ([5000, 300], [20, 5]),
                              ([3000], [600]))
         for d in (64, 128) for orders in (20, 24, 25, 26, 28)]
CASES += [([100001], [count], d, orders) for count in (1, 40) for d, orders in ((128, 25), (64, 26))]


@pytest.mark.parametrize("lens,counts,d,orders", CASES)
def test_small_weights_beside_a_sink_without_a_value(lens, counts, d, orders):
    require_gpu()
    heads = 8
    s = Setup(lens, counts, 1, d, 64, seed=d)
    rng = np.random.default_rng(orders)
    for b, n in enumerate(lens):
        k, v = 0.05 * rng.standard_normal((n, 1, d)), rng.uniform(1.0, 1.5, (n, 1, d))
        k[0, 0, 3], v[0] = 10.0, 0.0
        s.k[b], s.v[b] = (syn.f32_to_bf16_bits(x.astype(np.float32)) for x in (k, v))
    s.fill()
    q = 0.1 * rng.standard_normal((s.n_rows, heads, d))
    q[:, :, 3] = 8.0
    qb = syn.f32_to_bf16_bits(q.astype(np.float32))
    scale = orders * np.log(2.0) / 80.0  # the first key's score
    ws = s.cache.attention_workspace(s.rows(), heads)
    got = bf16_to_f64(host_bits(s.cache.attention(s.rows(), dev_bf16(qb), scale=scale, ws=ws)))
    s.check(ws)
    q, scale = bf16_to_f64(qb), float(np.float32(scale))
    for b, n in enumerate(counts):
        k, v = s.values(s.k[b], K_SCALE)[:, 0], s.values(s.v[b], V_SCALE)[:, 0]
        at = q[s.start[b]:s.start[b] + n]
        seen = np.arange(lens[b])[None] <= lens[b] - n + np.arange(n)[:, None]
        for h in range(heads):
            x = np.where(seen, at[:, h] @ k.T * scale, -np.inf)
            p = np.exp(x - x.max(1, keepdims=True))
            l = p.sum(1, keepdims=True)
            assert np.all(l < 1.2) and np.all(p[:, 0] == 1.0)
            ref = p @ v / l  # (v >= 0: the bound is relative to the result)
            ds = (d / 16 * 18 + 16) * 2.0 ** -23 * (np.abs(at[:, h]) @ np.abs(k).T * scale).max(1, keepdims=True) + 2.0 ** -19
            bound = 1.01 * ((2.0 ** -8 + 2.0 ** -11 + 2 * ds) * ref + 2.0 ** -32 * v.max() * seen.sum(1, keepdims=True) / l)
            bad = np.abs(got[s.start[b]:s.start[b] + n, h] - ref) - bound
            assert not np.any(~(bad <= 0)), (b, h, float((np.abs(bad + bound) / ref).max()))
