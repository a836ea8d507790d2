"""Calls of the token-step operators queued without a synchronisation between them: each kernel is resident before the one
ahead of it has ended, and still has to see what that one wrote."""
import numpy as np
import pytest
import torch

import oracle
from bit_video_dit_b200 import nvfp4 as nv
from bit_video_dit_b200 import synthetic as syn

from .gpu_util import dev_bf16, host_bits, require_gpu
from .test_gpu_paged import K_SCALE, V_SCALE, Setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,heads,d,page", [([1] * 40, 4, 128, 16), ([300, 7, 64], 2, 64, 48)])
def test_places_written_again_and_again_are_read_as_last_written(counts, heads, d, page):
    """append, gather, append, gather, ... of the same places, every step with other values: bit for bit."""
    require_gpu()
    s = Setup([n + 5 for n in counts], counts, heads, d, page, seed=d)
    rows = s.rows()
    kb = [syn.normal_bf16((s.n_rows, heads, d), seed=100 + i) for i in range(12)]
    vb = [syn.normal_bf16((s.n_rows, heads, d), seed=200 + i) for i in range(12)]
    k, v = [dev_bf16(x) for x in kb], [dev_bf16(x) for x in vb]
    out = [[torch.empty_like(k[0]) for _ in range(2)] for _ in k]
    torch.cuda.synchronize()
    for x, y, (ko, vo) in zip(k, v, out):
        s.cache.append(rows, x, y)
        s.cache.gather(rows, k_out=ko, v_out=vo)
    s.check()
    for x, y, o in zip(kb, vb, out):
        for bits, got, a in ((x, o[0], K_SCALE), (y, o[1], V_SCALE)):
            want = oracle.dequant_bf16(*oracle.quantize(bits.reshape(-1, d), alpha=a)).reshape(bits.shape)
            assert np.array_equal(host_bits(got), want)


@pytest.mark.parametrize("counts,lens", [([1, 1, 1], [700, 33, 90]), ([1, 2, 1], [5000, 4100, 60]), ([4, 8, 4], [60, 900, 30])])
def test_decoder_layers_in_one_queue(counts, lens):
    """gemv, append, attention and gemv over the same buffers, layer after layer: the same bits as with every call waited
    for (single tokens in one launch and in runs, and chunks)."""
    require_gpu()
    kv, heads, d, width = 2, 8, 128, 512
    s = Setup(lens, counts, kv, d, 16, seed=3).fill()
    rows, n = s.rows(), s.n_rows
    w_in = nv.quantize(dev_bf16(syn.normal_bf16(((heads + 2 * kv) * d, width), seed=1, std=0.06)))
    w_out = nv.quantize(dev_bf16(syn.normal_bf16((width, heads * d), seed=2, std=0.06)))
    ws = s.cache.attention_workspace(rows, heads)
    first = dev_bf16(syn.normal_bf16((n, width), seed=4))
    held = [t.clone() for t in (s.cache.k_codes, s.cache.k_scales, s.cache.v_codes, s.cache.v_scales)]

    def layers(wait):
        for t, h in zip((s.cache.k_codes, s.cache.k_scales, s.cache.v_codes, s.cache.v_scales), held):
            t.copy_(h)
        x, kept = first.clone(), []
        qkv = torch.empty((n, heads + 2 * kv, d), dtype=torch.bfloat16, device="cuda")
        o = torch.empty((n, heads, d), dtype=torch.bfloat16, device="cuda")
        results = [torch.empty_like(x) for _ in range(10)]
        torch.cuda.synchronize()
        for y in results:
            for call in (lambda: nv.gemv(x, w_in, out=qkv.view(n, -1)),
                         lambda: s.cache.append(rows, qkv[:, heads:heads + kv], qkv[:, heads + kv:]),
                         lambda: s.cache.attention(rows, qkv[:, :heads], out=o, ws=ws),
                         lambda: nv.gemv(o.view(n, -1), w_out, out=y, residual=x)):
                call()
                if wait:
                    torch.cuda.synchronize()
            kept.append(y)
            x = y
        s.check(), s.check(ws)
        return kept

    for a, b in zip(layers(True), layers(False)):
        assert torch.all(torch.isfinite(a)) and torch.equal(a, b)


def test_a_gemm_behind_the_kernel_that_writes_its_residual():
    """nvfp4_gemm with CTA pairs right behind the nvfp4_gemv that writes rows of its residual, and behind the nvfp4_gemm
    whose result is its residual: the same bits as with every call waited for."""
    require_gpu()
    m, n, k = 272, 4096, 512
    w = nv.quantize(dev_bf16(syn.normal_bf16((n, k), seed=1, std=0.06)))
    a = nv.quantize(dev_bf16(syn.normal_bf16((m, k), seed=2)))
    x = [dev_bf16(syn.normal_bf16((16, k), seed=10 + i)) for i in range(6)]
    ws = nv.workspace(nv.OP_GEMM, m, n, k)

    def queue(wait):
        y = torch.zeros((m, n), dtype=torch.bfloat16, device="cuda")
        out = [torch.empty_like(y) for _ in range(2 * len(x))]
        torch.cuda.synchronize()
        for i, t in enumerate(x):
            at = slice(16 * i, 16 * i + 16) if i % 2 else slice(m - 16 * i - 16, m - 16 * i)
            for call in (lambda: nv.gemv(t, w, out=y[at]), lambda: nv.gemm(a, w, out=out[2 * i], residual=y, ws=ws),
                         lambda: nv.gemm(a, w, out=out[2 * i + 1], residual=out[2 * i], ws=ws)):
                call()
                if wait:
                    torch.cuda.synchronize()
        assert nv.read_device_error(ws) == (nv.OK, 0)
        return out

    for p, q in zip(queue(True), queue(False)):
        assert torch.all(torch.isfinite(p)) and torch.equal(p, q)
