"""The token-step calls as Python programs make them: no rows, workspaces and tensors that do not fit, and where a call's
errors are read."""
import pytest
import torch

from bit_video_dit_b200 import nvfp4 as nv
from bit_video_dit_b200 import synthetic as syn

from .gpu_util import dev_bf16, require_gpu

pytestmark = pytest.mark.gpu


def _weight(n=96, k=256):
    return nv.quantize(dev_bf16(syn.normal_bf16((n, k), seed=1)))


def test_gemv_of_no_rows():
    require_gpu()
    w, x = _weight(), dev_bf16(syn.normal_bf16((4, 256), seed=2))
    bias = dev_bf16(syn.normal_bf16((96,), seed=3))
    for y in (nv.gemv(x[:0], w), nv.gemv(x[4:], w, bias=bias, act=nv.ACT_GELU_TANH),
              nv.gemv(x[:0], w, residual=torch.zeros((0, 96), dtype=torch.bfloat16, device="cuda"))):
        assert y.shape == (0, 96) and y.dtype == torch.bfloat16


def _step(counts, lens, page=16, heads=2, d=64):
    """A cache whose sequences have pages of their own, written with normal values, and the step's rows."""
    held = [-(-n // page) for n in lens]
    table = torch.full((len(lens), max(held) + 1), -1, dtype=torch.int32)
    for b, n in enumerate(held):
        table[b, :n] = sum(held[:b]) + torch.arange(n)
    cache = nv.PagedKVCache(sum(held), page, heads, d, k_scale=0.004, v_scale=0.004)

    def rows(n, table=table):
        start = torch.tensor([0, *n]).cumsum(0).to(torch.int32)
        return nv.PagedRows(start.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), n_rows=sum(n),
                            max_rows=max(n), max_len=max(lens))

    x = dev_bf16(syn.normal_bf16((sum(lens), heads, d), seed=7))
    cache.append(rows(lens), x, x)
    return cache, rows, table


@pytest.mark.parametrize("counts,lens", [([1, 1], [40, 60]), ([1, 2], [60, 3000]), ([1, 50], [60, 3000])])
def test_what_an_attention_without_a_workspace_finds_is_kept(counts, lens):
    """A bad page shows in the cache's own record, and stays there through later calls until it is read."""
    require_gpu()
    cache, rows, table = _step(counts, lens)
    q = dev_bf16(syn.normal_bf16((sum(counts), 4, 64), seed=3))
    good = rows(counts)
    want = cache.attention(good, q)
    assert nv.read_device_error(cache.ws_rows) == (nv.OK, 0)
    bad = table.clone()
    bad[1, 1] = cache.n_pages
    cache.attention(rows(counts, bad), q)
    assert torch.equal(cache.attention(good, q), want)
    assert nv.read_device_error(cache.ws_rows) == (nv.ERR_DEVICE, 1)
    assert nv.read_device_error(cache.ws_rows) == (nv.OK, 0)
    # a workspace that is given has the record of its calls
    ws = cache.attention_workspace(good, 4)
    cache.attention(rows(counts, bad), q, ws=ws)
    assert nv.read_device_error(cache.ws_rows) == (nv.OK, 0)
    assert nv.read_device_error(ws) == (nv.ERR_DEVICE, 1)


def test_a_captured_attention_without_a_workspace_reports_too():
    require_gpu()
    cache, rows, table = _step([1, 1], [40, 3000])
    q = dev_bf16(syn.normal_bf16((2, 4, 64), seed=3))
    r = rows([1, 1])
    want = cache.attention(r, q).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cache.attention(r, q)
    graph.replay()
    assert nv.read_device_error(cache.ws_rows) == (nv.OK, 0) and torch.equal(out, want)
    good = r.pages.clone()
    r.pages[1, 3] = -5
    graph.replay()
    assert nv.read_device_error(cache.ws_rows) == (nv.ERR_DEVICE, 1)
    r.pages.copy_(good)
    graph.replay()
    assert nv.read_device_error(cache.ws_rows) == (nv.OK, 0) and torch.equal(out, want)


def test_tensors_on_another_device_are_refused():
    """Here the host: a weight's scales and workspaces."""
    require_gpu()
    w, x = _weight(), dev_bf16(syn.normal_bf16((4, 256), seed=2))
    for part in ("codes", "scales", "global_scale"):
        parts = {name: getattr(w, name) for name in ("codes", "scales", "global_scale")}
        parts[part] = parts[part].cpu()
        with pytest.raises(ValueError):
            nv.gemv(x, nv.NVFP4Tensor(rows=w.rows, cols=w.cols, **parts))
    cache, rows, _ = _step([1, 1], [40, 60])
    r = rows([1, 1])
    k, q = dev_bf16(syn.normal_bf16((2, 2, 64), seed=3)), dev_bf16(syn.normal_bf16((2, 4, 64), seed=3))
    ws = cache.attention_workspace(r, 4)
    for bad in (ws.cpu(), ws[:1].expand(1 << 20), torch.zeros(2 * ws.numel(), dtype=torch.uint8, device="cuda")[::2]):
        for call in (lambda: cache.append(r, k, k, ws=bad), lambda: cache.gather(r, ws=bad),
                     lambda: cache.attention(r, q, ws=bad)):
            with pytest.raises(ValueError):
                call()


def test_a_workspace_of_words_counts_its_bytes():
    require_gpu()
    cache, rows, _ = _step([1, 1], [40, 3000])
    r, q = rows([1, 1]), dev_bf16(syn.normal_bf16((2, 4, 64), seed=3))
    ws = cache.attention_workspace(r, 4)
    words = torch.zeros(ws.numel() // 4, dtype=torch.int32, device="cuda")
    assert torch.equal(cache.attention(r, q, ws=words), cache.attention(r, q, ws=ws))
    with pytest.raises(nv.NVFP4Error):
        cache.attention(r, q, ws=words[:-1])


def test_numbers_beyond_32_bits_are_refused():
    """None of them may come out as its low bits (a window of 2^32 + 5 as one of 5)."""
    require_gpu()
    cache, rows, _ = _step([1, 1], [40, 60])
    r, q = rows([1, 1]), dev_bf16(syn.normal_bf16((2, 4, 64), seed=3))
    ws = cache.attention_workspace(r, 4)
    for kw in (dict(window=2 ** 32 + 5), dict(window=30, sinks=2 ** 32), dict(window=2 ** 31)):
        with pytest.raises(ValueError):
            cache.attention(r, q, ws=ws, **kw)
        with pytest.raises(ValueError):
            cache.attention_workspace(r, 4, **kw)
    with pytest.raises(ValueError):
        cache.attention_workspace(r, 2 ** 32 + 4)
    for kw in (dict(n_rows=2 ** 32 + 2), dict(max_rows=2 ** 32 + 1), dict(max_len=2 ** 32)):
        with pytest.raises(ValueError):
            nv.PagedRows(r.row_start, r.lens, r.pages, **{**dict(n_rows=2, max_rows=1, max_len=60), **kw})
