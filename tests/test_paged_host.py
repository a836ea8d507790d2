"""Host-side refusals of nvfp4_gemv and of the paged cache's calls, and the attention's workspace
query: every check runs before any launch, so none of this needs a GPU."""
import ctypes

import pytest

from bit_video_dit_b200 import build as nvbuild
from bit_video_dit_b200 import nvfp4 as nv

FAKE = 1 << 20  # never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def L():
    nvbuild.build()
    return nv.lib()


def _gemv(L, m=4, ldx=256, n=96, k=256, y=FAKE, ldy=96, x=FAKE, codes=FAKE, ep=None):
    w = nv.CTensor(codes, FAKE, FAKE, n, k)
    return L.nvfp4_gemv(x, m, ldx, ctypes.byref(w), y, ldy, None if ep is None else ctypes.byref(ep), None)


def test_gemv_refusals(L):
    assert L.nvfp4_gemv(FAKE, 1, 64, None, FAKE, 64, None, None) == nv.ERR_INVALID_ARG
    for kw, want in ((dict(m=17), nv.ERR_UNSUPPORTED), (dict(m=-1), nv.ERR_INVALID_ARG),
                     (dict(k=96, ldx=96), nv.ERR_UNSUPPORTED), (dict(n=0), nv.ERR_INVALID_ARG),
                     (dict(n=(1 << 30) + 1, ldy=1 << 31), nv.ERR_UNSUPPORTED), (dict(ldx=248), nv.ERR_INVALID_ARG),
                     (dict(ldx=260), nv.ERR_MISALIGNED), (dict(ldy=95), nv.ERR_INVALID_ARG),
                     (dict(y=None), nv.ERR_INVALID_ARG), (dict(x=None), nv.ERR_INVALID_ARG),
                     (dict(x=FAKE + 8), nv.ERR_MISALIGNED), (dict(codes=FAKE + 8), nv.ERR_MISALIGNED),
                     (dict(y=FAKE + 1), nv.ERR_MISALIGNED), (dict(m=0), nv.OK)):
        assert _gemv(L, **kw) == want, kw
    for ep, want in ((nv.CEpilogue(act=2), nv.ERR_INVALID_ARG), (nv.CEpilogue(debug_flags=1), nv.ERR_INVALID_ARG),
                     (nv.CEpilogue(residual=FAKE, ld_residual=95), nv.ERR_INVALID_ARG),
                     (nv.CEpilogue(out_codes=FAKE), nv.ERR_UNSUPPORTED), (nv.CEpilogue(out_amax=FAKE), nv.ERR_UNSUPPORTED),
                     (nv.CEpilogue(out_col0=64), nv.ERR_UNSUPPORTED), (nv.CEpilogue(bias=FAKE + 1), nv.ERR_MISALIGNED)):
        assert _gemv(L, ep=ep) == want


def _cache(**kw):
    a = dict(k_codes=FAKE, k_scales=FAKE, v_codes=FAKE, v_scales=FAKE, k_global=FAKE, v_global=FAKE, n_pages=8,
             page_size=16, kv_heads=2, head_dim=64)
    a.update(kw)
    return nv.CPagedCache(**a)


def _rows(**kw):
    a = dict(row_start=FAKE, lens=FAKE, pages=FAKE, n_seqs=3, max_pages=4, n_rows=5, max_rows=2, max_len=60)
    a.update(kw)
    return nv.CPagedRows(**a)


BAD = ((dict(head_dim=96), {}, nv.ERR_UNSUPPORTED), (dict(page_size=24), {}, nv.ERR_UNSUPPORTED),
       (dict(page_size=0), {}, nv.ERR_INVALID_ARG), (dict(kv_heads=0), {}, nv.ERR_INVALID_ARG),
       (dict(n_pages=0), {}, nv.ERR_INVALID_ARG), (dict(k_codes=None), {}, nv.ERR_INVALID_ARG),
       (dict(v_scales=FAKE + 8), {}, nv.ERR_MISALIGNED), (dict(k_global=FAKE + 2), {}, nv.ERR_MISALIGNED),
       ({}, dict(n_seqs=-1), nv.ERR_INVALID_ARG), ({}, dict(n_rows=-1), nv.ERR_INVALID_ARG),
       ({}, dict(n_rows=(1 << 30) + 1), nv.ERR_UNSUPPORTED), ({}, dict(lens=None), nv.ERR_INVALID_ARG),
       ({}, dict(pages=None), nv.ERR_INVALID_ARG), ({}, dict(row_start=FAKE + 2), nv.ERR_MISALIGNED),
       ({}, dict(max_len=-1), nv.ERR_INVALID_ARG))


@pytest.mark.parametrize("c,r,want", BAD)
def test_paged_calls_refuse_bad_caches_and_rows(L, c, r, want):
    cc, rr = _cache(**c), _rows(**r)
    a = (ctypes.byref(cc), ctypes.byref(rr))
    width = 2 * max(64, cc.head_dim)
    assert L.nvfp4_paged_append(*a, FAKE, width, FAKE, width, None, None, FAKE, 256, None) == want
    assert L.nvfp4_paged_gather(*a, FAKE, width, FAKE, width, FAKE, 256, None) == want
    assert L.nvfp4_paged_attention(*a, FAKE, 2 * width, 4, 0, 0, 0.0, FAKE, 2 * width, FAKE, 1 << 30, None) == want


def test_paged_row_call_refusals(L):
    cc, rr = _cache(), _rows()
    a = (ctypes.byref(cc), ctypes.byref(rr))
    app = L.nvfp4_paged_append
    assert app(*a, None, 128, FAKE, 128, None, None, FAKE, 256, None) == nv.ERR_INVALID_ARG
    assert app(*a, FAKE, 120, FAKE, 128, None, None, FAKE, 256, None) == nv.ERR_INVALID_ARG
    assert app(*a, FAKE, 132, FAKE, 128, None, None, FAKE, 256, None) == nv.ERR_MISALIGNED
    assert app(*a, FAKE + 8, 128, FAKE, 128, None, None, FAKE, 256, None) == nv.ERR_MISALIGNED
    assert app(*a, FAKE, 128, FAKE, 128, FAKE, None, FAKE, 256, None) == nv.ERR_INVALID_ARG  # half a table pair
    assert app(*a, FAKE, 128, FAKE, 128, FAKE + 4, FAKE, FAKE, 256, None) == nv.ERR_MISALIGNED
    assert app(*a, FAKE, 128, FAKE, 128, None, None, FAKE, 255, None) == nv.ERR_INVALID_ARG  # workspace
    assert app(*a, FAKE, 128, FAKE, 128, None, None, FAKE + 16, 256, None) == nv.ERR_MISALIGNED
    empty = _rows(n_rows=0, row_start=None, lens=None, pages=None)
    assert app(a[0], ctypes.byref(empty), None, 128, None, 128, None, None, FAKE, 256, None) == nv.OK
    assert L.nvfp4_paged_gather(*a, FAKE, 128, None, 128, FAKE, 256, None) == nv.ERR_INVALID_ARG


def test_paged_attention_refusals(L):
    cc, rr = _cache(), _rows()

    def att(q=FAKE, ld_q=256, heads=4, window=0, sinks=0, scale=0.0, o=FAKE, ld_o=256, ws=FAKE, n=1 << 30, r=rr):
        return L.nvfp4_paged_attention(ctypes.byref(cc), ctypes.byref(r), q, ld_q, heads, window, sinks, scale, o, ld_o,
                                       ws, n, None)

    for kw, want in ((dict(heads=3), nv.ERR_INVALID_ARG), (dict(heads=0), nv.ERR_INVALID_ARG),
                     (dict(window=-1), nv.ERR_INVALID_ARG), (dict(sinks=-1), nv.ERR_INVALID_ARG),
                     (dict(window=(1 << 30) + 1), nv.ERR_UNSUPPORTED), (dict(scale=-1.0), nv.ERR_INVALID_ARG),
                     (dict(scale=float("nan")), nv.ERR_INVALID_ARG), (dict(scale=float("inf")), nv.ERR_INVALID_ARG),
                     (dict(q=None), nv.ERR_INVALID_ARG), (dict(o=None), nv.ERR_INVALID_ARG),
                     (dict(ld_q=248), nv.ERR_INVALID_ARG), (dict(ld_o=260), nv.ERR_MISALIGNED),
                     (dict(q=FAKE + 8), nv.ERR_MISALIGNED), (dict(ws=None), nv.ERR_INVALID_ARG),
                     (dict(n=100), nv.ERR_INVALID_ARG), (dict(r=_rows(max_rows=0)), nv.OK),
                     (dict(r=_rows(n_seqs=0)), nv.OK),
                     (dict(r=_rows(max_rows=1 << 30, n_seqs=1 << 20)), nv.ERR_UNSUPPORTED)):
        assert att(**kw) == want, kw


def test_attention_workspace_query(L):
    def need(heads=4, window=0, sinks=0, c={}, **r):
        return L.nvfp4_paged_attention_workspace_bytes(ctypes.byref(_cache(**c)), ctypes.byref(_rows(**r)), heads, window,
                                                       sinks)

    # two pieces of a unit a CTA: no more for more sequences once every SM has its CTAs; larger for chunks
    assert need(max_len=100000) == need(max_len=200000) == need(n_seqs=700, n_rows=1000, max_len=100000) > need()
    assert need() == need(max_len=100000, window=100) == 256  # short spans are not cut into pieces
    assert need(max_len=100000) == need(max_len=100000, window=9000, n_seqs=1000)
    long = need(max_rows=100, max_len=100000)
    assert need(max_len=100000) < need(max_rows=8, max_len=100000) < long <= 40 << 20
    assert need(heads=3) == 0 and need(window=-1) == 0 and need(c=dict(head_dim=80)) == 0
    cc, rr = _cache(), _rows(max_rows=100, max_len=100000)
    # one byte less than the query says is refused
    assert L.nvfp4_paged_attention(ctypes.byref(cc), ctypes.byref(rr), FAKE, 256, 4, 0, 0, 0.0, FAKE, 256, FAKE,
                                   long - 1, None) == nv.ERR_INVALID_ARG
