"""Host-side answers of the token-step calls that need no GPU: nothing here reaches a launch."""
import ctypes

import pytest

from bit_video_dit_b200 import build as nvbuild
from bit_video_dit_b200 import nvfp4 as nv

FAKE = 1 << 20  # never dereferenced


@pytest.fixture(scope="module")
def L():
    nvbuild.build()
    return nv.lib()


def test_gemv_without_rows(L):
    """No rows are nothing to do, whatever the row tensors (an empty tensor has no address); a bad weight, row count,
    stride or epilogue is still refused."""
    def call(x=None, m=0, y=None, ldx=256, ldy=96, n=96, k=256, **ep):
        w = nv.CTensor(FAKE, FAKE, FAKE, n, k)
        e = nv.CEpilogue(**ep) if ep else None
        return L.nvfp4_gemv(x, m, ldx, ctypes.byref(w), y, ldy, None if e is None else ctypes.byref(e), None)

    assert call() == call(x=FAKE) == call(y=FAKE) == call(act=nv.ACT_GELU_TANH) == nv.OK
    assert call(ldx=192) == call(y=FAKE, ldy=95) == call(act=7) == nv.ERR_INVALID_ARG
    assert call(k=200) == call(out_codes=FAKE) == nv.ERR_UNSUPPORTED
    assert call(m=1, x=FAKE) == call(m=1, y=FAKE) == nv.ERR_INVALID_ARG


def test_attention_with_a_record_of_its_own(L):
    cache = nv.CPagedCache(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 8, 16, 2, 64)
    rows = nv.CPagedRows(FAKE, FAKE, FAKE, 3, 4, 5, 2, 60)

    def call(record=FAKE, ws=FAKE, n=1 << 30, heads=4, r=rows):
        return L.nvfp4_paged_attention_recorded(ctypes.byref(cache), ctypes.byref(r), FAKE, 256, heads, 0, 0, 0.0, FAKE, 256,
                                                ws, n, record, None)

    assert call(record=None) == call(heads=3) == call(ws=None) == call(n=255) == nv.ERR_INVALID_ARG
    assert call(record=FAKE + 16) == call(ws=FAKE + 16) == nv.ERR_MISALIGNED
    assert call(r=nv.CPagedRows(FAKE, FAKE, FAKE, 0, 4, 5, 2, 60)) == nv.OK  # no sequences
