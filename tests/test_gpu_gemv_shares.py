"""nvfp4_gemv over weights wide enough for every way of dealing the groups of 16 rows out to the CTAs (see the share and
pass rules in gemv.cu): single groups, aligned pairs, quads, whole quads with a rest, several passes; activations resident
in shared memory and streamed; a last 128-row tile that is partly padding."""
import pytest
import torch

from bit_video_dit_b200 import nvfp4 as nv
from bit_video_dit_b200 import synthetic as syn

from .gpu_util import bf16_to_f64, dev_bf16, require_gpu
from .test_gpu_gemv import _bound, _check, _weight

pytestmark = pytest.mark.gpu

# a CTA's groups: 1; 2; 4; a whole quad and 1, 2, 4; 3 quads and a rest; 4 quads and a rest; 8 quads and a rest (more
# than one pass of 3 quads, then of 4)
N = (2300, 4096, 6999, 10250, 13000, 17000, 29900, 38500, 76500)


@pytest.mark.parametrize("n", N)
@pytest.mark.parametrize("m", [1, 3, 8, 9, 16])
def test_resident_activations(m, n):
    require_gpu()
    k = 192
    w, wf = _weight(n, k, seed=n)
    xb = syn.activations_bf16(m, k, seed=m)
    x = bf16_to_f64(xb)
    y32 = torch.empty((m, n), dtype=torch.float32, device="cuda")
    out = nv.gemv(dev_bf16(xb), w, out_f32=y32)
    _check(y32, out, x @ wf.T, _bound(x, wf))


@pytest.mark.parametrize("m,n,k", [(m, n, k) for n in N[:7] for m, k in ((4, 6336), (8, 3200), (13, 2112))] + [(13, N[7], 2112)])
def test_streamed_activations(m, n, k):
    """chunks of 128 columns x rows above 195: the activations do not fit beside the rings."""
    require_gpu()
    assert -(-k // 128) * m > 195
    w, wf = _weight(n, k, seed=n)
    xb = syn.activations_bf16(m, k, seed=m)
    x = bf16_to_f64(xb)
    y32 = torch.empty((m, n), dtype=torch.float32, device="cuda")
    out = nv.gemv(dev_bf16(xb), w, out_f32=y32)
    _check(y32, out, x @ wf.T, _bound(x, wf))
