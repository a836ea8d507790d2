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
