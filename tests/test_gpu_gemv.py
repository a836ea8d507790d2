"""nvfp4_gemv against a 64-bit product of the same NVFP4 weight (the oracle's quantize and decode) and bf16 rows.

Bound of the binary32 result.  The operands are exact but for activations below 2^-28 of the largest of their row,
which move by at most 2^-25 2^-14 of it (half a binary16 step at 2^-14, under a scale that puts the maximum at 2^14 or
above).  A product passes through the 8 matrix instructions of each of a warp's chunks (8 or 16 warps share them) and
the sum of the warps.  An instruction sums 16 products and an accumulator and loses at most 18 units 2^-23 of their
magnitudes:
  |y - ref| <= (8 * 18 * ceil(chunks / 8) + 16) 2^-23 sum|x w| + 2^-39 max|x| sum|w|,
and the epilogue's own roundings, 2^-23 a step."""
import numpy as np
import pytest
import torch

import oracle
from bit_video_dit_b200 import nvfp4 as nv
from bit_video_dit_b200 import synthetic as syn

from .gpu_util import bf16_to_f64, dev_bf16, host_bits, require_gpu

pytestmark = pytest.mark.gpu


def _weight(n, k, seed):
    bits = syn.normal_bf16((n, k), seed=seed, std=0.05)
    w = nv.quantize(dev_bf16(bits))
    return w, oracle.dequant_f32(*oracle.quantize(bits)).astype(np.float64)


def _bound(x, w):
    k = x.shape[1]
    depth = 8 * 18 * -(-k // (128 * 8)) + 16
    return (depth * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T) +
            2.0 ** -39 * np.abs(x).max(1, keepdims=True) * np.abs(w).sum(1)[None])


def _check(y32, out, ref, bound):
    got = y32.cpu().numpy().astype(np.float64)
    bad = np.abs(got - ref) - bound
    assert np.all(bad <= 0), (np.unravel_index(np.argmax(bad), bad.shape), bad.max())
    assert np.array_equal(host_bits(out), host_bits(y32.to(torch.bfloat16)))


@pytest.mark.parametrize("m,n,k", [(1, 1, 64), (1, 64, 128), (2, 65, 192), (3, 129, 320), (5, 200, 1024), (7, 17, 4160),
                                   (8, 640, 2048), (9, 100, 2112), (12, 257, 640), (16, 1000, 4096), (1, 320, 16384),
                                   (16, 40000, 128)])
def test_products(m, n, k):
    require_gpu()
    w, wf = _weight(n, k, seed=n + k)
    xb = syn.activations_bf16(m, k, seed=m)
    x = bf16_to_f64(xb)
    y32 = torch.empty((m, n), dtype=torch.float32, device="cuda")
    out = nv.gemv(dev_bf16(xb), w, out_f32=y32)
    _check(y32, out, x @ wf.T, _bound(x, wf))
    # the plain call gives the same bf16
    assert torch.equal(nv.gemv(dev_bf16(xb), w), out)


def test_rows_of_very_different_size():
    """Rows near both ends of bf16's range, a zero row, and a row whose loud value hides the rest of its chunk."""
    require_gpu()
    n, k = 96, 512
    w, wf = _weight(n, k, seed=5)
    x = np.random.default_rng(6).standard_normal((6, k)).astype(np.float32)
    x[0] *= 2.0 ** 100
    x[1] *= 2.0 ** -120
    x[2] = 0.0
    x[3, 130] = 2.0 ** 40
    x[4] *= 2.0 ** np.random.default_rng(7).integers(-60, 60, k)
    xb = syn.f32_to_bf16_bits(x)
    x = bf16_to_f64(xb)
    y32 = torch.empty((6, n), dtype=torch.float32, device="cuda")
    out = nv.gemv(dev_bf16(xb), w, out_f32=y32)
    _check(y32, out, x @ wf.T, _bound(x, wf))
    assert not torch.any(out[2])


def test_zero_weight():
    require_gpu()
    w = nv.quantize(torch.zeros((70, 128), dtype=torch.bfloat16, device="cuda"))
    assert not torch.any(nv.gemv(torch.ones((2, 128), dtype=torch.bfloat16, device="cuda"), w))


@pytest.mark.parametrize("m", [1, 11])
def test_epilogue_and_strides(m):
    require_gpu()
    n, k = 150, 384
    w, wf = _weight(n, k, seed=9)
    xb = syn.normal_bf16((m, 400), seed=1)
    vecs = {v: syn.normal_bf16((n,), seed=20 + i) for i, v in enumerate(("bias", "mod_scale", "mod_shift", "gate"))}
    res = syn.normal_bf16((m, 200), seed=30)
    x = bf16_to_f64(xb)[:, :k]
    f = {v: bf16_to_f64(b) for v, b in vecs.items()}
    y = x @ wf.T
    e = _bound(x, wf)
    u = 2.0 ** -23
    y = y + f["bias"]
    e = e + u * np.abs(y)
    g = 0.5 * y * (1.0 + np.tanh(np.sqrt(2 / np.pi) * (y + 0.044715 * y ** 3)))
    # |gelu'| <= 1.13; tanh to 2 units, its argument's roundings (4 units, times |u| sech^2 u <= 0.45), the last steps
    e = 1.13 * e + 8 * u * np.abs(y)
    y = g * (1.0 + f["mod_scale"])
    e = e * np.abs(1.0 + f["mod_scale"]) + 2 * u * np.abs(y)
    y = y + f["mod_shift"]
    e = e + u * np.abs(y)
    y = f["gate"] * y
    e = e * np.abs(f["gate"]) + u * np.abs(y)
    y = bf16_to_f64(res)[:, :n] + y
    e = e + u * np.abs(y)
    y32 = torch.empty((m, n), dtype=torch.float32, device="cuda")
    whole = torch.full((m, 160), 7.0, dtype=torch.bfloat16, device="cuda")
    out = nv.gemv(dev_bf16(xb)[:, :k], w, out=whole[:, :n], out_f32=y32, act=nv.ACT_GELU_TANH,
                  residual=dev_bf16(res)[:, :n], **{v: dev_bf16(b) for v, b in vecs.items()})
    _check(y32, out, y, e)
    assert torch.all(whole[:, n:] == 7.0)


def test_captured_and_on_another_stream():
    require_gpu()
    w, _ = _weight(300, 1024, seed=3)
    x = dev_bf16(syn.normal_bf16((4, 1024), seed=2))
    want = nv.gemv(x, w)
    out = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        nv.gemv(x, w, out=out)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.gemv(x, w, out=out)
    x.copy_(dev_bf16(syn.normal_bf16((4, 1024), seed=8)))
    out.zero_()
    graph.replay()
    assert torch.equal(out, nv.gemv(x, w))


@pytest.mark.parametrize("m,k", [(3, 512), (5, 32768), (16, 640), (16, 16384)])
def test_what_is_not_finite_stays_in_its_row(m, k):
    require_gpu()
    w, _ = _weight(200, k, seed=k)
    x = dev_bf16(syn.activations_bf16(m, k, seed=m))
    want = nv.gemv(x, w)
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[1, 77] = bad
        got = nv.gemv(y, w)
        assert not torch.any(torch.isfinite(got[1]))
        got[1] = want[1]
        assert torch.equal(got, want)


def test_offsets_beyond_32_bits():
    """A weight of more than 4 GiB of codes, block scales all 1."""
    require_gpu()
    n, k, m = (1 << 20) + 150, 8192, 9
    w = nv.empty_nvfp4(n, k)
    assert w.codes.numel() > 1 << 32
    w.codes.zero_()
    w.scales.fill_(0x38)
    w.global_scale.fill_(0.125)
    rows = np.r_[0:3, n - 200:n]
    codes = np.random.default_rng(5).integers(0, 256, (rows.size, k // 2), dtype=np.uint8)
    w.codes[torch.from_numpy(rows).cuda()] = torch.from_numpy(codes).cuda()
    level = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
    wf = 0.125 * np.stack((level[codes & 15], level[codes >> 4]), -1).reshape(rows.size, k)
    xb = syn.activations_bf16(m, k, seed=3)
    x = bf16_to_f64(xb)
    y32 = torch.empty((m, n), dtype=torch.float32, device="cuda")
    out = nv.gemv(dev_bf16(xb), w, out_f32=y32)
    at = torch.from_numpy(rows).cuda()
    _check(y32[:, at], out[:, at], x @ wf.T, _bound(x, wf))
    assert not torch.any(out[:, 3:n - 200])


def test_given_streams():
    require_gpu()
    w, _ = _weight(1000, 2048, seed=1)
    xs = [dev_bf16(syn.activations_bf16(m, 2048, seed=m)) for m in (1, 4, 16)]
    want = [nv.gemv(x, w) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [(nv.gemv(x, w, stream=s), y) for _ in range(4) for x, s, y in zip(xs, streams, want)]
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a, b)


def test_python_refusals():
    require_gpu()
    w, _ = _weight(64, 128, seed=3)
    x = torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda")
    for bad in (x.float(), x[:, :64], x.T, x[0]):
        with pytest.raises(ValueError):
            nv.gemv(bad, w)
    with pytest.raises(ValueError):
        nv.gemv(x.cpu(), w)
    with pytest.raises(ValueError):
        nv.gemv(x, w, bias=torch.zeros(63, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        nv.gemv(x, w, bias=torch.zeros(64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        nv.gemv(x, w, out=torch.zeros((2, 64), device="cuda"))
    with pytest.raises(nv.NVFP4Error):
        nv.gemv(torch.zeros((17, 128), dtype=torch.bfloat16, device="cuda"), w)
