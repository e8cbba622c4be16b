"""GPU tests of the fused residual addition + RMS norm + FP8 quantization against float64.

Tolerance. The residual sum is exact up to one rounding to the dtype: compared bit for bit. With
|y_gpu - y| <= d |y|: a row's sum of squares is a chain of at most 64 + 6 + 16 float32 additions
of positive terms (each off by 2^-24 at most), halved by the square root, then a handful of single
roundings, so d = 2^-17 covers it twice over. A code times its scale is then within half an e4m3
step (2^-4 of the value, 2^-10 of the scale near zero) of y, plus 2 d |y| for y and the scale. A
UE8M0 scale may differ where amax / 448 is within d of a power of two."""

import numpy as np
import pytest
import torch

import block_scaled_fp8_bfp8_amd as bfp8
from oracle import e4m3, latent
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu
D = 2.0 ** -17


def _check(x, w, res, eps, q, s, h, e8):
    if res is not None:
        want_h = (x.float() + res.float()).to(x.dtype)
        assert torch.equal(h.cpu().view(torch.uint8), want_h.view(torch.uint8)), "h differs"
    else:
        want_h = x
    y = latent.rmsnorm_ref(want_h.double().numpy(), w.double().numpy(), eps)
    m, k = y.shape
    g = -(-k // 128)
    amax = np.abs(np.pad(y, ((0, 0), (0, g * 128 - k)))).reshape(m, g, 128).max(axis=2)
    want_s = np.maximum(amax, 1e-10) / 448
    s = s.cpu().contiguous()
    if e8:
        got_s = latent.e8m0_value(s.numpy())
        lo, hi = (np.exp2(np.ceil(np.log2(want_s * f))) for f in (1 - 2 * D, 1 + 2 * D))
        assert ((got_s == lo) | (got_s == hi)).all()
    else:
        got_s = s.double().numpy()
        assert (np.abs(got_s - want_s) <= 2 * D * want_s).all()
    sc = np.repeat(got_s, 128, axis=1)[:, :k]
    got = e4m3.decode(np.ascontiguousarray(q.cpu().numpy())) * sc
    bound = np.maximum(np.abs(y) * 2.0 ** -4, sc * 2.0 ** -10) + 2 * D * np.abs(y)
    over = np.abs(got - y) > bound
    assert not over.any(), f"{over.sum()} codes off, first at {np.argwhere(over)[0]}"


@pytest.mark.parametrize("e8", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("m,h,with_res", [
    (1, 16, True), (3, 128, False), (5, 144, True), (67, 512, True), (2, 528, False), (130, 1040, True), (3, 2048, True),
    (1, 2064, False), (1, 7168, True), (300, 4096, True), (2, 8208, True), (3, 16384, False), (2, 16400, True),
    (600, 2064, True), (520, 7168, True), (513, 16384, True), (1, 65536, True), (2, 65520, False)])
def test_against_float64(gpu, m, h, with_res, dtype, e8):
    announce("rmsnorm", m, h, with_res, dtype, e8)
    g = torch.Generator().manual_seed(m * 100003 + h)
    x = torch.randn(m, h, generator=g).to(dtype)
    res = (3 * torch.randn(m, h, generator=g)).to(dtype) if with_res else None
    w = (1 + 0.3 * torch.randn(h, generator=g)).to(dtype)
    call = bfp8.rmsnorm_quant_ue8m0 if e8 else bfp8.rmsnorm_quant
    q, s, hh = call(x.to(gpu), w.to(gpu), residual=None if res is None else res.to(gpu), eps=1e-6)
    assert q.shape == (m, h) and q.stride(0) == -(-h // 128) * 128 and s.shape == (m, -(-h // 128))
    _check(x, w, res, 1e-6, q, s, hh, e8)


def test_strides_and_in_place_stream(gpu):
    m, h = 37, 1040
    g = torch.Generator().manual_seed(5)
    x, res = torch.randn(m, h + 16, generator=g).bfloat16(), torch.randn(m, h + 48, generator=g).bfloat16()
    w = torch.randn(h, generator=g).bfloat16()
    announce("rmsnorm strided in place", m, h)
    xd, rd = x.to(gpu), res.to(gpu)
    q, s, out = bfp8.rmsnorm_quant(xd[:, :h], w.to(gpu), residual=rd[:, :h], out=rd[:, :h])
    assert out.data_ptr() == rd.data_ptr()
    _check(x[:, :h], w, res[:, :h], 1e-6, q, s, out.contiguous(), False)
    assert torch.equal(rd[:, h:].cpu(), res[:, h:])  # columns past the row are untouched


def test_zero_rows_large_values_and_nan(gpu):
    h = 512
    x = torch.zeros(4, h)
    x[1] = 1e18
    x[2, 5] = float("nan")
    x[3] = 1.0
    w = torch.ones(h)
    w[300] = float("inf")  # only the group of column 300 is affected
    announce("rmsnorm special values")
    q, s, _ = bfp8.rmsnorm_quant(x.to(gpu), w.to(gpu))
    v, sc = e4m3.decode(np.ascontiguousarray(q.cpu().numpy())), s.cpu().contiguous().numpy()
    floor = np.float32(1e-10) / np.float32(448)
    assert (v[0, :256] == 0).all() and (sc[0, [0, 1, 3]] == floor).all()
    assert np.isnan(v[0, 256:384]).all() and np.isnan(sc[0, 2])  # 0 * inf
    np.testing.assert_allclose(v[1, :256] * sc[1, 0], 1.0, rtol=2.0 ** -4)  # 1e18^2 is finite in float32
    assert np.isnan(v[2]).all() and np.isnan(sc[2]).all()
    assert np.isinf(sc[3, 2]) and np.isnan(v[3, 300]) and (np.delete(v[3, 256:384], 44) == 0).all()
    qe, e, _ = bfp8.rmsnorm_quant_ue8m0(x.to(gpu), w.to(gpu))
    assert (e.cpu()[2] == 255).all() and e.cpu()[3, 2] == 255 and (e.cpu()[3, [0, 1, 3]] == 127 - 8).all()


def test_feeds_the_gemms_as_the_quantizer_does(gpu):
    """With weights of one and rows of equal magnitude the norm divides by that magnitude exactly,
    so the codes are quant_act's of the signs; both GEMMs take them."""
    m, h, n = 5, 1024, 256
    g = torch.Generator().manual_seed(9)
    sign = torch.randint(0, 2, (m, h), generator=g).float() * 2 - 1
    x = (sign * 4).bfloat16().to(gpu)
    announce("rmsnorm into gemm")
    q, s, _ = bfp8.rmsnorm_quant(x, torch.ones(h, dtype=torch.bfloat16, device=gpu), eps=0.0)
    q2, s2 = bfp8.quant_act(sign.to(gpu))
    assert torch.equal(q, q2) and torch.equal(s, s2)
    b = torch.randint(0, 0x7F, (n, h), dtype=torch.uint8, generator=g).to(gpu)
    bs = torch.rand(n // 128, h // 128, generator=g).to(gpu)
    assert torch.equal(bfp8.gemm(q, s, b, bs), bfp8.gemm(q2, s2, b, bs))


def test_empty_and_refusals(gpu):
    w = torch.ones(256, dtype=torch.bfloat16, device=gpu)
    x = torch.zeros(0, 256, dtype=torch.bfloat16, device=gpu)
    q, s, _ = bfp8.rmsnorm_quant(x, w)
    assert q.shape == (0, 256) and s.shape == (0, 2)
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device=gpu)
    for call in (bfp8.rmsnorm_quant, bfp8.rmsnorm_quant_ue8m0):
        with pytest.raises(TypeError):
            call(x, w.float())
        with pytest.raises(ValueError):
            call(x, w[:128])
        with pytest.raises(ValueError):
            call(x, w, residual=x[:2])
        with pytest.raises(ValueError):
            call(x, w, out=x)  # no residual
        with pytest.raises(ValueError):
            call(x, w, residual=x, eps=-1.0)
        with pytest.raises(NotImplementedError):
            call(x[:, :200], w[:200])
        with pytest.raises(ValueError):
            call(x.t(), w[:4])


@pytest.mark.parametrize("e8", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,h", [(7, 256), (5, 512), (33, 1040), (6, 4096), (3, 7168), (5, 16400), (2, 65536)])
def test_stream_updated_in_place_of_x(gpu, m, h, dtype, e8):
    """out = x, with one wave, several waves and several chunks a row."""
    g = torch.Generator().manual_seed(m * 1009 + h)
    x, res = torch.randn(m, h, generator=g).to(dtype), (2 * torch.randn(m, h, generator=g)).to(dtype)
    w = (1 + 0.3 * torch.randn(h, generator=g)).to(dtype)
    announce("rmsnorm out = x", m, h, dtype, e8)
    call = bfp8.rmsnorm_quant_ue8m0 if e8 else bfp8.rmsnorm_quant
    xd = x.to(gpu)
    q, s, out = call(xd, w.to(gpu), residual=res.to(gpu), out=xd)
    assert out is xd
    _check(x, w, res, 1e-6, q, s, out, e8)
    want = call(x.to(gpu), w.to(gpu), residual=res.to(gpu))
    assert torch.equal(q, want[0]) and torch.equal(s, want[1]) and torch.equal(out, want[2])


@pytest.mark.parametrize("e8", [False, True])
@pytest.mark.parametrize("dtype,size", [(torch.bfloat16, 2.0 ** 62), (torch.bfloat16, 2.0 ** 110), (torch.bfloat16, 2.0 ** 125),
                                        (torch.float32, 2.0 ** 125)])
@pytest.mark.parametrize("m,h", [(3, 128), (2, 1040), (2, 7168), (1, 65536)])
def test_rows_whose_squares_pass_float32(gpu, m, h, dtype, size, e8):
    """Finite rows up to the type's range are normed as any other."""
    g = torch.Generator().manual_seed(h)
    x = (torch.randn(m, h, generator=g).clamp(-3.9, 3.9) * size).to(dtype)
    x[0, h // 2] = torch.finfo(dtype).max
    w = (1 + 0.3 * torch.randn(h, generator=g)).to(dtype)
    announce("rmsnorm large rows", m, h, dtype, size, e8)
    call = bfp8.rmsnorm_quant_ue8m0 if e8 else bfp8.rmsnorm_quant
    q, s, hh = call(x.to(gpu), w.to(gpu))
    _check(x, w, None, 1e-6, q, s, hh, e8)


@pytest.mark.parametrize("e8", [False, True])
@pytest.mark.parametrize("size,eps", [(2.0 ** -70, 0.0), (2.0 ** -100, 0.0), (2.0 ** -120, 0.0), (2.0 ** -60, 2.0 ** -121)])
@pytest.mark.parametrize("m,h", [(3, 128), (2, 1040), (2, 7168), (1, 65536)])
def test_rows_whose_squares_vanish_in_float32(gpu, m, h, size, eps, e8):
    """With an eps as small as the rows' mean square, or none, tiny rows are normed as any other."""
    g = torch.Generator().manual_seed(h + 1)
    x = (torch.randn(m, h, generator=g) * size).bfloat16()
    w = (1 + 0.3 * torch.randn(h, generator=g)).bfloat16()
    announce("rmsnorm tiny rows", m, h, size, eps, e8)
    call = bfp8.rmsnorm_quant_ue8m0 if e8 else bfp8.rmsnorm_quant
    q, s, hh = call(x.to(gpu), w.to(gpu), eps=eps)
    _check(x, w, None, eps, q, s, hh, e8)
