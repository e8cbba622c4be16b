"""GPU tests of the integer products at the ends of float32's range: tokens so large that the sum of their codes times
their scale passes it, while the channel's scale brings the output back."""

import pytest
import torch

import block_scaled_fp8_bfp8_amd as bfp8
from tests.gpu_util import announce
from tests.test_gpu_int8 import TYPES, _check_product, _codes

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k", [(1, 40, 256), (5, 100, 528), (40, 333, 2064), (300, 777, 640), (513, 1030, 144)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gemm_of_huge_tokens(gpu, m, n, k, dtype):
    """Every third token's scale is 2^97 to 2^127, channels' scales bring most outputs into the type's range. The others'
    outputs are what they are without such tokens, bit for bit."""
    g = torch.Generator().manual_seed(m + 7 * n + 31 * k)
    q, w = _codes((m, k), g).to(gpu), _codes((n, k), g).to(gpu)
    s = 0.02 * torch.exp(torch.randn(m, generator=g))
    huge = torch.arange(m) % 3 == 0
    s = torch.where(huge, torch.exp2(97 + 30 * torch.rand(m, generator=g)) * (1 - 2 * (torch.arange(m) % 2)), s).to(gpu)
    ws = torch.exp2(-126 + 20 * torch.rand(n, generator=g)).to(gpu)
    ws[1::2] = 0.0005
    ws[::7] = 0.0
    bias = torch.randn(n, generator=g).to(TYPES[dtype]).to(gpu) if n % 2 else None
    announce("gemm_int8 huge tokens", m, n, k, dtype)
    got = bfp8.gemm_int8(q, s, w, ws, bias=bias, dtype=TYPES[dtype])
    # outputs past the type's range are infinite; the rest within the product's tolerance
    exact = (q.double() @ w.double().t()) * s.double()[:, None] * ws.double() + (0.0 if bias is None else bias.double())
    past = exact.abs() > float(torch.finfo(TYPES[dtype]).max) * (1 + 2.0 ** -6)
    assert bool((got[past].double() == exact[past].sign() * float("inf")).all())
    near = ~past & (exact.abs() >= float(torch.finfo(TYPES[dtype]).max) * (1 - 2.0 ** -6))
    for i in torch.nonzero(~(past | near).all(dim=1)).flatten().tolist()[:64]:
        ok = ~(past | near)[i]
        _check_product(got[i:i + 1, ok], q[i:i + 1], s[i:i + 1], w[ok], ws[ok], None if bias is None else bias[ok], (m, n, k, i))
    small = ~huge.to(gpu)
    if bool(small.any()):
        calm = torch.where(small, s, 1.0)
        assert torch.equal(got[small], bfp8.gemm_int8(q, calm, w, ws, bias=bias, dtype=TYPES[dtype])[small])


@pytest.mark.parametrize("m,n,k", [(1, 64, 512), (4, 300, 1024), (8, 200, 2048), (9, 300, 1024), (200, 1000, 1024), (2100, 512, 1024)])
def test_linear_of_huge_tokens(gpu, m, n, k):
    """Whole layers in bf16: tokens of 10^37 and a weight of 10^-3 give finite outputs."""
    g = torch.Generator().manual_seed(m + n + k)
    x = (torch.randn(m, k, generator=g) * 2e36).to(torch.bfloat16).to(gpu)
    w, ws = bfp8.quant_act_int8((torch.randn(n, k, generator=g) * 1e-3).to(gpu))
    bias = torch.randn(n, generator=g).to(torch.bfloat16).to(gpu)
    announce("linear_int8 huge tokens", m, n, k)
    got = bfp8.linear_int8(x, w, ws, bias)
    q, s = bfp8.quant_act_int8(x)
    assert bool(got.isfinite().all())
    _check_product(got, q, s, w, ws, bias, (m, n, k))
    assert torch.equal(got, bfp8.gemm_int8(q, s, w, ws, bias=bias))
