"""GPU tests of every kernel of the integer product over a K that fills its stages or slots more than twice, with a whole
and with a partial last block (the tolerance is that of tests/test_gpu_int8.py). The library says which kernel a size runs,
so that another choice by size does not take one out of the tests unseen."""

import numpy as np
import pytest
import torch

import block_scaled_fp8_bfp8_amd as bfp8
from tests.gpu_util import announce
from tests.test_abi_int8_kernels import LONG
from tests.test_gpu_int8 import TYPES, _check_product, _codes

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kernel,m,n,k", LONG)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gemm_of_every_kernel_over_a_long_k(gpu, kernel, m, n, k, dtype):
    assert bfp8.gemm_int8_kernel_for(m, n, k) == kernel
    announce("gemm_int8", *kernel, m, n, k, dtype)
    g = torch.Generator().manual_seed(m + 7 * n + 31 * k)
    q, w = _codes((m, k), g).to(gpu), _codes((n, k), g).to(gpu)
    s, ws = (0.02 * torch.exp(torch.randn(m, generator=g))).to(gpu), (0.0005 * torch.exp(torch.randn(n, generator=g))).to(gpu)
    bias = torch.randn(n, generator=g).to(TYPES[dtype]).to(gpu) if k % 128 else None
    got = bfp8.gemm_int8(q, s, w, ws, bias=bias, dtype=TYPES[dtype])
    _check_product(got, q, s, w, ws, bias, (kernel, m, n, k, dtype))


def _steps(q, s, w, ws, bias):
    """The outputs in fp16 by the kernels' steps: the exact sum in float32, times the token's scale in float32, then the
    product with the channel's scale and the sum with the bias, rounded to fp16 once (numpy converts float64 so; 64 bits
    hold the product, and the sum to 2^-53)."""
    total = (q.double() @ w.double().t()).cpu().numpy().astype(np.float32)
    scaled = (total * s.cpu().numpy()[:, None]).astype(np.float64)
    return (scaled * ws.cpu().numpy().astype(np.float64) + bias.cpu().numpy().astype(np.float64)).astype(np.float16)


@pytest.mark.parametrize("kernel,m,n,k", LONG[1::2])
def test_every_kernel_rounds_fp16_alike(gpu, kernel, m, n, k):
    """A product's last bit does not go by the kernel that its size chooses."""
    m, n = (m, n) if m * n > 1 else (33, 257)
    announce("gemm_int8 fp16 steps", m, n, k)
    g = torch.Generator().manual_seed(m + n + k)
    q, w = _codes((m, k), g).to(gpu), _codes((n, k), g).to(gpu)
    s, ws = (0.02 * torch.exp(torch.randn(m, generator=g))).to(gpu), (0.0005 * torch.exp(torch.randn(n, generator=g))).to(gpu)
    bias = torch.randn(n, generator=g).to(torch.float16).to(gpu)
    got = bfp8.gemm_int8(q, s, w, ws, bias=bias, dtype=torch.float16).cpu().numpy()
    assert np.array_equal(got, _steps(q, s, w, ws, bias))


@pytest.mark.parametrize("m,n,k", [(1, 8192, 4096), (2, 8100, 2048), (4, 8192, 1024), (8, 8001, 528)])
def test_one_launch_rounds_fp16_alike(gpu, m, n, k):
    announce("linear_int8 fp16 steps", m, n, k)
    g = torch.Generator().manual_seed(m + n + k)
    w, ws = bfp8.quant_act_int8(torch.randn(n, k, generator=g).to(gpu))
    for _ in range(6):
        x = torch.randn(m, k, generator=g).to(torch.float16).to(gpu)
        bias = torch.randn(n, generator=g).to(torch.float16).to(gpu)
        q, s = bfp8.quant_act_int8(x)
        assert np.array_equal(bfp8.linear_int8(x, w, ws, bias).cpu().numpy(), _steps(q, s, w, ws, bias))
