"""GPU tests of every kernel of the integer product over a K that fills its stages or slots more than twice, with a whole
and with a partial last block (the tolerance is that of tests/test_gpu_int8.py). The library says which kernel a size runs,
so that another choice by size does not take one out of the tests unseen."""

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
