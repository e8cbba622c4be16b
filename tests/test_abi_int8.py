"""CPU tests of the integer products' entry points: host-side rejections, each before any device call, the documented
no-ops (fake pointers are never dereferenced, nothing is launched), and the binding's checks."""

import pytest
import torch

import block_scaled_fp8_bfp8_amd as bfp8
from block_scaled_fp8_bfp8_amd import _native

OK = _native.BFP8_OK
E_INV = _native.BFP8_ERR_INVALID_ARGUMENT
E_UNS = _native.BFP8_ERR_UNSUPPORTED
E_MIS = _native.BFP8_ERR_MISALIGNED
E_WS = _native.BFP8_ERR_WORKSPACE
BF16, F16, F32 = _native.BFP8_IN_BF16, _native.BFP8_IN_F16, _native.BFP8_IN_F32

P1, P2, P3, P4, P5, P6 = (0x10000000 * i for i in range(1, 7))  # fake, 256-byte aligned


@pytest.fixture(scope="module")
def lib():
    return _native.lib()


def _quant(lib, x=P1, dt=BF16, M=4, K=256, ldx=256, q=P2, ldq=256, s=P3):
    return lib.bfp8_quant_act_int8(x, dt, M, K, ldx, q, ldq, s, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), E_INV), (dict(K=0), E_INV), (dict(K=200), E_UNS), (dict(K=65552, ldx=65552, ldq=65552), E_UNS),
    (dict(dt=7), E_UNS), (dict(M=(1 << 30) + 1), E_UNS), (dict(x=None), E_INV), (dict(q=None), E_INV), (dict(s=None), E_INV),
    (dict(ldx=240), E_INV), (dict(ldq=240), E_INV), (dict(ldx=260), E_MIS), (dict(ldq=264), E_MIS), (dict(x=P1 + 8), E_MIS),
    (dict(q=P2 + 8), E_MIS), (dict(s=P3 + 2), E_MIS), (dict(ldx=1 << 31), E_UNS), (dict(dt=F32, ldx=258), E_MIS),
])
def test_quant_rejections(lib, kw, status):
    assert _quant(lib, **kw) == status, lib.bfp8_last_error_message()


def _gemm(lib, a=P1, lda=256, as_=P2, b=P3, ldb=256, bs=P4, bias=P5, c=P6, dt=BF16, ldc=64, M=4, N=64, K=256):
    return lib.bfp8_gemm_int8(a, lda, as_, b, ldb, bs, bias, c, dt, ldc, M, N, K, None)


GEMM = [
    (dict(M=-1), E_INV), (dict(N=0), E_INV), (dict(K=0), E_INV), (dict(K=8), E_UNS), (dict(K=65552, lda=65552, ldb=65552), E_UNS),
    (dict(M=(1 << 30) + 1), E_UNS), (dict(N=(1 << 30) + 1, ldc=1 << 31), E_UNS), (dict(M=1 << 30, N=1 << 20, ldc=1 << 20), E_UNS), (dict(N=(1 << 26) + 1, ldc=1 << 27), E_UNS), (dict(M=1 << 30, N=1), E_UNS),
    (dict(b=None), E_INV), (dict(bs=None), E_INV), (dict(c=None), E_INV), (dict(ldb=240), E_INV), (dict(ldc=63), E_INV),
    (dict(ldb=264), E_MIS), (dict(ldb=1 << 23), E_UNS), (dict(ldc=(1 << 30) + 1), E_UNS), (dict(b=P3 + 8), E_MIS),
    (dict(bs=P4 + 2), E_MIS), (dict(bias=P5 + 1), E_MIS), (dict(c=P6 + 1), E_MIS),
]


@pytest.mark.parametrize("kw,status", GEMM + [
    (dict(dt=F32), E_UNS), (dict(a=None), E_INV), (dict(as_=None), E_INV), (dict(lda=240), E_INV), (dict(lda=264), E_MIS),
    (dict(lda=1 << 23), E_UNS), (dict(a=P1 + 8), E_MIS), (dict(as_=P2 + 2), E_MIS),
])
def test_gemm_rejections(lib, kw, status):
    assert _gemm(lib, **kw) == status, lib.bfp8_last_error_message()


def _linear(lib, x=P1, dt=BF16, ldx=256, b=P3, ldb=256, bs=P4, bias=P5, c=P6, ldc=64, M=4, N=64, K=256, ws=P2, wsb=None, lda=None):
    if wsb is None:
        wsb = lib.bfp8_linear_int8_workspace_bytes(M, K)
    if K > 256 or K < 1:
        ldx = K
    return lib.bfp8_linear_int8(x, dt, M, K, ldx, b, ldb, bs, bias, c, ldc, N, ws, wsb, None)


@pytest.mark.parametrize("kw,status", GEMM + [
    (dict(dt=F32), E_UNS), (dict(x=None), E_INV), (dict(x=P1 + 8), E_MIS), (dict(ldx=240), E_INV), (dict(ws=None), E_WS),
    (dict(wsb=1024), E_WS), (dict(ws=P2 + 16), E_MIS),
])
def test_linear_rejections(lib, kw, status):
    assert _linear(lib, **kw) == status, lib.bfp8_last_error_message()


def test_no_rows_is_a_no_op(lib):
    assert _quant(lib, M=0, x=None, q=None, s=None) == OK
    assert _gemm(lib, M=0, a=None, as_=None, c=None) == OK
    assert _linear(lib, M=0, x=None, c=None, ws=None, wsb=0) == OK


def test_linear_workspace(lib):
    size = lib.bfp8_linear_int8_workspace_bytes
    assert size(0, 128) == 0 and size(-3, 128) == 0 and size(5, 0) == 0 and size(5, 1 << 20) == 0
    assert size(1, 16) == 512 and size(1000, 4096) == 1000 * 4096 + 4096
    assert size(1 << 30, 65536) > 1 << 45  # (no overflow)


def test_binding_refuses_on_the_host():
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError, match="GPU"):
        bfp8.quant_act_int8(x)
    with pytest.raises(NotImplementedError):
        bfp8.quant_act_int8(q)
    with pytest.raises(ValueError, match="GPU"):
        bfp8.gemm_int8(q, s, q, s)
    with pytest.raises(TypeError):
        bfp8.gemm_int8(q.view(torch.uint8), s, q, s)
    with pytest.raises(NotImplementedError):
        bfp8.gemm_int8(q, s, q, s, dtype=torch.float32)
    with pytest.raises(NotImplementedError):
        bfp8.linear_int8(x.float(), q, s)
