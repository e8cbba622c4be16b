"""GPU tests of the integer products against 64-bit arithmetic: the token quantizer bit for bit (its definition leaves no
freedom), the product and the linear layer to the rounding of their output.

Tolerance of a product: the sum is exact, so against exact arithmetic an output is off by its own rounding (eps / 2
relative: 2^-8 bf16, 2^-11 fp16, and half of the least step below the type's normal range) and by the float32 steps
before: conversion of the sum, two products, the sum with the bias, each 2^-24 relative to |product| + |bias|."""

import pytest
import torch

import block_scaled_fp8_bfp8_amd as bfp8
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _quant_ref(x):
    a = x.double().abs().amax(dim=1)
    finite = a < float("inf")
    a = a.clamp(min=torch.tensor(1e-10, dtype=torch.float32).item())  # the constant in float32
    q = torch.round(127.0 * x.double() / a[:, None])
    q = torch.where(finite[:, None], q, 0.0).nan_to_num(0.0).to(torch.int8)
    s = torch.where(finite, a.float() / torch.full_like(a, 127.0, dtype=torch.float32), float("nan"))
    return q, s


def _check_quant(x, q, s, what):
    q_ref, s_ref = _quant_ref(x.cpu())
    assert torch.equal(q.cpu(), q_ref), what
    assert torch.equal(s.cpu().nan_to_num(-1.0), s_ref.nan_to_num(-1.0)), what


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,k", [(1, 16), (5, 48), (3, 512), (7, 528), (2, 1024), (9, 2064), (4, 4096), (3, 7168), (2, 8208),
                                 (2, 16384), (1, 32784), (1, 65536), (1030, 144)])
def test_quant(gpu, dtype, m, k):
    announce("quant_act_int8", m, k, dtype)
    g = torch.Generator().manual_seed(m * 100003 + k)
    x = (torch.randn(m, k, generator=g) * torch.exp(torch.randn(m, 1, generator=g))).to(TYPES[dtype])
    q, s = bfp8.quant_act_int8(x.to(gpu))
    _check_quant(x, q, s, (m, k, dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,k", [(2049, 16), (2051, 1008), (2050, 1552), (2053, 2576), (2049, 4096), (2050, 5120), (2051, 5648), (2049, 7168),
                                 (2050, 7184)])
def test_quant_many_rows(gpu, dtype, m, k):
    """One to seven waves a row, and what follows them."""
    test_quant(gpu, dtype, m, k)


@pytest.mark.parametrize("dtype", TYPES)
def test_quant_middles_and_extremes(gpu, dtype):
    """Elements at the exact middle of two codes (ties to even) and next to it, tiny and huge rows, zeros, and rows that
    are not finite."""
    t = TYPES[dtype]
    steps = torch.arange(-254, 255, dtype=torch.float64) / 2  # every code and every middle, for a largest element of 127
    row = torch.zeros(528, dtype=torch.float64)
    row[:509] = steps
    rows = [row * 2.0 ** e for e in (-6, 0, 1, 8)]
    if dtype == "f32":
        near = row.clone()
        near[:509] *= 1 + 2.0 ** -23
        rows += [row * 2.0 ** 120, row * 2.0 ** -60, near, torch.nextafter(row.float(), torch.full((528,), 1000.0)).double(),
                 torch.nextafter(row.float(), torch.full((528,), -1000.0)).double()]
    rows.append(torch.zeros(528, dtype=torch.float64))
    rows.append(torch.full((528,), torch.finfo(t).max, dtype=torch.float64))
    rows.append(torch.full((528,), torch.finfo(t).smallest_normal / 8, dtype=torch.float64))
    x = torch.stack(rows).to(t)
    bad = x[:3].clone()
    bad[0, 5], bad[1, 300], bad[2, 527] = float("nan"), float("inf"), float("-inf")
    x = torch.cat([x, bad, x[1:2]])
    announce("quant_act_int8 middles", dtype)
    q, s = bfp8.quant_act_int8(x.to(gpu))
    _check_quant(x, q, s, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quant_strides(gpu, dtype):
    """Rows that lie apart, on both sides; columns past K stay as they were."""
    x = torch.randn(6, 320, generator=torch.Generator().manual_seed(3)).to(TYPES[dtype]).to(gpu)
    q = torch.full((6, 256), 99, dtype=torch.int8, device=gpu)
    announce("quant_act_int8 strides", dtype)
    got, s = bfp8.quant_act_int8(x[:, 32:240], q=q[:, 16:224])
    _check_quant(x[:, 32:240], got, s, dtype)
    assert bool((q[:, :16] == 99).all()) and bool((q[:, 224:] == 99).all())


def _codes(shape, g):
    q = torch.randint(-127, 128, shape, generator=g, dtype=torch.int8)
    q.view(-1)[:: 97] = -128  # weights from elsewhere may hold it
    return q


def _check_product(got, q, s, w, ws, bias, what):
    dt = got.dtype
    # (codes times codes sum to less than 2^53)
    y = (q.double() @ w.double().t()) * s.double()[:, None] * ws.double()
    add = torch.zeros_like(y) if bias is None else bias.double().expand_as(y)
    mag = y.abs() + add.abs()
    y = y + add
    tol = y.abs() * torch.finfo(dt).eps / 2 * (1 + 2.0 ** -20) + mag * 4 * 2.0 ** -24 + torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    bad = (got.double() - y).abs() > tol
    assert not bool(bad.any()), (what, int(bad.sum()), tuple(bad.nonzero()[0].tolist()))


# sizes on both sides of every choice of a kernel and a tile, odd ones, and partial last blocks of K
SIZES = [(1, 1, 16), (1, 64, 128), (2, 17, 48), (1, 576, 7168), (16, 100, 400), (17, 333, 1040), (31, 257, 272), (33, 4096, 512),
         (64, 95, 2064), (83, 576, 7168), (100, 640, 1168), (128, 129, 144), (129, 130, 640), (200, 1000, 384), (256, 515, 1024),
         (257, 129, 128), (300, 1111, 784), (513, 520, 4112), (1000, 2500, 256), (1024, 4096, 1040), (1100, 8200, 384),
         (2100, 4097, 528), (4096, 4096, 128), (4100, 4200, 272)]
# one whole and one partial last block of K for each of the 13 kernels that the choice may fall on
SIZES += [(5121, 1, 128), (4098, 1, 16), (3, 4402, 128), (1, 4471, 16), (17, 4838, 16), (36, 5690, 128), (4232, 34, 16), (2, 10717, 640),
          (1, 8942, 16), (294, 1732, 2304), (132, 2769, 2080), (171, 10944, 128), (385, 4935, 144), (7478, 556, 256), (6951, 1045, 32),
          (1483, 2798, 640), (415, 9425, 16), (3354, 2438, 128), (2982, 2737, 272), (198, 4658, 384), (135, 5905, 16), (72, 5772, 128),
          (19, 8799, 16)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gemm(gpu, m, n, k, dtype):
    announce("gemm_int8", m, n, k, dtype)
    g = torch.Generator().manual_seed(m + 7 * n + 31 * k)
    q, w = _codes((m, k), g).to(gpu), _codes((n, k), g).to(gpu)
    s, ws = (0.02 * torch.exp(torch.randn(m, generator=g))).to(gpu), (0.0005 * torch.exp(torch.randn(n, generator=g))).to(gpu)
    bias = torch.randn(n, generator=g).to(TYPES[dtype]).to(gpu) if (m + n) % 2 else None
    got = bfp8.gemm_int8(q, s, w, ws, bias=bias, dtype=TYPES[dtype])
    _check_product(got, q, s, w, ws, bias, (m, n, k, dtype))


def test_gemm_largest_sums(gpu):
    """The longest K with every code at its largest magnitude."""
    k = 65536
    q = torch.full((3, k), -128, dtype=torch.int8, device=gpu)
    w = torch.full((20, k), -128, dtype=torch.int8, device=gpu)
    w[::2] = 127
    s, ws = torch.full((3,), 2.0 ** -15, device=gpu), torch.full((20,), 2.0 ** -10, device=gpu)
    announce("gemm_int8 largest sums")
    _check_product(bfp8.gemm_int8(q, s, w, ws), q, s, w, ws, None, "largest")
    q = q.repeat(100, 1)
    s = s.repeat(100)
    _check_product(bfp8.gemm_int8(q, s, w, ws), q, s, w, ws, None, "largest, tiled")


@pytest.mark.parametrize("m", [3, 200])
def test_weight_past_4_gib(gpu, m):
    """Rows of a weight whose bytes lie past 2^32: the last channels against float64, and one in the middle."""
    n, k = 66000, 65536
    w = torch.randint(-128, 128, (n, k), dtype=torch.int8, device=gpu)
    q = torch.randint(-128, 128, (m, k), dtype=torch.int8, device=gpu)
    s, ws = torch.full((m,), 2.0 ** -10, device=gpu), torch.full((n,), 2.0 ** -10, device=gpu)
    announce("gemm_int8 past 4 GiB", m)
    got = bfp8.gemm_int8(q, s, w, ws)
    for at in (slice(n - 130, n), slice(32768 - 5, 32768 + 5), slice(65536 - 3, 65536 + 3)):
        _check_product(got[:, at], q, s, w[at], ws[at], None, at)


@pytest.mark.parametrize("m", [5, 300])
def test_gemm_views(gpu, m):
    """Operands with rows apart, whose gaps hold other codes, at the very end of their memory; an output with rows apart
    whose gaps stay as they were, aligned to 2 bytes only."""
    n, k = 150, 208
    g = torch.Generator().manual_seed(m)
    qa, wa = _codes((m, 320), g).to(gpu), _codes((n, 288), g).to(gpu)
    q, w = qa[:, 320 - k:], wa[:, 288 - k:]
    s, ws = (0.02 * torch.rand(m, generator=g)).to(gpu), (0.01 * torch.rand(n + 3, generator=g)).to(gpu)[3:]
    for lead, dt in ((0, torch.bfloat16), (1, torch.float16), (3, torch.bfloat16)):
        out = torch.full((m, n + 11), 7.0, dtype=dt, device=gpu)
        announce("gemm_int8 views", m, lead)
        got = bfp8.gemm_int8(q, s, w, ws, dtype=dt, out=out[:, lead:lead + n])
        _check_product(got, q, s, w, ws, None, (m, lead))
        assert bool((out[:, :lead] == 7).all()) and bool((out[:, lead + n:] == 7).all())


@pytest.mark.parametrize("m", [5, 300])
@pytest.mark.parametrize("pitch,lead,n", [(162, 2, 151), (162, 0, 150), (168, 8, 150), (164, 4, 145)])
def test_gemm_row_pitches(gpu, m, pitch, lead, n):
    """Outputs aligned to 4, 8 and 16 bytes, with columns that end inside such a piece."""
    g = torch.Generator().manual_seed(m + n)
    q, w = _codes((m, 208), g).to(gpu), _codes((n, 208), g).to(gpu)
    s, ws = (0.02 * torch.rand(m, generator=g)).to(gpu), (0.01 * torch.rand(n, generator=g)).to(gpu)
    out = torch.full((m, pitch), 7.0, dtype=torch.bfloat16, device=gpu)
    announce("gemm_int8 pitches", m, pitch, lead, n)
    _check_product(bfp8.gemm_int8(q, s, w, ws, out=out[:, lead:lead + n]), q, s, w, ws, None, (m, pitch, lead, n))
    assert bool((out[:, :lead] == 7).all()) and bool((out[:, lead + n:] == 7).all())


def test_bad_tokens_stay_alone(gpu):
    """A token that is not finite gives NaN outputs and leaves the others as they are, through the quantizer and all."""
    g = torch.Generator().manual_seed(8)
    for m in (4, 300):
        x = torch.randn(m, 256, generator=g).to(torch.bfloat16).to(gpu)
        w, ws = bfp8.quant_act_int8(torch.randn(96, 256, generator=g).to(gpu))
        clean = bfp8.linear_int8(x, w, ws)
        x[1, 17], x[2, 0] = float("inf"), float("nan")
        announce("linear_int8 with bad tokens", m)
        got = bfp8.linear_int8(x, w, ws)
        assert bool(got[1:3].isnan().all())
        keep = [i for i in range(m) if i not in (1, 2)]
        assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (1, 40, 16), (3, 576, 7168), (5, 5120, 8192), (8, 1000, 528), (9, 333, 1040),
                                   (64, 512, 2064), (300, 777, 640), (1000, 2048, 1024), (1, 4500, 65536), (2, 100, 32768), (2, 48, 32784),
                                   (4, 5000, 16384), (3, 130, 16400), (6, 77, 8192), (8, 4200, 8208), (7, 20, 112), (2, 1, 144),
                                   (1, 8192, 16384), (1, 8193, 144), (2, 77, 8192), (2, 77, 8208), (4, 500, 4096), (3, 500, 4112), (8, 19, 2048), (5, 8192, 2000)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_linear_is_quantizer_and_product(gpu, m, n, k, dtype):
    announce("linear_int8", m, n, k, dtype)
    g = torch.Generator().manual_seed(m + n + k)
    x = torch.randn(m, k, generator=g).to(TYPES[dtype]).to(gpu)
    w, ws = bfp8.quant_act_int8(torch.randn(n, k, generator=g).to(gpu))
    bias = torch.randn(n, generator=g).to(TYPES[dtype]).to(gpu)
    got = bfp8.linear_int8(x, w, ws, bias)
    q, s = bfp8.quant_act_int8(x)
    assert torch.equal(got, bfp8.gemm_int8(q, s, w, ws, bias=bias, dtype=TYPES[dtype]))
    q_ref, s_ref = _quant_ref(x.cpu())
    _check_product(got, q_ref.to(gpu), s_ref.to(gpu), w, ws, bias, (m, n, k, dtype))


def test_linear_in_graphs_of_one_stream(gpu):
    """Two captured calls and eager ones beside them: each replay equals its eager result."""
    g = torch.Generator().manual_seed(21)
    xs = [torch.randn(m, 1024, generator=g).to(torch.bfloat16).to(gpu) for m in (3, 40)]
    w, ws = bfp8.quant_act_int8(torch.randn(700, 1024, generator=g).to(gpu))
    want = [bfp8.linear_int8(x, w, ws) for x in xs]
    stream = torch.cuda.Stream()
    graphs, outs = [], []
    announce("linear_int8 in graphs")
    with torch.cuda.stream(stream):
        for x in xs:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                outs.append(bfp8.linear_int8(x, w, ws))
            graphs.append(graph)
        for _ in range(3):
            for graph, out, ref in zip(graphs, outs, want):
                out.zero_()
                graph.replay()
                big = bfp8.linear_int8(torch.cat([xs[1]] * 20), w, ws)
                stream.synchronize()
                assert torch.equal(out, ref) and torch.equal(big[:40], want[1])


def test_no_rows(gpu):
    w, ws = torch.zeros(8, 32, dtype=torch.int8, device=gpu), torch.ones(8, device=gpu)
    x = torch.zeros(0, 32, dtype=torch.bfloat16, device=gpu)
    q, s = bfp8.quant_act_int8(x)
    assert q.shape == (0, 32) and s.shape == (0,)
    assert bfp8.gemm_int8(q, s, w, ws).shape == (0, 8) and bfp8.linear_int8(x, w, ws).shape == (0, 8)


def test_refusals(gpu):
    w, ws = torch.zeros(8, 32, dtype=torch.int8, device=gpu), torch.ones(8, device=gpu)
    x = torch.zeros(4, 32, dtype=torch.bfloat16, device=gpu)
    q, s = bfp8.quant_act_int8(x)
    with pytest.raises(ValueError):
        bfp8.gemm_int8(q, s[:3], w, ws)
    with pytest.raises(ValueError):
        bfp8.gemm_int8(q, s, w[:, :16], ws)
    with pytest.raises(ValueError):
        bfp8.gemm_int8(q, s, w, ws, out=torch.empty(4, 9, dtype=torch.bfloat16, device=gpu))
    with pytest.raises(TypeError):
        bfp8.gemm_int8(q, s, w, ws, bias=torch.zeros(8, device=gpu))
    with pytest.raises(TypeError):
        bfp8.gemm_int8(q, s, w, ws, out=torch.empty(4, 8, dtype=torch.float16, device=gpu))
    with pytest.raises(ValueError):
        bfp8.gemm_int8(q, s, w, ws.cpu())
    with pytest.raises(NotImplementedError):
        bfp8.quant_act_int8(torch.zeros(2, 24, device=gpu))  # K not a multiple of 16
    with pytest.raises(ValueError):
        bfp8.quant_act_int8(torch.zeros(2, 34, device=gpu)[:, 2:])  # misaligned
    with pytest.raises(ValueError):
        bfp8.linear_int8(x, w, ws, workspace=torch.empty(16, dtype=torch.uint8, device=gpu))
