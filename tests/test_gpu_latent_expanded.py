"""GPU tests of latent attention in the expanded form (ragged, causal at the end) against float64.

Tolerance, per element, with u half a step of the dtype (2^-8 bf16, 2^-11 fp16) and A the weights'
average of |v|: u |o| for the output, u A for the weights (rounded before the second product, each
by at most u of itself; fp16 weights below 2^-14 of the running maximum are off by 2^-25 absolute,
1e-5 A at these lengths), 2 (e^d - 1) A for scores off by d = 2^-16 reach (192 products and their
float32 sums, reach the row's largest scale * sum |q||k|), and 2^-14 A for float32 sums."""

import numpy as np
import pytest
import torch

import block_scaled_fp8_bfp8_amd as bfp8
from oracle import latent
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def make(nq, nk, heads, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    tq, tk = sum(nq), sum(nk)
    c = dict(q=torch.randn(tq, heads, 192, generator=g).to(dtype), kv=torch.randn(tk, heads, 256, generator=g).to(dtype),
             rope=torch.randn(tk, 64, generator=g).to(dtype))
    c["cu_q"] = torch.tensor(np.concatenate([[0], np.cumsum(nq)]), dtype=torch.int32)
    c["cu_k"] = torch.tensor(np.concatenate([[0], np.cumsum(nk)]), dtype=torch.int32)
    return c


def run(c, gpu, scale=SCALE, **kw):
    d = {k: v.to(gpu) for k, v in c.items()}
    return bfp8.latent_attention_expanded(d["q"], d["kv"], d["rope"], d["cu_q"], d["cu_k"], scale, **kw)


def check(out, c, nq, nk, scale=SCALE, heads=None):
    u = U[out.dtype]
    got = out.double().cpu().numpy()
    q, kv, rope = (c[n].double().numpy() for n in ("q", "kv", "rope"))
    assert np.isfinite(got).all()
    aq = ak = 0
    for n, length in zip(nq, nk):
        for h in heads if heads is not None else range(q.shape[1]):
            k = np.concatenate([kv[ak:ak + length, h, :128], rope[ak:ak + length]], axis=1)
            o, mag, reach = latent.attention_ref(q[aq:aq + n, h], k, kv[ak:ak + length, h, 128:],
                                                 length - n + 1 + np.arange(n), scale)
            d = 2.0 ** -16 * reach[:, None]
            bound = u * np.abs(o) + (u + 2.0 ** -14 + 1e-5 + 2 * np.expm1(d)) * mag
            diff = np.abs(got[aq:aq + n, h] - o)
            assert (diff <= bound).all(), f"head {h}: worst {np.max(diff / np.maximum(bound, 1e-300))} of the bound"
        aq += n
        ak += length


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("nq,nk,heads", [
    ([1], [1], 1), ([1], [300], 3), ([31, 32, 33], [31, 32, 33], 2), ([64, 127, 128, 129], [64, 127, 128, 129], 1),
    ([5, 0, 70], [80, 9, 70], 4), ([200], [457], 5), ([300, 17], [300, 1000], 8), ([3] * 270, [4] * 270, 1),
    ([1, 260], [63, 321], 20)])
def test_against_float64(gpu, nq, nk, heads, dtype):
    announce("expanded", nq[:5], nk[:5], heads, dtype)
    c = make(nq, nk, heads, dtype, seed=sum(nq) + heads)
    check(run(c, gpu), c, nq, nk)


def test_long_prompt(gpu):
    c = make([1500], [1500], 2, torch.bfloat16, seed=1)
    announce("expanded long")
    out = run(c, gpu)
    check(out, c, [1500], [1500])
    assert torch.equal(out, run(c, gpu))


def test_rows_that_see_nothing(gpu):
    """More queries than keys, and no keys at all: the rows before the first key are zero."""
    nq, nk = [9, 140, 6], [4, 0, 6]
    c = make(nq, nk, 2, torch.bfloat16, seed=2)
    announce("expanded empty rows")
    out = run(c, gpu)
    assert (out[:5] == 0).all() and (out[9:149] == 0).all()
    check(out, c, nq, nk)
    c = make([3], [0], 2, torch.bfloat16, seed=3)
    assert (run(c, gpu) == 0).all()


def test_strides_and_untouched_rows(gpu):
    nq, nk, heads = [40, 20], [50, 20], 3
    c = make(nq, nk, heads, torch.bfloat16, seed=4)
    d = {k: v.to(gpu) for k, v in c.items()}
    want = bfp8.latent_attention_expanded(d["q"], d["kv"], d["rope"], d["cu_q"], d["cu_k"], SCALE)
    nan = float("nan")
    q = torch.full((62, heads + 1, 200), nan, dtype=torch.bfloat16, device=gpu)
    kv = torch.full((heads, 75, 264), nan, dtype=torch.bfloat16, device=gpu)  # heads outermost
    rope = torch.full((75, 80), nan, dtype=torch.bfloat16, device=gpu)
    q[:60, :heads, 8:] = d["q"]
    kv[:, :70, :256] = d["kv"].transpose(0, 1)
    rope[:70, 16:] = d["rope"]
    out = torch.full((62, heads + 2, 136), 7.0, dtype=torch.bfloat16, device=gpu)
    announce("expanded strides")
    bfp8.latent_attention_expanded(q[:, :heads, 8:], kv.transpose(0, 1)[:, :, :256], rope[:, 16:], d["cu_q"], d["cu_k"],
                                   SCALE, out=out[:, :heads, :128])
    assert torch.equal(out[:60, :heads, :128], want)
    assert (out[60:] == 7.0).all() and (out[:, heads:] == 7.0).all() and (out[:, :, 128:] == 7.0).all()


@pytest.mark.parametrize("scale", [0.0, -SCALE, 5.0])
def test_scales_of_the_softmax(gpu, scale):
    announce("expanded scale", scale)
    c = make([70], [90], 2, torch.float16, seed=5)
    check(run(c, gpu, scale), c, [70], [90], scale)


def test_neighbouring_sequences_do_not_leak(gpu):
    """NaN and infinite keys and values of one sequence leave the others as they were."""
    nq, nk, heads = [50, 30, 70], [50, 30, 75], 2
    c = make(nq, nk, heads, torch.bfloat16, seed=6)
    want = run(c, gpu)
    c["kv"][50:80] = float("nan")
    c["kv"][60:70, :, 128:] = float("inf")
    c["rope"][50:80] = float("-inf")
    announce("expanded neighbours")
    out = run(c, gpu)
    assert torch.equal(out[:50], want[:50]) and torch.equal(out[80:], want[80:])
    assert out[50:80].isnan().any()


def test_graph_follows_lengths(gpu):
    nq, nk, heads = [100, 28], [120, 28], 4
    c = {k: v.to(gpu) for k, v in make(nq, nk, heads, torch.bfloat16, seed=7).items()}
    out = torch.empty(128, heads, 128, dtype=torch.bfloat16, device=gpu)
    side, graph = torch.cuda.Stream(gpu), torch.cuda.CUDAGraph()

    def call(o):
        return bfp8.latent_attention_expanded(c["q"], c["kv"], c["rope"], c["cu_q"], c["cu_k"], SCALE, out=o)

    announce("expanded graph")
    with torch.cuda.stream(side):
        call(out)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            call(out)
    torch.cuda.synchronize()
    for cq, ck in [([0, 100, 128], [0, 120, 148]), ([0, 1, 128], [0, 20, 148]), ([0, 128, 128], [0, 148, 148])]:
        c["cu_q"].copy_(torch.tensor(cq, dtype=torch.int32))
        c["cu_k"].copy_(torch.tensor(ck, dtype=torch.int32))
        want = call(None)
        out.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_empty_and_refusals(gpu):
    c = {k: v.to(gpu) for k, v in make([4], [6], 2, torch.bfloat16, seed=8).items()}
    zero = torch.zeros(1, dtype=torch.int32, device=gpu)
    assert bfp8.latent_attention_expanded(c["q"][:0], c["kv"][:0], c["rope"][:0], zero, zero, SCALE).shape == (0, 2, 128)

    def call(**kw):
        a = {**c, "scale": SCALE, **kw}
        return bfp8.latent_attention_expanded(a["q"], a["kv"], a["rope"], a["cu_q"], a["cu_k"], a["scale"], out=a.get("out"))

    call()
    with pytest.raises(NotImplementedError):
        call(q=c["q"].float())
    for bad in [dict(kv=c["kv"].half()), dict(cu_q=c["cu_q"].long()), dict(cu_k=c["cu_k"].float())]:
        with pytest.raises(TypeError):
            call(**bad)
    for bad in [dict(q=c["q"][:, :, :128]), dict(kv=c["kv"][:, :1]), dict(rope=c["rope"][:3]), dict(cu_k=c["cu_k"][:1]),
                dict(kv=c["kv"].transpose(1, 2).contiguous().transpose(1, 2)), dict(scale=float("inf")),
                dict(out=torch.empty(4, 2, 64, dtype=torch.bfloat16, device=gpu)), dict(q=c["q"].cpu())]:
        with pytest.raises(ValueError):
            call(**bad)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("nq,nk,heads", [([100], [100], 2), ([40, 90], [77, 90], 3), ([700], [700], 2), ([300] * 9, [300] * 9, 30),
                                         ([130], [99], 2)])
def test_infinite_and_nan_values_reach_only_rows_that_see_them(gpu, nq, nk, heads, dtype):
    """A row that does not see a key keeps its bits whatever the key's values are; one that does has in each column
    what the sum of the formula gives: the infinity, or NaN for a NaN or infinities of both signs."""
    c = make(nq, nk, heads, dtype, seed=9)
    want = run(c, gpu)
    at = np.concatenate([[0], np.cumsum(nk)])[:-1]
    inf = float("inf")
    first = [(3 * n) // 5 for n in nk]  # no key before it is touched
    for a, f, n in zip(at, first, nk):
        v = c["kv"][a + f:a + n, :, 128:]
        v[0, :, 3] = inf
        v[1, :, 7] = -inf
        v[2, :, 5] = float("nan")
        v[4, :, 3] = -inf
        v[4, :, 64] = inf
        v[-1, :, 127] = inf  # the last key, which a partly filled tile repeats
    announce("expanded values not finite", nq[:3], nk[:3], heads, dtype)
    got = run(c, gpu).cpu()
    want = want.cpu()
    q, kv, rope = (c[n].double().numpy() for n in ("q", "kv", "rope"))
    aq = 0
    for a, f, n, length in zip(at, first, nq, nk):
        sees = length - n + 1 + np.arange(n)
        before = torch.from_numpy(sees <= f)
        assert torch.equal(got[aq:aq + n][before], want[aq:aq + n][before])
        for h in sorted({0, heads - 1}):
            k = np.concatenate([kv[a:a + length, h, :128], rope[a:a + length]], axis=1)
            with np.errstate(invalid="ignore"):
                o, _, _ = latent.attention_ref(q[aq:aq + n, h], k, kv[a:a + length, h, 128:], sees, SCALE)
            g = got[aq:aq + n, h].double().numpy()
            assert (np.isnan(g) == np.isnan(o)).all()
            assert (np.where(np.isinf(o), o, 0) == np.where(np.isinf(g), g, 0)).all()
            same = np.isfinite(o)
            assert (np.isfinite(g) == same).all()
            assert (g[same] == want[aq:aq + n, h].double().numpy()[same]).all()
        aq += n
