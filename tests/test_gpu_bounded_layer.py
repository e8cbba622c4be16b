"""The integer projections, the cache, attention with its masses and eviction, used together as a decoding layer: every step is
checked against float64 on what the cache then holds (the tolerances are those of the operators' own tests)."""

import numpy as np
import pytest
import torch

import block_scaled_fp8_bfp8_amd as bfp8
from examples.bounded_decoding import BoundedLayer, run
from tests import test_gpu_latent_attention as attention
from tests import test_gpu_latent_mass as mass_tests
from tests.gpu_util import announce
from tests.test_gpu_int8 import _check_product, _quant_ref
from tests.test_gpu_latent_evict import chosen

pytestmark = pytest.mark.gpu


def cached(layer):
    """The keys of every sequence in float64, and the bytes and codes of their rows."""
    keys, raw = [], []
    for b, n in enumerate(layer.lens.tolist()):
        t = torch.arange(n, device=layer.table.device)
        at = (layer.table[b, t // layer.page].long(), t % layer.page)
        rows, codes = layer.cache[at].cpu(), layer.scales[at].cpu()
        lat = rows[:, :512].contiguous().view(torch.float8_e4m3fn).double() * torch.exp2(codes.double() - 127)[:, None]
        keys.append(torch.cat([lat, rows[:, 512:].contiguous().view(torch.bfloat16).double()], dim=1).numpy())
        raw.append((rows, codes))
    return keys, raw


@pytest.mark.parametrize("batch,heads,page,budget,room", [(3, 8, 16, 20, 5), (2, 40, 7, 9, 1)])
def test_steps_against_float64(gpu, batch, heads, page, budget, room):
    layer = BoundedLayer(batch, 256, heads, budget + room, page, gpu, seed=heads)
    g = torch.Generator().manual_seed(5)
    for step in range(3 * (budget + room)):
        if int(layer.lens[0]) == budget + room:
            announce("bounded layer, eviction before step", step)
            _, raw = cached(layer)
            mass = layer.mass.clone().cpu()
            kept = layer.evict(budget, recent=budget // 2).cpu()
            _, now = cached(layer)
            for b in range(batch):
                stay = chosen(mass[b], budget + room, budget, budget // 2)
                assert kept[b].tolist() == stay and int(layer.lens[b]) == budget
                assert torch.equal(now[b][0], raw[b][0][stay]) and torch.equal(now[b][1], raw[b][1][stay])
                assert torch.equal(layer.mass[b, :budget].cpu(), mass[b][stay]) and not layer.mass[b, budget:].any()
        x = torch.randn(batch, 256, generator=g).to(torch.bfloat16)
        announce("bounded layer, step", step)
        before = layer.mass.clone()
        y = bfp8.linear_int8(x.to(gpu), *layer.w_in)
        q_ref, s_ref = _quant_ref(x)
        _check_product(y, q_ref.to(gpu), s_ref.to(gpu), *layer.w_in, None, step)
        got = layer.step(x.to(gpu))
        keys, _ = cached(layer)
        q, lens = y.view(batch, heads + 1, 576)[:, :heads], layer.lens.tolist()
        mass_tests.check(layer.mass, before, q, keys, lens, [1] * batch, layer.scale)
        out = bfp8.latent_attention(q, layer.cache, layer.scales, layer.table, layer.lens, layer.scale)
        attention.check(out, q, keys, lens, [1] * batch, layer.scale)
        assert torch.equal(got, bfp8.linear_int8(out.view(batch, -1), *layer.w_out))
    assert np.all([int(n) <= budget + room for n in layer.lens])


def test_captured_step(gpu):
    """A captured step, replayed, equals the eager one, before and after an eviction between replays."""
    a, b = (BoundedLayer(3, 512, 16, 48, 16, gpu, seed=1) for _ in range(2))
    g = torch.Generator().manual_seed(2)
    x = torch.zeros(3, 512, dtype=torch.bfloat16, device=gpu)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    announce("bounded layer captured")
    with torch.cuda.stream(stream):
        a.step(x), b.step(x)  # (what the step loads lazily is loaded)
        with torch.cuda.graph(graph, stream=stream):
            out = a.step(x)
        for step in range(60):
            if int(b.lens[0]) == 48:
                a.evict(24, 8), b.evict(24, 8)
            x.copy_(torch.randn(3, 512, generator=g).to(torch.bfloat16))
            graph.replay()
            want = b.step(x)
            stream.synchronize()
            assert torch.equal(out, want) and torch.equal(a.mass, b.mass) and torch.equal(a.lens, b.lens), step


def test_example_runs(gpu):
    """Nothing is evicted as long as the budget is not reached: both runs then agree bit for bit."""
    announce("bounded decoding example")
    bounded, whole = run(gpu, steps=50, budget=24, room=8)
    assert bounded.shape == whole.shape == (50, 4, 1024) and bool(bounded.isfinite().all())
    assert torch.equal(bounded[:32], whole[:32])
