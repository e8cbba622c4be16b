"""GPU tests of latent attention at the borders of its launch rules: rows a workgroup, cut and whole blocks, one and
eight waves a joined row, block orders. Tolerances are those of test_gpu_latent_attention.py and
test_gpu_latent_expanded.py."""

import numpy as np
import pytest
import torch

from tests import test_gpu_latent_attention as absorbed
from tests import test_gpu_latent_expanded as expanded
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,heads,width_extra", [
    ([256], 128, 0), ([257], 128, 0), ([256, 3, 0, 255], 33, 0),  # the last length that is not cut, and the next
    ([1111], 128, 520), ([2049, 10, 700], 128, 300),              # 64 rows a workgroup for a wide page table
    ([9000], 100, 0), ([6000], 128, 700), ([2100], 1, 1),         # many parts: eight waves join a row
    ([300, 1500, 0, 64, 65, 999, 1, 640], 128, 64), ([2048, 2049, 40], 16, 0)])
def test_absorbed_at_the_borders(gpu, lens, heads, width_extra):
    announce("latent attention plan", lens, heads, width_extra)
    c, keys = absorbed.make(gpu, lens, [1] * len(lens), heads, 64, seed=sum(lens) + heads, width_extra=width_extra)
    out = absorbed.attend(c)
    absorbed.check(out, c["q"], keys, lens, [1] * len(lens))
    assert torch.equal(out.view(torch.int16), absorbed.attend(c).view(torch.int16))


@pytest.mark.parametrize("width_extra", [0, 6, 40, 600])
def test_absorbed_chunks_in_wider_tables(gpu, width_extra):
    """A wider page table changes how the work is cut, not the answer beyond its tolerance."""
    lens, new, heads = [400, 90, 5], [20, 33, 5], 48
    announce("latent attention plan, chunks", width_extra)
    c, keys = absorbed.make(gpu, lens, new, heads, 64, seed=96, width_extra=width_extra)
    absorbed.check(absorbed.attend(c), c["q"], keys, lens, new)


def ragged(seed, n, top):
    rng = np.random.default_rng(seed)
    nq = [int(v) for v in rng.integers(0, top, n) * (rng.random(n) < 0.85)]
    return nq, [int(max(q + e, 0)) for q, e in zip(nq, rng.integers(-9, top, n) * (rng.random(n) < 0.6))]


@pytest.mark.parametrize("n,top,heads", [(33, 300, 3), (64, 90, 2), (65, 90, 2), (70, 40, 24), (12, 700, 5), (30, 70, 64)])
@pytest.mark.parametrize("seed", [1, 2])
def test_expanded_block_orders(gpu, n, top, heads, seed):
    """Sequences without queries or keys among others, fewer keys than queries, up to and beyond 64 sequences, and
    more workgroups than are ordered."""
    nq, nk = ragged(seed * 100 + n, n, top)
    announce("expanded order", n, top, heads, seed)
    c = expanded.make(nq, nk, heads, torch.bfloat16, seed=seed)
    out = expanded.run(c, gpu)
    expanded.check(out, c, nq, nk, heads=sorted({0, heads // 2, heads - 1}))
    assert torch.equal(out, expanded.run(c, gpu))


@pytest.mark.parametrize("lens,heads", [([1030] * 2, 32), ([600, 1500], 31), ([2050], 32)])
def test_expanded_around_one_workgroup_a_compute_unit(gpu, lens, heads):
    announce("expanded rows a workgroup", lens, heads)
    c = expanded.make(lens, lens, heads, torch.float16, seed=97)
    expanded.check(expanded.run(c, gpu), c, lens, lens, heads=[0, heads - 1])
