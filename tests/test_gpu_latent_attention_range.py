"""GPU tests of latent attention over the paged FP8 cache where the softmax's range is wide, and where there are
more blocks than workgroups run at once. Tolerances are those of test_gpu_latent_attention.py; the scores here
come from the rotary part alone (bf16 products, exact in float32 up to its rounding), so the bound's term for
scores does not hide anything."""

import numpy as np
import pytest
import torch

import block_scaled_fp8_bfp8_amd as bfp8
from oracle import e4m3, latent
from tests.gpu_util import announce
from tests.test_gpu_latent_attention import SCALE, attend, check, make

pytestmark = pytest.mark.gpu


def rotary_case(gpu, values, q_sizes, seed, latents=None):
    """One sequence whose key j has rotary part (values[j], 0, ...), and one token whose head h has (q_sizes[h], 0, ...)
    and no latent part."""
    n, heads = len(values), len(q_sizes)
    c, _ = make(gpu, [n], [1], heads, 16, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    kv = torch.randn(n, 576, generator=g).bfloat16()
    if latents is not None:
        kv[:, :512] = latents.bfloat16()
    kv[:, 512:] = 0
    kv[:, 512] = torch.tensor(values).bfloat16()
    i = torch.arange(n)
    slots = c["table"].cpu()[0, i // 16].long() * 16 + i % 16
    bfp8.latent_cache_write(kv.to(gpu), slots.to(gpu), c["cache"], c["scales"])
    rows = c["cache"].cpu()[slots // 16, slots % 16].numpy()
    codes = c["scales"].cpu()[slots // 16, slots % 16].numpy()
    lat = e4m3.decode(rows[:, :512].copy()) * latent.e8m0_value(codes)[:, None]
    c["q"].zero_()
    c["q"][0, :, 512] = torch.tensor(q_sizes).bfloat16().to(gpu)
    return c, [np.concatenate([lat, kv[:, 512:].double().numpy()], axis=1)]


@pytest.mark.parametrize("heads", [6, 40])
@pytest.mark.parametrize("order", ["rising", "falling", "peak in the middle", "steps"])
def test_scores_that_move_far_along_the_keys(gpu, order, heads):
    """Scores that rise or fall by up to 500 powers of two over ten tiles: the accumulator's reference moves, in
    rows of one block at different times and in opposite directions."""
    j = np.arange(600, dtype=np.float64)
    v = {"rising": 0.5 * j, "falling": -0.5 * j, "peak in the middle": -np.abs(j - 311), "steps": 45.0 * (j // 70)}[order]
    sizes = [16.0, -16.0, 1.0, 0.0, -4.0, 8.0] * 8
    announce("latent attention range", order, heads)
    c, keys = rotary_case(gpu, v, sizes[:heads], seed=91)
    check(attend(c), c["q"], keys, [600], [1])


@pytest.mark.parametrize("length", [65, 700, 4100])
def test_many_small_weights_beside_a_large_one(gpu, length):
    """One key 2^20 times the weight of each other: columns in which it is zero are the small weights' alone, and
    keep their relative accuracy."""
    v = [0.0] * length
    v[length // 3] = 12.0
    g = torch.Generator().manual_seed(92)
    lat = torch.randn(length, 512, generator=g)
    lat[:, :256] = 0
    lat[length // 3, :256] = torch.randn(256, generator=g)
    lat[length // 3, 256:] = 0
    announce("latent attention small weights", length)
    c, keys = rotary_case(gpu, v, [16.0] * 16, seed=93, latents=lat)
    out = attend(c)
    check(out, c["q"], keys, [length], [1])
    got = out[0, :, 256:].double().cpu().numpy()
    want = latent.attention_ref(c["q"][0].double().cpu().numpy(), keys[0], keys[0][:, :512], np.full(16, length), SCALE)[0][:, 256:]
    assert np.sqrt(((got - want) ** 2).sum()) <= 2.0 ** -8 * np.sqrt((want ** 2).sum())


@pytest.mark.parametrize("lens,new,heads,page", [
    ([90, 700, 10], [64, 64, 5], 128, 16), ([40] * 70, [4] * 70, 64, 16), ([333, 2000, 64, 65], [66, 70, 64, 1], 100, 64)])
def test_more_blocks_than_run_at_once(gpu, lens, new, heads, page):
    """The longest sequences start first (up to 64 of them), in the given order beyond."""
    announce("latent attention rounds", lens[:4], new[:4], heads)
    c, keys = make(gpu, lens, new, heads, page, seed=94)
    out = attend(c)
    check(out, c["q"], keys, lens, new)
    assert torch.equal(out.view(torch.int16), attend(c).view(torch.int16))


def test_one_sequence_cut_into_many_parts(gpu):
    """A long sequence alone: more parts than a wave has lanes are joined."""
    announce("latent attention many parts")
    c, keys = make(gpu, [20000], [1], 8, 64, seed=95)
    check(attend(c), c["q"], keys, [20000], [1])


@pytest.mark.parametrize("q_by,c_by", [(32.0, 1.0), (1.0, 32.0), (6.0, 6.0), (4096.0, 0.0)])
def test_outlier_channels(gpu, q_by, c_by):
    """A few channels of the queries, of the latents or of both far larger than the rest, and queries 2^12 larger where
    the latents are zero. The root mean square is held as ever; an element's scores to what the two windows can
    cost: products are off by 2^-13 of the largest of their group of 8 (of each of the query's two terms, together
    1.125 of it; 64 groups, so the 64 largest products of a key bound the sum), query elements by 2^-21 of their row's
    largest, and float32 sums by 2^-16 of their terms."""
    n, heads, channels = 400, 16, [5, 200, 511]
    announce("latent attention outliers", q_by, c_by)
    c, _ = make(gpu, [n], [1], heads, 16, seed=98)
    g = torch.Generator().manual_seed(99)
    kv = torch.randn(n, 576, generator=g)
    kv[:, channels] *= c_by
    kv = kv.bfloat16()
    i = torch.arange(n)
    slots = c["table"].cpu()[0, i // 16].long() * 16 + i % 16
    bfp8.latent_cache_write(kv.to(gpu), slots.to(gpu), c["cache"], c["scales"])
    rows = c["cache"].cpu()[slots // 16, slots % 16].numpy()
    codes = c["scales"].cpu()[slots // 16, slots % 16].numpy()
    lat = e4m3.decode(rows[:, :512].copy()) * latent.e8m0_value(codes)[:, None]
    keys = np.concatenate([lat, kv[:, 512:].double().numpy()], axis=1)
    c["q"][:, :, channels] *= q_by
    out = attend(c)
    check(out, c["q"], [keys], [n], [1])
    q, got = c["q"][0].double().cpu().numpy(), out[0].double().cpu().numpy()
    o, mag, _ = latent.attention_ref(q, keys, lat, np.full(heads, n), SCALE)
    for h in range(heads):
        terms = np.abs(q[h] * keys)
        windows = 2.0 ** -10 * 1.125 * np.sort(terms[:, :512], axis=1)[:, -64:].sum(axis=1)
        d = SCALE * (windows + 2.0 ** -21 * np.abs(q[h, :512]).max() * np.abs(lat).sum(axis=1) + 2.0 ** -16 * terms.sum(axis=1)).max()
        bound = 2.0 ** -8 * np.abs(o[h]) + (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -14 + 2 * np.expm1(d)) * mag[h]
        assert (np.abs(got[h] - o[h]) <= bound).all()


@pytest.mark.parametrize("lens,heads", [([5000] + [7 + 3 * i % 90 for i in range(259)], 16), ([70] * 129, 128), ([2000] + [100] * 140, 128)])
def test_many_blocks_of_uneven_lengths(gpu, lens, heads):
    """As many blocks as run at once or more, one sequence much longer than the rest, and one block too many."""
    announce("latent attention many uneven", len(lens), max(lens), heads)
    c, keys = make(gpu, lens, [1] * len(lens), heads, 64, seed=100)
    out = attend(c)
    check(out, c["q"], keys, lens, [1] * len(lens))
    assert torch.equal(out.view(torch.int16), attend(c).view(torch.int16))


def test_long_context(gpu):
    announce("latent attention long context")
    c, keys = make(gpu, [70001, 40], [1, 1], 8, 64, seed=101)
    check(attend(c), c["q"], keys, [70001, 40], [1, 1])
