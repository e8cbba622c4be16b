"""GPU tests of the attention weight that cached tokens gather, against float64.

Tolerance. A score is a sum of 576 exact products, added up in float32: off by at most d = 576 * 2^-23 of scale * sum |q||k|
(whatever the order, truncation included), and a weight so by expm1(2 d), itself and its row's sum. The exponentials, the
logarithm and the additions of float32 are each off by 2^-22 of a value at most: log2 values up to 2^7 in magnitude make
that 2^-15 of a weight, the additions of n weights n * 2^-24 of their sum. These are worst cases; errors of either sign make the root mean
square over all columns smaller, and it is held to 2^-15 of the root mean square of what was gathered (24 of the 576
steps' 2^-24 each, of scores of at most 2^4, are 2^-15.4)."""

import numpy as np
import pytest
import torch

import block_scaled_fp8_bfp8_amd as bfp8
from tests.gpu_util import announce
from tests.test_gpu_latent_attention import SCALE, make

pytestmark = pytest.mark.gpu


def reference(q, keys, lens, new, scale=SCALE):
    """Per sequence: the weight gathered by each key, and the largest scale * sum |q||k|."""
    q = q.double().cpu().numpy()
    heads, at, got = q.shape[1], 0, []
    for k, length, n in zip(keys, lens, new):
        total, reach = np.zeros(max(length, 0)), 0.0
        for i in range(n):
            seen = min(max(length - n + i + 1, 0), max(length, 0))
            if seen:
                s = q[at + i] @ k[:seen].T * scale
                p = np.exp(s - s.max(axis=1, keepdims=True))
                total[:seen] += (p / p.sum(axis=1, keepdims=True)).sum(axis=0)
                reach = max(reach, float((np.abs(q[at + i]) @ np.abs(k[:seen]).T).max()) * abs(scale))
        at += n
        got.append((total, reach, n * heads))
    return got


def check(got, before, q, keys, lens, new, scale=SCALE):
    got = got.double().cpu().numpy()
    before = np.zeros_like(got) if before is None else before.double().cpu().numpy()
    err = tot = 0.0
    for b, (total, reach, rows) in enumerate(reference(q, keys, lens, new, scale)):
        length = max(lens[b], 0)
        old = before[b, :length].copy()
        old[max(length - new[b], 0):] = 0.0
        want = old + total
        bound = total * (np.expm1(2 * 576 * 2.0 ** -23 * reach) + 2.0 ** -15 + rows * 2.0 ** -24) + 2.0 ** -24 * want
        diff = np.abs(got[b, :length] - want)
        assert (diff <= bound).all(), (b, int(np.argmax(diff - bound)), float((diff / np.maximum(bound, 1e-300)).max()))
        assert (got[b, length:] == 0).all()
        err += ((diff - 2.0 ** -24 * want).clip(0) ** 2).sum()
        tot += (total ** 2).sum()
    assert err <= 2.0 ** -30 * tot


CASES = [
    ([1], [1], 1, 1), ([1111], [1], 128, 64), ([500, 64, 7, 900], [1] * 4, 16, 64), ([127, 128, 129], [1] * 3, 33, 16),
    ([40, 300, 129], [40, 7, 129], 5, 37), ([100, 50, 9], [0, 3, 0], 8, 16), ([2, 0, 31], [5, 2, 31], 4, 16),
    ([600, 33], [65, 1], 20, 64), ([2000, 17, 1300], [1] * 3, 64, 16), ([700], [40], 128, 16), ([260] * 9, [2] * 9, 16, 37),
    ([4500], [1], 5, 1), ([900, 300, 70], [200, 2, 70], 32, 16),
]


@pytest.mark.parametrize("lens,new,heads,page", CASES)
def test_mass(gpu, lens, new, heads, page):
    announce("latent_attention_mass", lens, new, heads, page)
    c, keys = make(gpu, lens, new, heads, page, seed=len(lens) + heads, width_extra=2, gap=1)
    want = bfp8.latent_attention(c["q"], c["cache"], c["scales"], c["table"], c["lens"], SCALE, cu_q=c["cu"])
    out, mass = bfp8.latent_attention_mass(c["q"], c["cache"], c["scales"], c["table"], c["lens"], SCALE, cu_q=c["cu"])
    assert torch.equal(out, want)  # (zeros where a row sees no key)
    assert mass.shape == (len(lens), c["table"].shape[1] * page)
    check(mass, None, c["q"], keys, lens, new)
    # again on top of that: wider rows, apart, then in place
    g = torch.Generator().manual_seed(5)
    wide = torch.rand(len(lens), mass.shape[1] + 300, generator=g).to(gpu)
    before = wide[:, 7:7 + mass.shape[1] + 3]
    kept = before.clone()
    _, more = bfp8.latent_attention_mass(c["q"], c["cache"], c["scales"], c["table"], c["lens"], SCALE, mass=before, cu_q=c["cu"])
    assert torch.equal(before, kept) and more.shape == before.shape
    check(more, kept, c["q"], keys, lens, new)
    _, same = bfp8.latent_attention_mass(c["q"], c["cache"], c["scales"], c["table"], c["lens"], SCALE, mass=before, cu_q=c["cu"],
                                         out_mass=before)
    assert same is before and torch.equal(same, more)


def test_every_row_gives_one(gpu):
    """A row's weights add up to one, so a sequence gathers as much as it has rows."""
    lens, new, heads = [3000, 900, 1], [3, 9, 1], 48
    c, _ = make(gpu, lens, new, heads, 64, seed=3)
    _, mass = bfp8.latent_attention_mass(c["q"], c["cache"], c["scales"], c["table"], c["lens"], SCALE, cu_q=c["cu"])
    for row, n in zip(mass.double().sum(dim=1).tolist(), new):
        assert abs(row - n * heads) <= 2.0 ** -15 * n * heads


def test_strides_and_one_token_each(gpu):
    """Queries and outputs that lie apart, without cu_q, and scores of a large range (scale 3, negative scale)."""
    lens, heads = [77, 300, 512], 12
    c, keys = make(gpu, lens, [1, 1, 1], heads, 16, seed=9)
    wide = torch.zeros(3, heads + 2, 584, dtype=torch.bfloat16, device=gpu)
    wide[:, 1:-1, :576] = c["q"]
    q = wide[:, 1:-1, :576]
    for scale in (SCALE, 0.3, -0.2):
        announce("latent_attention_mass strides", scale)
        _, mass = bfp8.latent_attention_mass(q, c["cache"], c["scales"], c["table"], c["lens"], scale)
        check(mass, None, q, keys, lens, [1, 1, 1], scale)


def test_keys_that_are_nan_or_missing(gpu):
    """A NaN key, a page that is none and a length past the table reach the rows that see them and no other sequence; rows
    that end before the bad key stay as they were."""
    lens, new, heads, page = [200, 150, 90, 40], [1, 4, 1, 1], 6, 16
    c, keys = make(gpu, lens, new, heads, page, seed=12)
    args = (c["q"], c["cache"], c["scales"], c["table"], c["lens"], SCALE)
    _, clean = bfp8.latent_attention_mass(*args, cu_q=c["cu"])
    table, lens_t, scales = c["table"].clone(), c["lens"].clone(), c["scales"].clone()
    scales[table[0, 3], 5] = 255     # a NaN key of sequence 0
    table[1, 149 // page] = -1       # the last tokens of sequence 1 (144 .. 149) lie nowhere: none of its rows is without them
    table[2, 2] = c["cache"].shape[0]
    lens_t[3] = table.shape[1] * page + 9
    announce("latent_attention_mass with bad keys")
    out, mass = bfp8.latent_attention_mass(c["q"], c["cache"], scales, table, lens_t, SCALE, cu_q=c["cu"])
    for b, length in enumerate((200, 150, 90)):
        assert bool(mass[b, :length].isnan().all()) and bool((mass[b, length:] == 0).all())
    assert bool(mass[3].isnan().all()) and bool(out.isnan().all())
    # the last new token alone sees the bad key: the others' weights are what they were without it
    scales = c["scales"].clone()
    scales[c["table"][1, 149 // page], 149 % page] = 255
    _, part = bfp8.latent_attention_mass(c["q"], c["cache"], scales, c["table"], c["lens"], SCALE, cu_q=c["cu"])
    assert bool(part[1, :150].isnan().all()) and torch.equal(part[0], clean[0]) and torch.equal(part[2:], clean[2:])


def test_nan_query_and_stale_cache(gpu):
    """A NaN query row adds NaN to the tokens that it sees; what the cache holds past a sequence does not matter."""
    lens, new, heads = [130, 61], [3, 1], 4
    c, keys = make(gpu, lens, new, heads, 64, seed=4)  # (NaN bytes wherever nothing is written)
    q = c["q"].clone()
    q[0, 2, 100] = float("nan")  # the first new token of sequence 0 does not see its last two
    announce("latent_attention_mass nan query")
    _, mass = bfp8.latent_attention_mass(q, c["cache"], c["scales"], c["table"], c["lens"], SCALE, cu_q=c["cu"])
    _, clean = bfp8.latent_attention_mass(c["q"], c["cache"], c["scales"], c["table"], c["lens"], SCALE, cu_q=c["cu"])
    assert bool(mass[0, :128].isnan().all()) and torch.equal(mass[0, 128:], clean[0, 128:]) and torch.equal(mass[1], clean[1])


def test_no_new_tokens(gpu):
    lens = [100, 3]
    c, _ = make(gpu, lens, [1, 1], 4, 16, seed=2)
    before = torch.rand(2, 130, device=gpu)
    cu = torch.zeros(3, dtype=torch.int32, device=gpu)
    out, mass = bfp8.latent_attention_mass(c["q"][:0], c["cache"], c["scales"], c["table"], c["lens"], SCALE, mass=before, cu_q=cu)
    assert out.shape[0] == 0
    for b, n in enumerate(lens):
        assert torch.equal(mass[b, :n], before[b, :n]) and bool((mass[b, n:] == 0).all())


@pytest.mark.parametrize("b,length,heads,width", [(520, 2200, 1, 36), (520, 2200, 150, 36), (17, 700, 8, 1 << 14), (300, 700, 16, 11)])
def test_many_sequences_of_shared_pages(gpu, b, length, heads, width):
    """520 sequences on the pages of one, so that none is cut and each walks more than 2048 keys; a page table that reaches
    far further than its sequences (2^20 tokens, too many for scores to be kept); 300 sequences, some of which are cut."""
    c, keys = make(gpu, [length], [1], 1, 64, seed=77)
    table = torch.full((b, width), -1, dtype=torch.int32, device=gpu)
    table[:, :c["table"].shape[1]] = c["table"]
    lens = torch.full((b,), length, dtype=torch.int32, device=gpu)
    g = torch.Generator().manual_seed(6)
    q = torch.randn(b, heads, 576, generator=g).to(torch.bfloat16).to(gpu)
    announce("latent_attention_mass shared pages", heads, width)
    _, mass = bfp8.latent_attention_mass(q, c["cache"], c["scales"], table, lens, SCALE)
    some = [0, 1, b // 2, b - 1]
    check(mass[some], None, q[some], keys * 4, [length] * 4, [1] * 4)
    assert bool(((mass.double().sum(dim=1) - heads).abs() <= 2.0 ** -15 * heads).all())


def test_far_pages(gpu):
    """Pages that lie past 4 GiB and 8 GiB of the cache."""
    lens, heads, page = [300, 77], 16, 64
    c, keys = make(gpu, lens, [1, 1], heads, page, seed=41)
    pages = 220000
    big = torch.empty(pages, page, 640, dtype=torch.uint8, device=gpu)
    scales = torch.empty(pages, page, dtype=torch.uint8, device=gpu)
    table = torch.full_like(c["table"], -1)
    for b, n in enumerate(lens):
        for i in range(-(-n // page)):
            to = pages - 1 - 7 * i if b == 0 else 110000 + 3 * i
            table[b, i] = to
            big[to], scales[to] = c["cache"][c["table"][b, i]], c["scales"][c["table"][b, i]]
    announce("latent_attention_mass far pages")
    _, mass = bfp8.latent_attention_mass(c["q"], big, scales, table, c["lens"], SCALE)
    check(mass, None, c["q"], keys, lens, [1, 1])


def test_captured_beside_eager_calls(gpu):
    """A replay follows later lengths, and larger eager calls on the stream do not disturb it."""
    lens, new, heads = [900, 400, 33], [1, 1, 1], 16
    c, keys = make(gpu, lens, new, heads, 64, seed=30)
    big, _ = make(gpu, [3000] * 4, [8] * 4, 32, 64, seed=31)
    before = torch.rand(3, c["table"].shape[1] * 64, device=gpu)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    announce("latent_attention_mass captured")
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            out, mass = bfp8.latent_attention_mass(c["q"], c["cache"], c["scales"], c["table"], c["lens"], SCALE, mass=before)
        for cut in (0, 7, 300):
            c["lens"].copy_(torch.tensor([max(n - cut, 1) for n in lens], dtype=torch.int32))
            bfp8.latent_attention_mass(big["q"], big["cache"], big["scales"], big["table"], big["lens"], SCALE, cu_q=big["cu"])
            graph.replay()
            want = bfp8.latent_attention_mass(c["q"], c["cache"], c["scales"], c["table"], c["lens"], SCALE, mass=before)
            stream.synchronize()
            assert torch.equal(out, want[0]) and torch.equal(mass, want[1])


def test_refusals(gpu):
    c, _ = make(gpu, [100, 3], [1, 1], 4, 16, seed=2)
    args = (c["q"], c["cache"], c["scales"], c["table"], c["lens"], SCALE)
    reach = c["table"].shape[1] * 16
    with pytest.raises(ValueError):
        bfp8.latent_attention_mass(*args, mass=torch.zeros(2, reach - 1, device=gpu))
    with pytest.raises(ValueError):
        bfp8.latent_attention_mass(*args, mass=torch.zeros(3, reach, device=gpu))
    with pytest.raises(ValueError):
        bfp8.latent_attention_mass(*args, mass=torch.zeros(2, reach, device=gpu), out_mass=torch.zeros(2, reach + 1, device=gpu))
    with pytest.raises(TypeError):
        bfp8.latent_attention_mass(*args, mass=torch.zeros(2, reach, dtype=torch.float64, device=gpu))
    with pytest.raises(ValueError):
        bfp8.latent_attention_mass(*args, workspace=torch.zeros(256, dtype=torch.uint8, device=gpu))
    with pytest.raises(ValueError):
        bfp8.latent_attention_mass(*args, mass=torch.zeros(2, reach))
