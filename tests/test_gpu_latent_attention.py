"""GPU tests of latent attention over the paged FP8 cache (absorbed form) against float64.

Tolerance, per element, with A = the weights' average of |c| and reach = the row's largest
scale * sum |q||k|:
  2^-8 |o|           the output's rounding to bf16
  2^-8 A             the weights' rounding to 8 significant bits (each off by at most 2^-8 of itself)
  2^-10 A            the FP8 block dot drops what lies 13 binades below a product's group of 8:
                     8 * 2^-13 of the group's largest product, summed over the groups
  2 (e^d - 1) A      scores off by d = 2^-10 reach (the same window) move a weight and its sum
  2^-14 A            float32 sums
These are worst cases of errors of either sign; so the root mean square over all elements is also
held: bf16 rounding (2^-8 / sqrt 3 of a value at most), weights (2^-10) and scores (2^-11) together
stay below 2^-8 of the root mean square of o."""

import numpy as np
import pytest
import torch

import block_scaled_fp8_bfp8_amd as bfp8
from oracle import e4m3, latent
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


def make(gpu, lens, new, heads, page, seed, spread=0.7, width_extra=0, gap=0):
    """A case on the GPU and its float64 keys: dict of tensors, and per sequence [L, 576]."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(n, 0) // page) for n in lens]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g).int()
    table = torch.full((len(lens), max(need + [1]) + width_extra), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    full = torch.full((pages, page + gap, 640), 0xFF, dtype=torch.uint8, device=gpu)  # NaN wherever nothing is written
    fsc = torch.full((pages, page + gap), 0xFF, dtype=torch.uint8, device=gpu)
    cache, sc = full[:, :page], fsc[:, :page]
    keys = []
    for b, n in enumerate(lens):
        if n <= 0:
            keys.append(np.zeros((0, 576)))
            continue
        kv = torch.randn(n, 576, generator=g) * torch.exp(spread * torch.randn(n, 1, generator=g))
        kv = kv.bfloat16()
        i = torch.arange(n)
        slots = table[b, i // page].long() * page + i % page
        bfp8.latent_cache_write(kv.to(gpu), slots.to(gpu), cache, sc)
        rows = cache.cpu()[slots // page, slots % page].numpy()
        codes = sc.cpu()[slots // page, slots % page].numpy()
        lat = e4m3.decode(rows[:, :512].copy()) * latent.e8m0_value(codes)[:, None]
        keys.append(np.concatenate([lat, kv[:, 512:].double().numpy()], axis=1))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
    q = torch.randn(int(cu[-1]), heads, 576, generator=g).bfloat16()
    return dict(q=q.to(gpu), cache=cache, scales=sc, table=table.to(gpu),
                lens=torch.tensor(lens, dtype=torch.int32, device=gpu), cu=cu.to(gpu)), keys


def check(out, q, keys, lens, new, scale=SCALE):
    got, q = out.double().cpu().numpy(), q.double().cpu().numpy()
    heads = q.shape[1]
    assert np.isfinite(got).all()
    at, err, tot = 0, 0.0, 0.0
    for k, length, n in zip(keys, lens, new):
        if n == 0:
            continue
        rows = q[at:at + n].reshape(n * heads, 576)
        sees = np.repeat(length - n + 1 + np.arange(n), heads)
        o, mag, reach = latent.attention_ref(rows, k, k[:, :512], sees, scale)
        diff = np.abs(got[at:at + n].reshape(n * heads, 512) - o)
        d = 2.0 ** -10 * reach[:, None]
        bound = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -14 + 2 * np.expm1(d)) * mag
        assert (diff <= bound).all(), f"worst {np.max(diff / np.maximum(bound, 1e-300))} of the bound"
        err += (diff ** 2).sum()
        tot += (o ** 2).sum()
        at += n
    assert at == got.shape[0]
    assert err <= 2.0 ** -16 * tot, f"rms error {np.sqrt(err / max(tot, 1e-300))}"


def attend(c, with_cu=True, scale=SCALE, **kw):
    return bfp8.latent_attention(c["q"], c["cache"], c["scales"], c["table"], c["lens"], scale,
                                 cu_q=c["cu"] if with_cu else None, **kw)


@pytest.mark.parametrize("lens,heads,page", [
    ([1], 1, 1), ([2], 16, 64), ([63, 64, 65], 5, 16), ([1, 127, 128, 129], 16, 37), ([300], 128, 64), ([1000, 3, 511], 40, 16),
    ([700, 650], 128, 1), ([2500], 8, 64), ([130, 131], 17, 64), ([257] * 9, 32, 37), ([5] * 300, 16, 16)])
def test_one_new_token(gpu, lens, heads, page):
    announce("latent attention decode", lens[:5], heads, page)
    c, keys = make(gpu, lens, [1] * len(lens), heads, page, seed=len(lens) * 31 + heads)
    out = attend(c, with_cu=False)
    check(out, c["q"], keys, lens, [1] * len(lens))
    assert torch.equal(out.view(torch.int16), attend(c).view(torch.int16))  # the same with cu_q, and again


@pytest.mark.parametrize("lens,new,heads,page", [
    ([5], [5], 1, 4), ([70, 64], [70, 3], 16, 16), ([300, 40, 129], [2, 40, 17], 128, 64), ([900], [7], 40, 37),
    ([200, 333], [33, 0], 5, 16), ([600, 10], [1, 4], 64, 1), ([1100], [66], 3, 64)])
def test_chunks(gpu, lens, new, heads, page):
    announce("latent attention chunk", lens, new, heads, page)
    c, keys = make(gpu, lens, new, heads, page, seed=sum(new) + heads)
    check(attend(c), c["q"], keys, lens, new)


def test_rows_that_see_nothing(gpu):
    """Empty sequences, and chunks longer than their sequences: rows before the first key are zero."""
    lens, new, heads = [0, 3, -5, 40], [2, 5, 1, 40], 16
    announce("latent attention empty rows")
    c, keys = make(gpu, lens, new, heads, 16, seed=77)
    out = attend(c)
    assert (out[:2] == 0).all() and (out[2:4] == 0).all() and (out[7] == 0).all()
    check(out, c["q"], keys, [max(n, 0) for n in lens], new)


def test_strides_page_gaps_and_untouched_rows(gpu):
    lens, new, heads = [90, 33], [4, 2], 7
    announce("latent attention strides")
    c, keys = make(gpu, lens, new, heads, 16, seed=78, width_extra=5, gap=1)
    want = attend(c)
    t = 6
    big = torch.full((t + 2, heads + 3, 640), float("nan"), dtype=torch.bfloat16, device=gpu)
    big[1:t + 1, 1:heads + 1, 8:584] = c["q"]
    c["q"] = big[1:t + 3, 1:heads + 1, 8:584]  # one row that no sequence owns
    out = torch.full((t + 1, heads + 1, 520), 7.0, dtype=torch.bfloat16, device=gpu)
    wide = torch.full((2, c["table"].shape[1] + 3), 99, dtype=torch.int32, device=gpu)
    wide[:, :c["table"].shape[1]] = c["table"]
    c["table"] = wide[:, :c["table"].shape[1]]
    attend(c, out=out[:, :heads, :512])
    assert torch.equal(out[:t, :heads, :512], want)
    assert (out[t] == 7.0).all() and (out[:, heads] == 7.0).all() and (out[:, :, 512:] == 7.0).all()
    check(want, c["q"][:t], keys, lens, new)


@pytest.mark.parametrize("scale", [0.0, -SCALE, 3.0])
def test_scales_of_the_softmax(gpu, scale):
    """No temperature, a negative one, and one sharp enough to leave one or two keys."""
    announce("latent attention scale", scale)
    c, keys = make(gpu, [200], [3], 16, 16, seed=79)
    check(attend(c, scale=scale), c["q"], keys, [200], [3], scale)


def test_token_scales_far_apart(gpu):
    """Tokens 2^70 apart in size: a key of huge values under a tiny weight, and the reverse. Queries
    look along the rotary key alone, so that scores stay moderate."""
    heads, n = 4, 96
    c, keys = make(gpu, [n], [1], heads, 16, seed=80)
    g = torch.Generator().manual_seed(81)
    size = torch.exp2(torch.randint(-38, 33, (n, 1), generator=g).float())
    kv = (torch.randn(n, 576, generator=g) * torch.cat([size.expand(n, 512), torch.full((n, 64), 2.0)], dim=1)).bfloat16()
    i = torch.arange(n)
    slots = c["table"].cpu()[0, i // 16].long() * 16 + i % 16
    announce("latent attention token scales")
    bfp8.latent_cache_write(kv.to(gpu), slots.to(gpu), c["cache"], c["scales"])
    rows = c["cache"].cpu()[slots // 16, slots % 16].numpy()
    codes = c["scales"].cpu()[slots // 16, slots % 16].numpy()
    lat = e4m3.decode(rows[:, :512].copy()) * latent.e8m0_value(codes)[:, None]
    keys = [np.concatenate([lat, kv[:, 512:].double().numpy()], axis=1)]
    c["q"][:, :, :512] = 0
    out = attend(c)
    check(out, c["q"], keys, [n], [1])


def test_far_below_and_above_one(gpu):
    """Query rows of very different size, zero rows among them."""
    c, keys = make(gpu, [150], [1], 6, 16, seed=82)
    c["q"][0, 1] *= 2.0 ** -60
    c["q"][0, 2] = 0
    c["q"][0, 3] *= 2.0 ** -9
    c["q"][0, 4, :512] *= 2.0 ** -30
    c["q"][0, 5, 1:] *= 2.0 ** -12
    announce("latent attention query sizes")
    check(attend(c), c["q"], keys, [150], [1])


def test_nan_stays_where_it_is_seen(gpu):
    """A NaN query row, a token stored as NaN and a NaN rotary key reach the rows that see them and
    no others; so does a page that does not exist."""
    lens, new, heads = [40, 30], [8, 3], 2
    c, keys = make(gpu, lens, new, heads, 4, seed=83)
    want = attend(c)
    kv = torch.zeros(2, 576, dtype=torch.bfloat16)
    kv[0, 3] = float("inf")   # token 36 of sequence 0: rows of tokens 36 .. 39
    kv[1, 575] = float("nan")  # token 38
    tab = c["table"].cpu()
    slots = torch.tensor([int(tab[0, 9]) * 4, int(tab[0, 9]) * 4 + 2])
    announce("latent attention nan")
    bfp8.latent_cache_write(kv.to(gpu), slots.to(gpu), c["cache"], c["scales"])
    c["q"][9, 1, 100] = float("nan")
    out = attend(c)
    assert out[4:8].isnan().all()  # tokens 36 .. 39
    assert out[9, 1].isnan().all()
    same = torch.ones(11, heads, dtype=torch.bool)
    same[4:8] = False
    same[9, 1] = False
    assert torch.equal(out.cpu()[same], want.cpu()[same])
    c["table"][1, 2] = c["cache"].shape[0] + 5
    assert attend(c)[8:].isnan().all()


def test_batches_that_are_cut(gpu):
    """One long sequence among many short ones: blocks cut along their keys and joined."""
    lens = [9000] + [64 * i + 1 for i in range(6)]
    announce("latent attention cut")
    c, keys = make(gpu, lens, [1] * 7, 16, 64, seed=84)
    out = attend(c, with_cu=False)
    check(out, c["q"], keys, lens, [1] * 7)
    for _ in range(3):  # the same bits again
        assert torch.equal(out, attend(c, with_cu=False))


def test_own_workspace_and_side_stream(gpu):
    lens = [500, 700]
    c, keys = make(gpu, lens, [1, 1], 128, 64, seed=85)
    want = attend(c)
    need = bfp8.latent_attention_workspace_bytes(2, 2, 128, c["table"].shape[1] * 64)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=gpu)
    side = torch.cuda.Stream(gpu)
    side.wait_stream(torch.cuda.current_stream())
    announce("latent attention side stream")
    with torch.cuda.stream(side):
        out = attend(c, workspace=ws)
    side.synchronize()
    assert torch.equal(out, want)
    with pytest.raises(ValueError):
        attend(c, workspace=ws[:need - 1])


def test_graph_follows_lengths(gpu):
    """A captured call, replayed after the lengths and the queries changed in place."""
    lens = [900, 200]
    c, keys = make(gpu, lens, [1, 1], 16, 16, seed=86)
    out = torch.empty(2, 16, 512, dtype=torch.bfloat16, device=gpu)
    announce("latent attention graph")
    side = torch.cuda.Stream(gpu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        attend(c, out=out)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            attend(c, out=out)
    torch.cuda.synchronize()
    for a, b in [(900, 200), (17, 199), (640, 1), (0, 128)]:
        c["lens"].copy_(torch.tensor([a, b], dtype=torch.int32))
        c["q"].mul_(0.75)
        want = attend(c)
        out.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_cache_past_four_gib(gpu):
    """Pages far apart, the last one past 2^32 bytes from the first."""
    page, stride = 16, 1 << 30
    pages = 6
    big = torch.empty((pages - 1) * stride + page * 640, dtype=torch.uint8, device=gpu)
    cache = big.as_strided((pages, page, 640), (stride, 640, 1))
    sc = torch.empty(pages, page, dtype=torch.uint8, device=gpu)
    g = torch.Generator().manual_seed(87)
    kv = torch.randn(page, 576, generator=g).bfloat16().to(gpu)
    announce("latent attention 4 GiB")
    small, ssc = torch.zeros(1, page, 640, dtype=torch.uint8, device=gpu), torch.zeros(1, page, dtype=torch.uint8, device=gpu)
    i = torch.arange(page, device=gpu)
    bfp8.latent_cache_write(kv, i, small, ssc)
    bfp8.latent_cache_write(kv, i + (pages - 1) * page, cache, sc)
    q = torch.randn(1, 16, 576, generator=g).bfloat16().to(gpu)
    lens = torch.tensor([page], dtype=torch.int32, device=gpu)
    want = bfp8.latent_attention(q, small, ssc, torch.zeros(1, 1, dtype=torch.int32, device=gpu), lens, SCALE)
    got = bfp8.latent_attention(q, cache, sc, torch.full((1, 1), pages - 1, dtype=torch.int32, device=gpu), lens, SCALE)
    assert torch.equal(got, want)
    cu = torch.tensor([0, page], dtype=torch.int32, device=gpu)
    far = torch.full((1, 1), pages - 1, dtype=torch.int32, device=gpu)
    assert torch.equal(bfp8.latent_cache_read(cache, sc, far, cu, page),
                       bfp8.latent_cache_read(small, ssc, torch.zeros_like(far), cu, page))


def test_empty_and_refusals(gpu):
    c, _ = make(gpu, [10], [1], 4, 4, seed=88)
    empty = bfp8.latent_attention(c["q"][:0], c["cache"], c["scales"], c["table"][:0], c["lens"][:0], SCALE)
    assert empty.shape == (0, 4, 512)
    q, rest = c["q"], (c["cache"], c["scales"], c["table"], c["lens"], SCALE)
    with pytest.raises(TypeError):
        bfp8.latent_attention(q.half(), *rest)
    with pytest.raises(ValueError):
        bfp8.latent_attention(q[:, :, :512], *rest)
    with pytest.raises(ValueError):
        bfp8.latent_attention(q.expand(2, 4, 576), *rest)  # two tokens, one sequence, no cu_q
    with pytest.raises(ValueError):
        bfp8.latent_attention(q, *rest, cu_q=c["cu"][:1])
    with pytest.raises(TypeError):
        bfp8.latent_attention(q, *rest, cu_q=c["cu"].long())
    with pytest.raises(ValueError):
        bfp8.latent_attention(q, *rest[:3], c["lens"].expand(2).contiguous(), SCALE)
    with pytest.raises(ValueError):
        bfp8.latent_attention(q, *rest, out=torch.empty(1, 4, 511, dtype=torch.bfloat16, device=gpu))
    with pytest.raises(ValueError):
        bfp8.latent_attention(q, *rest[:4], float("nan"))
    with pytest.raises(ValueError):
        bfp8.latent_attention(q.cpu(), *rest)


@pytest.mark.parametrize("heads", [2, 40])
@pytest.mark.parametrize("how", ["no page of the cache", "past the table"])
def test_missing_page_reaches_only_rows_that_see_it(gpu, heads, how):
    """A chunk whose last tokens alone lie on a missing page: the rows before them are as they were, whatever bytes
    the cache's first row holds (here the e4m3 codes of NaN)."""
    lens, new = [200, 30], [9, 2]
    c, keys = make(gpu, lens, new, heads, 4, seed=89)
    nan_page = torch.full_like(c["cache"][:1], 0xFF), torch.full_like(c["scales"][:1], 0xFF)
    c["cache"] = torch.cat([nan_page[0], c["cache"]])
    c["scales"] = torch.cat([nan_page[1], c["scales"]])
    c["table"] = torch.where(c["table"] >= 0, c["table"] + 1, c["table"])
    want = attend(c)
    check(want, c["q"], keys, lens, new)
    if how == "past the table":
        c["table"] = c["table"][:, :49].contiguous()  # token 196 on (tokens 191 .. 199 are new)
    else:
        c["table"][0, 49] = c["cache"].shape[0]
    announce("latent attention missing page", heads, how)
    out = attend(c)
    if how == "past the table":  # (a narrower table may be cut in another way)
        check(out[:5], c["q"][:5], [keys[0][:196]], [196], [5])
        check(out[9:], c["q"][9:], keys[1:], lens[1:], new[1:])
    else:
        assert torch.equal(out[:5], want[:5]) and torch.equal(out[9:], want[9:])
    assert out[5:9].isnan().all()


@pytest.mark.parametrize("length", [2 ** 31 - 1, 2 ** 31 - 64, 2 ** 30, 65, 96])
@pytest.mark.parametrize("heads", [2, 128])
def test_lengths_past_the_table(gpu, length, heads):
    """A length that the page table does not hold makes the rows that see past it NaN, soon and whatever the length,
    and leaves the other sequences as they were."""
    lens, new = [64, 30], [3, 2]
    c, keys = make(gpu, lens, new, heads, 16, seed=90)
    want = attend(c)
    c["lens"][0] = length
    announce("latent attention length past the table", length, heads)
    out = attend(c)
    assert torch.equal(out[3:], want[3:])
    past = [min(length, 1000) - 3 + i + 1 > 64 for i in range(3)]
    assert out[:3][torch.tensor(past)].isnan().all()
    if not all(past):
        check(out[:2], c["q"][:2], [keys[0]], [64], [2])
