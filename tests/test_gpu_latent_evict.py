"""GPU tests of eviction from the latent cache: what stays is compared with a sort on the host, and every byte of the cache with
what it should hold (nothing is computed, so there is no tolerance)."""

import pytest
import torch

import block_scaled_fp8_bfp8_amd as bfp8
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu


def make(lens, page, seed, spare=0, gap=0, extra=1):
    """A cache of random bytes (on the host), page tables for the lengths and for `spare` tokens a sequence."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(n, 0) // page) for n in lens]
    more = -(-spare // page)
    pages = sum(need) + more * len(lens) + 2
    order = torch.randperm(pages, generator=g).int()
    table = torch.full((len(lens), max(need + [0]) + extra), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    to = order[at:at + more * len(lens)].view(len(lens), more).contiguous() if more else None
    full = torch.randint(0, 256, (pages, page + gap, 640), generator=g, dtype=torch.uint8)
    codes = torch.randint(0, 256, (pages, page + gap), generator=g, dtype=torch.uint8)
    return full, codes, table, to, g


def chosen(mass, n, budget, recent):
    """The tokens that stay, from the definition."""
    if n <= budget:
        return list(range(n))
    worth = [float("inf") if m != m else m for m in mass[:n - recent].tolist()]
    nan_first = [0 if m != m else 1 for m in mass[:n - recent].tolist()]
    order = sorted(range(n - recent), key=lambda j: (nan_first[j], -worth[j], j))
    return sorted(order[:budget - recent]) + list(range(n - recent, n))


def run(gpu, lens, page, budget, recent, mass, seed=0, onto=False, gap=0, in_place_mass=False):
    reach_lens = lens
    full, codes, table, to, _ = make(lens, page, seed, spare=min(budget, max(lens)) if onto else 0, gap=gap)
    want, want_codes = full.clone(), codes.clone()
    cache, scales = full.to(gpu), codes.to(gpu)
    m = mass.to(gpu)
    lens_t = torch.tensor(lens, dtype=torch.int32, device=gpu)
    kept, new, moved = bfp8.latent_cache_evict(cache[:, :page], scales[:, :page], table.to(gpu), lens_t, m, budget, recent=recent,
                                               out_table=to.to(gpu) if onto else None, out_mass=m if in_place_mass else None)
    kept, new, moved = kept.cpu(), new.cpu(), moved.cpu()
    for b, n in enumerate(reach_lens):
        stay = chosen(mass[b], n, budget, recent)
        assert new[b] == len(stay)
        assert kept[b, :len(stay)].tolist() == stay and bool((kept[b, len(stay):] == -1).all()), b
        ref = torch.zeros_like(mass[b])
        ref[:len(stay)] = mass[b][stay]
        assert torch.equal(moved[b].view(torch.int32), ref.view(torch.int32)), b
        where = to if onto else table
        for i, j in enumerate(stay):
            src, dst = (table[b, j // page], j % page), (where[b, i // page], i % page)
            want[dst], want_codes[dst] = full[src], codes[src]
    got, got_codes = cache.cpu(), scales.cpu()
    if not onto:  # rows past the new length hold what they held, or what moved over them: nothing is said of them
        for b, n in enumerate(lens):
            for i in range(int(new[b]), n):
                at = (table[b, i // page], i % page)
                want[at], want_codes[at] = got[at], got_codes[at]
    assert torch.equal(got, want) and torch.equal(got_codes, want_codes)


CASES = [
    ([1], 1, 1, 0), ([2], 1, 1, 0), ([2], 1, 1, 1), ([100, 5, 64], 16, 64, 0), ([100, 65, 64, 63], 16, 64, 64), ([300, 0, 77], 37, 50, 13),
    ([1111], 64, 1024, 128), ([1030, 2100, 1023], 64, 1000, 7), ([700] * 5, 16, 1, 0), ([2500, 900], 37, 2047, 500), ([600, 600], 16, 599, 3),
]


@pytest.mark.parametrize("onto", [False, True])
@pytest.mark.parametrize("lens,page,budget,recent", CASES)
def test_evict(gpu, lens, page, budget, recent, onto):
    announce("latent_cache_evict", lens, page, budget, recent, onto)
    g = torch.Generator().manual_seed(budget + recent)
    width = (-(-max(lens) // page) + 1) * page + 5
    mass = torch.exp(3 * torch.randn(len(lens), width, generator=g))
    mass[torch.rand(mass.shape, generator=g) < 0.3] = 0.0
    run(gpu, lens, page, budget, recent, mass, seed=budget, onto=onto, gap=1 if page > 1 else 0)


@pytest.mark.parametrize("onto", [False, True])
def test_long_sequences(gpu, onto):
    """More tokens than a workgroup holds masses of at once, and more chunks than one of moves."""
    lens = [20011, 8192, 8193]
    g = torch.Generator().manual_seed(1)
    mass = torch.rand(3, 20011 + 64 + 64, generator=g).round(decimals=2)  # (many equal ones)
    announce("latent_cache_evict long", onto)
    run(gpu, lens, 64, 8000, 100, mass, onto=onto, in_place_mass=True)


@pytest.mark.parametrize("kind", ["equal", "zeros", "nan", "signs", "infinite", "bits", "falling", "rising"])
def test_orders(gpu, kind):
    n, width = 700, 800
    g = torch.Generator().manual_seed(3)
    mass = torch.rand(2, width, generator=g)
    if kind == "equal":
        mass[:] = 0.37
    elif kind == "zeros":
        mass = torch.where(torch.rand(2, width, generator=g) < 0.5, 0.0, -0.0)
    elif kind == "nan":
        mass[torch.rand(2, width, generator=g) < 0.2] = float("nan")
        mass[0, 4] = -float("nan")
        mass[0, 9] = float("inf")
    elif kind == "signs":
        mass = torch.randn(2, width, generator=g)
    elif kind == "infinite":
        mass[torch.rand(2, width, generator=g) < 0.2] = float("inf")
        mass[torch.rand(2, width, generator=g) < 0.5] = -float("inf")
    elif kind == "bits":  # neighbours in the last bits, and subnormals
        mass = (0x3f800000 + torch.randint(0, 5, (2, width), generator=g)).int().view(torch.float32).clone()
        mass[1] = torch.randint(0, 7, (width,), generator=g).int().view(torch.float32)
    else:
        mass = torch.arange(width).float().repeat(2, 1)
        if kind == "falling":
            mass = -mass
    announce("latent_cache_evict order", kind)
    for budget, recent in ((1, 0), (100, 0), (350, 31), (699, 0), (699, 699)):
        run(gpu, [n, n - 13], 16, budget, recent, mass.clone(), seed=budget)


def test_bad_lengths_and_pages(gpu):
    """Lengths below zero and past the table; a token whose page is none reads as NaN where it goes, and one whose new page is none is
    not stored."""
    page, budget = 16, 40
    full, codes, table, to, g = make([96, 96, 96, 96], page, 5, spare=budget, extra=0)
    table[2, 1] = -1
    table[3, 5] = full.shape[0]
    to[3, 1] = -7
    mass = torch.rand(4, 96, generator=g)
    mass[2, 16:32] += 2  # the tokens without a page stay
    lens = torch.tensor([-5, 1 << 30, 96, 96], dtype=torch.int32, device=gpu)
    cache, scales = full.to(gpu), codes.to(gpu)
    announce("latent_cache_evict bad lengths and pages")
    kept, new, _ = bfp8.latent_cache_evict(cache, scales, table.to(gpu), lens, mass.to(gpu), budget, recent=4, out_table=to.to(gpu))
    assert new.tolist() == [0, 40, 40, 40]
    got, got_codes = cache.cpu(), scales.cpu()
    want, want_codes = full.clone(), codes.clone()
    for b in (1, 2, 3):
        stay = chosen(mass[b], 96, budget, 4)
        assert kept[b].tolist() == stay
        for i, j in enumerate(stay):
            src, dst = int(table[b, j // page]), int(to[b, i // page])
            if dst < 0:
                continue
            if 0 <= src < full.shape[0]:
                want[dst, i % page], want_codes[dst, i % page] = full[src, j % page], codes[src, j % page]
            else:
                want[dst, i % page, :512], want[dst, i % page, 512::2], want[dst, i % page, 513::2] = 0, 0xFF, 0x7F
                want_codes[dst, i % page] = 255
    assert torch.equal(got, want) and torch.equal(got_codes, want_codes)


@pytest.mark.parametrize("onto", [False, True])
def test_far_pages(gpu, onto):
    """From and to pages past 4 GiB of the cache."""
    page, pages, n, budget = 64, 110000, 200, 130
    g = torch.Generator().manual_seed(9)
    cache = torch.zeros(pages, page, 640, dtype=torch.uint8, device=gpu)
    scales = torch.zeros(pages, page, dtype=torch.uint8, device=gpu)
    table = torch.tensor([[pages - 1, 3, pages - 7, 105000]], dtype=torch.int32)
    to = torch.tensor([[106000, pages - 2, 12]], dtype=torch.int32)
    rows = torch.randint(0, 256, (4, page, 640), generator=g, dtype=torch.uint8)
    codes = torch.randint(0, 256, (4, page), generator=g, dtype=torch.uint8)
    for i, p in enumerate(table[0].tolist()):
        cache[p], scales[p] = rows[i].to(gpu), codes[i].to(gpu)
    mass = torch.rand(1, 256, generator=g)
    announce("latent_cache_evict far pages", onto)
    bfp8.latent_cache_evict(cache, scales, table.to(gpu), torch.tensor([n], dtype=torch.int32, device=gpu), mass.to(gpu), budget,
                            recent=20, out_table=to.to(gpu) if onto else None)
    stay = chosen(mass[0], n, budget, 20)
    where = (to if onto else table)[0].tolist()
    for i, j in enumerate(stay):
        assert torch.equal(cache[where[i // page], i % page].cpu(), rows[j // page, j % page])
        assert int(scales[where[i // page], i % page]) == int(codes[j // page, j % page])


def test_captured(gpu):
    """A captured call follows later masses and lengths."""
    lens, page, budget = [400, 300], 16, 200
    full, codes, table, to, g = make(lens, page, 6, spare=budget)
    cache, scales, table, to = full.to(gpu), codes.to(gpu), table.to(gpu), to.to(gpu)
    mass, lens_t = torch.rand(2, 416, generator=g).to(gpu), torch.tensor(lens, dtype=torch.int32, device=gpu)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    announce("latent_cache_evict captured")
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            got = bfp8.latent_cache_evict(cache, scales, table, lens_t, mass, budget, recent=10, out_table=to)
        for i in range(3):
            mass.copy_(torch.rand(2, 416, generator=g))
            lens_t.copy_(torch.tensor([400 - 90 * i, 300], dtype=torch.int32))
            graph.replay()
            stream.synchronize()
            kept, new, _ = (t.clone() for t in got)
            rows = cache.clone()
            want = bfp8.latent_cache_evict(cache, scales, table, lens_t, mass, budget, recent=10, out_table=to)
            stream.synchronize()
            assert torch.equal(kept, want[0]) and torch.equal(new, want[1]) and torch.equal(rows, cache)


def test_empty_and_refusals(gpu):
    full, codes, table, to, g = make([40, 40], 16, 7, spare=16)
    cache, scales, table, to = full.to(gpu), codes.to(gpu), table.to(gpu), to.to(gpu)
    mass, lens = torch.rand(2, 64, generator=g).to(gpu), torch.tensor([40, 40], dtype=torch.int32, device=gpu)
    kept, new, m = bfp8.latent_cache_evict(cache, scales, table[:0], lens[:0], mass[:0], 8)
    assert kept.shape == (0, 8) and new.shape == (0,) and m.shape == (0, 64)
    for kw in (dict(budget=0), dict(budget=8, recent=9), dict(budget=8, recent=-1), dict(budget=8, out_table=to[:1]),
               dict(budget=8, out_table=to[:, :0]), dict(budget=8, out_mass=torch.zeros(2, 65, device=gpu))):
        with pytest.raises(ValueError):
            bfp8.latent_cache_evict(cache, scales, table, lens, mass, **kw)
    with pytest.raises(ValueError):
        bfp8.latent_cache_evict(cache, scales, table, lens, mass[:, :63], 8)
    with pytest.raises(TypeError):
        bfp8.latent_cache_evict(cache, scales, table, lens, mass.double(), 8)
    with pytest.raises(ValueError):
        bfp8.latent_cache_evict(cache, scales, table, lens, mass.cpu(), 8)
