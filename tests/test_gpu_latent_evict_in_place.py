"""GPU tests of eviction within a sequence's own pages: pages that are none, lengths that are none, lengths updated where they lie,
and the widest masses."""

import pytest
import torch

import block_scaled_fp8_bfp8_amd as bfp8
from block_scaled_fp8_bfp8_amd import _native
from tests.gpu_util import announce
from tests.test_gpu_latent_evict import chosen, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page,n,budget", [(16, 96, 40), (16, 1300, 700), (37, 1299, 1298), (1, 70, 33)])
def test_bad_pages_and_lengths_in_place(gpu, page, n, budget):
    """A token without a page that moves reads as NaN where it goes; one whose new place is on no page is not stored; one that
    stays is left alone. Lengths below zero and past the table count as none and as the table's reach."""
    recent = 4
    full, codes, table, _, g = make([n, n, n, n], page, 5, extra=0)
    last = table.shape[1] - 1
    table[1, last // 2] = -1                    # tokens that move lie nowhere
    table[2, 1] = full.shape[0]                 # and others would move there
    table[2, last // 3] = -(1 << 31)
    reach = table.shape[1] * page
    mass = torch.rand(4, reach, generator=g)
    mass[1, last // 2 * page:(last // 2 + 1) * page] += 2
    lens = [-3, n, n, (1 << 31) - 1]
    cache, scales = full.to(gpu), codes.to(gpu)
    announce("latent_cache_evict in place, bad pages", page, n, budget)
    kept, new, _ = bfp8.latent_cache_evict(cache, scales, table.to(gpu), torch.tensor(lens, dtype=torch.int32, device=gpu),
                                           mass.to(gpu), budget, recent=recent)
    got, got_codes = cache.cpu(), scales.cpu()
    want, want_codes = full.clone(), codes.clone()
    for b, length in enumerate((0, n, n, reach)):
        stay = chosen(mass[b], length, budget, recent)
        assert int(new[b]) == len(stay) and kept[b, :len(stay)].tolist() == stay
        for i, j in enumerate(stay):
            src, dst = int(table[b, j // page]), int(table[b, i // page])
            if i == j or not 0 <= dst < full.shape[0]:
                continue
            if 0 <= src < full.shape[0]:
                want[dst, i % page], want_codes[dst, i % page] = full[src, j % page], codes[src, j % page]
            else:
                want[dst, i % page, :512], want[dst, i % page, 512::2], want[dst, i % page, 513::2] = 0, 0xFF, 0x7F
                want_codes[dst, i % page] = 255
        for i in range(len(stay), length):  # (nothing is said of rows past the new length)
            at = (int(table[b, i // page]), i % page)
            if 0 <= at[0] < full.shape[0]:
                want[at], want_codes[at] = got[at], got_codes[at]
    assert torch.equal(got, want) and torch.equal(got_codes, want_codes)


@pytest.mark.parametrize("onto", [False, True])
def test_lengths_and_masses_where_they_lie(gpu, onto):
    """lens_out may be seq_lens, mass_out the masses: the C entry, with the results of separate ones."""
    lens, page, budget, recent = [500, 90, 1030], 16, 100, 7
    full, codes, table, to, g = make(lens, page, 8, spare=budget if onto else 0)
    mass = torch.rand(3, table.shape[1] * page, generator=g).to(gpu)
    table = table.to(gpu)
    to = to.to(gpu) if onto else None
    caches = [(full.to(gpu), codes.to(gpu)) for _ in range(2)]
    lens_t = torch.tensor(lens, dtype=torch.int32, device=gpu)
    announce("latent_cache_evict lengths in place", onto)
    kept, new, moved = bfp8.latent_cache_evict(*caches[0], table, lens_t, mass, budget, recent=recent, out_table=to)
    cache, scales = caches[1]
    kept2 = torch.empty_like(kept)
    st = _native.lib().bfp8_latent_cache_evict(
        cache.data_ptr(), cache.stride(0), scales.data_ptr(), scales.stride(0), cache.shape[0], page, table.data_ptr(), table.stride(0),
        table.shape[1], lens_t.data_ptr(), 3, mass.data_ptr(), mass.stride(0), mass.shape[1], budget, recent,
        to.data_ptr() if onto else None, to.stride(0) if onto else 0, to.shape[1] if onto else 0, kept2.data_ptr(), lens_t.data_ptr(),
        mass.data_ptr(), mass.stride(0), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == _native.BFP8_OK
    assert torch.equal(kept, kept2) and torch.equal(new, lens_t) and torch.equal(moved, mass)
    if onto:
        assert torch.equal(caches[0][0], cache) and torch.equal(caches[0][1], scales)
    else:
        for b, n in enumerate(new.tolist()):
            for i in range(n):
                at = (int(table[b, i // page]), i % page)
                assert torch.equal(caches[0][0][at], cache[at]) and int(caches[0][1][at]) == int(scales[at])


def test_widest_masses(gpu):
    """The most columns that are accepted, 65537 below 2^31, in place."""
    n, page, budget, width = 100, 16, 40, (1 << 31) - 1 - 65536
    full, codes, table, _, g = make([n], page, 9)
    mass = torch.rand(1, table.shape[1] * page, generator=g)
    wide = torch.full((1, width), 7.0, device=gpu)
    wide[:, :mass.shape[1]] = mass.to(gpu)
    announce("latent_cache_evict widest")
    kept, new, got = bfp8.latent_cache_evict(full.to(gpu), codes.to(gpu), table.to(gpu), torch.tensor([n], dtype=torch.int32, device=gpu),
                                             wide, budget, recent=3, out_mass=wide)
    stay = chosen(mass[0], n, budget, 3)
    assert got is wide and kept[0].tolist() == stay and int(new[0]) == budget
    assert torch.equal(got[0, :budget].cpu(), mass[0][stay])
    assert max(float(p.abs().max()) for p in got[0, budget:].split(1 << 28)) == 0.0
