"""GPU tests of the paged FP8 latent cache: writing (with and without the norm), reading back and
gathering, against float64. Without the norm the stored bytes are exact: the scale code and the
e4m3 rounding of an exact quotient. With it, y is off by at most d = 2^-17 of itself (a chain of
8 + 6 float32 additions, a square root and a few roundings), as in the norm's own tests."""

import numpy as np
import pytest
import torch

import block_scaled_fp8_bfp8_amd as bfp8
from oracle import e4m3, latent
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu
D = 2.0 ** -17


def _kv(t, seed):
    g = torch.Generator().manual_seed(seed)
    kv = torch.randn(t, 576, generator=g) * torch.exp(2 * torch.randn(t, 1, generator=g))
    return kv.bfloat16()


def _empty_cache(gpu, pages, page, gap=0):
    """A cache filled with NaN codes whose pages are `gap` rows apart."""
    full = torch.full((pages, page + gap, 640), 0xFF, dtype=torch.uint8, device=gpu)
    sc = torch.full((pages, page + gap), 0xFF, dtype=torch.uint8, device=gpu)
    return full, sc, full[:, :page], sc[:, :page]


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("t,pages,page,gap", [(1, 1, 1, 0), (3, 5, 1, 0), (67, 9, 16, 0), (200, 7, 37, 3), (1000, 17, 64, 1)])
def test_write(gpu, t, pages, page, gap, norm):
    announce("latent write", t, pages, page, gap, norm)
    kv = _kv(t, t)
    w = (1 + 0.3 * torch.randn(512, generator=torch.Generator().manual_seed(1))).bfloat16() if norm else None
    full, fsc, cache, sc = _empty_cache(gpu, pages, page, gap)
    perm = torch.randperm(pages * page, generator=torch.Generator().manual_seed(2))[:t]
    bfp8.latent_cache_write(kv.to(gpu), perm.to(gpu), cache, sc, norm_weight=None if w is None else w.to(gpu), eps=1e-6)
    torch.cuda.synchronize()
    y = kv[:, :512].double().numpy()
    if norm:
        y = latent.rmsnorm_ref(y, w.double().numpy(), 1e-6)
    rows = cache.cpu()[perm // page, perm % page].numpy()
    codes = sc.cpu()[perm // page, perm % page].numpy().astype(np.int64)
    want = latent.token_code_ref(y)
    if norm:
        assert ((codes == latent.token_code_ref(y * (1 - D))) | (codes == latent.token_code_ref(y * (1 + D)))).all()
        s = latent.e8m0_value(codes)[:, None]
        bound = np.maximum(np.abs(y) * 2.0 ** -4, s * 2.0 ** -10) + D * np.abs(y)
        assert (np.abs(e4m3.decode(rows[:, :512].copy()) * s - y) <= bound).all()
    else:
        np.testing.assert_array_equal(codes, want)
        np.testing.assert_array_equal(rows[:, :512], e4m3.encode(y / latent.e8m0_value(want)[:, None]))
    np.testing.assert_array_equal(rows[:, 512:], kv[:, 512:].contiguous().view(torch.uint8).numpy())
    # every other row, and the gaps, are as they were
    left = torch.ones(pages, page + gap, dtype=torch.bool)
    left[perm // page, perm % page] = False
    assert (full.cpu()[left] == 0xFF).all() and (fsc.cpu()[left] == 0xFF).all()


def test_write_skips_padding_and_out_of_range_slots(gpu):
    kv = _kv(6, 3).to(gpu)
    full, fsc, cache, sc = _empty_cache(gpu, 2, 4)
    slots = torch.tensor([-1, 5, 8, 1 << 40, 0, -(1 << 62)], device=gpu)
    announce("latent write padding slots")
    bfp8.latent_cache_write(kv, slots, cache, sc)
    one, osc = torch.full_like(full, 0xFF), torch.full_like(fsc, 0xFF)
    bfp8.latent_cache_write(kv[[1, 4]].contiguous(), slots[[1, 4]].contiguous(), one, osc)
    assert torch.equal(full, one) and torch.equal(fsc, osc)
    written = (fsc != 0xFF).flatten().nonzero().flatten().tolist()
    assert written == [0, 5]


def test_write_special_values_and_strided_rows(gpu):
    big = torch.zeros(6, 640, dtype=torch.bfloat16)
    big[0, 7] = float("nan")
    big[1, 9] = float("inf")
    big[2, :512] = 3.0e38       # past 2^40 * 448: saturates
    big[3, :512] = 1.0e-30      # far below the scale floor
    big[4, 512] = float("nan")  # a NaN in the rotary key is stored as it is
    big[5, :576] = 1.0
    announce("latent write special values")
    _, _, cache, sc = _empty_cache(gpu, 1, 6)
    bfp8.latent_cache_write(big.to(gpu)[:, :576], torch.arange(6, device=gpu), cache, sc)
    rows, codes = cache.cpu()[0].numpy(), sc.cpu()[0].tolist()
    assert codes[:2] == [255, 255] and (rows[:2, :512] == 0).all()
    assert codes[2] == 167 and (rows[2, :512] == 0x7E).all()
    assert codes[3] == 85 and (rows[3, :512] == 0).all()
    assert torch.equal(torch.from_numpy(rows[4, 512:].copy()), big[4, 512:576].contiguous().view(torch.uint8))
    assert codes[5] == 127 - 8 and (e4m3.decode(rows[5, :512].copy()) == 256).all()


def _filled(gpu, lens, page, seed, width_extra=0):
    """(cache, scales, table, tokens [sum(lens), 576] float64) with sequences on shuffled pages."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    rng = np.random.default_rng(seed)
    order = rng.permutation(pages)
    table = np.full((len(lens), max(need + [1]) + width_extra), -7, dtype=np.int32)
    slots, at = [], 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        i = np.arange(n)
        slots.append(table[b, i // page].astype(np.int64) * page + i % page)
    _, _, cache, sc = _empty_cache(gpu, pages, page, 1)
    slots = torch.from_numpy(np.concatenate(slots))
    kv = _kv(len(slots), seed)
    bfp8.latent_cache_write(kv.to(gpu), slots.to(gpu), cache, sc)
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    rows = cache.cpu()[slots // page, slots % page].numpy()
    codes = sc.cpu()[slots // page, slots % page].numpy()
    return cache, sc, torch.from_numpy(table).to(gpu), cu.to(gpu), rows, codes


@pytest.mark.parametrize("lens,page", [([1], 1), ([5, 0, 33], 16), ([0, 0, 7], 4), ([100, 37, 1, 74], 37),
                                       ([64, 65, 63, 300], 64)])
def test_read_and_gather(gpu, lens, page):
    announce("latent read", lens, page)
    cache, sc, table, cu, rows, codes = _filled(gpu, lens, page, seed=len(lens))
    t = sum(lens)
    out = bfp8.latent_cache_read(cache, sc, table, cu, t)
    q, e, rope = bfp8.latent_cache_gather(cache, sc.view(torch.float8_e8m0fnu), table, cu, t)
    torch.cuda.synchronize()
    exact = e4m3.decode(rows[:, :512].copy()) * latent.e8m0_value(codes)[:, None]
    np.testing.assert_array_equal(out.cpu()[:, :512].double().numpy(), exact)  # 4 significant bits: exact in bf16
    np.testing.assert_array_equal(out.cpu()[:, 512:].contiguous().view(torch.uint8).numpy(), rows[:, 512:])
    np.testing.assert_array_equal(q.cpu().numpy(), rows[:, :512])
    np.testing.assert_array_equal(e.cpu().numpy(), np.repeat(codes[:, None], 4, axis=1))
    np.testing.assert_array_equal(rope.cpu().view(torch.uint8).numpy(), rows[:, 512:])


def test_read_of_missing_pages_is_nan(gpu):
    """A table entry that is no page of the cache, and positions past the table, read as NaN."""
    cache, sc, table, cu, rows, codes = _filled(gpu, [8, 8], 4, seed=11)
    table = table.clone()
    table[0, 1] = -1
    table[1, 0] = cache.shape[0]
    cu = torch.tensor([0, 8, 18], dtype=torch.int32, device=gpu)  # two tokens past the table's 2 pages
    announce("latent read missing pages")
    out = bfp8.latent_cache_read(cache, sc, table, cu, 20, out=torch.full((20, 576), 5.0, dtype=torch.bfloat16, device=gpu))
    q, e, rope = bfp8.latent_cache_gather(cache, sc, table, cu, 18)
    bad = torch.tensor([4, 5, 6, 7, 8, 9, 10, 11, 16, 17])
    good = torch.tensor([0, 1, 2, 3, 12, 13, 14, 15])
    assert out.cpu()[bad].isnan().all() and out.cpu()[good].isfinite().all()
    assert (out.cpu()[18:] == 5.0).all()  # past cu[B]: not written
    assert (q.cpu()[bad] == 0).all() and (e.cpu()[bad] == 255).all() and rope.cpu()[bad].isnan().all()
    assert torch.equal(q.cpu()[good], torch.from_numpy(rows[[0, 1, 2, 3, 12, 13, 14, 15], :512]))


def test_gather_feeds_the_ue8m0_gemm(gpu):
    """gather -> gemm_ue8m0 equals, bit for bit, the GEMM of the same rows laid out by the host."""
    n, lens = 256, [70, 130]
    cache, sc, table, cu, rows, codes = _filled(gpu, lens, 64, seed=21)
    g = torch.Generator().manual_seed(22)
    w = torch.randn(n, 512, generator=g).to(torch.float8_e4m3fn).view(torch.uint8).to(gpu)
    w_e = bfp8.ue8m0_scales(torch.randint(120, 130, (n // 128, 4), dtype=torch.uint8, generator=g).to(gpu))
    announce("latent gather into gemm")
    q, e, _ = bfp8.latent_cache_gather(cache, sc, table, cu, 200)
    host_e = torch.from_numpy(np.repeat(codes[None], 4, axis=0).copy()).to(gpu).t()
    want = bfp8.gemm_ue8m0(torch.from_numpy(rows[:, :512].copy()).to(gpu), host_e, w, w_e)
    assert torch.equal(bfp8.gemm_ue8m0(q, e, w, w_e).view(torch.int16), want.view(torch.int16))
    assert want.isfinite().all() and want.abs().max() > 0


def test_empty_and_refusals(gpu):
    _, _, cache, sc = _empty_cache(gpu, 2, 4)
    kv = torch.zeros(3, 576, dtype=torch.bfloat16, device=gpu)
    slots = torch.arange(3, device=gpu)
    table = torch.zeros(1, 2, dtype=torch.int32, device=gpu)
    cu = torch.tensor([0, 3], dtype=torch.int32, device=gpu)
    bfp8.latent_cache_write(kv[:0], slots[:0], cache, sc)
    assert bfp8.latent_cache_read(cache, sc, table, cu, 0).shape == (0, 576)
    assert bfp8.latent_cache_gather(cache, sc, table, cu, 0)[1].shape == (0, 4)
    with pytest.raises(TypeError):
        bfp8.latent_cache_write(kv.float(), slots, cache, sc)
    with pytest.raises(TypeError):
        bfp8.latent_cache_write(kv, slots.int(), cache, sc)
    with pytest.raises(ValueError):
        bfp8.latent_cache_write(kv[:, :512], slots, cache, sc)
    with pytest.raises(ValueError):
        bfp8.latent_cache_write(kv, slots[:2], cache, sc)
    with pytest.raises(ValueError):
        bfp8.latent_cache_write(kv, slots, cache[:, :, :512], sc)
    with pytest.raises(ValueError):
        bfp8.latent_cache_write(kv, slots, cache, sc[:1])
    with pytest.raises(ValueError):
        bfp8.latent_cache_write(kv, slots, cache.cpu(), sc)
    with pytest.raises(NotImplementedError):
        bfp8.latent_cache_write(kv, slots, cache, sc.int())
    with pytest.raises(ValueError):
        bfp8.latent_cache_read(cache, sc, table, cu[:1], 3)
    with pytest.raises(TypeError):
        bfp8.latent_cache_read(cache, sc, table.long(), cu, 3)
    with pytest.raises(ValueError):
        bfp8.latent_cache_read(cache, sc, table, cu, 3, out=torch.empty(2, 576, dtype=torch.bfloat16, device=gpu))


@pytest.mark.parametrize("size", [2.0 ** 62, 2.0 ** 110, 2.0 ** 125])
def test_write_norms_tokens_whose_squares_pass_float32(gpu, size):
    t = 9
    kv = torch.randn(t, 576, generator=torch.Generator().manual_seed(31)).clamp(-3.9, 3.9)
    kv[:, :512] *= size
    kv = kv.bfloat16()
    kv[3, 200] = torch.finfo(torch.bfloat16).max
    w = (1 + 0.3 * torch.randn(512, generator=torch.Generator().manual_seed(32))).bfloat16()
    announce("latent write large tokens", size)
    _, _, cache, sc = _empty_cache(gpu, 1, t)
    bfp8.latent_cache_write(kv.to(gpu), torch.arange(t, device=gpu), cache, sc, norm_weight=w.to(gpu), eps=1e-6)
    y = latent.rmsnorm_ref(kv[:, :512].double().numpy(), w.double().numpy(), 1e-6)
    rows, codes = cache.cpu()[0].numpy(), sc.cpu()[0].numpy().astype(np.int64)
    assert ((codes == latent.token_code_ref(y * (1 - D))) | (codes == latent.token_code_ref(y * (1 + D)))).all()
    s = latent.e8m0_value(codes)[:, None]
    bound = np.maximum(np.abs(y) * 2.0 ** -4, s * 2.0 ** -10) + D * np.abs(y)
    assert (np.abs(e4m3.decode(rows[:, :512].copy()) * s - y) <= bound).all()


@pytest.mark.parametrize("size", [2.0 ** -70, 2.0 ** -100, 2.0 ** -120])
def test_write_norms_tokens_whose_squares_vanish_in_float32(gpu, size):
    t = 9
    kv = torch.randn(t, 576, generator=torch.Generator().manual_seed(33))
    kv[:, :512] *= size
    kv = kv.bfloat16()
    w = (1 + 0.3 * torch.randn(512, generator=torch.Generator().manual_seed(34))).bfloat16()
    announce("latent write tiny tokens", size)
    _, _, cache, sc = _empty_cache(gpu, 1, t)
    bfp8.latent_cache_write(kv.to(gpu), torch.arange(t, device=gpu), cache, sc, norm_weight=w.to(gpu), eps=0.0)
    y = latent.rmsnorm_ref(kv[:, :512].double().numpy(), w.double().numpy(), 0.0)
    rows, codes = cache.cpu()[0].numpy(), sc.cpu()[0].numpy().astype(np.int64)
    assert ((codes == latent.token_code_ref(y * (1 - D))) | (codes == latent.token_code_ref(y * (1 + D)))).all()
    s = latent.e8m0_value(codes)[:, None]
    bound = np.maximum(np.abs(y) * 2.0 ** -4, s * 2.0 ** -10) + D * np.abs(y)
    assert (np.abs(e4m3.decode(rows[:, :512].copy()) * s - y) <= bound).all()
