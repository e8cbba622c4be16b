"""CPU tests of the bounded cache's entry points: host-side rejections, each before any device call, and the documented
no-ops (fake pointers are never dereferenced, nothing is launched)."""

import pytest

from block_scaled_fp8_bfp8_amd import _native

OK = _native.BFP8_OK
E_INV = _native.BFP8_ERR_INVALID_ARGUMENT
E_UNS = _native.BFP8_ERR_UNSUPPORTED
E_MIS = _native.BFP8_ERR_MISALIGNED
E_WS = _native.BFP8_ERR_WORKSPACE

P = [0x10000000 * i for i in range(1, 14)]  # fake, 256-byte aligned


@pytest.fixture(scope="module")
def lib():
    return _native.lib()


SHARED = [
    (dict(rows=None), E_INV), (dict(sc=None), E_INV), (dict(pages=0), E_INV), (dict(ps=64 * 640 + 64), E_MIS), (dict(B=-1), E_INV),
    (dict(table=None), E_INV), (dict(tw=-1), E_INV), (dict(ts=3), E_INV), (dict(lens=None), E_INV), (dict(lens=P[4] + 2), E_MIS),
    (dict(width=255), E_INV), (dict(width=(1 << 31) - 1, ms=1 << 31, mos=1 << 31), E_UNS), (dict(mo=None), E_INV), (dict(mos=255), E_INV),
    (dict(ms=255), E_INV), (dict(m=P[5] + 2), E_MIS), (dict(mo=P[6] + 2), E_MIS), (dict(tw=1 << 28, ts=1 << 28), E_UNS),
    (dict(B=(1 << 24) + 1), E_UNS), (dict(B=(1 << 19) + 1), E_UNS),
]


def _mass(lib, q=P[0], T=4, H=16, qt=16 * 576, qh=576, rows=P[1], ps=64 * 640, sc=P[2], ss=64, pages=10, page=64, table=P[3], ts=4,
          tw=4, lens=P[4], B=4, cu=None, scale=0.1, out=P[7], ot=16 * 512, oh=512, m=P[5], ms=256, mo=P[6], mos=256, width=256, ws=P[8],
          wsb=None):
    if cu is None and B != 4:
        cu = P[9]
    if wsb is None:
        wsb = lib.bfp8_latent_attention_mass_workspace_bytes(max(T, 1), max(B, 1), max(H, 1), max(tw, 0) * max(page, 0))
    return lib.bfp8_latent_attention_mass(q, T, H, qt, qh, rows, ps, sc, ss, pages, page, table, ts, tw, lens, B, cu, scale, out, ot, oh,
                                          m, ms, mo, mos, width, ws, wsb, None)


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(T=-1), E_INV), (dict(H=0), E_INV), (dict(T=1 << 20, H=1 << 20), E_UNS), (dict(q=None), E_INV), (dict(out=None), E_INV),
    (dict(T=3), E_INV), (dict(scale=float("nan")), E_INV), (dict(qt=568), E_INV), (dict(qh=580), E_MIS), (dict(out=P[7] + 8), E_MIS),
    (dict(ws=None), E_WS), (dict(wsb=1000), E_WS), (dict(ws=P[8] + 64), E_MIS), (dict(cu=P[9] + 2), E_MIS),
])
def test_mass_rejections(lib, kw, status):
    assert _mass(lib, **kw) == status, lib.bfp8_last_error_message()


def test_mass_workspace(lib):
    size, attention = lib.bfp8_latent_attention_mass_workspace_bytes, lib.bfp8_latent_attention_workspace_bytes
    assert size(0, 4, 16, 256) == 0 and size(4, 4, 0, 256) == 0 and size(4, 4, 16, -1) == 0
    for t, b, h, keys in ((4, 4, 16, 256), (1, 1, 128, 4096), (300, 6, 128, 3501), (5, 5, 7, 0), (64, 64, 16, 1 << 20), (2048, 3, 128, 8192)):
        rest = size(t, b, h, keys) - attention(t, b, h, keys)
        pitch = -(-keys // 32) * 32
        scores = 4 * t * h * pitch
        kept = t * h <= 1024 * b and scores <= (512 if t * h <= 32 * b else 192) << 20
        need = scores if kept else 4 * (t * h // 128 + b + 1) * pitch
        assert need <= rest <= need + 1024 * (t * h // 128 + b + 512 + 16) + 8 * b + 4 * 256


def _evict(lib, rows=P[1], ps=64 * 640, sc=P[2], ss=64, pages=10, page=64, table=P[3], ts=4, tw=4, lens=P[4], B=4, m=P[5], ms=256,
           width=256, budget=100, recent=10, to=None, tos=4, tow=4, kept=P[8], lo=P[9], mo=P[6], mos=256):
    return lib.bfp8_latent_cache_evict(rows, ps, sc, ss, pages, page, table, ts, tw, lens, B, m, ms, width, budget, recent, to, tos, tow,
                                       kept, lo, mo, mos, None)


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(budget=0), E_INV), (dict(recent=-1), E_INV), (dict(recent=101), E_INV), (dict(budget=(1 << 30) + 1), E_UNS),
    (dict(m=None), E_INV), (dict(kept=None), E_INV), (dict(lo=None), E_INV), (dict(kept=P[8] + 1), E_MIS), (dict(lo=P[9] + 1), E_MIS),
    (dict(to=P[10], tos=3), E_INV), (dict(to=P[10] + 1), E_MIS), (dict(to=P[10], tow=-1), E_INV), (dict(mo=P[5], mos=300), E_INV),
])
def test_evict_rejections(lib, kw, status):
    assert _evict(lib, **kw) == status, lib.bfp8_last_error_message()


def test_no_sequences_is_a_no_op(lib):
    assert _evict(lib, B=0, rows=None) == OK
    assert _mass(lib, T=0, B=0, rows=None) == OK
