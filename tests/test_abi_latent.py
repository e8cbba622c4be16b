"""CPU tests of the C entry points of the norm, the latent cache and latent attention: the host-side
rejections, each before any device call, and the documented no-ops (fake pointers are never
dereferenced, nothing is launched)."""

import random

import pytest

from block_scaled_fp8_bfp8_amd import _native

OK = _native.BFP8_OK
E_INV = _native.BFP8_ERR_INVALID_ARGUMENT
E_UNS = _native.BFP8_ERR_UNSUPPORTED
E_MIS = _native.BFP8_ERR_MISALIGNED
E_WS = _native.BFP8_ERR_WORKSPACE
BF16, F16, F32 = _native.BFP8_IN_BF16, _native.BFP8_IN_F16, _native.BFP8_IN_F32

P1, P2, P3, P4, P5, P6, P7 = (0x10000000 * i for i in range(1, 8))  # fake, 256-byte aligned
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return _native.lib()


def _norm(entry, x=P1, dt=BF16, M=4, H=256, ldx=256, res=P2, ld_res=256, w=P3, eps=1e-6, h=P4, ld_h=256, q=P5, ldq=256,
          as_=P6, ld_as=4):
    return entry(x, dt, M, H, ldx, res, ld_res, w, eps, h, ld_h, q, ldq, as_, ld_as, None)


@pytest.mark.parametrize("e8", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), E_INV), (dict(H=0), E_INV), (dict(H=200, ldx=256), E_UNS), (dict(H=65552, ldx=65552, ldq=65552), E_UNS),
    (dict(dt=7), E_UNS), (dict(M=(1 << 30) + 1, ld_as=1 << 31), E_UNS), (dict(x=None), E_INV), (dict(w=None), E_INV),
    (dict(q=None), E_INV), (dict(as_=None), E_INV), (dict(h=None), E_INV), (dict(ldx=128), E_INV), (dict(ld_res=240), E_INV),
    (dict(ld_h=240), E_INV), (dict(ldq=128), E_INV), (dict(ld_as=3), E_INV), (dict(ldx=260), E_MIS), (dict(ld_res=260), E_MIS),
    (dict(ld_h=260), E_MIS), (dict(ldq=264), E_MIS), (dict(x=P1 + 8), E_MIS), (dict(res=P2 + 8), E_MIS),
    (dict(w=P3 + 8), E_MIS), (dict(h=P4 + 8), E_MIS), (dict(q=P5 + 8), E_MIS), (dict(eps=-1.0), E_INV), (dict(eps=NAN), E_INV),
    (dict(eps=INF), E_INV),
])
def test_norm_rejections(lib, e8, kw, status):
    entry = lib.bfp8_rmsnorm_quant_ue8m0 if e8 else lib.bfp8_rmsnorm_quant
    assert _norm(entry, **kw) == status, lib.bfp8_last_error_message()


def test_norm_m_zero_is_a_no_op(lib):
    for entry in (lib.bfp8_rmsnorm_quant, lib.bfp8_rmsnorm_quant_ue8m0):
        assert _norm(entry, M=0, x=None, res=None, w=None, h=None, q=None, as_=None) == OK


CACHE = dict(rows=P1, ps=64 * 640, sc=P2, ss=64, pages=10, page=64)
BAD_CACHE = [
    (dict(rows=None), E_INV), (dict(sc=None), E_INV), (dict(pages=0), E_INV), (dict(page=0), E_INV), (dict(pages=-1), E_INV),
    (dict(pages=1 << 26), E_UNS), (dict(ps=63 * 640), E_INV), (dict(ps=64 * 640 + 64), E_MIS), (dict(ss=63), E_INV),
    (dict(rows=P1 + 8), E_MIS), (dict(ps=1 << 36), E_UNS), (dict(ps=1 << 62), E_UNS),
]


def _write(lib, kv=P3, T=4, ld_kv=576, w=P4, eps=1e-6, slots=P5, **kw):
    c = {**CACHE, **kw}
    return lib.bfp8_latent_cache_write(kv, T, ld_kv, w, eps, slots, c["rows"], c["ps"], c["sc"], c["ss"], c["pages"],
                                       c["page"], None)


@pytest.mark.parametrize("kw,status", BAD_CACHE + [
    (dict(T=-1), E_INV), (dict(T=(1 << 30) + 1), E_UNS), (dict(kv=None), E_INV), (dict(slots=None), E_INV),
    (dict(ld_kv=575), E_INV), (dict(ld_kv=580), E_MIS), (dict(kv=P3 + 8), E_MIS), (dict(w=P4 + 8), E_MIS),
    (dict(slots=P5 + 4), E_MIS), (dict(eps=-1.0), E_INV), (dict(eps=NAN), E_INV),
])
def test_write_rejections(lib, kw, status):
    assert _write(lib, **kw) == status, lib.bfp8_last_error_message()


def test_write_t_zero_is_a_no_op(lib):
    assert _write(lib, T=0, kv=None, slots=None, rows=None) == OK


TABLE = dict(table=P3, ts=8, tw=8, B=3)
BAD_TABLE = [
    (dict(table=None), E_INV), (dict(ts=7), E_INV), (dict(tw=-1), E_INV), (dict(B=-1), E_INV), (dict(table=P3 + 2), E_MIS),
    (dict(tw=1 << 31, ts=1 << 31), E_UNS), (dict(B=1 << 31), E_UNS),
]


def _read(lib, cu=P4, T=100, out=P5, ld_out=576, **kw):
    c = {**CACHE, **TABLE, **kw}
    return lib.bfp8_latent_cache_read(c["rows"], c["ps"], c["sc"], c["ss"], c["pages"], c["page"], c["table"], c["ts"],
                                      c["tw"], c["B"], cu, T, out, ld_out, None)


@pytest.mark.parametrize("kw,status", BAD_CACHE + BAD_TABLE + [
    (dict(T=-1), E_INV), (dict(T=(1 << 30) + 1), E_UNS), (dict(B=0), E_INV), (dict(cu=None), E_INV), (dict(out=None), E_INV),
    (dict(cu=P4 + 2), E_MIS), (dict(ld_out=575), E_INV), (dict(ld_out=580), E_MIS), (dict(out=P5 + 8), E_MIS),
])
def test_read_rejections(lib, kw, status):
    assert _read(lib, **kw) == status, lib.bfp8_last_error_message()


def _gather(lib, cu=P4, T=100, q=P5, ldq=512, as_=P6, ld_as=100, rope=P7, ld_rope=64, **kw):
    c = {**CACHE, **TABLE, **kw}
    return lib.bfp8_latent_cache_gather(c["rows"], c["ps"], c["sc"], c["ss"], c["pages"], c["page"], c["table"], c["ts"],
                                        c["tw"], c["B"], cu, T, q, ldq, as_, ld_as, rope, ld_rope, None)


@pytest.mark.parametrize("kw,status", BAD_CACHE + BAD_TABLE + [
    (dict(T=-1), E_INV), (dict(T=(1 << 30) + 1), E_UNS), (dict(B=0), E_INV), (dict(cu=None), E_INV), (dict(q=None), E_INV),
    (dict(as_=None), E_INV), (dict(rope=None), E_INV), (dict(ldq=511), E_INV), (dict(ld_as=99), E_INV),
    (dict(ld_rope=63), E_INV), (dict(cu=P4 + 2), E_MIS), (dict(ldq=520), E_MIS), (dict(q=P5 + 8), E_MIS),
    (dict(rope=P7 + 8), E_MIS), (dict(ld_rope=68), E_MIS),
])
def test_gather_rejections(lib, kw, status):
    assert _gather(lib, **kw) == status, lib.bfp8_last_error_message()


def test_read_and_gather_t_zero_are_no_ops(lib):
    assert _read(lib, T=0, cu=None, out=None, rows=None, table=None) == OK
    assert _gather(lib, T=0, cu=None, q=None, as_=None, rope=None, rows=None, table=None) == OK


def _attend(lib, q=P3, T=3, H=16, qt=16 * 576, qh=576, lens=P4, B=3, cu=None, scale=0.1, out=P5, ot=16 * 512, oh=512, ws=P6,
            wsb=None, table=P7, ts=8, tw=8, **kw):
    c = {**CACHE, **kw}
    if wsb is None:
        wsb = lib.bfp8_latent_attention_workspace_bytes(max(T, 1), max(B, 1), max(H, 1), max(tw, 0) * max(c["page"], 0))
    return lib.bfp8_latent_attention(q, T, H, qt, qh, c["rows"], c["ps"], c["sc"], c["ss"], c["pages"], c["page"], table, ts,
                                     tw, lens, B, cu, scale, out, ot, oh, ws, wsb, None)


@pytest.mark.parametrize("kw,status", BAD_CACHE + [
    (dict(T=-1), E_INV), (dict(H=0), E_INV), (dict(T=1 << 20, B=1 << 20, H=1 << 11), E_UNS), (dict(q=None), E_INV),
    (dict(out=None), E_INV), (dict(lens=None), E_INV), (dict(T=4), E_INV), (dict(B=0), E_INV), (dict(qh=575), E_INV),
    (dict(qt=575), E_INV), (dict(oh=511), E_INV), (dict(ot=511), E_INV), (dict(qh=580), E_MIS), (dict(ot=16 * 512 + 4), E_MIS),
    (dict(q=P3 + 8), E_MIS), (dict(out=P5 + 8), E_MIS), (dict(lens=P4 + 2), E_MIS), (dict(cu=P4 + 2), E_MIS),
    (dict(scale=NAN), E_INV), (dict(scale=INF), E_INV), (dict(ws=None), E_WS), (dict(wsb=1024), E_WS), (dict(ws=P6 + 128), E_MIS),
    (dict(table=None), E_INV), (dict(ts=7), E_INV), (dict(tw=-1), E_INV), (dict(B=1 << 31, T=1 << 31), E_UNS),
    (dict(tw=1 << 26, ts=1 << 26), E_UNS), (dict(table=P7 + 2), E_MIS), (dict(qt=-8), E_INV),
])
def test_attention_rejections(lib, kw, status):
    assert _attend(lib, **kw) == status, lib.bfp8_last_error_message()


def test_attention_t_zero_is_a_no_op_and_workspace_sizes(lib):
    assert _attend(lib, T=0, q=None, out=None, lens=None, rows=None, ws=None) == OK
    size = lib.bfp8_latent_attention_workspace_bytes
    assert size(1, 1, 16, 64) == 0  # one tile: nothing is cut
    assert size(0, 1, 16, 640) == size(1, 1, 0, 640) == size(1, 1, 1, -1) == size(1 << 20, 1, 1 << 11, 64) == 0
    last = 0
    for t in (1, 8, 64, 512, 4096):  # grows with the work up to a bound
        n = size(t, t, 128, 1 << 20)
        assert n % 256 == 0 and last <= n <= 136 << 20
        last = n


def _expanded(lib, q=P1, dt=BF16, Tq=10, H=4, qt=768, qh=192, kv=P2, Tk=12, kt=1024, kh=256, rope=P3, ldr=64, cq=P4, ck=P5,
              B=2, scale=0.1, out=P6, ot=512, oh=128):
    return lib.bfp8_latent_attention_expanded(q, dt, Tq, H, qt, qh, kv, Tk, kt, kh, rope, ldr, cq, ck, B, scale, out, ot, oh,
                                              None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=F32), E_UNS), (dict(dt=9), E_UNS), (dict(Tq=-1), E_INV), (dict(Tk=-1), E_INV), (dict(H=0), E_INV),
    (dict(B=0), E_INV), (dict(Tq=1 << 31), E_UNS), (dict(Tk=1 << 31), E_UNS), (dict(Tq=1 << 30, H=1 << 10), E_UNS),
    (dict(q=None), E_INV), (dict(kv=None), E_INV), (dict(rope=None), E_INV), (dict(out=None), E_INV), (dict(cq=None), E_INV),
    (dict(ck=None), E_INV), (dict(qt=184), E_INV), (dict(qh=184), E_INV), (dict(kt=248), E_INV), (dict(kh=248), E_INV),
    (dict(ldr=56), E_INV), (dict(ot=120), E_INV), (dict(oh=120), E_INV), (dict(Tq=1, qt=-8), E_INV), (dict(qt=772), E_MIS),
    (dict(kh=260), E_MIS), (dict(ldr=68), E_MIS), (dict(oh=132), E_MIS), (dict(q=P1 + 8), E_MIS), (dict(kv=P2 + 8), E_MIS),
    (dict(rope=P3 + 8), E_MIS), (dict(out=P6 + 8), E_MIS), (dict(cq=P4 + 2), E_MIS), (dict(ck=P5 + 1), E_MIS),
    (dict(scale=NAN), E_INV), (dict(scale=-INF), E_INV),
])
def test_expanded_rejections(lib, kw, status):
    assert _expanded(lib, **kw) == status, lib.bfp8_last_error_message()


def test_expanded_t_zero_is_a_no_op(lib):
    assert _expanded(lib, Tq=0, q=None, kv=None, rope=None, out=None, cq=None, ck=None) == OK


def test_attention_workspace_stays_below_its_stated_bound(lib):
    """256 parts of 64 rows: their float32 states, statistics and descriptors, whatever the sizes."""
    size = lib.bfp8_latent_attention_workspace_bytes
    bound = 256 * 64 * (512 + 2) * 4 + 2304
    rng = random.Random(5)
    most = 0
    for _ in range(20000):
        t, h, keys = (int(2 ** rng.uniform(0, top)) for top in (22, 8, 31))
        b = rng.choice([t, max(1, t // rng.randint(1, 64)), 1])
        n = size(t, b, h, min(keys, 2 ** 31 - 1))
        assert n <= bound, (t, b, h, keys)
        most = max(most, n)
    assert most == bound < 33 << 20
