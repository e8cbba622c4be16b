"""Measured cases of the latent-attention operators: residual add + RMS norm + FP8 quantization, the
paged FP8 latent cache (write, read, gather) and attention over it in the absorbed and the expanded
form. `run` computes each operator either in plain torch steps or, with `own`, through the package."""

from __future__ import annotations

import torch

own = False

LATENT, ROPE = 512, 64  # the cached latent vector and the shared rotary key of a token
NOPE, VDIM = 128, 128   # expanded keys (without the rotary part) and values of a head
ROW = LATENT + 2 * ROPE  # bytes of a cache row: e4m3 codes, then the rotary key in bf16
EPS = 1e-6
SCALE = (NOPE + ROPE) ** -0.5

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One decoded token between two layers: pure latency.
        {"name": "norm 1x7168", "op": "norm", "m": 1, "h": 7168, "dtype": "bf16", "res": True, "e8": False},
        # A prefill batch's residual stream; power-of-two scales for the hardware-scaled GEMM.
        {"name": "norm 8192x7168 e8", "op": "norm", "m": 8192, "h": 7168, "dtype": "bf16", "res": True, "e8": True},
        # One decode step of 67 sequences: each token's latent goes to its own page.
        {"name": "write 67", "op": "write", "t": 67, "pages": 300, "page": 64, "norm": True},
        # A prefill batch of prompts is cached.
        {"name": "write 16384", "op": "write", "t": 16384, "pages": 1100, "page": 16, "norm": True},
        # A short cached prefix is read back for a host-side or torch consumer.
        {"name": "read 5x777", "op": "read", "b": 5, "lo": 33, "hi": 777, "page": 16, "raw": False},
        # Long cached prefixes become the expanding GEMM's operands (chunked prefill).
        {"name": "gather 16x8192", "op": "read", "b": 16, "lo": 2000, "hi": 8192, "page": 64, "raw": True},
        # One sequence, one new token, all heads: the latency case of decoding.
        {"name": "decode 1x128h", "op": "attend", "b": 1, "heads": 128, "q": 1, "lo": 1111, "hi": 1111, "page": 64},
        # A tensor-parallel rank's 16 heads over ragged long contexts: reading the cache is the work.
        {"name": "decode 64x16h", "op": "attend", "b": 64, "heads": 16, "q": 1, "lo": 500, "hi": 8000, "page": 64},
        # A data-parallel rank's decode batch with all heads: the matrix cores are the work.
        {"name": "decode 128x128h", "op": "attend", "b": 128, "heads": 128, "q": 1, "lo": 2500, "hi": 4096, "page": 64},
        # Chunks of new tokens behind cached prefixes, in the absorbed form.
        {"name": "chunk 6x40", "op": "attend", "b": 6, "heads": 128, "q": 40, "lo": 700, "hi": 3500, "page": 16},
        # Short prompts of a small model shard, expanded form.
        {"name": "expanded 5x8h", "op": "expand", "b": 5, "heads": 8, "qlo": 17, "qhi": 300, "ctx": 0, "dtype": "bf16"},
        # Ragged long prompts, expanded form.
        {"name": "expanded 4x32h", "op": "expand", "b": 4, "heads": 32, "qlo": 2100, "qhi": 4090, "ctx": 0,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "write", "read", "attend", "attend", "expand"])
    if op == "norm":
        h = 16 * _log(rng, 8, 1024)
        return {"op": op, "m": _log(rng, 1, min(8192, (1 << 25) // h)), "h": h,
                "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]), "res": rng.random() < 0.7,
                "e8": rng.random() < 0.4}
    if op == "write":
        t, page = _log(rng, 1, 16384), rng.choice([1, 16, 37, 64])
        return {"op": op, "t": t, "pages": t // page + rng.randint(1, 50), "page": page, "norm": rng.random() < 0.6}
    if op == "read":
        hi = _log(rng, 1, 8192)
        return {"op": op, "b": _log(rng, 1, 16), "lo": rng.randint(1, hi), "hi": hi, "page": rng.choice([1, 16, 37, 64]),
                "raw": rng.random() < 0.5}
    if op == "attend":
        heads = rng.choice([1, 5, 8, 16, 16, 32, 40, 64, 128, 128])
        q = rng.choice([1, 1, 1, 2, 4, rng.randint(5, 96)])
        hi = _log(rng, 1, 8192)
        b = _log(rng, 1, 128)
        while b > 1 and b * heads * q * hi > 128 * 128 * 2048:
            b //= 2
        return {"op": op, "b": b, "heads": heads, "q": q, "lo": rng.randint(max(1, hi // 4), hi), "hi": hi,
                "page": rng.choice([1, 16, 37, 64])}
    heads = rng.choice([1, 4, 8, 20, 32, 128])
    qhi = _log(rng, 1, 4000)
    ctx = rng.choice([0, 0, _log(rng, 1, 1500)])
    b = _log(rng, 1, 8)
    while b > 1 and b * heads * qhi * (qhi + ctx) > 2 * 32 * 4000 * 4000:
        b //= 2
    if heads * qhi * (qhi + ctx) > 2 * 32 * 4000 * 4000:
        heads = 8
    return {"op": op, "b": b, "heads": heads, "qlo": rng.randint(max(1, qhi // 2), qhi), "qhi": qhi, "ctx": ctx,
            "dtype": rng.choice(["bf16", "bf16", "f16"])}


def _lens(n, lo, hi):
    """n lengths in [lo, hi], spread evenly and out of order; the same for every seed, so that a
    case's work is its own. The last is hi."""
    return [lo + int((hi - lo) * ((0.6180339887 * (i + 1)) % 1.0)) for i in range(n - 1)] + [hi]


def _read_lens(c):
    return _lens(c["b"], c["lo"], c["hi"])


def _attend_lens(c):
    """(lengths of the whole sequences, lengths of their chunks of new tokens)"""
    lens = _read_lens(c)
    return lens, [min(c["q"], n) for n in lens]


def _expand_lens(c):
    """(new tokens, keys) of each sequence: the keys are a context of ctx tokens, then the new ones."""
    q = _lens(c["b"], c["qlo"], c["qhi"])
    return q, [n + c["ctx"] for n in q]


# ---------------------------------------------------------------- inputs

def _ints(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _starts(lens):
    s = [0]
    for n in lens:
        s.append(s[-1] + n)
    return s


def _quantize_rows(y):
    """Codes and UE8M0 scale codes of latent rows y [T, LATENT] float32: one power of two a row."""
    amax = y.abs().amax(dim=1)
    s = torch.clamp(amax, min=1e-10) / torch.full_like(amax, 448.0)
    e = (((s.view(torch.int32) + 0x7FFFFF) >> 23) & 0xFF).clamp(127 - 42, 127 + 40)
    inv = torch.ldexp(torch.ones_like(s), 127 - e)
    codes = (y * inv[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), e.to(torch.uint8)


def _filled_cache(lens, page, g, dev):
    """A paged cache that holds sequences of these lengths on shuffled pages, and its page table."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    first = _starts(need)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=dev)
    for b, n in enumerate(need):
        table[b, :n] = order[first[b]:first[b] + n]
    cache = torch.empty(pages * page, ROW, dtype=torch.uint8, device=dev)
    scales = torch.empty(pages * page, dtype=torch.uint8, device=dev)
    for i in range(0, pages * page, 65536):
        n = min(65536, pages * page - i)
        y = torch.randn(n, LATENT, generator=g, device=dev)
        y *= torch.exp(0.5 * torch.randn(n, 1, generator=g, device=dev))  # tokens differ in size
        cache[i:i + n, :LATENT], scales[i:i + n] = _quantize_rows(y)
        r = torch.randn(n, ROPE, generator=g, device=dev).to(torch.bfloat16)
        cache[i:i + n, LATENT:] = r.view(torch.uint8)
    return cache.view(pages, page, ROW), scales.view(pages, page), table


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    if op == "norm":
        m, h, dt = case["m"], case["h"], DTYPES[case["dtype"]]
        st["x"] = torch.randn(m, h, generator=g, device=dev).to(dt)
        st["res"] = (3 * torch.randn(m, h, generator=g, device=dev)).to(dt) if case["res"] else None
        st["w"] = (1 + 0.3 * torch.randn(h, generator=g, device=dev)).to(dt)
    elif op == "write":
        t, slots = case["t"], case["pages"] * case["page"]
        st["kv"] = (2 * torch.randn(t, LATENT + ROPE, generator=g, device=dev)).to(torch.bfloat16)
        st["w"] = (1 + 0.3 * torch.randn(LATENT, generator=g, device=dev)).to(torch.bfloat16) if case["norm"] else None
        st["slots"] = torch.randperm(slots, generator=g, device=dev)[:t]
        st["cache"] = torch.zeros(case["pages"], case["page"], ROW, dtype=torch.uint8, device=dev)
        st["scales"] = torch.full((case["pages"], case["page"]), 127, dtype=torch.uint8, device=dev)
    elif op == "read":
        lens = _read_lens(case)
        st["cache"], st["scales"], st["table"] = _filled_cache(lens, case["page"], g, dev)
        st["cu"], st["total"] = _ints(_starts(lens), dev), sum(lens)
    elif op == "attend":
        lens, new = _attend_lens(case)
        st["cache"], st["scales"], st["table"] = _filled_cache(lens, case["page"], g, dev)
        st["lens"], st["cu"] = _ints(lens, dev), _ints(_starts(new), dev)
        st["q"] = torch.randn(sum(new), case["heads"], LATENT + ROPE, generator=g, device=dev).to(torch.bfloat16)
        st["max_q"], st["max_len"] = max(new), max(lens)
    else:
        new, keys = _expand_lens(case)
        dt, heads = DTYPES[case["dtype"]], case["heads"]
        st["q"] = torch.randn(sum(new), heads, NOPE + ROPE, generator=g, device=dev).to(dt)
        st["kv"] = torch.randn(sum(keys), heads, NOPE + VDIM, generator=g, device=dev).to(dt)
        st["rope"] = torch.randn(sum(keys), ROPE, generator=g, device=dev).to(dt)
        st["cu_q"], st["cu_k"] = _ints(_starts(new), dev), _ints(_starts(keys), dev)
        st["max_q"], st["max_k"] = max(new), max(keys)
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    return (_own if own else _plain)(st)


def _f8(codes):
    return codes.view(torch.float8_e4m3fn)


def _e8(codes):
    return codes.view(torch.float8_e8m0fnu)


def _cache_values(cache, scales):
    """What a cache holds: codes, rotary keys and scales as the numbers they stand for."""
    return {"codes": _f8(cache[:, :, :LATENT]), "rope": cache[:, :, LATENT:].view(torch.bfloat16), "scales": _e8(scales)}


def _own(st):
    import block_scaled_fp8_bfp8_amd as bfp8

    c = st["case"]
    if c["op"] == "norm":
        call = bfp8.rmsnorm_quant_ue8m0 if c["e8"] else bfp8.rmsnorm_quant
        q, s, h = call(st["x"], st["w"], residual=st["res"], eps=EPS)
        return {"q": _f8(q), "s": _e8(s) if c["e8"] else s, "h": h if c["res"] else None}
    if c["op"] == "write":
        bfp8.latent_cache_write(st["kv"], st["slots"], st["cache"], st["scales"], norm_weight=st["w"], eps=EPS)
        return _cache_values(st["cache"], st["scales"])
    if c["op"] == "read":
        if not c["raw"]:
            return bfp8.latent_cache_read(st["cache"], st["scales"], st["table"], st["cu"], st["total"])
        q, s, rope = bfp8.latent_cache_gather(st["cache"], st["scales"], st["table"], st["cu"], st["total"])
        return {"q": _f8(q), "s": _e8(s), "rope": rope}
    if c["op"] == "attend":
        return bfp8.latent_attention(st["q"], st["cache"], st["scales"], st["table"], st["lens"], SCALE, cu_q=st["cu"])
    return bfp8.latent_attention_expanded(st["q"], st["kv"], st["rope"], st["cu_q"], st["cu_k"], SCALE)


def _rms(x, w):
    return x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * w


def _rows_of(st, cu, total):
    """Cache rows of the tokens of all sequences one after the other."""
    pos = torch.arange(total, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), pos.to(torch.int32), right=True)
    p = pos - cu[b]
    page = st["case"]["page"]
    return st["table"][b, p // page].long() * page + p % page


def _dequantized(cache, scales, rows):
    """float32 [..., LATENT + ROPE] of the cache rows `rows`."""
    raw = cache.reshape(-1, ROW)[rows]
    e = scales.reshape(-1)[rows].to(torch.int32) - 127
    lat = torch.ldexp(_f8(raw[..., :LATENT]).float(), e[..., None])
    return torch.cat([lat, raw[..., LATENT:].contiguous().view(torch.bfloat16).float()], dim=-1)


def _softmax_product(s, seen, v):
    """softmax over the seen keys of the scores s [..., R, L], times v [..., L, D]; rows that see no key are zero."""
    s = s.masked_fill(~seen, float("-inf"))
    top = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(dim=-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)


def _plain(st):
    c = st["case"]
    if c["op"] == "norm":
        dt, w = st["x"].dtype, st["w"].float()
        h = st["x"].float() if st["res"] is None else (st["x"].float() + st["res"].float()).to(dt).float()
        y = _rms(h, w)
        m, k = y.shape
        groups = -(-k // 128)
        y = torch.nn.functional.pad(y, (0, groups * 128 - k)).view(m, groups, 128)
        s = torch.clamp(y.abs().amax(dim=2), min=1e-10)
        s = s / torch.full_like(s, 448.0)
        if c["e8"]:
            s = ((s.view(torch.int32) + 0x7FFFFF) & ~0x7FFFFF).view(torch.float32)
        q = (y / s[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(m, groups * 128)[:, :k]
        s = _e8((s.view(torch.int32) >> 23).to(torch.uint8)) if c["e8"] else s
        return {"q": q, "s": s, "h": None if st["res"] is None else h.to(dt)}
    if c["op"] == "write":
        y = st["kv"][:, :LATENT].float()
        if c["norm"]:
            y = _rms(y, st["w"].float())
        codes, e = _quantize_rows(y)
        rope = st["kv"][:, LATENT:].contiguous().view(torch.uint8)
        st["cache"].view(-1, ROW)[st["slots"]] = torch.cat([codes, rope], dim=1)
        st["scales"].view(-1)[st["slots"]] = e
        return _cache_values(st["cache"], st["scales"])
    if c["op"] == "read":
        rows = _rows_of(st, st["cu"], st["total"])
        if not c["raw"]:
            return _dequantized(st["cache"], st["scales"], rows).to(torch.bfloat16)
        raw = st["cache"].view(-1, ROW)[rows]
        e = st["scales"].view(-1)[rows]
        return {"q": _f8(raw[:, :LATENT]), "s": _e8(e[:, None].expand(-1, LATENT // 128).contiguous()),
                "rope": raw[:, LATENT:].contiguous().view(torch.bfloat16)}
    if c["op"] == "attend":
        return _plain_attend(st)
    return _plain_expand(st)


def _padded(cu, longest):
    """[B, longest] places of the tokens of each sequence in the packed order (clipped), and which exist."""
    at = torch.arange(longest, device=cu.device)
    n = (cu[1:] - cu[:-1]).long()
    return torch.minimum(cu[:-1, None].long() + at, cu[-1].long() - 1), at < n[:, None]


def _plain_attend(st):
    c = st["case"]
    lens, cu, page = st["lens"].long(), st["cu"], st["case"]["page"]
    at = torch.arange(st["max_len"], device=lens.device)
    pages = st["table"][:, at // page].long().clamp(min=0)
    k = _dequantized(st["cache"], st["scales"], pages * page + at % page)  # [B, L, 576]
    where, exists = _padded(cu, st["max_q"])
    q = st["q"][where].float()  # [B, Q, H, 576]
    b, nq, heads, d = q.shape
    s = torch.matmul(q.view(b, nq * heads, d), k.transpose(1, 2)) * SCALE
    n = (cu[1:] - cu[:-1]).long()
    last = (lens - n)[:, None] + torch.arange(nq, device=lens.device)  # the last key that a new token sees
    seen = at <= last[:, :, None]
    seen = seen[:, :, None, :].expand(b, nq, heads, -1).reshape(b, nq * heads, -1)
    o = _softmax_product(s, seen, k[:, :, :LATENT]).view(b, nq, heads, LATENT)
    return o[exists].to(torch.bfloat16)


def _plain_expand(st):
    cu_q, cu_k = st["cu_q"], st["cu_k"]
    wq, eq = _padded(cu_q, st["max_q"])
    wk, ek = _padded(cu_k, st["max_k"])
    q = st["q"][wq].float().transpose(1, 2)  # [B, H, Q, 192]
    kv = st["kv"][wk].float().transpose(1, 2)  # [B, H, K, 256]
    rope = st["rope"][wk].float()[:, None].expand(-1, kv.shape[1], -1, -1)
    k = torch.cat([kv[..., :NOPE], rope], dim=-1)
    s = torch.matmul(q, k.transpose(2, 3)) * SCALE
    nq, nk = (cu_q[1:] - cu_q[:-1]).long(), (cu_k[1:] - cu_k[:-1]).long()
    last = (nk - nq)[:, None] + torch.arange(st["max_q"], device=nq.device)
    seen = (torch.arange(st["max_k"], device=nq.device) <= last[:, :, None]) & ek[:, None, :]
    o = _softmax_product(s, seen[:, None], kv[..., NOPE:])
    return o.transpose(1, 2)[eq].to(st["q"].dtype)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "norm":
        m, h, size = case["m"], case["h"], {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]]
        n = m * h
        return {"bytes": n * size * (3 if case["res"] else 1) + n + h * size + m * -(-h // 128) * (1 if case["e8"] else 4),
                "flops": 8 * n}
    if op == "write":
        return {"bytes": case["t"] * (2 * (LATENT + ROPE) + 8 + ROW + 1), "flops": case["t"] * 6 * LATENT}
    if op == "read":
        n = sum(_read_lens(case))
        out = ROW + LATENT // 128 if case["raw"] else 2 * (LATENT + ROPE)
        return {"bytes": n * (ROW + 1 + out), "flops": n * LATENT}
    if op == "attend":
        lens, new = _attend_lens(case)
        pairs = sum(m * (n - m) + m * (m + 1) // 2 for n, m in zip(lens, new)) * case["heads"]
        return {"bytes": sum(lens) * (ROW + 1) + sum(new) * case["heads"] * 2 * (2 * LATENT + ROPE),
                "flops": pairs * 2 * (2 * LATENT + ROPE)}
    new, keys = _expand_lens(case)
    size, heads = 2, case["heads"]
    pairs = sum(m * (n - m) + m * (m + 1) // 2 for n, m in zip(keys, new)) * heads
    return {"bytes": size * (sum(new) * heads * (NOPE + ROPE + VDIM) + sum(keys) * (heads * (NOPE + VDIM) + ROPE)),
            "flops": pairs * 2 * (NOPE + ROPE + VDIM)}


# ---------------------------------------------------------------- the definition in 64 bits

def _e4m3_value(code):
    """The number that an e4m3 code (uint8) stands for, from the format's definition."""
    code = code.long()
    sign = torch.where(code >= 128, -1.0, 1.0).double()
    exp, man = (code >> 3) & 15, (code & 7).double()
    return sign * torch.where(exp == 0, man * 2.0 ** -9, (1 + man / 8) * torch.exp2((exp - 7).double()))


def _cache_row(st, b, length):
    """(latent, rotary key) of the first `length` tokens of sequence b in float64."""
    page = st["cache"].shape[1]
    t = torch.arange(length, device=st["cache"].device)
    p, o = st["table"][b, t // page].long(), t % page
    raw = st["cache"][p, o]
    lat = _e4m3_value(raw[:, :LATENT]) * torch.exp2(st["scales"][p, o].double() - 127)[:, None]
    return lat, raw[:, LATENT:].contiguous().view(torch.bfloat16).double()


def _attention64(q, k, v, first):
    """One head or one group of rows: q [R, D], k [L, D], v [L, E], first [R] = keys that row r sees."""
    s = q @ k.t() * SCALE
    s[torch.arange(k.shape[0], device=k.device)[None, :] >= first[:, None]] = float("-inf")
    return torch.softmax(s, dim=-1) @ v


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        # codes before their rounding to 8 bits; with power-of-two scales 2^ceil(log2(amax / 448))
        x = st["x"].double()
        if st["res"] is not None:
            # the sum of two numbers of 24 bits or fewer, rounded to the stream's type
            x = (x + st["res"].double()).to(st["x"].dtype).double()
        y = x / torch.sqrt(x.square().sum(1, keepdim=True) / x.shape[1] + EPS) * st["w"].double()
        s = torch.stack([p.abs().amax(1).clamp(min=1e-10) / 448 for p in y.split(128, dim=1)], dim=1)
        if case["e8"]:
            s = torch.exp2(torch.ceil(torch.log2(s)))
        q = y / s.repeat_interleave(128, dim=1)[:, :y.shape[1]]
        return {"q": q, "s": s, "h": None if st["res"] is None else x}
    if op == "write":
        y = st["kv"][:, :LATENT].double()
        if st["w"] is not None:
            y = y / torch.sqrt(y.square().sum(1, keepdim=True) / LATENT + EPS) * st["w"].double()
        s = torch.exp2(torch.ceil(torch.log2(y.abs().amax(1).clamp(min=1e-10) / 448)))
        codes = _f8(st["cache"][:, :, :LATENT]).double()
        rope = st["cache"][:, :, LATENT:].contiguous().view(torch.bfloat16).double()
        scales = torch.exp2(st["scales"].double() - 127)
        page = case["page"]
        at, off = st["slots"] // page, st["slots"] % page
        codes[at, off], scales[at, off] = y / s[:, None], s
        rope[at, off] = st["kv"][:, LATENT:].double()
        return {"codes": codes, "rope": rope, "scales": scales}
    if op == "read":
        rows, scales = [], []
        for b, n in enumerate(_read_lens(case)):
            rows.append(_cache_row(st, b, n))
            t = torch.arange(n, device=st["cache"].device)
            scales.append(torch.exp2(st["scales"][st["table"][b, t // case["page"]].long(), t % case["page"]].double() - 127))
        if not case["raw"]:
            return torch.cat([torch.cat(r, dim=1) for r in rows])
        s = torch.cat(scales)[:, None]
        return {"q": torch.cat([r[0] for r in rows]) / s, "s": s.repeat(1, LATENT // 128), "rope": torch.cat([r[1] for r in rows])}
    if op == "attend":
        lens, new = _attend_lens(case)
        first, out = _starts(new), []
        for b, (n, m) in enumerate(zip(lens, new)):
            lat, rope = _cache_row(st, b, n)
            q = st["q"][first[b]:first[b + 1]].double().flatten(0, 1)
            sees = (n - m + 1 + torch.arange(m, device=q.device)).repeat_interleave(case["heads"])
            out.append(_attention64(q, torch.cat([lat, rope], dim=1), lat, sees).view(m, case["heads"], LATENT))
        return torch.cat(out)
    new, keys = _expand_lens(case)
    fq, fk = _starts(new), _starts(keys)
    out = torch.empty(sum(new), case["heads"], VDIM, dtype=torch.float64, device=st["q"].device)
    for b, (m, n) in enumerate(zip(new, keys)):
        sees = n - m + 1 + torch.arange(m, device=out.device)
        rope = st["rope"][fk[b]:fk[b + 1]].double()
        for h in range(case["heads"]):
            kv = st["kv"][fk[b]:fk[b + 1], h].double()
            k = torch.cat([kv[:, :NOPE], rope], dim=1)
            out[fq[b]:fq[b + 1], h] = _attention64(st["q"][fq[b]:fq[b + 1], h].double(), k, kv[:, NOPE:], sees)
    return out
