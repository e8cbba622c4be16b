"""Measured cases of the 8-bit integer products (token quantizer, product with scales for each token
and channel, linear layer) and of a bounded latent cache (attention that accumulates its weights,
eviction by them). `run` computes each operator either in plain torch steps or, with `own`, through
the package."""

from __future__ import annotations

import torch

own = False

LATENT, ROPE = 512, 64   # the cached latent vector and the shared rotary key of a token
ROW = LATENT + 2 * ROPE  # bytes of a cache row: e4m3 codes, then the rotary key in bf16
SCALE = (128 + ROPE) ** -0.5

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One decoded token in front of a projection: pure latency.
        {"name": "quant 1x7168", "op": "quant", "m": 1, "k": 7168, "dtype": "bf16"},
        # A prefill batch in front of the hidden-5120 projections.
        {"name": "quant 8192x5120", "op": "quant", "m": 8192, "k": 5120, "dtype": "bf16"},
        # One decoded token through a square projection: reading the weights is the work.
        {"name": "gemm 1x4096x4096", "op": "gemm", "m": 1, "n": 4096, "k": 4096, "dtype": "bf16", "bias": False},
        # An odd batch against a narrow weight with a long inner dimension.
        {"name": "gemm 83x576x7168", "op": "gemm", "m": 83, "n": 576, "k": 7168, "dtype": "f16", "bias": True},
        # A prefill batch through the QKV projection at hidden 5120: the matrix cores are the work.
        {"name": "gemm 8192x10240x5120", "op": "gemm", "m": 8192, "n": 10240, "k": 5120, "dtype": "bf16", "bias": False},
        # A small decode batch through a layer as a model calls it: 16-bit activations in, 16-bit out.
        {"name": "linear 5x5120x8192", "op": "linear", "m": 5, "n": 5120, "k": 8192, "dtype": "bf16", "bias": True},
        # A medium prefill chunk, likewise.
        {"name": "linear 1000x4096x4096", "op": "linear", "m": 1000, "n": 4096, "k": 4096, "dtype": "bf16", "bias": True},
        # One sequence, one new token, all heads: the latency case of decoding with a bounded cache.
        {"name": "mass 1x128h", "op": "mass", "b": 1, "heads": 128, "q": 1, "lo": 1111, "hi": 1111, "page": 64},
        # A tensor-parallel rank's 16 heads over ragged contexts: reading the cache is the work.
        {"name": "mass 64x16h", "op": "mass", "b": 64, "heads": 16, "q": 1, "lo": 500, "hi": 8000, "page": 64},
        # Chunks of new tokens behind cached prefixes: the matrix cores are the work.
        {"name": "mass 6x40x128h", "op": "mass", "b": 6, "heads": 128, "q": 40, "lo": 700, "hi": 3500, "page": 16},
        # One sequence that has just passed its budget.
        {"name": "evict 1x1111", "op": "evict", "b": 1, "lo": 1111, "hi": 1111, "page": 64, "budget": 1024, "recent": 128},
        # Prompts of a batch are cut down to what decoding keeps, onto pages of their own.
        {"name": "evict 64x8000", "op": "evict", "b": 64, "lo": 500, "hi": 8000, "page": 64, "budget": 4096, "recent": 512},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["quant", "gemm", "gemm", "linear", "mass", "mass", "evict"])
    if op == "quant":
        k = 16 * _log(rng, 1, 1024)
        return {"op": op, "m": _log(rng, 1, min(8192, max(1, (1 << 25) // k))), "k": k,
                "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
    if op in ("gemm", "linear"):
        n, k = _log(rng, 8, 25600), 16 * _log(rng, 4, 1600)
        m = _log(rng, 1, 8192)
        while m > 1 and m * n * k > 8192 * 10240 * 5120:
            m //= 2
        return {"op": op, "m": m, "n": n, "k": k, "dtype": rng.choice(["bf16", "bf16", "f16"]),
                "bias": rng.random() < 0.5}
    hi = _log(rng, 1, 8000)
    page, b = rng.choice([1, 16, 37, 64]), _log(rng, 1, 64)
    lo = rng.randint(max(1, hi // 8), hi)
    if op == "mass":
        heads = rng.choice([1, 5, 8, 16, 16, 32, 40, 64, 128, 128])
        q = rng.choice([1, 1, 1, 2, 4, rng.randint(5, 96)])
        while b > 1 and b * heads * q * hi > 6 * 40 * 128 * 2048:
            b //= 2
        if heads * q * hi > 6 * 40 * 128 * 2048:
            q = 1
        return {"op": op, "b": b, "heads": heads, "q": q, "lo": lo, "hi": hi, "page": page}
    budget = _log(rng, 1, 4096)
    return {"op": op, "b": b, "lo": lo, "hi": hi, "page": page, "budget": budget,
            "recent": rng.choice([0, budget, rng.randint(0, budget)])}


def _lens(n, lo, hi):
    """n lengths in [lo, hi], spread evenly and out of order; the same for every seed, so that a
    case's work is its own. The last is hi."""
    return [lo + int((hi - lo) * ((0.6180339887 * (i + 1)) % 1.0)) for i in range(n - 1)] + [hi]


def _cache_lens(c):
    return _lens(c["b"], c["lo"], c["hi"])


def _new_tokens(c):
    """Tokens of each sequence that are new in the call: the last of it."""
    return [min(c["q"], n) for n in _cache_lens(c)]


# ---------------------------------------------------------------- inputs

def _ints(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _starts(lens):
    s = [0]
    for n in lens:
        s.append(s[-1] + n)
    return s


def _activations(m, k, dtype, g, dev):
    """Tokens of different sizes, with a few channels that stand out in all of them."""
    x = torch.randn(m, k, generator=g, device=dev)
    x *= torch.exp(0.5 * torch.randn(m, 1, generator=g, device=dev))
    x *= torch.where(torch.rand(k, generator=g, device=dev) < 0.01, 20.0, 1.0)
    return x.to(dtype)


def _weights(n, k, g, dev):
    """int8 codes of weights and the scale of each channel, as a checkpoint holds them."""
    q = (30 * torch.randn(n, k, generator=g, device=dev)).round().clamp(-127, 127).to(torch.int8)
    s = 0.002 * torch.exp(0.3 * torch.randn(n, generator=g, device=dev))
    return q, s


def _page_table(lens, page, order, dev):
    need = [-(-n // page) for n in lens]
    first = _starts(need)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=dev)
    for b, n in enumerate(need):
        table[b, :n] = order[first[b]:first[b] + n]
    return table


def _filled_cache(lens, page, extra, g, dev):
    """A paged cache that holds sequences of these lengths on shuffled pages, its page table, and
    `extra` further pages."""
    used = sum(-(-n // page) for n in lens)
    pages = used + extra
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = _page_table(lens, page, order, dev)
    cache = torch.empty(pages * page, ROW, dtype=torch.uint8, device=dev)
    scales = torch.empty(pages * page, dtype=torch.uint8, device=dev)
    for i in range(0, pages * page, 65536):
        n = min(65536, pages * page - i)
        y = torch.randn(n, LATENT, generator=g, device=dev)
        y *= torch.exp(0.5 * torch.randn(n, 1, generator=g, device=dev))  # tokens differ in size
        s = torch.clamp(y.abs().amax(dim=1), min=1e-10) / 448.0
        e = ((s.view(torch.int32) + 0x7FFFFF) >> 23) & 0xFF  # the next power of two
        y = torch.ldexp(y, (127 - e)[:, None]).clamp(-448.0, 448.0)
        cache[i:i + n, :LATENT] = y.to(torch.float8_e4m3fn).view(torch.uint8)
        scales[i:i + n] = e.to(torch.uint8)
        r = torch.randn(n, ROPE, generator=g, device=dev).to(torch.bfloat16)
        cache[i:i + n, LATENT:] = r.view(torch.uint8)
    return cache.view(pages, page, ROW), scales.view(pages, page), table, order[used:]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    if op == "quant":
        st["x"] = _activations(case["m"], case["k"], DTYPES[case["dtype"]], g, dev)
    elif op in ("gemm", "linear"):
        m, n, k, dt = case["m"], case["n"], case["k"], DTYPES[case["dtype"]]
        st["w"], st["ws"] = _weights(n, k, g, dev)
        st["bias"] = torch.randn(n, generator=g, device=dev).to(dt) if case["bias"] else None
        if op == "linear":
            st["x"] = _activations(m, k, dt, g, dev)
        else:
            st["q"] = (30 * torch.randn(m, k, generator=g, device=dev)).round().clamp(-127, 127).to(torch.int8)
            st["qs"] = 0.02 * torch.exp(0.5 * torch.randn(m, generator=g, device=dev))
    else:
        lens, page = _cache_lens(case), case["page"]
        kept = [min(n, case["budget"]) for n in lens] if op == "evict" else []
        extra = sum(-(-n // page) for n in kept) + 3
        st["cache"], st["scales"], st["table"], spare = _filled_cache(lens, page, extra, g, dev)
        st["lens"] = _ints(lens, dev)
        # weights accumulated so far: of very different sizes, some tokens never looked at
        width = st["table"].shape[1] * page
        mass = torch.exp(2.0 * torch.randn(case["b"], width, generator=g, device=dev))
        st["mass"] = torch.where(torch.rand(case["b"], width, generator=g, device=dev) < 0.2, 0.0, mass)
        if op == "mass":
            new = _new_tokens(case)
            st["cu"] = _ints(_starts(new), dev)
            st["q"] = torch.randn(sum(new), case["heads"], LATENT + ROPE, generator=g, device=dev).to(torch.bfloat16)
            st["max_q"], st["max_len"] = max(new), max(lens)
        else:
            st["to"] = _page_table(kept, page, spare, dev)
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    return (_own if own else _plain)(st)


def _cache_values(cache, scales):
    """What a cache holds: codes, rotary keys and scales as the numbers they stand for."""
    return {"codes": cache[:, :, :LATENT].view(torch.float8_e4m3fn), "rope": cache[:, :, LATENT:].view(torch.bfloat16),
            "scales": scales.view(torch.float8_e8m0fnu)}


def _own(st):
    import block_scaled_fp8_bfp8_amd as bfp8

    c = st["case"]
    if c["op"] == "quant":
        q, s = bfp8.quant_act_int8(st["x"])
        return {"q": q, "s": s}
    if c["op"] == "gemm":
        return bfp8.gemm_int8(st["q"], st["qs"], st["w"], st["ws"], bias=st["bias"], dtype=DTYPES[c["dtype"]])
    if c["op"] == "linear":
        return bfp8.linear_int8(st["x"], st["w"], st["ws"], st["bias"])
    if c["op"] == "mass":
        out, mass = bfp8.latent_attention_mass(st["q"], st["cache"], st["scales"], st["table"], st["lens"], SCALE,
                                               mass=st["mass"], cu_q=st["cu"])
        return {"out": out, "mass": mass}
    kept, lens, mass = bfp8.latent_cache_evict(st["cache"], st["scales"], st["table"], st["lens"], st["mass"],
                                               c["budget"], recent=c["recent"], out_table=st["to"])
    return {"kept": kept, "lens": lens, "mass": mass, **_cache_values(st["cache"], st["scales"])}


def _plain(st):
    c = st["case"]
    if c["op"] == "quant":
        q, s = _plain_quant(st["x"])
        return {"q": q.to(torch.int8), "s": s}
    if c["op"] == "gemm":
        return _plain_product(st["q"].float(), st["qs"], st).to(DTYPES[c["dtype"]])
    if c["op"] == "linear":
        return _plain_product(*_plain_quant(st["x"]), st).to(st["x"].dtype)
    return _plain_mass(st) if c["op"] == "mass" else _plain_evict(st)


def _plain_quant(x):
    """Codes (float32) and scales of tokens. The codes are decided in 64 bits: x may lie at the middle of two."""
    a = x.float().abs().amax(dim=1).clamp(min=1e-10)
    q = torch.round(x.double() * 127.0 / a.double()[:, None])
    return q.float(), a / torch.full_like(a, 127.0)


def _plain_product(q, s, st):
    y = torch.matmul(q, st["w"].float().t()) * s[:, None] * st["ws"]
    return y if st["bias"] is None else y + st["bias"].float()


def _padded(cu, longest):
    """[B, longest] places of the tokens of each sequence in the packed order (clipped), and which exist."""
    at = torch.arange(longest, device=cu.device)
    n = (cu[1:] - cu[:-1]).long()
    return torch.minimum(cu[:-1, None].long() + at, cu[-1].long() - 1), at < n[:, None]


def _plain_mass(st):
    c = st["case"]
    lens, cu, page = st["lens"].long(), st["cu"], c["page"]
    at = torch.arange(st["max_len"], device=lens.device)
    rows = st["table"][:, at // page].long().clamp(min=0) * page + at % page
    raw = st["cache"].view(-1, ROW)[rows]
    e = st["scales"].view(-1)[rows].to(torch.int32) - 127
    v = torch.ldexp(raw[..., :LATENT].view(torch.float8_e4m3fn).float(), e[..., None])
    k = torch.cat([v, raw[..., LATENT:].contiguous().view(torch.bfloat16).float()], dim=-1)  # [B, L, 576]
    where, exists = _padded(cu, st["max_q"])
    q = st["q"][where].float()  # [B, Q, H, 576]
    b, nq, heads, d = q.shape
    s = torch.matmul(q.view(b, nq * heads, d), k.transpose(1, 2)) * SCALE
    n = (cu[1:] - cu[:-1]).long()
    last = (lens - n)[:, None] + torch.arange(nq, device=lens.device)  # the last key that a new token sees
    seen = (at <= last[:, :, None]) & exists[:, :, None]
    s = s.view(b, nq, heads, -1).masked_fill(~seen[:, :, None], float("-inf"))
    top = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(dim=-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    o = torch.matmul(p.view(b, nq * heads, -1), v).view(b, nq, heads, LATENT)
    mass = torch.zeros_like(st["mass"])
    old = at < (lens - n)[:, None]
    mass[:, :st["max_len"]] = torch.where(old, st["mass"][:, :st["max_len"]], 0.0) + p.sum(dim=(1, 2))
    return {"out": o[exists].to(torch.bfloat16), "mass": mass}


def _plain_evict(st):
    c = st["case"]
    lens, mass, page, budget, recent = st["lens"].long(), st["mass"], c["page"], c["budget"], c["recent"]
    b, width = mass.shape
    at = torch.arange(width, device=mass.device).expand(b, width)
    exists = at < lens[:, None]
    # rank every token: the recent ones first, then by mass, the earlier of two equals first
    worth = torch.where(at >= (lens - recent)[:, None], float("inf"), mass)
    worth = torch.where(exists, worth, float("-inf"))
    order = torch.sort(worth, dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, at.contiguous())
    keep = exists & (rank < budget)
    place = torch.cumsum(keep, dim=1) - 1
    kept = torch.full((b, budget), -1, dtype=torch.int32, device=mass.device)
    new_mass = torch.zeros_like(mass)
    seq, pos = torch.nonzero(keep, as_tuple=True)
    to = place[seq, pos]
    kept[seq, to] = pos.to(torch.int32)
    new_mass[seq, to] = mass[seq, pos]
    src = st["table"][seq, pos // page].long() * page + pos % page
    dst = st["to"][seq, to // page].long() * page + to % page
    st["cache"].view(-1, ROW)[dst] = st["cache"].view(-1, ROW)[src]
    st["scales"].view(-1)[dst] = st["scales"].view(-1)[src]
    return {"kept": kept, "lens": lens.clamp(max=budget).to(torch.int32), "mass": new_mass,
            **_cache_values(st["cache"], st["scales"])}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "quant":
        n, size = case["m"] * case["k"], {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]]
        return {"bytes": n * (size + 1) + 4 * case["m"], "flops": 3 * n}
    if op in ("gemm", "linear"):
        m, n, k = case["m"], case["n"], case["k"]
        rows = m * k * 2 if op == "linear" else m * (k + 4)
        return {"bytes": rows + n * (k + 4) + 2 * m * n + (2 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    lens = _cache_lens(case)
    width = -(-max(lens) // case["page"]) * case["page"]
    if op == "mass":
        new = _new_tokens(case)
        pairs = sum(m * (n - m) + m * (m + 1) // 2 for n, m in zip(lens, new)) * case["heads"]
        return {"bytes": sum(lens) * (ROW + 1 + 4) + sum(new) * case["heads"] * 2 * (2 * LATENT + ROPE) + case["b"] * width * 4,
                "flops": pairs * 2 * (2 * LATENT + ROPE)}
    kept = sum(min(n, case["budget"]) for n in lens)
    return {"bytes": 2 * kept * (ROW + 1) + sum(lens) * 4 + case["b"] * (width + case["budget"]) * 4, "flops": sum(lens)}


# ---------------------------------------------------------------- the definition in 64 bits

def _e4m3_value(code):
    """The number that an e4m3 code (uint8) stands for, from the format's definition."""
    code = code.long()
    sign = torch.where(code >= 128, -1.0, 1.0).double()
    exp, man = (code >> 3) & 15, (code & 7).double()
    return sign * torch.where(exp == 0, man * 2.0 ** -9, (1 + man / 8) * torch.exp2((exp - 7).double()))


def _codes64(x):
    a = x.double().abs().max(dim=1, keepdim=True).values.clamp(min=1e-10)
    return (127 * x.double() / a).round(), (a / 127)[:, 0]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        q, s = _codes64(st["x"])
        return {"q": q.to(torch.int8), "s": s}
    if op in ("gemm", "linear"):
        q, s = _codes64(st["x"]) if op == "linear" else (st["q"].double(), st["qs"].double())
        w = st["w"].double() * st["ws"].double()[:, None]
        out = (q * s[:, None]) @ w.t()
        return out if st["bias"] is None else out + st["bias"].double()
    lens, page = _cache_lens(case), case["page"]
    if op == "mass":
        new = _new_tokens(case)
        first = _starts(new)
        out, mass = [], torch.zeros(st["mass"].shape, dtype=torch.float64, device=st["mass"].device)
        for b, (n, m) in enumerate(zip(lens, new)):
            t = torch.arange(n, device=mass.device)
            p, o = st["table"][b, t // page].long(), t % page
            raw = st["cache"][p, o]
            lat = _e4m3_value(raw[:, :LATENT]) * torch.exp2(st["scales"][p, o].double() - 127)[:, None]
            keys = torch.cat([lat, raw[:, LATENT:].contiguous().view(torch.bfloat16).double()], dim=1)
            mass[b, :n - m] = st["mass"][b, :n - m].double()
            for i in range(m):  # a new token: all its heads see the same keys
                sees = n - m + i + 1
                p = torch.softmax(st["q"][first[b] + i].double() @ keys[:sees].t() * SCALE, dim=-1)
                out.append(p @ lat[:sees])
                mass[b, :sees] += p.sum(dim=0)
        return {"out": torch.stack(out), "mass": mass}
    budget, recent = case["budget"], case["recent"]
    kept = torch.full((case["b"], budget), -1, dtype=torch.int32, device=st["mass"].device)
    mass = torch.zeros(st["mass"].shape, dtype=torch.float64, device=kept.device)
    cache, scales = st["cache"].clone(), st["scales"].clone()
    for b, n in enumerate(lens):
        old = max(n - recent, 0) if n > budget else n
        # by falling mass, then by rising position
        best = sorted(range(old), key=lambda j, w=st["mass"][b].tolist(): (-w[j], j))[:min(n, budget) - (n - old)]
        pos = torch.tensor(sorted(best) + list(range(old, n)), device=kept.device)
        to = torch.arange(len(pos), device=kept.device)
        kept[b, :len(pos)] = pos.to(torch.int32)
        mass[b, :len(pos)] = st["mass"][b, pos].double()
        src, dst = st["table"][b, pos // page].long(), st["to"][b, to // page].long()
        cache[dst, to % page], scales[dst, to % page] = st["cache"][src, pos % page], st["scales"][src, pos % page]
    return {"kept": kept, "lens": torch.tensor([min(n, budget) for n in lens], dtype=torch.int32, device=kept.device),
            "mass": mass, "codes": _e4m3_value(cache[:, :, :LATENT]),
            "rope": cache[:, :, LATENT:].contiguous().view(torch.bfloat16).double(),
            "scales": torch.exp2(scales.double() - 127)}
