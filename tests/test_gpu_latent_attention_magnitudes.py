"""GPU tests of latent attention with scores of every magnitude in float32's range: where all of a row's lie below -10^30, and at each
power of two, where the highest score stands far above the others."""

import pytest
import torch

import block_scaled_fp8_bfp8_amd as bfp8
from tests.gpu_util import announce
from tests.test_gpu_latent_attention import SCALE

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,tokens,heads", [(1, 1, 1), (90, 1, 16), (1500, 1, 128), (1500, 3, 5), (300, 40, 64)])
@pytest.mark.parametrize("with_rope", [False, True])
def test_scores_below_every_common_bound(gpu, n, tokens, heads, with_rope):
    """Key j has first[j] as its first latent, 448 as its second (which holds the scale at one) and rope[j] as its first
    rotary value; queries see the first dimensions alone and make finite scores of -10^31 and less of them. The keys whose
    scores are highest, which all have 1 as their first latent, share the weight (the next are 2^100 lower), so the output
    is their value, to its rounding."""
    page = 16
    pages = -(-n // page)
    kv = torch.zeros(n, 576, dtype=torch.bfloat16)
    kv[:, 0] = torch.tensor([[1.0, 2.5, 1.0, 4.0, 28.0][j % 5] for j in range(n)])
    kv[:, 1] = 448.0
    if with_rope:
        kv[:, 512] = torch.tensor([[1.0, 1.0, 8.0, 0.5, 2.0][j % 5] for j in range(n)])
    cache = torch.zeros(pages, page, 640, dtype=torch.uint8, device=gpu)
    scales = torch.full((pages, page), 127, dtype=torch.uint8, device=gpu)
    bfp8.latent_cache_write(kv.to(gpu), torch.arange(n, device=gpu), cache, scales)
    table = torch.arange(pages, dtype=torch.int32, device=gpu)[None]
    q = torch.zeros(tokens, heads, 576, dtype=torch.bfloat16)
    by = -torch.exp2(torch.tensor([108.0 + h % 5 for h in range(heads)]))
    q[:, :, 0] = by
    if with_rope:
        q[:, :, 512] = by
    announce("latent attention low scores", n, tokens, heads, with_rope)
    out = bfp8.latent_attention(q.to(gpu), cache, scales, table, torch.tensor([n], dtype=torch.int32, device=gpu), SCALE,
                                cu_q=torch.tensor([0, tokens], dtype=torch.int32, device=gpu))
    want = torch.zeros(512)
    want[0], want[1] = 1.0, 448.0
    got = out.float().cpu()
    assert bool(((got - want).abs() <= want * 2.0 ** -8).all()), got[0, 0, :4]


@pytest.mark.parametrize("n,tokens", [(7, 1), (90, 1), (90, 5), (1500, 1)])
def test_scores_of_every_magnitude(gpu, n, tokens):
    """Keys as above; a head's queries are 2^10 .. 2^118 of either sign, with different mantissas, so that the keys with the
    highest score share the weight (the next are 2^100 times less) and the output is their value. The attention's masses lie on them in
    equal shares (one division and one product a row, 2^-22; additions of rows 2^-24 each)."""
    page, level = 16, [1.0, 2.5, 1.0, 4.0, 28.0]
    pages = -(-n // page)
    first = torch.tensor([level[j % 5] for j in range(n)])
    kv = torch.zeros(n, 576, dtype=torch.bfloat16)
    kv[:, 0] = first
    kv[:, 1] = 448.0
    cache = torch.zeros(pages, page, 640, dtype=torch.uint8, device=gpu)
    scales = torch.full((pages, page), 127, dtype=torch.uint8, device=gpu)
    bfp8.latent_cache_write(kv.to(gpu), torch.arange(n, device=gpu), cache, scales)
    by = torch.tensor([s * 2.0 ** e * (1 + (e * 5 % 8) / 8) for e in range(10, 119) for s in (1.0, -1.0)])
    heads = len(by)
    q = torch.zeros(tokens, heads, 576, dtype=torch.bfloat16)
    q[:, :, 0] = by
    announce("latent attention magnitudes", n, tokens)
    args = (q.to(gpu), cache, scales, torch.arange(pages, dtype=torch.int32, device=gpu)[None],
            torch.tensor([n], dtype=torch.int32, device=gpu), SCALE)
    out, mass = bfp8.latent_attention_mass(*args, cu_q=torch.tensor([0, tokens], dtype=torch.int32, device=gpu))
    want = torch.zeros(tokens, heads, 512)
    shares = torch.zeros(n, dtype=torch.float64)
    for t in range(tokens):
        seen = first[:n - tokens + t + 1]
        for best, sign in ((seen.max(), 1.0), (seen.min(), -1.0)):
            want[t, by.sign() == sign, 0] = float(best)
            shares[:len(seen)] += heads / 2 * (seen == best).double() / (seen == best).sum()
    want[:, :, 1] = 448.0
    got = out.float().cpu()
    bad = ((got - want).abs() <= want * 2.0 ** -8).all(dim=-1).logical_not()
    assert not bool(bad.any()), [(float(by[h]), got[t, h, :3].tolist()) for t, h in bad.nonzero().tolist()[:8]]
    assert bool(((mass[0, :n].double().cpu() - shares).abs() <= shares * (2.0 ** -22 + tokens * heads * 2.0 ** -24)).all())
