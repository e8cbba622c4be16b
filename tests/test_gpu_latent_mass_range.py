"""GPU tests of the accumulated attention weights at the ends of their ranges: the widest masses, and the
lowest scores."""

import pytest
import torch

import block_scaled_fp8_bfp8_amd as bfp8
from tests.gpu_util import announce
from tests.test_gpu_latent_attention import SCALE, make
from tests.test_gpu_latent_mass import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,heads", [(0, 16), (1, 16), (1, 64), (20, 64)])
def test_widest_masses(gpu, tokens, heads):
    """The most columns that are accepted, 65537 below 2^31: a step of the last launch's workgroups past the last of them
    goes beyond 2^31. The sequence's masses are held to the tolerance of narrow ones (not to their bits: how many workgroups
    there are decides how many waves add up the rows), those that no new token adds to are as they were, and every other
    column is zero."""
    length, width = 100, (1 << 31) - 1 - 65536
    c, keys = make(gpu, [length], [max(tokens, 1)], heads, 16, seed=61)
    args = (c["q"][:tokens], c["cache"], c["scales"], c["table"], c["lens"], SCALE)
    cu = torch.tensor([0, tokens], dtype=torch.int32, device=gpu)
    reach = c["table"].shape[1] * 16
    g = torch.Generator().manual_seed(62)
    before = torch.rand(1, reach, generator=g).to(gpu)
    announce("latent_attention_mass widest", tokens, heads)
    wide = torch.full((1, width), 7.0, device=gpu)
    wide[:, :reach] = before
    _, got = bfp8.latent_attention_mass(*args, mass=wide, cu_q=cu, out_mass=wide)
    torch.cuda.synchronize()
    assert got is wide
    if tokens:
        check(got[:, :reach], before, c["q"], keys, [length], [tokens])
    else:
        assert torch.equal(got[:, :length], before[:, :length])
    past = got[0, length:]
    assert max(float(p.abs().max()) for p in past.split(1 << 28)) == 0.0


def low_case(gpu, first, heads, tokens, rope=None):
    """One sequence whose key j has first[j] (an e4m3 value) as its first latent, 448 as its second, which holds the scale
    at one, and rope[j] as its first rotary value; queries see the first dimensions alone: -2^by of the token's head, of
    which scores below -10^30 are made."""
    n, page = len(first), 16
    pages = -(-n // page)
    kv = torch.zeros(n, 576, dtype=torch.bfloat16)
    kv[:, 0] = torch.tensor(first)
    kv[:, 1] = 448.0
    if rope is not None:
        kv[:, 512] = torch.tensor(rope)
    cache = torch.zeros(pages, page, 640, dtype=torch.uint8, device=gpu)
    scales = torch.full((pages, page), 127, dtype=torch.uint8, device=gpu)
    bfp8.latent_cache_write(kv.to(gpu), torch.arange(n, device=gpu), cache, scales)
    table = torch.arange(pages, dtype=torch.int32, device=gpu)[None]
    q = torch.zeros(tokens, heads, 576, dtype=torch.bfloat16)
    by = torch.tensor([108.0 + h % 5 for h in range(heads)])
    q[:, :, 0] = -torch.exp2(by)
    if rope is not None:
        q[:, :, 512] = -torch.exp2(by)
    return (q.to(gpu), cache, scales, table, torch.tensor([n], dtype=torch.int32, device=gpu), SCALE)


@pytest.mark.parametrize("tokens,heads", [(1, 1), (1, 16), (1, 64), (3, 48), (20, 64), (33, 40)])
@pytest.mark.parametrize("with_rope", [False, True])
def test_scores_below_every_common_bound(gpu, tokens, heads, with_rope):
    """Finite scores of -10^31 and less, in float32's range: each row's weights add up to one and lie, in equal shares, on
    the keys whose scores are highest (the next are 2^100 lower). Scores kept (1024 rows or fewer) and scored twice.

    Tolerance: a row's shares are 1 / n of equal scores, by one division and one product (2^-23), rows add up to rows *
    2^-24 relative."""
    n = 150
    first = [[1.0, 2.5, 1.0, 4.0, 28.0][j % 5] for j in range(n)]
    rope = [[1.0, 1.0, 8.0, 0.5, 2.0][j % 5] for j in range(n)] if with_rope else None
    args = low_case(gpu, first, heads, tokens, rope)
    cu = torch.tensor([0, tokens], dtype=torch.int32, device=gpu)
    announce("latent_attention_mass low scores", tokens, heads, with_rope)
    _, mass = bfp8.latent_attention_mass(*args, cu_q=cu)
    level = torch.tensor(first) + (torch.tensor(rope) if with_rope else 0.0)
    want = torch.zeros(n, dtype=torch.float64)
    for t in range(tokens):
        seen = level[:n - tokens + t + 1]
        best = (seen == seen.min()).double()
        want[:len(seen)] += heads * best / best.sum()
    got = mass[0, :n].double().cpu()
    assert bool((mass[0, n:] == 0).all())
    assert bool(((got - want).abs() <= want * (2.0 ** -22 + tokens * heads * 2.0 ** -24)).all()), (got - want).abs().max()


@pytest.mark.parametrize("tokens", [1, 40])
def test_low_scores_leave_other_rows_as_they_are(gpu, tokens):
    """Such rows beside ordinary ones of the same sequence: what the sequence gathers is one a row, and a sequence beside it
    gathers what it does without them."""
    lens, new, heads = [300, 200], [tokens, tokens], 40
    c, _ = make(gpu, lens, new, heads, 16, seed=63)
    args = (c["cache"], c["scales"], c["table"], c["lens"], SCALE)
    _, clean = bfp8.latent_attention_mass(c["q"], *args, cu_q=c["cu"])
    q = c["q"].clone()
    q[:tokens, ::3] *= 2.0 ** 104
    announce("latent_attention_mass low rows beside others", tokens)
    _, mass = bfp8.latent_attention_mass(q, *args, cu_q=c["cu"])
    assert torch.equal(mass[1], clean[1])
    assert abs(float(mass[0].double().sum()) - tokens * heads) <= 2.0 ** -15 * tokens * heads


@pytest.mark.parametrize("tokens,heads", [(1, 16), (20, 64)])
def test_scores_that_are_minus_infinity(gpu, tokens, heads):
    """A row all of whose scores are minus infinity has no softmax: NaN for the keys that it sees and no others. Where some
    are finite, the others' weights are zero."""
    n = 100
    args = low_case(gpu, [1.0] * 40 + [2.0] * 60, heads, tokens)
    cu = torch.tensor([0, tokens], dtype=torch.int32, device=gpu)
    q = args[0].clone()
    q[:, :, 0] = float("-inf")
    announce("latent_attention_mass minus infinity", tokens, heads)
    _, mass = bfp8.latent_attention_mass(q, *args[1:], cu_q=cu)
    assert bool(mass[0, :n].isnan().all()) and bool((mass[0, n:] == 0).all())
    q = args[0].clone()
    q[0, 0, 0] = float("-inf")  # the first new token does not see the others
    _, mass = bfp8.latent_attention_mass(q, *args[1:], cu_q=cu)
    seen = n - tokens + 1
    assert bool(mass[0, :seen].isnan().all()) and not bool(mass[0, seen:].isnan().any())
    # -2^127 * 2 passes float32 for the later keys alone
    q = args[0].clone()
    q[:, :, 0] = -2.0 ** 127
    _, mass = bfp8.latent_attention_mass(q, *args[1:5], 0.69, cu_q=cu)
    want = tokens * heads / 40
    assert bool(((mass[0, :40] - want).abs() <= want * (2.0 ** -22 + tokens * heads * 2.0 ** -24)).all())
    assert bool((mass[0, 40:] == 0).all())
