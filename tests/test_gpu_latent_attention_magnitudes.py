"""GPU tests of latent attention with scores of every magnitude in float32's range: where all of a row's lie below -10^30."""

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
