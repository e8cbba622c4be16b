"""GPU tests of the accumulated attention weights at the ends of their ranges: the widest masses."""

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
