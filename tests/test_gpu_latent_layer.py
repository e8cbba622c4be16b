"""The example's layer: norm and quantization, projections, the cache and both forms of attention together.

The absorbed and the expanded form of a decoded token differ by roundings to bf16, each at most 2^-8 of a
value: the expanded keys and values, the absorbed query and output, and both forms' weights and outputs.
Uncorrelated, seven of them at 2^-8 / sqrt 3 each stay within 7 * 2^-8 of the norm."""

import pytest
import torch

from examples.latent_attention import run
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,heads,page", [((37, 130, 1, 64), 16, 16), ((3,), 8, 64), ((300, 2), 40, 37)])
def test_decoded_tokens_agree_in_both_forms(gpu, lens, heads, page):
    announce("latent layer", lens, heads, page)
    assert run(gpu, lens=lens, heads=heads, page=page, steps=3) <= 7 * 2.0 ** -8


def test_the_same_twice(gpu):
    announce("latent layer twice")
    torch.manual_seed(0)
    assert run(gpu, steps=2) == run(gpu, steps=2)
