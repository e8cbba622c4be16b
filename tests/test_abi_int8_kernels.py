"""CPU tests of what the library says about the integer product's kernels, and of the linear layer's workspace."""

import pytest

import block_scaled_fp8_bfp8_amd as bfp8
from block_scaled_fp8_bfp8_amd import _native

# LDS stages of a tile, or slots of a wave that shares K with seven others
STAGES = {("tiled", 256, 256): 2, ("tiled", 256, 128): 3, ("tiled", 128, 256): 3, ("tiled", 128, 128): 4, ("tiled", 64, 128): 4,
          ("tiled", 64, 64): 4, ("split_k", 16, 16): 2, ("split_k", 16, 32): 2, ("split_k", 32, 16): 3, ("split_k", 32, 32): 2,
          ("split_k", 64, 16): 1, ("split_k", 32, 64): 1, ("split_k", 64, 64): 1}
# For every kernel a K of more blocks than twice its stages (for each of eight waves, more than its slots), a multiple of the
# block's 128 and none.
LONG = [
    (("tiled", 256, 256), 4764, 1668, 768), (("tiled", 256, 256), 2316, 3381, 672), (("tiled", 256, 128), 4138, 1682, 1024),
    (("tiled", 256, 128), 1650, 3750, 960), (("tiled", 128, 256), 2313, 1682, 1152), (("tiled", 128, 256), 1719, 2323, 928),
    (("tiled", 128, 128), 1108, 1823, 1408), (("tiled", 128, 128), 1180, 1694, 1168), (("tiled", 64, 128), 1338, 808, 1280),
    (("tiled", 64, 128), 1082, 1003, 1168), (("tiled", 64, 64), 473, 1034, 1408), (("tiled", 64, 64), 529, 899, 1200),
    (("split_k", 16, 16), 1, 1, 3456), (("split_k", 16, 16), 1, 1, 3344), (("split_k", 16, 32), 218, 361, 3456),
    (("split_k", 16, 32), 145, 405, 3408), (("split_k", 32, 16), 289, 244, 4736), (("split_k", 32, 16), 365, 182, 4368),
    (("split_k", 32, 32), 284, 470, 3584), (("split_k", 32, 32), 310, 410, 3408), (("split_k", 64, 16), 335, 753, 2560),
    (("split_k", 64, 16), 324, 760, 2496), (("split_k", 32, 64), 732, 361, 2432), (("split_k", 32, 64), 559, 458, 2416),
    (("split_k", 64, 64), 738, 703, 2432), (("split_k", 64, 64), 513, 949, 2352),
]


@pytest.mark.parametrize("kernel", STAGES)
def test_long_sizes_reach_every_kernel(kernel):
    rest = set()
    for _, m, n, k in [c for c in LONG if c[0] == kernel]:
        assert bfp8.gemm_int8_kernel_for(m, n, k) == kernel
        blocks, stages = -(-k // 128), STAGES[kernel]
        assert blocks >= 2 * stages + 2 if kernel[0] == "tiled" else blocks // 8 > stages
        rest.add(k % 128 > 0)
    assert rest == {False, True}


def test_sizes_without_a_kernel():
    assert bfp8.gemm_int8_kernel_for(0, 64, 128) is None and bfp8.gemm_int8_kernel_for(4, 0, 128) is None
    assert bfp8.gemm_int8_kernel_for(4, 64, 120) is None and bfp8.gemm_int8_kernel_for(4, 64, 65552) is None
    assert bfp8.gemm_int8_kernel_for(1 << 30, 1, 128) is None and bfp8.gemm_int8_kernel_for(4, (1 << 26) + 1, 128) is None
    assert bfp8.gemm_int8_kernel_for(1, 1, 16) == ("split_k", 16, 16) and bfp8.gemm_int8_kernel_for(8192, 10240, 5120) == ("tiled", 256, 256)


def test_linear_workspace_of_padded_rows():
    """Codes lie in rows of whole 128-byte lines, then the scales, each from a multiple of 256 bytes on."""
    size = _native.lib().bfp8_linear_int8_workspace_bytes
    for m, k in ((3, 16), (3, 144), (1000, 4112), (7, 65520), (5, 128), (64, 6832)):
        row = -(-k // 128) * 128
        assert size(m, k) == -(-m * row // 256) * 256 + -(-m * 4 // 256) * 256 == bfp8.linear_int8_workspace_bytes(m, k)
