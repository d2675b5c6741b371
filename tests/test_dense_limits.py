"""Sizes at the ends of int's range, refused or taken on the host without a GPU."""
import pytest
import torch

import mixture_experts_fp32_b200 as moe
from mixture_experts_fp32_b200 import build as moe_build


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.load()


@pytest.mark.parametrize("gated", [0, 1])
def test_quantise_columns_whose_groups_would_overflow(lib, gated):
    """ceil(cols / 128) takes cols + 127: columns above 2^31 - 128 are refused as a shape, before a
    device is looked for; those below get as far as the device."""
    def call(cols):
        return lib.moe_quantize_groups(0x1000, moe.MOE_T_BF16, 1, cols, 2 * 2 ** 31, gated, None,
                                       0x8000, 0x9000, None)

    most = 2 ** 31 - 128
    for cols in (2 ** 31 - 16, 2 ** 31 - 112):
        assert call(cols) == moe.MOE_ERR_UNSUPPORTED
    assert call(most + 8) == moe.MOE_ERR_UNSUPPORTED       # no multiple of 16 either way
    if not torch.cuda.is_available():                      # the addresses above are made up
        assert call(most) == moe.MOE_ERR_CUDA
