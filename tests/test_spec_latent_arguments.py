"""CPU tests of arguments of the calls over latents: what is not looked at may be left out, and what
is given has to be known."""

import pytest
import torch

import segmented_gather_gemm_amd as sgg
from test_spec_capi import BF16, C, E4M3, FP16, _err


@pytest.mark.parametrize("dtype", [-1, 3, 99])
def test_workspace_of_an_unknown_cache_type(dtype):
    size = C.spec_latent_attention_workspace_bytes
    assert size(4, 16, 512, dtype, 1, 5000) == -1 and "cache dtype" in _err()


def test_workspace_of_every_cache_type():
    size = C.spec_latent_attention_workspace_bytes
    for dtype in (BF16, FP16, E4M3):
        assert size(4, 16, 512, dtype, 1, 5000) > 0
    # 8-bit latents come in pieces of 16
    assert size(4, 16, 504, BF16, 1, 5000) > 0 and size(4, 16, 504, E4M3, 1, 5000) == -1


def test_prefill_needs_no_bound_of_the_keys():
    """Nothing is divided over the keys, so that a bound of theirs shapes nothing."""
    x, i = torch.zeros((2, 2, 64), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    for bound in ((), (5,)):
        with pytest.raises(ValueError, match="ROCm"):
            sgg.spec_latent_prefill(x, x, x, x[0], i, i, 1, *bound)
