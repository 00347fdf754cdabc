"""Arguments of the speculative decoding calls that have to be refused before a kernel follows
them, on the CPU."""

import pytest
import torch

from segmented_gather_gemm_amd import speculative


def test_workspace_of_a_caller_is_checked():
    """A workspace in host memory, on another device, or in pieces would be written by a kernel."""
    for dev in (0, -1):
        with pytest.raises(ValueError, match="workspace"):
            speculative._given_workspace(torch.zeros(64, dtype=torch.uint8), dev)
    with pytest.raises(TypeError, match="workspace"):
        speculative._given_workspace(bytes(64), 0)
