"""Arguments of the speculative decoding calls that have to be refused before a kernel follows
them, on the CPU."""

import types

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


def test_fork_compares_the_devices_of_cache_and_table(monkeypatch):
    """Two devices stand in for each other here: the cache's own checks are passed over."""
    monkeypatch.setattr(speculative, "_cache", lambda k, v: (b"", (1, 4, 16, 2, 64)))
    cache, table = (types.SimpleNamespace(get_device=lambda d=d: d) for d in (1, 0))
    with pytest.raises(ValueError, match="device"):
        speculative.spec_kv_fork(cache, cache, table, *[None] * 5)
