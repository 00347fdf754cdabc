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


def test_bounded_writes_need_the_counts():
    """spec_kv_write_held and spec_kv_compact_held refuse what the plain calls refuse, and a
    missing page_counts."""
    import struct

    from segmented_gather_gemm_amd import _lib
    calls, F = _lib.spec_calls(), 0x10000
    cache = struct.pack("=QQ4q4qq6i", F, F, *((0, 16384, 1024, 128) * 2), 64, 1, 16, 8, 128, 0, 0)

    def write(table=F, counts=F, bs=2, c=cache):
        return calls.spec_kv_write_held(F, 1024, 128, F, 1024, 128, 0, c, table, 8, 8, 4, counts, F,
                                        F, F, bs, 4, 0, 0, 0)

    def compact(table=F, counts=F, bs=2, c=cache):
        return calls.spec_kv_compact_held(c, table, 8, 8, 4, counts, F, F, F, 4, 4, F, F, bs, 0)
    for call in (write, compact):
        for kw, text in ((dict(counts=0), "page_counts"), (dict(table=0), "page_table"),
                         (dict(bs=-1), "negative"), (dict(c=0), "cache")):
            assert call(**kw) == -1 and text in _lib.lib().lora_last_error().decode()
        assert call(bs=0) == 0
