"""Attention over the paged cache on paths that take particular batches: against the oracle,
with the shape of the launch that each case is meant for read from the library."""

import ctypes

import numpy as np
import pytest
import torch

from segmented_gather_gemm_amd import _lib
from test_spec_gpu import Setup, tree

pytestmark = pytest.mark.gpu

TYPES = [("bf16", None), ("fp16", None), ("bf16", "e4m3"), ("fp16", "e4m3")]


def shape(s, q, kv):
    """The division of the work that the host computes for the batch of a Setup."""
    out = (ctypes.c_int64 * 6)()
    fn = ctypes.CDLL(_lib.LIB).sgg_spec_attention_shape
    fn.argtypes = [ctypes.c_int32] * 6 + [ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)]
    fn(len(s.kv), s.hq, s.hkv, s.d, s.dev[0].element_size(), q, kv, out)
    return dict(zip(("rows", "keys", "min_tiles", "ranges", "slots", "grid"), out))


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("d,q,group,hkv,kv", [(64, 1, 4, 1, 40001), (128, 7, 4, 2, 20011),
                                              (128, 13, 4, 3, 20011), (256, 3, 4, 1, 20011),
                                              (256, 15, 4, 1, 20011)])
def test_pieces_joined_in_two_levels(dtype, cache, d, q, group, hkv, kv):
    """A request in more pieces than one level joins, for every way in which waves share rows
    and keys: a piece that goes on to the second level writes into a slot that was read in the
    first."""
    rng = np.random.default_rng(d + q)
    s = Setup([kv], [q], hkv * group, hkv, d, ps=64, dtype=dtype, cache=cache,
              trees=[tree(q, rng)], seed=q)
    assert shape(s, q, kv + q)["ranges"] > 32
    out = s.call()
    s.check(out)
    for _ in range(3):
        assert torch.equal(s.call(), out)
