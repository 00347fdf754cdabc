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


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("d", [64, 72, 128])
@pytest.mark.parametrize("q,skew", [(1, False), (4, False), (1, True), (4, True)])
def test_two_waves_a_workgroup(dtype, cache, d, q, skew):
    """Many requests of at most 16 rows; with a request far longer than the others the keys of all
    are cut into ranges, else each workgroup takes a request."""
    if cache and d == 72:
        d = 80
    rng = np.random.default_rng(d + q)
    kv = [int(x) for x in rng.integers(0, 150, 70)]
    kv[17] = 7000 if skew else 150
    ql = [q] + [int(x) for x in rng.integers(0, q + 1, 69)]
    ql[17] = q
    s = Setup(kv, ql, 32, 8, d, dtype=dtype, cache=cache, rows=True, seed=q,
              trees=[tree(n, rng) for n in ql] if q > 1 else None)
    at = shape(s, q, max(kv) + q)
    assert (at["rows"], at["keys"]) == (16, 64) and at["ranges"] > 1
    out = s.call()
    s.check(out)
    assert torch.equal(s.call(), out)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("bs,q,trees", [(300, 3, True), (700, 1, False), (520, 20, True),
                                        (1100, 40, False)])
def test_more_requests_than_threads(dtype, cache, bs, q, trees):
    """A thread of the scan over the batch has several requests, some of them empty."""
    rng = np.random.default_rng(bs)
    kv = [int(x) for x in rng.integers(0, 90, bs)]
    ql = [int(x) for x in rng.integers(0, q + 1, bs) * (rng.random(bs) < 0.4)]
    ql[3] = q
    kv[bs // 2], ql[bs // 2] = 3000, q
    s = Setup(kv, ql, 2, 2, 64, dtype=dtype, cache=cache, rows=True, seed=bs,
              trees=[tree(n, rng) for n in ql] if trees else None)
    s.check(s.call())
    s.check(s.call(max_q_len=1, max_kv_len=1))


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("d,bs,q,group,trees", [(64, 44, 40, 8, True), (128, 44, 40, 8, False),
                                                (256, 22, 40, 8, True), (256, 22, 40, 8, False),
                                                (96, 128, 80, 2, False)])
def test_a_workgroup_for_every_row_block(dtype, cache, d, bs, q, group, trees):
    """Batches with more row blocks than the GPU holds workgroups: no keys are cut."""
    rng = np.random.default_rng(d + bs)
    kv = [int(x) for x in rng.integers(0, 200, bs)]
    ql = [q] + [int(x) for x in rng.integers(0, q // 2, bs - 1)]
    ql[bs // 2], kv[bs // 2] = q, 700
    s = Setup(kv, ql, 8 * group if bs < 100 else 4 * group, 8 if bs < 100 else 4, d, dtype=dtype,
              cache=cache, seed=d, trees=[tree(n, rng) for n in ql] if trees else None)
    at = shape(s, q, max(kv) + q)
    assert at["ranges"] == 0 and q * group > at["rows"]
    out = s.call()
    s.check(out)
    assert torch.equal(s.call(), out)
