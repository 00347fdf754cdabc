"""Paths of many values of one chunk, in trees of every order; tolerances as in test_spec_probs_gpu."""

import numpy as np
import pytest
import torch

from test_spec_gpu import DEV, _i32, _sgg
from test_spec_probs_gpu import Batch

pytestmark = pytest.mark.gpu


def branches(n, k):
    """k branches from the root, their nodes in turn."""
    return [-1] + [max(i - k, 0) for i in range(1, n)]


def one_after_another(n, k):
    """k branches from the root, each whole before the next."""
    per = max(1, (n - 1 + k - 1) // k)
    return [-1] + [0 if (i - 1) % per == 0 else i - 1 for i in range(1, n)]


def roots(n):
    """Chains of 50 under roots of their own, parents that are none among them."""
    return [(-1, i, n + 3, -7)[i // 50 % 4] if i % 50 == 0 else i - 1 for i in range(n)]


def back(n, rng):
    """A chain whose nodes go back now and then."""
    return [-1] + [i - 1 if rng.random() < 0.9 else int(rng.integers(max(0, i - 40), i))
                   for i in range(1, n)]


@pytest.mark.parametrize("V", [3, 50, 2600])
@pytest.mark.parametrize("shape", ["two", "five", "whole", "roots", "back"])
def test_long_paths_of_trees(shape, V):
    s = Batch([330, 1, 75], V, seed=V, history=20)
    make = {"two": lambda n: branches(n, 2), "five": lambda n: branches(n, 5),
            "whole": lambda n: one_after_another(n, 3), "roots": roots,
            "back": lambda n: back(n, s.rng)}[shape]
    s.trees = [make(n) for n in s.ql]
    # values that fall into the first chunk for some nodes and outside of the vocabulary for others
    s.tokens = np.where(s.rng.random(406) < 0.8, s.rng.integers(0, min(V, 9), 406),
                        s.rng.integers(-2, V + 2, 406))
    got = s.call()
    s.check(got)
    assert torch.equal(s.call(), got)


def test_long_and_short_paths_in_turn():
    """Two branches in turn: one's values all in the chunk, the other's outside of the vocabulary."""
    s = Batch([200], 1500, seed=1, history=0)
    s.trees = [branches(200, 2)]
    s.tokens = np.where(np.arange(200) % 2 == 0, s.rng.integers(0, 1500, 200), -1)
    s.check(s.call())


def test_past_the_nodes_kept_in_lds():
    s = Batch([1300], 40, seed=2, history=0)
    for tree in (branches(1300, 3), list(range(-1, 1299))):
        s.trees = [tree]
        s.check(s.call())


def test_a_chain_given_by_its_parents_takes_little_longer_than_one_given_by_none():
    """4096 nodes of one chunk: 100 times as long where one thread walks every node's path, about 5
    where a node that follows the last one adds itself to that one's counts."""
    n, V = 4096, 1000
    x = torch.zeros((n, V), device=DEV)
    tok, ptr = torch.arange(n, dtype=torch.int32, device=DEV) % 40, _i32([0, n])
    presence = torch.full((1,), 0.1, device=DEV)
    parents = torch.arange(-1, n - 1, dtype=torch.int32, device=DEV)

    def least(parents):
        times = []
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            got = _sgg().spec_target_probs(x, ptr, n, tokens=tok, parents=parents, presence=presence)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times), got

    (chain, p), (none, q) = least(parents), least(None)
    assert torch.equal(p, q) and chain < 20 * none, (chain, none)
