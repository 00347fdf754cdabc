"""Verification of requests of a thousand nodes and more, against the oracle."""

import numpy as np
import pytest

from test_spec_gpu import _verify_case, _verify_check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("n", [1023, 1024, 1025, 2500])
def test_chain_accepted_to_its_end(drawn, n):
    c = _verify_case([4, n], 60, drawn, n, chain=True)
    c["u"][:] = 0.0                                  # every candidate with mass is taken
    assert _verify_check(c)[1] == n
    _verify_check(c, width=1100)
    c["u"][4 + n - 3] = np.nextafter(np.float32(1), np.float32(0))
    c["p"][4 + n - 4, c["tokens"][4 + n - 3]] = 0.0  # and one without mass is not
    assert _verify_check(c)[1] == n - 3


@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("n", [1023, 1024, 1025, 1600])
def test_children_far_from_their_parent(drawn, n):
    """The root's first child has no mass, and a long branch follows it; the root's other children
    are the last nodes, with children of their own."""
    for seed in range(6):
        c = _verify_case([3, n, 5], 80, drawn, seed, spread=1.0)
        c["trees"][1] = [-1, 0] + [int(i) for i in range(1, n - 8)] + [0] * 3 + \
            [n - 7, n - 5, n - 6, n - 4]
        assert len(c["trees"][1]) == n
        c["p"][3, c["tokens"][4]] = 0.0
        c["u"][3 + n - 7:3 + n] *= 0.7
        _verify_check(c)


@pytest.mark.parametrize("n,V", [(1023, 3000), (1025, 3000), (1026, 700), (1500, 9001), (2600, 3000)])
def test_many_candidates_of_one_node(n, V):
    """More candidates refused at one node than its list holds: they stay out of what is left, and
    count once however often they come."""
    for seed, top in ((0, 1.0), (1, 0.9), (2, 0.0)):
        rng = np.random.default_rng(seed)
        c = _verify_case([2, n], V, False, seed, spread=0.5, chain=True)
        c["trees"][1] = [-1] + [0] * (n - 1)
        c["tokens"][2:] = rng.permutation(np.arange(n) % V) if seed != 2 else \
            rng.integers(0, V, n)                    # repeated ones
        c["u"][:] = 1.0 - 2.0 ** -24
        if top < 1.0:
            c["u"][-1] = top                         # the last candidate may be taken
        for uf in (0.0, 0.5, float(np.nextafter(np.float32(1), np.float32(0)))):
            c["uf"][:] = uf
            _verify_check(c)
