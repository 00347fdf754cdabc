"""Logits of the type's lowest value are numbers: they stay apart from -inf, NaN and what a grammar
does not allow.

Where the largest of a row stands n times beside numbers far below it, its weights are 1 and the others
0; the sum of n < 2^24 ones is n, and its inverse is rounded once: 2^-24 of 1 / n.
"""

import numpy as np
import pytest
import torch

from test_spec_gpu import DEV, _i32, _sgg

pytestmark = pytest.mark.gpu
LOW = torch.finfo(torch.float32).min


def probs(x, heat, **kw):
    n = x.shape[0]
    t = None if heat is None else torch.tensor([heat], device=DEV)
    return _sgg().spec_target_probs(x.to(DEV), _i32([0, n]), n, temperature=t, **kw)


def uniform(row, places):
    got, want = row.double().cpu().numpy(), np.zeros(row.numel())
    want[places] = 1.0 / len(places)
    assert (np.abs(got - want) <= 2.0 ** -24 * want).all(), np.abs(got - want).max()


@pytest.mark.parametrize("V", [1, 30, 2048, 5000])
@pytest.mark.parametrize("heat", [None, 0.5, 1e-30, 3.0])
def test_rows_of_the_lowest_value(V, heat):
    inf = float("inf")
    x = torch.full((6, V), LOW)
    x[1, 1:] = -inf                              # beside -inf
    x[2, :-1] = -inf
    x[3, :V // 2] = float("nan")
    x[4, V // 3] = 0.0                           # beside a number
    x[5] = -inf
    got = probs(x, heat)
    uniform(got[0], range(V))
    uniform(got[1], [0])
    uniform(got[2], [V - 1])
    uniform(got[3], range(V // 2, V))
    uniform(got[4], [V // 3])
    assert not got[5].any()


@pytest.mark.parametrize("V", [40, 5000])
def test_only_the_lowest_is_allowed(V):
    x = torch.full((2, V), LOW)
    x[:, ::3] = 1.0
    bits = torch.ones((2, V), dtype=torch.bool)
    bits[:, ::3] = False
    bits[:, :8] = False
    words = np.packbits(np.pad(bits.numpy(), ((0, 0), (0, -V % 32))), axis=1, bitorder="little")
    allowed = torch.from_numpy(words.view(np.int32)).to(DEV)
    at = [v for v in range(8, V) if v % 3]
    got = probs(x, 1.0, allowed=allowed)
    uniform(got[0], at)
    uniform(got[1], at)
    got = probs(x, 0.0, allowed=allowed)         # greedy: the first of them
    assert got.argmax(1).tolist() == [8, 8] and got.sum(1).tolist() == [1, 1]


def test_the_lowest_in_other_chunks_and_a_greedy_row():
    V = 7000
    x = torch.full((3, V), -float("inf"))
    x[0, 6500:] = LOW                            # chunks of nothing before and between
    x[1, 100], x[1, 6999] = LOW, LOW
    x[2] = LOW
    got = probs(x, 0.0)
    assert got.argmax(1).tolist() == [6500, 100, 0] and got.sum(1).tolist() == [1, 1, 1]
    got = probs(x, 1.0)
    uniform(got[0], range(6500, 7000))
    uniform(got[1], [100, 6999])
    uniform(got[2], range(V))
