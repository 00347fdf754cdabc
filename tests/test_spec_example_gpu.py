"""The speculative decoding example, run as a user runs it."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "speculative_decode.py")
    spec = importlib.util.spec_from_file_location("speculative_decode", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_greedy_follows_the_dense_model(example):
    """Every emitted token is the dense float32 model's choice, up to what 16-bit activations
    move a logit: some ten roundings of 2^-8 on a path of unit size, under a tenth of the
    logits' spread."""
    model, seqs, starts, adapters, counts = example.decode(steps=8)
    for r, seq in enumerate(seqs):
        assert len(seq) - starts[r] == sum(counts[r])
        assert example.behind(model, seq, starts[r], *adapters[r]) < 0.1
    assert seqs[4] == seqs[0]            # a greedy sample forked from a greedy one
    assert sum(map(sum, counts)) > 8 * 5    # some drafts are accepted


def test_sampled_runs_and_repeats(example):
    a = example.decode(steps=6, temperature=0.7, seed=3)
    b = example.decode(steps=6, temperature=0.7, seed=3)
    assert a[1] == b[1] and a[4] == b[4]
    assert all(0 <= t < example.VOCAB for s in a[1] for t in s)
    assert sum(map(sum, a[4])) > 6 * 5
