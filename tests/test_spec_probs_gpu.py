"""From logits to the target's probabilities, against the oracle.

Tolerance, relative to the probability p of a value whose x (before the softmax) lies z below the
row's largest, in units of the temperature T, with X the largest magnitude on the way to any x of
the row: x takes at most 7 roundings of 2^-24 X, twice in a difference, 2^-20 X / T; the exponent's
own roundings and the hardware's exponential 2^-21 + 2^-22 z; the same again for the sum, where z
counts with its probability and is below 32: 2^-18 + 2^-19 X / T + 2^-21 z in all.
"""

import numpy as np
import pytest
import torch

from oracle import latent as ola
from test_spec_gpu import DEV, _i32, _sgg, f64, tree

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _f32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.float32, device=DEV)


class Batch:
    def __init__(self, ql, V, dtype="fp32", history=40, seed=0, chain=False, pad=0, bias=True,
                 grammar=True):
        rng = self.rng = np.random.default_rng(seed)
        bs, n = len(ql), sum(ql)
        self.ql, self.V, self.ptr = ql, V, np.concatenate([[0], np.cumsum(ql)])
        wide = torch.from_numpy(rng.normal(size=(n, V + pad)) * 4).to(TYPES[dtype])
        self.logits = wide.to(DEV)[:, :V]
        self.trees = [tree(k, rng, chain) for k in ql]
        self.rows = rng.permutation(bs + 2)[:bs]
        self.text = rng.integers(-3, min(V + 3, 60), (bs + 2, history + 5))
        self.lens = rng.integers(0, history + 1, bs + 2)
        self.prompt = rng.integers(0, history + 1, bs + 2)
        self.tokens = rng.integers(0, min(V, 40), n)
        self.temp = np.where(rng.random(bs) < 0.25, 0.0, rng.uniform(0.4, 2.0, bs))
        self.rep, self.pres = rng.uniform(0.8, 1.6, bs), rng.uniform(-0.5, 1.0, bs)
        self.freq = rng.uniform(-0.2, 0.5, bs)
        k = rng.integers(0, min(V, 150), bs) if bias else np.zeros(bs, np.int64)
        self.bptr = np.concatenate([[0], np.cumsum(k)])
        self.bids = np.concatenate([rng.integers(-2, V + 2, j) for j in k] + [[]])   # some twice
        self.bval = rng.normal(size=len(self.bids)) * 3
        words = (V + 31) // 32
        self.bits = rng.random((n, 32 * words)) < 0.3 if grammar else None
        for name in ("temp", "rep", "pres", "freq", "bval"):
            setattr(self, name, getattr(self, name).astype(np.float32))

    def call(self, **kw):
        a = dict(temperature=_f32(self.temp), tokens=_i32(self.tokens),
                 parents=_i32(np.concatenate([t for t in self.trees if t] or [[]])),
                 history=_i32(self.text), history_lens=_i32(self.lens),
                 prompt_lens=_i32(self.prompt), rows=_i32(self.rows), repetition=_f32(self.rep),
                 presence=_f32(self.pres), frequency=_f32(self.freq), bias_indptr=_i32(self.bptr),
                 bias_ids=_i32(self.bids), bias_values=_f32(self.bval), allowed=None)
        if self.bits is not None:
            a["allowed"] = torch.from_numpy(
                np.packbits(self.bits, axis=1, bitorder="little").view(np.int32)).to(DEV)
        a.update(kw)
        return _sgg().spec_target_probs(self.logits, _i32(self.ptr), max(self.ql + [0]), **a)

    def request(self, r, **kw):
        at = slice(self.ptr[r], self.ptr[r + 1])
        row = self.rows[r]
        b = slice(self.bptr[r], self.bptr[r + 1])
        a = dict(tokens=self.tokens[at], parents=self.trees[r],
                 text=self.text[row][:self.lens[row]], prompt=self.prompt[row],
                 temperature=self.temp[r], repetition=self.rep[r], presence=self.pres[r],
                 frequency=self.freq[r], bias=list(zip(self.bids[b].astype(int),
                                                       self.bval[b].astype(float))),
                 allowed=None if self.bits is None else self.bits[at][:, :self.V])
        a.update(kw)
        return ola.target_probs(f64(self.logits[at]), **a), a["temperature"]

    def check(self, got, requests=None, **kw):
        for r in requests or range(len(self.ql)):
            (want, x), heat = self.request(r, **kw)
            y = f64(got[self.ptr[r]:self.ptr[r + 1]])
            if not heat > 0:
                assert np.array_equal(y, want), r
                continue
            logit = np.abs(f64(self.logits[self.ptr[r]:self.ptr[r + 1]]))
            extra = np.abs(self.bval[self.bptr[r]:self.bptr[r + 1]]).sum()
            for i in range(len(y)):
                fin = np.isfinite(x[i])
                if not fin.any():
                    assert np.array_equal(y[i], want[i])
                    continue
                X = 1.6 * logit[i].max() + 60 + extra
                z = np.where(fin, (x[i][fin].max() - np.where(fin, x[i], 0)) / heat, 0)
                tol = want[i] * (2.0 ** -18 + 2.0 ** -19 * X / heat + 2.0 ** -21 * z) + 1e-37
                assert (np.abs(y[i] - want[i]) <= tol).all(), (r, i, np.abs(y[i] - want[i]).max())


CASES = [
    # nodes, vocab, dtype, history, chain, pad
    ([1], 5, "fp32", 3, False, 0), ([5], 2048, "fp32", 40, True, 0),
    ([4, 0, 7], 2049, "bf16", 100, False, 0), ([3, 2], 4100, "fp16", 1000, False, 0),
    ([2, 3], 3001, "bf16", 50, False, 7), ([2], 6143, "fp32", 50, True, 1),
    ([40, 1], 2500, "fp32", 300, False, 0),      # groups of nodes
    ([50], 1000, "fp32", 20, True, 0),           # long paths of few values
    ([1] * 30, 777, "fp16", 64, False, 0),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_target_probs(case):
    ql, V, dtype, history, chain, pad = case
    s = Batch(ql, V, dtype, history, seed=V, chain=chain, pad=pad)
    got = s.call()
    s.check(got)
    assert torch.equal(s.call(), got)


def test_what_is_not_given_does_nothing():
    s = Batch([3, 2], 2100, seed=1, grammar=False)
    none = dict(temperature=None, repetition=None, presence=None, frequency=None, bias_indptr=None,
                bias_ids=None, bias_values=None)
    got = s.call(tokens=None, parents=None, history=None, history_lens=None, prompt_lens=None, **none)
    assert torch.allclose(got.double(), torch.softmax(s.logits.double(), 1), rtol=2.0 ** -16, atol=0)
    s.bids, s.bval = s.bids[:0], s.bval[:0]
    s.bptr[:] = 0
    # nodes alone, then the text alone, all of it since the prompt; no parents: a chain
    s.check(s.call(history=None, history_lens=None, prompt_lens=None), text=[], prompt=0)
    s.check(s.call(tokens=None, parents=None, prompt_lens=None), tokens=None, prompt=0)
    s.check(s.call(parents=None), parents=None)
    # rows given by the requests' own numbers
    s.rows = np.arange(2)
    s.check(s.call(rows=None))


def test_a_path_of_many_entries_in_one_chunk():
    """Over 32 nodes of a path in the same values: counted by walking it again."""
    s = Batch([90], 3000, seed=2, chain=True)
    s.tokens[:] = 7
    s.check(s.call(), temperature=s.temp[0])
    s = Batch([1100], 50, seed=3, chain=True, history=5)     # past the nodes kept in LDS
    s.check(s.call())


def test_ties_and_special_values():
    V = 5000
    s = Batch([6], V, "bf16", seed=4, bias=False, grammar=False)
    off = dict(repetition=None, presence=None, frequency=None, tokens=None, parents=None,
               history=None, history_lens=None, prompt_lens=None)
    x = torch.zeros((6, V))
    x[0, [4000, 17, 2050]] = 3.0                        # a tie: the first
    x[1] = float("-inf")
    x[2, 3] = float("nan")
    x[2, 100] = 1.0
    x[3, [5, 4999]] = float("inf")
    x[4] = float("nan")
    x[5, 8:] = float("-inf")
    s.logits = x.bfloat16().to(DEV)
    for heat in (0.0, -1.0, float("nan")):
        got = s.call(temperature=_f32([heat]), **off)
        first = got.argmax(1).tolist()
        assert [first[i] for i in (0, 2, 3, 5)] == [17, 100, 5, 0]
        assert got.sum(1).tolist() == [1, 0, 1, 1, 0, 1] and ((got == 0) | (got == 1)).all()
    for heat in (1.0, float("inf"), 1e-30):
        got = s.call(temperature=_f32([heat]), **off)
        assert not got.isnan().any()
        assert not got[1].any() and not got[4].any() and got[2, 3] == 0
        assert got[3, 5] == 0.5 and got[3, 4999] == 0.5 and got[3].sum() == 1
        assert torch.allclose(got[5, :8], torch.full((8,), 0.125, device=DEV)) and not got[5, 8:].any()
        if heat == 1e-30:
            assert torch.allclose(got[0, [17, 2050, 4000]], torch.tensor(1 / 3, device=DEV))
    # a mask that allows nothing, and one that allows one value
    bits = torch.zeros((6, (V + 31) // 32), dtype=torch.int32, device=DEV)
    bits[2, 4096 // 32] = 1
    got = s.call(temperature=_f32([1.0]), allowed=bits, **off)
    assert got[2, 4096] == 1 and got.sum() == 1


def test_bad_rows_and_what_is_left_alone():
    s = Batch([2, 3, 1], 2500, seed=5)
    want = s.call()
    out = torch.full((6, 2600), 9.0, device=DEV)
    got = s.call(out=out[:, 50:2550])
    assert torch.equal(got, want) and (out[:, :50] == 9).all() and (out[:, 2550:] == 9).all()
    # a row out of range has no text; boundaries that do not fit are no request
    rows = s.rows.copy()
    rows[1] = 99
    got = s.call(rows=_i32(rows))
    s.check(got, [1], text=[], prompt=0)
    assert torch.equal(got[:2], want[:2]) and torch.equal(got[5:], want[5:])
    out.fill_(9.0)
    for ptr in ([0, 7, 7, 7], [-1, 0, 0, 0], [3, 2, 2, 1]):
        _sgg().spec_target_probs(s.logits, _i32(ptr), 3, out=out[:, :2500])
    assert (out == 9.0).all()
    # rows behind the last request
    _sgg().spec_target_probs(s.logits, _i32([0, 2]), 2, out=out[:, :2500])
    assert not (out[:2, :2500] == 9.0).any() and (out[2:] == 9.0).all()
    # a bound below the longest request
    assert torch.equal(_sgg().spec_target_probs(s.logits, _i32([0, 6]), 0),
                       _sgg().spec_target_probs(s.logits, _i32([0, 6]), 6))


def test_probabilities_go_into_the_verification():
    """Logits, probabilities, verification in one stream: greedy candidates along the largest."""
    s = Batch([4, 4], 3000, seed=6, chain=True)
    s.temp[:] = 0.0
    p = s.call()
    top = p.argmax(1)
    # every draft is what the target says after its parent, but the second request's last
    tok = torch.from_numpy(s.tokens).int().to(DEV)
    for r in (0, 4):
        for i in range(3):
            s.tokens[r + i + 1] = int(top[r + i])
            p = s.call()
            top = p.argmax(1)
    tok = _i32(s.tokens)
    tok[7] = (tok[7] + 1) % 3000
    s.tokens[7] = int(tok[7])
    p = s.call()
    u, f = torch.full((8,), 0.5, device=DEV), torch.full((2,), 0.5, device=DEV)
    path, accept, nxt = _sgg().spec_verify(tok, _i32(np.concatenate(s.trees)), _i32(s.ptr), p, u, f, 4)
    assert accept.tolist() == [4, 3] and nxt.tolist() == [int(p[3].argmax()), int(p[6].argmax())]


def test_biases_of_one_value_are_added_in_their_order():
    """Sums whose float32 value depends on the order, several to a batch of 64 and across batches.

    The sums are exact copies, so what is left is the softmax: below 2^-18 of each as in check."""
    rng = np.random.default_rng(8)
    ids = rng.integers(0, 5, 333)
    values = rng.choice([1.0, -1.0, 2.0 ** 24, -2.0 ** 24, 0.25], 333).astype(np.float32)
    want, back = np.zeros(5, np.float32), np.zeros(5, np.float32)
    for i in range(333):
        want[ids[i]] += values[i]
        back[ids[332 - i]] += values[332 - i]
    assert (want != back).any()
    # down to a few units, so that every sum shows
    ids = np.concatenate([ids, np.arange(5)])
    values = np.concatenate([values, rng.integers(-2, 3, 5) - want]).astype(np.float32)
    want += values[333:]
    assert np.abs(want).max() <= 4
    got = _sgg().spec_target_probs(torch.zeros((1, 5), device=DEV), _i32([0, 1]), 1,
                                   bias_indptr=_i32([0, 338]), bias_ids=_i32(ids),
                                   bias_values=_f32(values))
    e = np.exp(want.astype(np.float64))
    assert (np.abs(f64(got[0]) - e / e.sum()) <= 2.0 ** -18 * e / e.sum()).all()


@pytest.mark.parametrize("V", [700, 5000])
def test_long_paths_of_many_values(V):
    """Paths of more values than a list holds, of trees and of chains with and without parents."""
    s = Batch([300, 3, 90], V, seed=9, chain=False, history=30)
    s.tokens = s.rng.integers(-2, V + 2, 393)
    s.check(s.call())
    s.trees = [list(range(-1, k - 1)) for k in s.ql]
    got = s.call()
    s.check(got)
    assert torch.equal(s.call(parents=None), got)
