"""The speculative decoding calls against the oracle, on the GPU.

Tolerance of the attention, per element, from the way it is computed.  With r
the half step of the 16-bit type (2^-8 bf16, 2^-11 fp16), A the sum of weight
times |value| and o the exact result:
  - the weights are rounded to 16 bits (relative r each):        r A
  - the result is rounded once:                                  r |o| (and half a subnormal)
  - a score is off by (D + 4) 2^-24 of its sum of |q k| and a few 2^-24 of
    itself, its exponential by 2^-21 (hardware exp2, argument):  2 e A, numerator and sum,
    e = (D + 4) 2^-24 sum|q k| + 2^-22 |s| + 2^-21
  - sums over S keys in 32 bits:                                 S 2^-24 A
Verification, masks and pages are whole numbers or moved rows: equal.
"""

import numpy as np
import pytest
import torch

from oracle import spec as osp

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}


def _sgg():
    import segmented_gather_gemm_amd as sgg
    return sgg


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32, device=DEV)


def _bits(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def f64(x):
    return x.detach().cpu().double().numpy()


def tree(n, rng, chain=False):
    return [-1 if i == 0 else i - 1 if chain else int(rng.integers(max(0, i - 5), i))
            for i in range(n)]


class Setup:
    """A batch over a paged cache with every row's pages in a random order, the slots that no
    token holds filled with NaN."""

    def __init__(self, kv, ql, hq, hkv, d, ps=16, dtype="bf16", cache=None, heads_first=False,
                 trees=None, seed=0, rows=False, fill=float("nan")):
        rng = self.rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        bs = len(kv)
        self.kv, self.ql, self.ps, self.hkv, self.d = kv, ql, ps, hkv, d
        self.rows = rng.permutation(bs + 2)[:bs] if rows else np.arange(bs)
        R = bs + 2 if rows else bs
        counts = [-(-(a + b) // ps) for a, b in zip(kv, ql)]
        pages = sum(counts) + 2
        width = max(max(counts), 1)
        table = np.full((R, width), 1 << 30)      # entries past the counts lie outside the pool
        order, at = rng.permutation(pages), 0
        for r, c in zip(self.rows, counts):
            table[r, :c] = order[at:at + c]
            at += c
        self.table = table
        lens = np.zeros(R, np.int64)
        lens[self.rows] = kv
        ct = TYPES[cache or dtype]
        shape = (pages, hkv, ps, d) if heads_first else (pages, ps, hkv, d)
        self.host = []                            # (bs) lists of (S, Hkv, D) in 64 bits
        self.dev = []
        scale = 12.0 if cache == "e4m3" else 1.0
        for _ in range(2):
            vals = [(torch.randn((a + b, hkv, d), generator=gen) * scale).to(ct)
                    for a, b in zip(kv, ql)]
            x = torch.full(shape, fill, dtype=torch.float32).to(ct)
            if heads_first:
                x = x.transpose(1, 2)
            for r, y in zip(self.rows, vals):
                pos = np.arange(len(y))
                if len(y):
                    _bits(x)[torch.from_numpy(table[r, pos // ps]), torch.from_numpy(pos % ps)] = \
                        _bits(y)
            self.host.append([f64(y) for y in vals])
            x = x.transpose(1, 2).contiguous().transpose(1, 2) if heads_first else x
            self.dev.append(x.to(DEV) if not heads_first
                            else x.transpose(1, 2).to(DEV).transpose(1, 2))
        self.ks = self.vs = None
        if cache == "e4m3":
            self.ks = torch.rand(hkv, generator=gen) * 0.05 + 0.05
            self.vs = torch.rand(hkv, generator=gen) * 0.05 + 0.05
        n = sum(ql)
        self.q = torch.randn((n, hq, d), generator=gen).to(TYPES[dtype])
        self.ptr = np.concatenate([[0], np.cumsum(ql)])
        self.trees = trees
        self.dtype, self.hq = dtype, hq
        self.lens = lens

    def seen(self, r):
        kv, n = self.kv[r], self.ql[r]
        m = np.ones((n, kv + n), bool)
        m[:, kv:] = osp.ancestors(self.trees[r]) if self.trees else np.tril(np.ones((n, n)))
        return m

    def mask(self, words=None):
        if self.trees is None:
            return None
        w = words or max(1, -(-max(self.ql) // 64))
        m = [osp.mask_words(osp.ancestors(t), w) for t in self.trees if len(t)]
        return torch.from_numpy(np.concatenate(m)).to(DEV)

    def call(self, **kw):
        a = dict(tree_mask=self.mask(), rows=None if len(self.rows) == len(self.lens) else
                 _i32(self.rows), max_q_len=max(self.ql),
                 max_kv_len=max(x + y for x, y in zip(self.kv, self.ql)))
        if self.ks is not None:
            a.update(k_scale=self.ks.to(DEV), v_scale=self.vs.to(DEV))
        a.update(kw)
        q = a.pop("q", None)
        return _sgg().spec_attention(self.q.to(DEV) if q is None else q, self.dev[0], self.dev[1],
                                     _i32(self.table), _i32(self.lens), _i32(self.ptr), **a)

    def check(self, out, scale=None, seen=None, only=None):
        scale = self.d ** -0.5 if scale is None else scale
        r16 = torch.finfo(TYPES[self.dtype]).eps / 2
        info = torch.finfo(TYPES[self.dtype])
        tiny = info.smallest_normal * info.eps      # the smallest subnormal
        got, q = f64(out), f64(self.q)
        for r in range(len(self.kv)):
            if only is not None and r not in only:
                continue
            k, v = self.host[0][r], self.host[1][r]
            if self.ks is not None:
                k = k * f64(self.ks)[None, :, None]
                v = v * f64(self.vs)[None, :, None]
            at = slice(self.ptr[r], self.ptr[r + 1])
            o, mag, prod, top = osp.attention(q[at], k, v,
                                              self.seen(r) if seen is None else seen(r), scale)
            e = (self.d + 4) * 2.0 ** -24 * prod + 2.0 ** -22 * top + 2.0 ** -21
            tol = r16 * (mag + np.abs(o)) + 2 * e[:, :, None] * mag + \
                len(k) * 2.0 ** -24 * mag + tiny
            bad = ~(np.abs(got[at] - o) <= tol)
            assert not bad.any(), (r, int(bad.sum()), np.abs(got[at] - o)[bad].max(),
                                   np.argwhere(bad)[:5].tolist())


def batch(bs, top, q, seed, trees=True):
    rng = np.random.default_rng(seed)
    kv = [int(x) for x in rng.integers(0, top + 1, bs)]
    kv[0] = top
    ql = [int(x) for x in rng.integers(1, q + 1, bs)]
    ql[0] = q
    return kv, ql, [tree(n, rng) for n in ql] if trees else None


# every instance of the kernel: row block (tokens x group) by head_dim by type
@pytest.mark.parametrize("dtype,cache", [("bf16", None), ("fp16", None), ("bf16", "e4m3"),
                                         ("fp16", "e4m3")])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q,group", [(1, 4), (4, 7), (13, 4), (30, 4), (20, 8)])
def test_attention_shapes(dtype, cache, d, q, group):
    kv, ql, trees = batch(3, 300, q, d + q, trees=q > 1)
    s = Setup(kv, ql, 2 * group, 2, d, dtype=dtype, cache=cache, trees=trees, seed=q)
    s.check(s.call())


@pytest.mark.parametrize("d,cache", [(8, None), (16, "e4m3"), (72, None), (80, "e4m3"), (96, None),
                                     (136, None), (192, None), (240, "e4m3")])
@pytest.mark.parametrize("q", [1, 9, 25])
def test_attention_odd_head_dims(d, cache, q):
    kv, ql, trees = batch(2, 150, q, d, trees=True)
    s = Setup(kv, ql, 6, 2, d, cache=cache, trees=trees, seed=d + q)
    s.check(s.call())


@pytest.mark.parametrize("ps", [1, 2, 8, 32, 128, 1024])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("q", [1, 6])
def test_attention_pages_and_layouts(ps, heads_first, q):
    kv, ql, trees = batch(3, 700, q, ps, trees=True)
    s = Setup(kv, ql, 12, 3, 64, ps=ps, trees=trees, heads_first=heads_first, rows=True, seed=ps)
    s.check(s.call())


@pytest.mark.parametrize("q", [2, 40, 65, 150])
@pytest.mark.parametrize("kv", [0, 1, 63, 200])
def test_attention_causal_chunks(q, kv):
    s = Setup([kv, kv + 1], [q, max(1, q // 2)], 8, 2, 64, dtype="fp16", seed=q + kv)
    s.check(s.call())


@pytest.mark.parametrize("n", [63, 64, 65, 130])
def test_attention_wide_trees(n):
    rng = np.random.default_rng(n)
    for kv in (0, 61, 129):
        s = Setup([kv], [n], 4, 2, 64, trees=[tree(n, rng)], seed=kv)
        s.check(s.call())


def test_attention_lengths_around_every_border():
    """Context lengths on both sides of tile, page and chunk borders, in one ragged batch."""
    kv = [0, 1, 15, 16, 17, 30, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513]
    for q, trees in ((1, False), (5, True)):
        rng = np.random.default_rng(q)
        s = Setup(kv, [q] * len(kv), 8, 2, 128, trees=[tree(q, rng) for _ in kv] if trees else None,
                  rows=True, seed=q)
        s.check(s.call())


@pytest.mark.parametrize("cache", [None, "e4m3"])
def test_attention_split_over_a_long_axis(cache):
    for q, group in ((1, 1), (3, 4), (17, 4)):
        rng = np.random.default_rng(q)
        s = Setup([5003, 2, 1200], [q, q, q], 2 * group, 2, 128, ps=64, cache=cache,
                  trees=[tree(q, rng) for _ in range(3)], seed=q)
        out = s.call()
        s.check(out)
        # bounds only shape the launch: too small, and far too large
        for mq, mkv in ((1, 1), (1, 6000), (q, 300), (300, 100000)):
            s.check(s.call(max_q_len=mq, max_kv_len=mkv))
        # the same bits on every run
        assert torch.equal(s.call(), out)


def test_attention_empty_requests_and_rows():
    rng = np.random.default_rng(0)
    trees = [tree(n, rng) for n in (3, 0, 2, 0)]
    s = Setup([40, 10, 0, 0], [3, 0, 2, 0], 8, 2, 64, trees=trees, seed=1)
    s.check(s.call())
    # a mask that leaves rows empty: with a context they see it, without one they are zero
    mask = s.mask()
    mask[1] = 0
    mask[3] = 0
    out = torch.full_like(s.q.to(DEV), 7.0)
    s.call(tree_mask=mask, out=out)

    def seen(r):
        m = s.seen(r)
        if r == 0:
            m[1, 40:] = False
        if r == 2:
            m[0] = False       # row 3 of the batch is token 0 of request 2
        return m
    s.check(out, seen=seen)
    assert not out[3].any()


def test_attention_any_mask():
    """A mask need not be a tree: tokens may see later ones; bits past the tokens mean nothing."""
    rng = np.random.default_rng(5)
    s = Setup([33, 0], [20, 9], 8, 2, 64, trees=[tree(20, rng), tree(9, rng)], seed=2)
    m = [rng.random((n, n)) < 0.5 for n in (20, 9)]
    words = np.concatenate([osp.mask_words(x, 1) for x in m])
    words |= np.int64(-1) << np.int64(25)
    out = s.call(tree_mask=torch.from_numpy(words).to(DEV))

    def seen(r):
        x = s.seen(r)
        x[:, s.kv[r]:] = m[r]
        return x
    s.check(out, seen=seen)
    # two words a row, the second empty
    two = np.concatenate([words & ((1 << 25) - 1), np.zeros_like(words)], 1)
    assert torch.equal(s.call(tree_mask=torch.from_numpy(two).to(DEV)), out)


@pytest.mark.parametrize("dtype,cache", [("bf16", None), ("fp16", None), ("bf16", "e4m3")])
@pytest.mark.parametrize("d,q,group", [(64, 7, 2), (128, 7, 8), (96, 7, 1), (128, 17, 8)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_attention_hidden_keys_hold_anything(dtype, cache, d, q, group, bad):
    """Infinities and NaN in a drafted token that only its own branch sees."""
    if cache and not np.isnan(bad):
        bad = float("nan")                     # the 8-bit type has no infinity
    par = [-1, 0, 0, 1, 2, 4, 0] + [0] * (q - 7)
    s = Setup([50, 0], [q, q], 2 * group, 2, d, dtype=dtype, cache=cache, trees=[par, par], seed=4)
    seen_by = osp.ancestors(par)[:, 2]         # token 2 and its descendants 4, 5
    for r in range(2):
        pos = s.kv[r] + 2
        page = int(s.table[s.rows[r], pos // s.ps])
        for x in s.dev:
            _bits(x)[page, pos % s.ps] = _bits(torch.full((2, d), bad).to(x.dtype).to(DEV))
        for x in s.host:
            x[r][pos] = bad
    out = s.call()
    got = f64(out)
    for r in range(2):
        rows = got[s.ptr[r]:s.ptr[r + 1]]
        assert np.isfinite(rows[~seen_by]).all()
        if np.isnan(bad):
            assert np.isnan(rows[seen_by]).all()
        else:
            assert not np.isfinite(rows[seen_by]).any()
    # the finite rows are right (the others are set to zero, a row that sees nothing)
    out[torch.from_numpy(np.tile(seen_by, 2)).to(DEV)] = 0

    def hidden(r):
        m = s.seen(r)
        m[seen_by] = False
        return m
    s.check(out, seen=hidden)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_attention_values_with_infinities_in_sight(dtype):
    """An infinite value in sight makes its column infinite, in a drafted key and in the context."""
    s = Setup([20], [3], 4, 2, 64, dtype=dtype, trees=[[-1, 0, 1]], seed=9)
    for pos, col in ((22, 3), (5, 10)):
        page = int(s.table[0, pos // 16])
        s.dev[1][page, pos % 16, :, col] = float("inf")
    got = f64(s.call())
    assert np.isinf(got[2, :, 3]).all() and np.isfinite(got[:2, :, 3]).all()
    assert np.isinf(got[:, :, 10]).all()
    rest = np.delete(got, [3, 10], axis=2)
    assert np.isfinite(rest).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("kv", [0, 70])
def test_attention_causal_rows_before_an_infinity(dtype, kv):
    """A causal call over several row blocks: an infinity in a drafted token's value and a NaN in
    its key reach the rows from that token on and no other, whichever steps a block sees in full."""
    s = Setup([kv], [200], 8, 2, 128, ps=16, dtype=dtype, seed=kv)
    want = s.call()
    s.check(want)
    for tok in (0, 31, 32, 150, 199):
        held = [x.clone() for x in s.dev]
        page, at = int(s.table[0, (kv + tok) // 16]), (kv + tok) % 16
        s.dev[1][page, at, 1, 5] = float("inf")
        s.dev[0][page, at, 0, 7] = float("nan")
        got = s.call()
        assert torch.equal(got[:tok], want[:tok])
        assert not torch.isfinite(got[tok, 4:, 5]).any()
        assert torch.isnan(got[tok:, :4]).all()
        keep = [c for c in range(128) if c != 5]
        assert torch.equal(got[:, 4:][..., keep], want[:, 4:][..., keep])
        s.dev = held
    assert torch.equal(s.call(), want)


def test_attention_large_scores():
    """Scores of thousands: the running maximum keeps the exponentials in range."""
    s = Setup([300], [4], 8, 2, 128, trees=[[-1, 0, 0, 1]], seed=3)
    out = s.call(scale=40.0)
    s.check(out, scale=40.0)
    out = s.call(scale=0.0)
    s.check(out, scale=0.0)
    out = s.call(scale=-0.5)
    s.check(out, scale=-0.5)


def test_attention_strided_q_and_out():
    """q as a slice of a packed qkv row, out as a slice of a wider one: only its columns change."""
    s = Setup([70, 9], [5, 3], 8, 2, 64, trees=[tree(5, np.random.default_rng(1)),
                                               tree(3, np.random.default_rng(2))], seed=6)
    n = 8
    packed = torch.randn((n, 8 * 64 + 4 * 64), dtype=torch.bfloat16, device=DEV)
    packed[:, :512] = s.q.to(DEV).reshape(n, 512)
    wide = torch.full((n, 10, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    s.call(q=packed[:, :512].view(n, 8, 64), out=wide[:, 1:9])
    s.check(wide[:, 1:9])
    assert (wide[:, 0] == 3).all() and (wide[:, 9] == 3).all()
    # heads outermost
    qt = s.q.to(DEV).transpose(0, 1).contiguous().transpose(0, 1)
    s.check(s.call(q=qt))


def test_attention_bad_page_ids_stay_inside():
    """Page ids outside the pool read some page of it; the other requests are right."""
    s = Setup([200, 100], [2, 2], 4, 2, 64, trees=[[-1, 0], [-1, 0]], seed=8, fill=0.0)
    s.table[0, 3] = -5
    s.table[0, 5] = 1 << 30
    out = s.call()
    s.check(out, only=[1])
    assert torch.isfinite(out).all()


def test_attention_offsets_past_32_bits():
    """A cache of over 4 GiB, its last pages in use."""
    pages, ps, hkv, d = (1 << 17) + 64, 16, 8, 128
    k = torch.empty((pages, ps, hkv, d), dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    assert k.numel() * 2 > 1 << 32
    s = Setup([500], [3], 16, hkv, d, trees=[[-1, 0, 0]], seed=7)
    n = s.dev[0].shape[0]
    k[pages - n:] = s.dev[0]
    v[pages - n:] = s.dev[1]
    s.table = s.table + (pages - n)
    s.dev = [k, v]
    s.check(s.call())


def test_attention_on_another_stream_and_in_a_graph():
    s = Setup([700, 30], [4, 2], 8, 2, 128, trees=[[-1, 0, 0, 1], [-1, 0]], seed=5)
    want = s.call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = s.call()
    side.synchronize()
    assert torch.equal(got, want)
    q, args = s.q.to(DEV), (s.dev[0], s.dev[1], _i32(s.table), _i32(s.lens), _i32(s.ptr))
    kw = dict(tree_mask=s.mask(), max_q_len=4, max_kv_len=704)
    sgg = _sgg()
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        sgg.spec_attention(q, *args, out=out, **kw)
    for i in range(3):
        q.copy_(s.q.to(DEV) if i != 1 else -s.q.to(DEV))
        eager = sgg.spec_attention(q, *args, **kw)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), i
    # lengths are device data: a replay follows them
    args[3].copy_(_i32([100, 7]))
    eager = sgg.spec_attention(q, *args, **kw)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)


# ------------------------------------------------------------------- verification

def _verify_case(ql, V, drawn, seed, chain=False, spread=5.0, flat=False):
    rng = np.random.default_rng(seed)
    n = sum(ql)
    logits = rng.normal(size=(n, V)) * spread
    guess = logits + rng.normal(size=(n, V))
    soft = lambda x: (np.exp(x - x.max(1, keepdims=True)) /                      # noqa: E731
                      np.exp(x - x.max(1, keepdims=True)).sum(1, keepdims=True)).astype(np.float32)
    p, q = soft(logits), soft(guess)
    trees = [tree(k, rng, chain) for k in ql]
    tokens = np.zeros(n, np.int64)
    at = 0
    for t in trees:
        for i, par in enumerate(t):
            if par >= 0:
                row = q[at + par].astype(np.float64)
                tokens[at + i] = rng.choice(V, p=row / row.sum())
        at += len(t)
    u = rng.random(n).astype(np.float32)
    uf = rng.random(len(ql)).astype(np.float32)
    return dict(ql=ql, trees=trees, tokens=tokens, p=p, q=q if drawn else None, u=u, uf=uf)


def _verify_call(c, width=None, workspace=None):
    sgg = _sgg()
    par = np.concatenate([np.asarray(t, np.int64) for t in c["trees"]] or [np.zeros(0)])
    return sgg.spec_verify(
        _i32(c["tokens"]), _i32(par), _i32(np.concatenate([[0], np.cumsum(c["ql"])])),
        torch.from_numpy(c["p"]).to(DEV), torch.from_numpy(c["u"]).to(DEV),
        torch.from_numpy(c["uf"]).to(DEV), width or max(max(c["ql"]), 1),
        draft_probs=None if c["q"] is None else torch.from_numpy(c["q"]).to(DEV),
        workspace=workspace)


def _verify_want(c, width=None):
    width = width or max(max(c["ql"]), 1)
    paths, counts, nxt, at = [], [], [], 0
    for r, (n, t) in enumerate(zip(c["ql"], c["trees"])):
        s = slice(at, at + n)
        path, x = osp.verify(c["tokens"][s], t, c["p"][s], None if c["q"] is None else c["q"][s],
                             c["u"][s], c["uf"][r], width)
        paths.append(path + [-1] * (width - len(path)))
        counts.append(len(path))
        nxt.append(x)
        at += n
    return (paths, counts, nxt)


def _verify_check(c, width=None, workspace=None):
    path, count, nxt = _verify_call(c, width, workspace)
    want = _verify_want(c, width)
    assert path.tolist() == want[0]
    assert count.tolist() == want[1]
    assert nxt.tolist() == want[2]
    return count.tolist()


@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("V", [1, 2, 63, 1000, 4097, 20011])
def test_verify_vocabularies(drawn, V):
    for seed in range(4):
        _verify_check(_verify_case([1, 5, 12, 2, 7], V, drawn, seed, chain=seed == 3))


@pytest.mark.parametrize("drawn", [False, True])
def test_verify_many_trees(drawn):
    counts = []
    for seed in range(12):
        rng = np.random.default_rng(seed)
        ql = [int(x) for x in rng.integers(0, 20, 24)]
        counts += _verify_check(_verify_case(ql, 301, drawn, seed, spread=1.0 + seed % 4))
    assert max(counts) >= 4 and counts.count(1) > 10     # paths of all lengths were met


@pytest.mark.parametrize("drawn", [False, True])
def test_verify_coins_at_the_ends(drawn):
    for u, uf in ((0.0, 0.0), (np.nextafter(np.float32(1), np.float32(0)),) * 2):
        c = _verify_case([6, 9], 500, drawn, 3)
        c["u"][:] = u
        c["uf"][:] = uf
        _verify_check(c)


def test_verify_greedy_rows():
    """Rows with all their mass on one token: the walk follows exactly those tokens."""
    c = _verify_case([9, 9, 1], 64, False, 5)
    best = c["p"].argmax(1)
    c["p"] = np.eye(64, dtype=np.float32)[best]
    assert _verify_check(c)
    at = 0
    for t in c["trees"]:                                  # make the first child right everywhere
        for i in range(len(t) - 1, 0, -1):
            c["tokens"][at + i] = best[at + t[i]]
        at += len(t)
    assert min(_verify_check(c)[:2]) > 1


@pytest.mark.parametrize("drawn", [False, True])
def test_verify_repeated_and_bad_tokens(drawn):
    """The same candidate twice, tokens outside the vocabulary, parents that are none."""
    c = _verify_case([8, 8], 40, drawn, 11, spread=1.0)
    c["trees"] = [[-1, 0, 0, 0, 0, 1, 2, 7], [-1, 0, 0, 5, -3, 0, 0, 0]]
    c["tokens"][:] = [0, 7, 7, 3, 7, 1, 1, 1, 0, -1, 40, 2, 2, 1 << 30, 5, 5]
    for seed in range(20):
        c["u"] = np.random.default_rng(seed).random(16).astype(np.float32) * 1.0
        c["uf"] = np.random.default_rng(seed).random(2).astype(np.float32)
        _verify_check(c)


@pytest.mark.parametrize("drawn", [False, True])
def test_verify_rows_that_hold_nothing(drawn):
    c = _verify_case([3, 3, 3], 100, drawn, 2)
    c["p"][0:3] = 0.0                                     # no mass: -1
    c["p"][3:6] = np.nan
    c["p"][3:6, 41] = 0.25                                # NaN counts as nothing
    c["p"][6:9, ::2] = np.inf
    _verify_check(c)
    if drawn:                                             # q covers p: the residual is empty
        c = _verify_case([2], 10, True, 1)
        c["q"][:] = 1.0
        c["tokens"][1] = 3
        c["u"][:] = 0.999
        _verify_check(c)


def test_verify_path_width_ends_the_walk():
    c = _verify_case([10], 30, False, 4, chain=True)
    c["u"][:] = 0.0                                       # every candidate with mass is taken
    for w in (1, 2, 5, 10, 14):
        assert _verify_check(c, w) == [min(w, 10)]


def test_verify_waits_end_without_the_others():
    """With no poll allowed, every workgroup adds up its request's parts by itself: the same
    results, and the same again afterwards (the counters are back at zero)."""
    sgg = _sgg()
    c = [_verify_case([9, 4, 12], 9000 + i, True, i, spread=2.0) for i in range(6)]
    want = [tuple(x.tolist() for x in _verify_call(x)) for x in c]
    assert want == [_verify_want(x) for x in c]
    old = sgg.spec_set_option("verify_spin_limit", 0)
    try:
        for x, w in zip(c, want):
            assert tuple(y.tolist() for y in _verify_call(x)) == w
    finally:
        sgg.spec_set_option("verify_spin_limit", old)
    for x, w in zip(c, want):
        assert tuple(y.tolist() for y in _verify_call(x)) == w


@pytest.mark.parametrize("drawn", [False, True])
@pytest.mark.parametrize("bs", [1, 3, 300])
def test_verify_batch_sizes(drawn, bs):
    """One request over many workgroups, and more requests than workgroups."""
    ql = [int(x) for x in np.random.default_rng(bs).integers(1, 9, bs)]
    for seed in range(3):
        _verify_check(_verify_case(ql, 30011 if bs < 10 else 1500, drawn, seed, spread=3.0))


def test_attention_and_verify_share_a_workspace():
    """Calls of both kinds in turn on one workspace: what has to be zero for one is not where
    the other leaves its partial results."""
    sgg = _sgg()
    s = Setup([40001, 700], [3, 2], 2, 1, 64, ps=64, trees=[tree(3, None, True), tree(2, None, True)],
              seed=4)
    want = s.call()
    s.check(want)
    many = _verify_case([int(x) for x in np.random.default_rng(1).integers(1, 5, 300)], 1500, True,
                        5, spread=3.0)
    few = _verify_case([9, 4, 12], 30011, True, 6, spread=2.0)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        for c in (many, few):
            _verify_check(c, workspace=ws)
            assert torch.equal(s.call(workspace=ws), want)


def test_verify_strided_rows_and_graph():
    sgg = _sgg()
    c = _verify_case([5, 7, 3], 777, True, 8)
    want = _verify_want(c)
    wide = torch.zeros((15, 2, 1000), device=DEV)
    wide[:, 0, :777] = torch.from_numpy(c["p"]).to(DEV)
    wide[:, 1, :777] = torch.from_numpy(c["q"]).to(DEV)
    par = _i32(np.concatenate([np.asarray(t) for t in c["trees"]]))
    args = (_i32(c["tokens"]), par, _i32([0, 5, 12, 15]), wide[:, 0, :777],
            torch.from_numpy(c["u"]).to(DEV), torch.from_numpy(c["uf"]).to(DEV), 7)
    path, count, nxt = sgg.spec_verify(*args, draft_probs=wide[:, 1, :777])
    assert (path.tolist(), count.tolist(), nxt.tolist()) == want
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = sgg.spec_verify(*args, draft_probs=wide[:, 1, :777])
    for i in range(4):
        c["u"] = np.random.default_rng(i).random(15).astype(np.float32)
        args[4].copy_(torch.from_numpy(c["u"]))
        for x in got:
            x.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        assert tuple(x.tolist() for x in got) == tuple(_verify_want(c)), i
        eager = sgg.spec_verify(*args, draft_probs=wide[:, 1, :777])
        assert all(torch.equal(a, b) for a, b in zip(got, eager))


# -------------------------------------------------------------------------- pages

def _pool(R, width, pages, ps, rng, held):
    table = rng.integers(-5, pages + 5, (R, width))
    counts, lens, refs = np.zeros(R, int), np.zeros(R, int), np.zeros(pages, int)
    order, at = rng.permutation(pages), 0
    for r in range(R):
        n = int(held[r])
        c = -(-n // ps)
        table[r, :c] = order[at:at + c]
        refs[table[r, :c]] = 1
        counts[r], lens[r] = c, n
        at += c
    return table, counts, lens, refs


def _same(pool, table, counts, lens, refs):
    assert counts.tolist() == pool.counts.tolist()
    assert lens.tolist() == pool.lens.tolist()
    assert refs.tolist() == pool.refs.tolist()
    assert table.tolist() == pool.table.tolist()


@pytest.mark.parametrize("pages,ps", [(40, 16), (5000, 1), (9000, 8)])
def test_resize_follows_the_oracle(pages, ps):
    sgg = _sgg()
    rng = np.random.default_rng(pages)
    R, width = 17, 30 if pages < 100 else 400
    held = rng.integers(0, 20 if pages < 100 else 150, R)
    state = _pool(R, width, pages, ps, rng, held)
    pool = osp.Pool(state[0], state[1], state[2], state[3], ps)
    table, counts, lens, refs = (_i32(x) for x in state)
    for step in range(12):
        n = int(rng.integers(1, R + 1))
        rows = rng.permutation(R)[:n]
        new = rng.integers(0, (40 if pages < 100 else 300), n)
        if step == 5:
            rows[0], new[n // 2] = R + 3, -1           # left alone
        if step == 7:
            new[0] = width * ps + 1
        commit = step % 2 == 0
        st = sgg.spec_kv_resize(table, counts, refs, _i32(rows), _i32(new), ps,
                                kv_lens=lens if commit else None)
        assert st.tolist() == list(pool.resize(rows, new, commit)), step
        _same(pool, table, counts, lens, refs)


@pytest.mark.parametrize("R,pages", [(300, 600), (3, 70000), (1500, 70000), (4096, 9000)])
def test_resize_many_rows_and_large_pools(R, pages):
    """The lowest free pages lie behind 32768 taken ones, or few are left."""
    sgg = _sgg()
    rng = np.random.default_rng(R)
    table, counts, lens, refs = _pool(R, 40, pages, 4, rng, np.zeros(R, int))
    refs[:] = 1                                   # held by nobody here
    refs[rng.permutation(pages)[:2 * R + 5] if pages < 10000 else
         np.r_[10:20, pages - 2 * R - 5:pages]] = 0
    pool = osp.Pool(table, counts, lens, refs, 4)
    table, counts, lens, refs = (_i32(x) for x in (table, counts, lens, refs))
    order = rng.permutation(R)
    for top, commit in ((9, True), (13, False), (5, True), (9, False), (1, True)):
        new = rng.integers(0, top, R)
        st = sgg.spec_kv_resize(table, counts, refs, _i32(order), _i32(new), 4,
                                kv_lens=lens if commit else None)
        assert st.tolist() == list(pool.resize(order, new, commit))
        _same(pool, table, counts, lens, refs)


@pytest.mark.parametrize("n,pages", [(2, 9000), (300, 2000), (1100, 5000)])
def test_fork_many_pairs(n, pages):
    sgg = _sgg()
    rng = np.random.default_rng(n)
    R, ps, d = 20 + n, 4, 8
    state = _pool(R, 30, pages, ps, rng, np.r_[rng.integers(0, 60, 20), np.zeros(n, int)])
    pool = osp.Pool(state[0], state[1], state[2], state[3], ps)
    table, counts, lens, refs = (_i32(x) for x in state)
    k, v = (torch.randint(-9, 9, (2, pages, ps, 1, d), device=DEV).to(torch.bfloat16)
            for _ in range(2))
    before = [x.cpu().clone() for x in (k, v)]
    src, dst = rng.integers(0, 20, n), 20 + rng.permutation(n)
    st = sgg.spec_kv_fork(k, v, table, counts, refs, lens, _i32(src), _i32(dst))
    missing, refused, copies = pool.fork(src, dst)
    assert st.tolist() == [missing, refused] == [0, 0]
    _same(pool, table, counts, lens, refs)
    for x, want in zip((k, v), before):
        for a, b, m in copies:
            want[:, b, :m] = want[:, a, :m]
        assert torch.equal(x.cpu(), want)


def test_resize_whole_rows_and_exhaustion():
    sgg = _sgg()
    rng = np.random.default_rng(1)
    R, ps, pages = 6, 4, 30
    state = _pool(R, 20, pages, ps, rng, [16, 9, 0, 0, 40, 3])
    pool = osp.Pool(state[0], state[1], state[2], state[3], ps)
    table, counts, lens, refs = (_i32(x) for x in state)
    for new in ([16, 9, 40, 40, 40, 3], [80, 0, 0, 0, 0, 36], [0] * 6, [80, 40, 0, 0, 0, 0]):
        st = sgg.spec_kv_resize(table, counts, refs, None, _i32(new), ps, kv_lens=lens)
        assert st.tolist() == list(pool.resize(range(R), new, True))
        _same(pool, table, counts, lens, refs)


@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("e4m3", 80), ("fp16", 8)])
def test_fork_shares_and_copies(heads_first, dtype, d):
    sgg = _sgg()
    rng = np.random.default_rng(d)
    R, ps, pages, L, H = 12, 8, 60, 3, 2
    state = _pool(R, 9, pages, ps, rng, [20, 8, 1, 0, 33, 0, 0, 0, 0, 0, 0, 0])
    pool = osp.Pool(state[0], state[1], state[2], state[3], ps)
    table, counts, lens, refs = (_i32(x) for x in state)
    shape = (L, pages, H, ps, d) if heads_first else (L, pages, ps, H, d)
    k, v = (torch.randint(0, 256, (*shape, TYPES[dtype].itemsize), dtype=torch.uint8, device=DEV)
            .view(TYPES[dtype]).reshape(shape) for _ in range(2))
    if heads_first:
        k, v = k.transpose(2, 3), v.transpose(2, 3)
    before = [x.contiguous().view(torch.uint8).cpu().clone() for x in (k, v)]
    # row 3 is empty; the last three pairs are left alone: dst not empty, out of range, itself
    src, dst = [0, 0, 1, 2, 3, 4, 4, 0, 2], [5, 6, 7, 8, 9, 10, 1, 12, 2]
    st = sgg.spec_kv_fork(k, v, table, counts, refs, lens, _i32(src), _i32(dst))
    missing, refused, copies = pool.fork(src, dst)
    assert copies and st.tolist() == [missing, refused] == [0, 3]
    _same(pool, table, counts, lens, refs)
    for x, old in zip((k, v), before):
        want = old.clone()
        for a, b, n in copies:
            want[:, b, :n] = old[:, a, :n]
        assert torch.equal(x.contiguous().view(torch.uint8).cpu(), want)


def test_fork_without_room_does_nothing():
    sgg = _sgg()
    rng = np.random.default_rng(2)
    state = _pool(8, 4, 7, 4, rng, [9, 5, 3, 0, 0, 0, 0, 0])
    pool = osp.Pool(state[0], state[1], state[2], state[3], 4)
    table, counts, lens, refs = (_i32(x) for x in state)
    k = torch.randn((2, 7, 4, 2, 64), device=DEV).bfloat16()
    v = k.clone()
    old = k.clone()
    for src, dst in (([0, 1, 2], [3, 4, 5]), ([0], [3])):
        st = sgg.spec_kv_fork(k, v, table, counts, refs, lens, _i32(src), _i32(dst))
        missing, refused, copies = pool.fork(src, dst)
        assert st.tolist() == [missing, refused]
        _same(pool, table, counts, lens, refs)
        for a, b, n in copies:
            old[:, b, :n] = old[:, a, :n].clone()
        assert torch.equal(k, old) and torch.equal(v, old)


@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("dtype,d,ps", [("bf16", 128, 16), ("e4m3", 16, 1), ("fp16", 24, 32)])
def test_copy_pages(heads_first, dtype, d, ps):
    sgg = _sgg()
    L, P, H = 2, 20, 3
    shape = (L, P, H, ps, d) if heads_first else (L, P, ps, H, d)
    k, v = ((torch.randn(shape, device=DEV) * 50).to(TYPES[dtype]) for _ in range(2))
    if heads_first:
        k, v = k.transpose(2, 3), v.transpose(2, 3)
    want = [x.contiguous().view(torch.uint8).clone() for x in (k, v)]
    src, dst = [3, 3, 0, 19, -1, 4, 20], [5, 6, 7, 8, 9, -2, 10]
    sgg.spec_kv_copy_pages(k, v, _i32(src), _i32(dst))
    for w, x in zip(want, (k, v)):
        for a, b in zip(src[:4], dst[:4]):
            w[:, b] = w[:, a].clone()
        assert torch.equal(x.contiguous().view(torch.uint8), w)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("cache", [None, "e4m3"])
@pytest.mark.parametrize("heads_first", [False, True])
def test_write_places_rows(dtype, cache, heads_first):
    sgg = _sgg()
    rng = np.random.default_rng(3)
    R, ps, P, H, d = 6, 8, 40, 3, 48
    lens = [0, 7, 8, 30, 5, 2]
    held = [x + 11 for x in lens]
    state = _pool(R, 6, P, ps, rng, held)
    rows, ql = [4, 1, 3, 0], [5, 0, 11, 1]
    n = sum(ql)
    new = (torch.randn((n, 2 * H, d), device=DEV) * 30).to(TYPES[dtype])
    knew, vnew = new[:, :H], new[:, H:]                       # strided
    shape = (P, H, ps, d) if heads_first else (P, ps, H, d)
    ct = TYPES[cache or dtype]
    k, v = ((torch.randn(shape, device=DEV) * 9).to(ct) for _ in range(2))
    if heads_first:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    want = [x.contiguous().view(torch.uint8).clone().view(ct) for x in (k, v)]
    scales = [torch.rand(H, device=DEV) + 0.01 for _ in range(2)] if cache else [None, None]
    sgg.spec_kv_write(knew, vnew, k, v, _i32(state[0]), _i32(lens),
                      _i32(np.concatenate([[0], np.cumsum(ql)])), rows=_i32(rows),
                      k_scale=scales[0], v_scale=scales[1])
    for w, x, y, s in zip(want, (k, v), (knew, vnew), scales):
        if cache:
            y = (y.float() / s[:, None]).clamp(-448, 448).to(ct)
        at = 0
        for r, m in zip(rows, ql):
            for i in range(m):
                pos = lens[r] + i
                w[int(state[0][r, pos // ps]), pos % ps] = y[at]
                at += 1
        assert torch.equal(x.contiguous().view(torch.uint8), w.view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_write_rounds_every_value_like_the_type(dtype):
    """All 65536 values of the 16-bit type through the 8-bit cache: nearest even, saturated,
    NaN kept."""
    sgg = _sgg()
    x = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(TYPES[dtype])
    x = x.to(DEV).view(32, 16, 128)
    k = torch.zeros((2, 16, 16, 128), dtype=torch.float8_e4m3fn, device=DEV)
    v = torch.zeros_like(k)
    one, third = torch.ones(16, device=DEV), torch.full((16,), 0.3, device=DEV)
    sgg.spec_kv_write(x, x, k, v, _i32([[1, 0]]), _i32([0]), _i32([0, 32]), k_scale=one,
                      v_scale=third)
    for got, s in ((k, one), (v, third)):
        want = (x.float() / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        got = torch.cat([got[1], got[0]])
        assert torch.equal(torch.isnan(got.float()), torch.isnan(want.float()))
        fine = ~torch.isnan(want.float())
        assert torch.equal(got.view(torch.uint8)[fine], want.view(torch.uint8)[fine])


def test_write_without_room_is_skipped():
    """Tokens whose position has no page leave the cache alone; the others land."""
    sgg = _sgg()
    k = torch.zeros((3, 4, 1, 64), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    x = torch.ones((6, 1, 64), dtype=torch.bfloat16, device=DEV)
    # row 0: pages 2 and one outside the pool; six tokens from position 3 on
    sgg.spec_kv_write(x, x, k, v, _i32([[2, 9]]), _i32([3]), _i32([0, 6]))
    assert k[2, 3].eq(1).all() and k.sum() == 64 and v.sum() == 64
    k.zero_()
    sgg.spec_kv_write(x, x, k, v, _i32([[2, 9]]), _i32([-9]), _i32([0, 6]))
    sgg.spec_kv_write(x, x, k, v, _i32([[2, 1]]), _i32([0]), _i32([0, 6]), rows=_i32([1]))
    assert not k.any()


@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("dtype,H,d", [("bf16", 8, 128), ("e4m3", 2, 64), ("fp16", 5, 40)])
def test_compact_moves_accepted_rows(heads_first, dtype, H, d):
    sgg = _sgg()
    rng = np.random.default_rng(d)
    R, ps, P, L = 7, 4, 80, 3
    lens = [0, 5, 3, 17, 30, 8, 1]
    state = _pool(R, 16, P, ps, rng, [x + 20 for x in lens])
    shape = (L, P, H, ps, d) if heads_first else (L, P, ps, H, d)
    k, v = ((torch.randn(shape, device=DEV) * 50).to(TYPES[dtype]) for _ in range(2))
    if heads_first:
        k, v = k.transpose(2, 3), v.transpose(2, 3)
    want = [x.contiguous().view(torch.uint8).clone().view(x.dtype) for x in (k, v)]
    rows = [3, 0, 6, 1, 5]
    paths = [[0, 1, 2, 7, 9, 19], [0], [], list(range(0, 20, 2)), [4, 5, 6]]
    W = 12
    path = np.full((5, W), -1)
    for i, w in enumerate(paths):
        path[i, :len(w)] = w
    new = sgg.spec_kv_compact(k, v, _i32(state[0]), _i32(lens), _i32(path),
                              _i32([len(w) for w in paths]), rows=_i32(rows))
    assert new.tolist() == [lens[r] + len(w) for r, w in zip(rows, paths)]
    place = lambda r, pos: (int(state[0][r, pos // ps]), pos % ps)                # noqa: E731
    for w, x in zip(want, (k, v)):
        for r, way in zip(rows, paths):
            for j, i in enumerate(way):
                a, b = place(r, lens[r] + i), place(r, lens[r] + j)
                w[:, b[0], b[1]] = w[:, a[0], a[1]].clone()
        assert torch.equal(x.contiguous().view(torch.uint8), w.view(torch.uint8))


def test_compact_skips_what_is_out_of_range():
    sgg = _sgg()
    k = torch.randn((1, 4, 4, 2, 64), device=DEV).bfloat16()
    v = torch.randn_like(k)
    old = [k.clone(), v.clone()]
    path = _i32([[0, 0, 3, -1], [0, 900, 1 << 30, 2], [0, 1, 2, 3]])
    new = sgg.spec_kv_compact(k, v, _i32([[0, 1], [2, -1], [3, 7]]), _i32([0, 0, 2]), path,
                              _i32([3, 4, -5]))
    assert new.tolist() == [3, 4, 2]
    for x, y in zip((k, v), old):
        y[0, 0, 2] = y[0, 0, 3].clone()          # row 0: path entry 3 -> place 2
        assert torch.equal(x, y)


@pytest.mark.parametrize("words", [1, 2, 3])
def test_tree_mask(words):
    sgg = _sgg()
    rng = np.random.default_rng(words)
    ql = [1, 0, 64, 65, 130, 7]
    trees = [tree(n, rng) if n else [] for n in ql]
    trees[5] = [-1, 5, 0, 3, -9, 2, 1 << 30]     # parents that are none
    lens, rows = [5, 0, 11, 2, 9, 0, 77], [3, 0, 1, 6, 2, 4]
    par = np.concatenate([np.asarray(t, np.int64) for t in trees])
    mask, pos = sgg.spec_tree_mask(_i32(par), _i32(np.concatenate([[0], np.cumsum(ql)])),
                                   _i32(lens), words, rows=_i32(rows))
    want = [osp.ancestors(t) for t in trees if t]
    assert torch.equal(mask.cpu(), torch.from_numpy(
        np.concatenate([osp.mask_words(m, words) for m in want])))
    depth = [m.sum(1) - 1 + lens[r] for m, r in zip(want, [r for r, n in zip(rows, ql) if n])]
    assert pos.tolist() == np.concatenate(depth).tolist()


def test_one_step_end_to_end():
    """reserve, write, attend, compact, commit, fork and release through PagedKVCache: after the
    step, ordinary attention over the accepted tokens equals attention over a cache that never
    held the others."""
    sgg = _sgg()
    torch.manual_seed(0)
    H, D, hq = 2, 64, 8
    c = sgg.PagedKVCache(2, 64, 8, H, D, 6, 8, device=DEV)
    rows, zero = _i32([4, 1]), _i32([0, 13, 26])
    first = [torch.randn((26, H, D), device=DEV).bfloat16() for _ in range(4)]
    assert c.reserve(rows, _i32([13, 13])).tolist() == [0, 0]
    for layer in range(2):
        c.write(layer, first[2 * layer], first[2 * layer + 1], zero, rows)
    c.commit(rows, _i32([13, 13]))
    par = _i32([-1, 0, 0, 2, 1, -1, 0, 1])
    ind = _i32([0, 5, 8])
    mask, pos = sgg.spec_tree_mask(par, ind, c.kv_lens, 1, rows=rows)
    assert pos.tolist() == [13, 14, 14, 15, 15, 13, 14, 15]
    c.reserve(rows, _i32([18, 16]))
    new = [torch.randn((8, H, D), device=DEV).bfloat16() for _ in range(4)]
    for layer in range(2):
        c.write(layer, new[2 * layer], new[2 * layer + 1], ind, rows)
        q = torch.randn((8, hq, D), device=DEV).bfloat16()
        tree_out = c.attention(layer, q, ind, 5, 18, tree_mask=mask, rows=rows)
        assert torch.isfinite(tree_out).all()
    lens = c.compact(_i32([[0, 2, 3, -1, -1], [0, 1, 2, -1, -1]]), _i32([3, 3]), rows=rows)
    assert lens.tolist() == [16, 16]
    c.commit(rows, lens)
    assert c.page_counts.tolist() == [0, 2, 0, 0, 2, 0] and int(c.ref_counts.sum()) == 4
    # the same tokens in a cache of their own
    d = sgg.PagedKVCache(2, 64, 8, H, D, 2, 8, device=DEV)
    d.reserve(None, _i32([16, 16]))
    pick = [0, 2, 3, 5, 6, 7]
    for layer in range(2):
        for i in (0, 1):
            full = [torch.cat([first[2 * layer + i][13 * r:13 * r + 13],
                               new[2 * layer + i][pick[3 * r:3 * r + 3]]]) for r in range(2)]
            if i == 0:
                ks = torch.cat(full)
            else:
                vs = torch.cat(full)
        d.write(layer, ks, vs, _i32([0, 16, 32]))
    for x, y, r, t in ((c.k, d.k, 4, 0), (c.k, d.k, 1, 1), (c.v, d.v, 4, 0), (c.v, d.v, 1, 1)):
        for pg in range(2):
            assert torch.equal(x[:, int(c.page_table[r, pg])], y[:, int(d.page_table[t, pg])])
    # a fork goes on without touching its source
    assert c.fork(_i32([4, 4]), _i32([0, 2])).tolist() == [0, 0]
    assert c.kv_lens.tolist() == [16, 16, 16, 0, 16, 0]
    c.commit(_i32([0, 2, 4, 1]), _i32([0, 0, 0, 0]))
    assert not c.ref_counts.any() and not c.page_counts.any() and not c.kv_lens.any()
