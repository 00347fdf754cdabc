"""Attention over a paged cache of latents and over expanded latents, against the oracle.

Tolerance per element as derived in test_spec_gpu, with the D = latent + rope (or nope + rope)
columns of a score: r A for the rounded weights, r |o| for the result, 2 e A for the exponentials,
e = (D + 4) 2^-24 sum|q k| + 2^-22 |s| + 2^-21, S 2^-24 A for the sums.
"""

import numpy as np
import pytest
import torch

from oracle import spec as osp
from test_spec_gpu import DEV, TYPES, _bits, _i32, _sgg, f64, tree

pytestmark = pytest.mark.gpu

STEP = {"bf16": (2.0 ** -8, 2.0 ** -134), "fp16": (2.0 ** -11, 2.0 ** -25)}


def hold(got, q, k, v, seen, scale, dtype, unit=1.0):
    """got (T, H, dv) against the oracle of q (T, H, D), k (S, Hkv, D), v (S, Hkv, dv)."""
    o, mag, prod, top = osp.attention(q, k * unit, v * unit, seen, scale)
    half, tiny = STEP[dtype]
    D, S = q.shape[2], k.shape[0]
    e = (D + 4) * 2.0 ** -24 * prod + 2.0 ** -22 * top + 2.0 ** -21
    tol = half * (mag + np.abs(o)) * (1 + half) + (2 * e + S * 2.0 ** -24)[:, :, None] * mag + tiny
    off = np.abs(got - o)
    assert (off <= tol).all(), (float((off - tol).max()), np.argwhere(~(off <= tol))[:4].tolist())


class Latents:
    """A batch over a paged cache of latents, pages in random order, slots of no token NaN."""

    def __init__(self, kv, ql, H, latent=512, rope=64, ps=16, dtype="bf16", cache=None, trees=None,
                 seed=0, spread=1.0):
        rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        bs = len(kv)
        self.kv, self.ql, self.dtype, self.trees, self.latent = kv, ql, dtype, trees, latent
        self.rows = rng.permutation(bs + 1)[:bs]
        counts = [-(-(a + b) // ps) for a, b in zip(kv, ql)]
        pages = sum(counts) + 1
        self.table = np.full((bs + 1, max(counts + [1])), 1 << 30)
        order, at = rng.permutation(pages), 0
        self.lens = np.zeros(bs + 1, np.int64)
        x = torch.full((pages, ps, latent + rope), float("nan")).to(TYPES[cache or dtype])
        self.host = []
        for row, c, a, b in zip(self.rows, counts, kv, ql):
            self.table[row, :c] = order[at:at + c]
            self.lens[row], at = a, at + c
            y = (torch.randn((a + b, latent + rope), generator=gen)
                 * (12.0 if cache else spread)).to(x.dtype)
            p = np.arange(a + b)
            if a + b:
                _bits(x)[torch.from_numpy(self.table[row, p // ps]), torch.from_numpy(p % ps)] = \
                    _bits(y)
            self.host.append(f64(y))
        self.cache = x.to(DEV)
        self.unit = torch.tensor([0.07]) if cache else None
        self.ptr = np.concatenate([[0], np.cumsum(ql)])
        self.q = torch.randn((int(self.ptr[-1]), H, latent + rope), generator=gen).to(TYPES[dtype])
        self.scale = (128 + rope) ** -0.5

    def seen(self, r):
        kv, n = self.kv[r], self.ql[r]
        m = np.ones((n, kv + n), bool)
        m[:, kv:] = osp.ancestors(self.trees[r]) if self.trees else np.tril(np.ones((n, n)))
        return m

    def mask(self):
        if self.trees is None:
            return None
        w = max(1, -(-max(self.ql) // 64))
        m = [osp.mask_words(osp.ancestors(t), w) for t in self.trees if len(t)]
        return torch.from_numpy(np.concatenate(m)).to(DEV)

    def call(self, **kw):
        a = dict(tree_mask=self.mask(), max_q_len=max(self.ql), rows=_i32(self.rows),
                 max_kv_len=max(x + y for x, y in zip(self.kv, self.ql)),
                 cache_scale=None if self.unit is None else self.unit.to(DEV), scale=self.scale,
                 q=self.q.to(DEV), page_table=_i32(self.table), kv_lens=_i32(self.lens),
                 q_indptr=_i32(self.ptr))
        a.update(kw)
        return _sgg().spec_latent_attention(cache=self.cache, latent_dim=self.latent, **a)

    def check(self, got, requests=None, scale=None, tokens=None):
        got = f64(got)
        for r in requests or range(len(self.kv)):
            at = slice(self.ptr[r], self.ptr[r + 1])
            pick = slice(None) if tokens is None else tokens
            k = self.host[r][:, None]
            hold(got[at][pick], f64(self.q[at])[pick], k, k[:, :, :self.latent],
                 self.seen(r)[pick], self.scale if scale is None else scale, self.dtype,
                 1.0 if self.unit is None else float(self.unit))


CASES = [
    # kv, ql, heads, latent, rope, ps, dtype, cache, tree
    ([0], [1], 16, 512, 64, 16, "bf16", None, False),
    ([31], [1], 1, 512, 64, 16, "bf16", None, False),
    ([500], [1], 16, 512, 64, 16, "fp16", None, False),
    ([17, 0, 64, 300], [1, 0, 1, 1], 16, 512, 64, 8, "bf16", "e4m3", False),
    ([100, 7], [5, 9], 16, 512, 64, 16, "bf16", None, True),          # 144 rows: two blocks of 128
    ([40, 3, 0], [2, 1, 2], 16, 512, 64, 32, "fp16", "e4m3", True),   # 32 rows
    ([90, 128], [3, 4], 12, 512, 64, 16, "bf16", None, True),         # 48 rows of 64
    ([33, 70], [1, 2], 128, 512, 64, 64, "bf16", None, False),
    ([33, 70], [1, 2], 128, 512, 64, 64, "fp16", "e4m3", False),
    ([200, 15], [3, 30], 7, 256, 32, 8, "fp16", None, False),
    ([200, 15], [3, 2], 8, 256, 64, 8, "bf16", "e4m3", True),
    ([65, 64, 63], [1, 1, 1], 8, 384, 64, 1, "bf16", None, False),
    ([50], [70], 4, 40, 8, 4, "fp16", None, True),                    # a mask of two words
    ([1200], [6], 16, 512, 64, 1, "bf16", None, True),                # more pages than the window
    ([1500, 3], [2, 1], 64, 256, 64, 2, "bf16", "e4m3", False),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_latent_attention(case):
    kv, ql, H, latent, rope, ps, dtype, cache, drafts = case
    rng = np.random.default_rng(H)
    s = Latents(kv, ql, H, latent, rope, ps, dtype, cache,
                [tree(n, rng) for n in ql] if drafts else None, seed=latent + H)
    got = s.call()
    s.check(got)
    assert torch.equal(s.call(), got)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_blocks_of_a_long_launch(case):
    """The same requests in a launch for long ones, which takes the row blocks that hold them."""
    kv, ql, H, latent, rope, ps, dtype, cache, drafts = case
    rng = np.random.default_rng(H)
    s = Latents(kv, ql, H, latent, rope, ps, dtype, cache,
                [tree(n, rng) for n in ql] if drafts else None, seed=latent + H + 1)
    got = s.call(max_kv_len=1 << 20)
    s.check(got)
    assert torch.equal(s.call(max_kv_len=1 << 20), got)


@pytest.mark.parametrize("kv,ql,H,cache", [
    ([5000], [1], 16, None), ([9000, 40], [2, 1], 16, "e4m3"), ([4097], [4], 32, None),
    ([3333, 2000], [1, 2], 64, None), ([2500], [3], 128, "e4m3")])
def test_long_requests_in_pieces(kv, ql, H, cache):
    s = Latents(kv, ql, H, cache=cache, ps=64, seed=H)
    s.check(s.call())


def test_many_requests():
    """More units than workgroups, one unit each, and equal ranges over uneven requests."""
    for bs, H, top in ((300, 16, 40), (520, 4, 20), (40, 16, 900), (150, 40, 33)):
        rng = np.random.default_rng(bs)
        kv = [int(x) for x in rng.integers(0, top, bs)]
        s = Latents(kv, [1 + i % 2 for i in range(bs)], H, 256, 32, seed=bs)
        s.check(s.call(), requests=range(0, bs, 17))


def test_bounds_shape_only_the_launch():
    s = Latents([700, 20, 0], [3, 40, 9], 16, 256, 32, seed=3)
    want = s.call()
    s.check(want)
    for q, kv in ((1, 1), (1, 4000), (40, 1), (0, 0)):
        s.check(s.call(max_q_len=q, max_kv_len=kv))


def test_strides_scales_and_what_is_left_alone():
    s = Latents([77, 5], [3, 2], 6, 256, 64, seed=4)
    n = int(s.ptr[-1])
    want = s.call()
    q = torch.full((8, n + 3, 352), float("nan"), dtype=torch.bfloat16, device=DEV)
    q[:6, :n, 16:336] = s.q.to(DEV).transpose(0, 1)
    out = torch.full((8, n + 3, 320), 4.0, dtype=torch.bfloat16, device=DEV)
    o = out[:6, :, 8:264].transpose(0, 1)
    got = s.call(q=q[:6, :, 16:336].transpose(0, 1), out=o)     # three rows behind the last request
    assert got is o and torch.equal(got[:n], want)
    out[:6, :n, 8:264] = 4.0
    assert (out == 4.0).all()
    for scale in (-0.05, 0.0, 1.5):
        s.check(s.call(scale=scale), scale=scale)


def test_rows_that_see_nothing_and_hidden_values():
    bf = torch.bfloat16
    s = Latents([0, 9], [3, 2], 16, trees=[[-1, 0, 0], [-1, 0]], seed=5)
    mask = s.mask()
    mask[1] = 0                                # no key at all
    got = s.call(tree_mask=mask)
    assert not got[1].any() and not got.isnan().any()
    # what a row does not see may hold anything
    for bad in (float("nan"), float("inf"), -float("inf")):
        t = Latents([40, 9], [6, 2], 16, trees=[[-1, 0, 0, 1, 2, 2], [-1, 0]], seed=6)
        want = t.call()
        p = 43                                 # drafted token 3, which 0, 1, 2, 4, 5 do not see
        t.cache[int(t.table[t.rows[0], p // 16]), p % 16] = torch.full((576,), bad, dtype=bf)
        got = t.call()
        keep = [0, 1, 2, 4, 5, 6, 7]
        assert torch.equal(got[keep], want[keep])
        c = Latents([3], [40], 8, 256, 32, seed=7)
        want = c.call()
        c.cache[int(c.table[c.rows[0], 33 // 16]), 33 % 16] = torch.full((288,), bad, dtype=bf)
        assert torch.equal(c.call()[:30], want[:30])


def test_large_scores_and_far_values():
    """Scores of thousands: the weights' reference moves, and nothing overflows."""
    s = Latents([900], [4], 16, dtype="fp16", seed=8, spread=6.0)
    got = s.call(scale=2.0)
    s.check(got, scale=2.0)
    assert torch.isfinite(got).all()


def test_bad_indices_do_no_harm():
    s = Latents([40, 9, 5], [2, 2, 1], 16, 256, 32, seed=9)
    want = s.call()
    n = int(s.ptr[-1])
    out = torch.full((n, 16, 256), 2.0, dtype=torch.bfloat16, device=DEV)
    rows = s.rows.copy()
    rows[1] = 77
    s.call(rows=_i32(rows), out=out)
    assert (out[2:4] == 2.0).all() and torch.equal(out[:2], want[:2]) and torch.equal(out[4:], want[4:])
    table = s.table.copy()
    table[s.rows[1], 0] = -3
    got = s.call(page_table=_i32(table))
    assert torch.equal(got[:2], want[:2]) and torch.equal(got[4:], want[4:])
    lens = s.lens.copy()
    lens[s.rows[2]] = -8
    assert torch.equal(s.call(kv_lens=_i32(lens))[:4], want[:4])


def test_a_cache_past_32_bits():
    """Pages behind 4 GiB of the pool."""
    pages = 60000
    cache = torch.empty((pages, 64, 576), dtype=torch.bfloat16, device=DEV)   # 4.4 GB
    gen = torch.Generator(DEV).manual_seed(1)
    at = [59999, 3, 58260]
    for p in at:
        cache[p] = torch.randn((64, 576), generator=gen, device=DEV)
    q = torch.randn((1, 16, 576), generator=gen, device=DEV).bfloat16()
    got = _sgg().spec_latent_attention(q, cache, _i32([at]), _i32([149]), _i32([0, 1]), 1, 150, 512,
                                       0.07)
    k = f64(torch.cat([cache[p] for p in at]))[:150, None]
    hold(f64(got), f64(q), k, k[:, :, :512], np.ones((1, 150), bool), 0.07, "bf16")


# ------------------------------------------------------------------- the expanded form

def prefill(ql, kl, H, dn, dr, dv, dtype, seed, extra=0):
    gen = torch.Generator().manual_seed(seed)
    n, m = sum(ql) + extra, sum(kl) + extra
    t = TYPES[dtype]
    kv = torch.randn((m, H, dn + dv), generator=gen).to(t).to(DEV)
    rows = torch.randn((m, 64 + dr), generator=gen).to(t).to(DEV)
    return dict(q=torch.randn((n, H, dn + dr), generator=gen).to(t).to(DEV), k=kv[:, :, :dn],
                v=kv[:, :, dn:], k_pe=rows[:, 64:], q_indptr=_i32(np.cumsum([0] + ql)),
                kv_indptr=_i32(np.cumsum([0] + kl)), max_q_len=max(ql), max_kv_len=max(kl))


def check_prefill(got, x, ql, kl, dtype, requests=None, pick=None):
    q0, k0 = np.cumsum([0] + ql), np.cumsum([0] + kl)
    q, k, v, kr = (f64(x[name]) for name in ("q", "k", "v", "k_pe"))
    scale = x.get("scale", q.shape[2] ** -0.5)
    for r in requests or range(len(ql)):
        if not ql[r]:
            continue
        a, b = slice(q0[r], q0[r + 1]), slice(k0[r], k0[r + 1])
        key = np.concatenate([k[b], np.repeat(kr[b][:, None], q.shape[1], 1)], 2)
        seen = np.arange(kl[r])[None] <= (kl[r] - ql[r] + np.arange(ql[r]))[:, None]
        p = slice(None) if pick is None else pick
        hold(f64(got)[a][p], q[a][p], key, v[b], seen[p], scale, dtype)


PREFILL = [
    ([1], [1], 4, 128, 64, 128, "bf16"), ([5, 0, 33], [5, 7, 40], 3, 128, 64, 128, "fp16"),
    ([100], [100], 16, 128, 64, 128, "bf16"), ([64, 65], [64, 300], 7, 64, 32, 64, "bf16"),
    ([129], [200], 2, 96, 32, 96, "fp16"), ([31, 1], [95, 129], 5, 128, 64, 64, "bf16"),
    ([40], [33], 2, 128, 64, 128, "bf16"),           # queries ahead of the first key see nothing
    ([3, 3], [0, 2], 2, 64, 64, 64, "fp16"), ([20], [50], 2, 8, 8, 24, "bf16"),
]


@pytest.mark.parametrize("ql,kl,H,dn,dr,dv,dtype", PREFILL)
def test_prefill(ql, kl, H, dn, dr, dv, dtype):
    x = prefill(ql, kl, H, dn, dr, dv, dtype, seed=dn + H, extra=2)
    got = _sgg().spec_latent_prefill(**x)
    check_prefill(got, x, ql, kl, dtype)
    out = torch.full_like(got, 6.0)
    _sgg().spec_latent_prefill(**x, out=out)
    assert torch.equal(out[:sum(ql)], got[:sum(ql)]) and (out[sum(ql):] == 6.0).all()


def test_prefill_large_launches_and_bounds():
    ql, kl = [700, 130, 257], [900, 130, 1300]
    x = prefill(ql, kl, 40, 128, 64, 128, "bf16", seed=11)      # 128 rows a workgroup
    got = _sgg().spec_latent_prefill(**x)
    check_prefill(got, x, ql, kl, "bf16", pick=slice(None, None, 61))
    x.update(max_q_len=1, max_kv_len=0)
    check_prefill(_sgg().spec_latent_prefill(**x), x, ql, kl, "bf16", pick=slice(None, None, 61))
    for scale in (-0.1, 0.0):
        x.update(scale=scale)
        check_prefill(_sgg().spec_latent_prefill(**x), x, ql, kl, "bf16", [1],
                      pick=slice(None, None, 13))


def test_prefill_strides_and_hidden_values():
    x = prefill([70], [90], 2, 128, 64, 128, "fp16", seed=12)
    want = _sgg().spec_latent_prefill(**x)
    y = dict(x, q=x["q"].transpose(0, 1).contiguous().transpose(0, 1),
             k=x["k"].transpose(0, 1).contiguous().transpose(0, 1))
    assert torch.equal(_sgg().spec_latent_prefill(**y), want)
    for bad in (float("nan"), float("inf")):
        for name in ("k", "v", "k_pe"):
            z = {**x, name: x[name].clone()}
            z[name][60] = bad                       # token 60 is query 40's
            got = _sgg().spec_latent_prefill(**z)
            assert torch.equal(got[:40], want[:40])
        z = {**x, "v": x["v"].clone()}
        z["v"][60, 0, 5] = bad                      # and is seen from there on, in its column
        got = _sgg().spec_latent_prefill(**z)
        assert not torch.isfinite(got[40:, 0, 5]).any()
        keep = torch.ones(128, dtype=torch.bool)
        keep[5] = False
        assert torch.equal(got[:, :, keep.to(DEV)], want[:, :, keep.to(DEV)])


# --------------------------------------------------------- both forms are the same attention

def test_absorbed_and_expanded_forms_agree():
    """A chunk behind a context through the pages: written, gathered, expanded and attended, and
    attended in the absorbed form, against the dense attention in 64 bits.

    Beside the tolerance above, the expanded keys and values and the absorbed queries are rounded to
    16 bits: relative r each, so a score is off by 2 r sum|q k| at most and a result by 3 r A."""
    sgg, gen = _sgg(), torch.Generator().manual_seed(13)
    L, R, H, dn, dv, kv, T = 128, 32, 4, 64, 64, 45, 9
    c = sgg.PagedLatentCache(2, 12, 8, L, R, 3, 10, torch.float16, DEV)
    rows = _i32([2])
    lat = (torch.randn((kv + T, L), generator=gen) * 0.5).half().to(DEV)
    kr = torch.randn((kv + T, R), generator=gen).half().to(DEV)
    inv = torch.rand(R // 2, generator=gen).to(DEV)
    wk, wv = (torch.randn((H, L, d), generator=gen) * L ** -0.5 for d in (dn, dv))
    qn, qr = (torch.randn((kv + T, H, d), generator=gen).half().to(DEV) for d in (dn, R))
    turned = torch.empty_like(qr)
    for a, b in ((0, kv), (kv, kv + T)):
        assert not c.reserve(rows, _i32([b])).any()
        turned[a:b] = c.write(1, qr[a:b], lat[a:b], kr[a:b], inv, _i32([0, b - a]), rows)
        if a == 0:
            c.commit(rows, _i32([b]))
    got_lat, got_kr = c.gather(1, _i32([0, kv + T]), kv + T, rows)
    assert torch.equal(got_lat, lat)
    k = torch.einsum("tl,hld->thd", f32(got_lat), wk).half().to(DEV)
    v = torch.einsum("tl,hld->thd", f32(got_lat), wv).half().to(DEV)
    q = torch.cat([qn, turned], 2)[kv:]
    scale = (dn + R) ** -0.5
    full = sgg.spec_latent_prefill(q, k, v, got_kr, _i32([0, T]), _i32([0, kv + T]), T, kv + T)
    qa = torch.cat([torch.einsum("thd,hld->thl", f32(qn[kv:]), wk).half().to(DEV), turned[kv:]], 2)
    o = c.attention(1, qa, _i32([0, T]), T, kv + T, scale, rows=rows)
    folded = np.einsum("thl,hld->thd", f64(o), wv.double().numpy())
    key = np.concatenate([np.einsum("tl,hld->thd", f64(lat), wk.double().numpy()),
                          np.repeat(f64(got_kr)[:, None], H, 1)], 2)
    val = np.einsum("tl,hld->thd", f64(lat), wv.double().numpy())
    size = np.einsum("tl,hld->thd", np.abs(f64(lat)), np.abs(wv.double().numpy()))
    seen = np.arange(kv + T)[None] <= (kv + np.arange(T))[:, None]
    want, mag, prod, top = osp.attention(f64(q), key, val, seen, scale)
    wide = osp.attention(f64(q), key, size, seen, scale)[0]
    r = 2.0 ** -11
    # (the absorbed query's products with the latent add up to more than the score's own)
    each = np.einsum("thd,hld->thl", np.abs(f64(qn[kv:])), np.abs(wk.double().numpy()))
    prod = np.maximum(prod, scale * np.einsum("thl,sl->ths", each, np.abs(f64(lat))).max(2) + prod)
    tol = 5 * r * wide + (2 * 2 * r * prod)[:, :, None] * wide + 2.0 ** -20
    assert (np.abs(f64(full) - want) <= tol).all()
    assert (np.abs(folded - want) <= tol).all()


def f32(x):
    return x.detach().cpu().float()
