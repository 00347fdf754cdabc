"""Rotation on the way into a paged cache, and rows of a cache of latents, against the oracle.

Tolerance per element: with r the half step of the type it is rounded to (2^-8 bf16, 2^-11 fp16,
2^-4 e4m3; half a subnormal step beside it), r |o| for the rounding, and (|a| + |b|) factor 2^-20
for the pair: a sine and a cosine of a fraction of a turn in 32 bits (2^-21 together with the
fraction's own rounding, 2 pi 2^-25), two products and a sum.  What is not rotated is equal.
"""

import numpy as np
import pytest
import torch

from oracle import latent as ola
from test_spec_gpu import DEV, TYPES, _bits, _i32, _sgg, f64

pytestmark = pytest.mark.gpu

HALF = {"bf16": (2.0 ** -8, 2.0 ** -134), "fp16": (2.0 ** -11, 2.0 ** -25),
        "e4m3": (2.0 ** -4, 2.0 ** -10)}


def fill(shape, dtype, gen, scale=1.0):
    return (torch.randn(shape, generator=gen) * scale).to(TYPES[dtype])


class Pages:
    """Pages for ql new tokens behind kv held ones; pages of context alone are one page."""

    def __init__(self, kv, ql, ps, seed, extra=0):
        rng = np.random.default_rng(seed)
        bs = len(kv)
        self.rows = rng.permutation(bs + 2)[:bs]
        self.kv, self.ql, self.ps = kv, ql, ps
        counts = [-(-(a + b) // ps) for a, b in zip(kv, ql)]
        first = [a // ps for a in kv]
        self.pages = sum(c - f for c, f in zip(counts, first)) + 2
        self.table = np.full((bs + 2, max(counts + [1])), 1 << 30)
        order, at = 1 + rng.permutation(self.pages - 1), 0
        self.lens, self.held = np.zeros(bs + 2, np.int64), np.zeros(bs + 2, np.int64)
        for row, f, c, a in zip(self.rows, first, counts, kv):
            self.table[row, :f] = 0
            self.table[row, f:c] = order[at:at + c - f]
            self.lens[row], self.held[row] = a, c
            at += c - f
        self.ptr = np.concatenate([[0], np.cumsum(ql)])
        self.n = int(self.ptr[-1]) + extra    # rows behind the last request

    def args(self):
        return dict(page_table=_i32(self.table), kv_lens=_i32(self.lens),
                    q_indptr=_i32(self.ptr), rows=_i32(self.rows))

    def places(self):
        for r, row in enumerate(self.rows):
            for i in range(self.ql[r]):
                p = self.kv[r] + i
                yield int(self.ptr[r]) + i, p, int(self.table[row, p // self.ps]), p % self.ps


def near(got, want, pair, dtype, scale=None):
    half, tiny = HALF[dtype]
    if scale is not None:
        want, pair = np.clip(want / scale, -448, 448), pair / scale
    tol = half * np.abs(want) + tiny + pair * 2.0 ** -20 * (1 + half)
    assert (np.abs(got - want) <= tol).all(), np.abs(got - want).max()


def pair_sizes(x, rot, start, interleaved, factor):
    """|a| + |b| of the pair that each column belongs to, 0 where it is not rotated."""
    size = np.zeros(x.shape)
    part = np.abs(x[..., start:start + rot])
    if interleaved:
        s = np.repeat(part.reshape(*part.shape[:-1], rot // 2, 2).sum(-1), 2, axis=-1)
    else:
        s = np.tile(part[..., :rot // 2] + part[..., rot // 2:], 2)
    size[..., start:start + rot] = s * abs(factor)
    return size


CASES = [
    # kv, ql, ps, hq, hkv, d, rot, start, interleaved, dtype, cache, positions
    ([5], [1], 16, 4, 2, 64, 64, 0, False, "bf16", None, False),
    ([0, 33, 7], [3, 0, 9], 8, 8, 2, 128, 128, 0, False, "fp16", None, True),
    ([100, 0], [1, 5], 16, 4, 4, 128, 64, 64, True, "bf16", "e4m3", True),
    ([31, 2], [2, 40], 32, 6, 2, 96, 24, 72, False, "bf16", None, False),     # pairs one by one
    ([31, 2], [2, 40], 32, 3, 1, 96, 24, 0, False, "fp16", "e4m3", False),
    ([9], [4], 1, 2, 2, 64, 10, 7, True, "bf16", None, False),
    ([9], [4], 1, 2, 2, 64, 10, 7, False, "fp16", "e4m3", True),
    ([12], [7], 8, 2, 1, 256, 256, 0, True, "fp16", None, False),
    ([499990, 123456], [17, 3], 1024, 2, 2, 64, 64, 0, False, "fp16", None, False),
    ([400], [2500], 64, 2, 1, 64, 32, 16, False, "bf16", None, False),        # several a workgroup
    ([3] * 300, [1] * 300, 16, 2, 1, 64, 64, 0, True, "bf16", None, False),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_rope_write(case):
    kv, ql, ps, hq, hkv, d, rot, start, inter, dtype, cache, given = case
    gen = torch.Generator().manual_seed(len(kv) + d)
    g = Pages(kv, ql, ps, seed=d + rot, extra=2)
    x = fill((g.n, hq + 2 * hkv, d), dtype, gen).to(DEV)     # as one projection leaves them
    q, k, v = x.split([hq, hkv, hkv], 1)
    inv = (10000.0 ** (-torch.arange(0, rot, 2) / rot)).float()
    ks = vs = None
    if cache:
        ks, vs = torch.rand(hkv) * 0.01 + 0.004, torch.rand(hkv) * 0.01 + 0.004
    kc, vc = (fill((g.pages, ps, hkv, d), cache or dtype, gen).to(DEV) for _ in range(2))
    before = [f64(kc), f64(vc)]
    pos = None
    if given:
        pos = np.random.default_rng(1).integers(0, 5000, g.n)
    out = torch.full((g.n, hq, d), 7.0, dtype=x.dtype, device=DEV)
    keep = x.clone()
    got = _sgg().spec_rope_write(
        q, k, v, inv.to(DEV), kc, vc, **g.args(), positions=None if pos is None else _i32(pos),
        rope_start=start, interleaved=inter, factor=1.25,
        k_scale=None if ks is None else ks.to(DEV), v_scale=None if vs is None else vs.to(DEV),
        page_counts=_i32(g.held), q_out=out)
    assert got is out and torch.equal(x, keep)
    hx, after = f64(x), [f64(kc), f64(vc)]
    wq = np.full((g.n, hq, d), 7.0)
    wk, wv = before
    pq, pk = np.zeros(wq.shape), np.zeros(wk.shape)
    new = np.zeros(wk.shape[:2], bool)
    unit = np.ones((1, hkv, 1)) if ks is None else f64(ks)[None, :, None]
    for n, p, page, off in g.places():
        at = p if pos is None else int(pos[n])
        turned = ola.rotate(hx[n, :hq + hkv], at, inv.numpy(), start, inter, 1.25)
        size = pair_sizes(hx[n, :hq + hkv], rot, start, inter, 1.25)
        wq[n], pq[n] = turned[:hq], size[:hq]
        wk[page, off], pk[page, off] = turned[hq:], size[hq:]
        wv[page, off] = hx[n, hq + hkv:]
        new[page, off] = True
    near(f64(out), wq, pq, dtype)
    still = np.ones(d, bool)
    still[start:start + rot] = False
    assert np.array_equal(f64(out)[..., still], wq[..., still])
    assert np.array_equal(after[0][~new], wk[~new]) and np.array_equal(after[1][~new], wv[~new])
    if cache is None:
        near(after[0][new], wk[new], pk[new], dtype)
        assert np.array_equal(after[0][new][..., still], wk[new][..., still])
        assert np.array_equal(after[1][new], wv[new])
    else:
        near(after[0][new], wk[new], pk[new], "e4m3", unit)
        near(after[1][new], wv[new], 0 * pk[new], "e4m3", f64(vs)[None, :, None])


def test_rope_in_place_and_keys_alone():
    gen = torch.Generator().manual_seed(5)
    g = Pages([4, 20], [3, 2], 8, seed=2)
    q, k, v = (fill((g.n, h, 64), "bf16", gen).to(DEV) for h in (4, 2, 2))
    inv = torch.rand(16, generator=gen).to(DEV)
    kc, vc = (fill((g.pages, 8, 2, 64), "bf16", gen).to(DEV) for _ in range(2))
    k1, v1, k2, v2 = kc.clone(), vc.clone(), kc.clone(), vc.clone()
    for inter in (False, True):
        a = dict(interleaved=inter, rope_start=8)
        want = _sgg().spec_rope_write(q, k, v, inv, kc, vc, **g.args(), **a)
        place = q.clone()
        assert _sgg().spec_rope_write(place, k, v, inv, k1, v1, **g.args(), q_out=place, **a) is place
        assert torch.equal(place, want) and torch.equal(k1, kc) and torch.equal(v1, vc)
        assert _sgg().spec_rope_write(None, k, v, inv, k2, v2, **g.args(), **a) is None
        assert torch.equal(k2, kc) and torch.equal(v2, vc)


def test_rope_without_angles_is_the_plain_write():
    """Position 0 rotates by nothing: the same bits as spec_kv_write, special values included."""
    gen = torch.Generator().manual_seed(6)
    for cache in ("bf16", "e4m3"):
        g = Pages([0, 9], [5, 3], 4, seed=3)
        k, v = (fill((g.n, 2, 64), "bf16", gen, 40.0).to(DEV) for _ in range(2))
        v[0, 0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 1e30])
        s = torch.full((2,), 0.3, device=DEV)
        sc = dict(k_scale=s, v_scale=s) if cache == "e4m3" else {}
        kc, vc = (torch.zeros((g.pages, 4, 2, 64), dtype=TYPES[cache], device=DEV) for _ in range(2))
        k1, v1 = kc.clone(), vc.clone()
        _sgg().spec_kv_write(k, v, kc, vc, **g.args(), **sc)
        _sgg().spec_rope_write(None, k, v, torch.ones(32, device=DEV), k1, v1, **g.args(), **sc,
                               positions=_i32(np.zeros(g.n)))
        assert torch.equal(_bits(kc).view(torch.uint8), _bits(k1).view(torch.uint8))
        assert torch.equal(_bits(vc).view(torch.uint8), _bits(v1).view(torch.uint8))


def test_rope_bad_rows_and_missing_pages():
    gen = torch.Generator().manual_seed(7)
    q, k, v = (fill((6, 2, 64), "bf16", gen).to(DEV) for _ in range(3))
    kc, vc = (torch.zeros((5, 4, 2, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    inv = torch.ones(32, device=DEV)
    table = _i32([[0, 1, 2], [3, 4, 1 << 30], [-1, 9, 9], [0, 0, 0]])
    a = dict(page_table=table, kv_lens=_i32([2, 7, 0, 1]), q_indptr=_i32([0, 2, 4, 5, 6]))
    out = torch.full_like(q, 3.0)
    # row 9 is no row; row 1's tokens fall on its page 1 and past its pages; row 2 has a bad page
    _sgg().spec_rope_write(q, k, v, inv, kc, vc, **a, rows=_i32([9, 1, 2, 3]), q_out=out,
                           page_counts=_i32([3, 3, 3, 0]))
    assert (out[:2] == 3.0).all() and not (out[2:] == 3.0).all(-1).any()
    assert (kc[4, 3] != 0).any() and (vc[4, 3] == v[2]).all()
    kc[4, 3], vc[4, 3] = 0, 0
    assert not kc.any() and not vc.any()
    # boundaries that do not fit: nothing is touched
    out.fill_(3.0)
    for ind in ([0, 7, 7, 7, 7], [-1, 0, 0, 0, 0], [4, 2, 2, 1, 0]):
        _sgg().spec_rope_write(q, k, v, inv, kc, vc, **{**a, "q_indptr": _i32(ind)}, q_out=out)
    assert (out == 3.0).all() and not kc.any() and not vc.any()


@pytest.mark.parametrize("latent,rope,dtype,cache,ps,inter", [
    (512, 64, "bf16", None, 16, True), (256, 32, "fp16", "e4m3", 8, False),
    (384, 64, "bf16", "e4m3", 64, True), (40, 8, "fp16", None, 1, True),
    (16, 24, "bf16", None, 4, False)])
def test_latent_write_and_gather(latent, rope, dtype, cache, ps, inter):
    sgg, gen = _sgg(), torch.Generator().manual_seed(latent)
    kv, ql, H = [3, 0, 40, 17], [2, 4, 0, 30], 5
    rng = np.random.default_rng(latent)
    counts = [-(-(a + b) // ps) for a, b in zip(kv, ql)]
    pages = sum(counts) + 2
    rows = rng.permutation(6)[:4]
    table, at, order = np.full((6, max(counts)), -5), 0, rng.permutation(pages)
    lens, held = np.zeros(6), np.zeros(6)
    for row, c, a in zip(rows, counts, kv):
        table[row, :c] = order[at:at + c]
        lens[row], held[row], at = a, c, at + c
    n = sum(ql)
    wide = torch.full((n, latent + 8), 9.0, dtype=TYPES[dtype])
    wide[:, :latent] = fill((n, latent), dtype, gen)
    lat = wide.to(DEV)[:, :latent]
    kpe = fill((n, rope), dtype, gen).to(DEV)
    qa = fill((n, H, latent + rope), dtype, gen).to(DEV) if latent % 8 == 0 else None
    qpe, inv = qa[:, :, latent:], torch.rand(rope // 2, generator=gen).to(DEV)
    scale = torch.tensor([0.02], device=DEV) if cache else None
    x = fill((pages, ps, latent + rope), cache or dtype, gen).to(DEV)
    before, hq, hk, hl = f64(x), f64(qpe), f64(kpe), f64(lat)
    rest = qa[:, :, :latent].clone()
    ptr = np.concatenate([[0], np.cumsum(ql)])
    args = dict(rows=_i32(rows), page_counts=_i32(held), cache_scale=scale)
    got = sgg.spec_latent_write(qpe, lat, kpe, inv, x, _i32(table), _i32(lens), _i32(ptr),
                                interleaved=inter, q_out=qpe, **args)
    assert got is qpe and torch.equal(qa[:, :, :latent], rest)
    after, new, pair = f64(x), np.zeros((pages, ps), bool), np.zeros(before.shape)
    wq, pq = np.zeros(hq.shape), np.zeros(hq.shape)
    for r, row in enumerate(rows):
        for i in range(ql[r]):
            t, p = ptr[r] + i, kv[r] + i
            wq[t] = ola.rotate(hq[t], p, f64(inv), 0, inter, 1.0)
            pq[t] = pair_sizes(hq[t], rope, 0, inter, 1.0)
            page, off = table[row, p // ps], p % ps
            before[page, off, :latent] = hl[t]
            before[page, off, latent:] = ola.rotate(hk[t][None], p, f64(inv), 0, inter, 1.0)[0]
            pair[page, off, latent:] = pair_sizes(hk[t][None], rope, 0, inter, 1.0)[0]
            new[page, off] = True
    near(f64(qpe), wq, pq, dtype)
    assert np.array_equal(after[~new], before[~new])
    near(after[new], before[new], pair[new], cache or dtype, f64(scale)[0] if cache else None)
    if not cache:
        assert np.array_equal(after[new][:, :latent], before[new][:, :latent])
    # rows out of the pages; two more than the requests have stay as they were
    total = [a + b for a, b in zip(kv, ql)]
    ends = np.concatenate([[0], np.cumsum(total)])
    out = torch.full((ends[-1] + 2, latent + rope), 5.0, dtype=TYPES[dtype], device=DEV)
    sgg.spec_latent_gather(x, _i32(table), _i32(ends), ends[-1] + 2, out=out, **args)
    unit = 1.0 if scale is None else f64(scale)[0]
    half, tiny = HALF[dtype]
    for r, row in enumerate(rows):
        p = np.arange(total[r])
        want = after[table[row, p // ps], p % ps] * unit
        y = f64(out)[ends[r]:ends[r + 1]]
        assert (np.abs(y - want) <= (0 if scale is None else half * np.abs(want) + tiny)).all()
    assert (out[-2:] == 5.0).all()
    # a page less: its positions are zeros
    held[rows[3]] -= 1
    args["page_counts"] = _i32(held)
    less = sgg.spec_latent_gather(x, _i32(table), _i32(ends), ends[-1], dtype=TYPES[dtype], **args)
    lost = ends[3] + (counts[3] - 1) * ps
    assert torch.equal(less[:lost], out[:lost]) and not less[lost:].any()
