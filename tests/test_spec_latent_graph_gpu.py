"""A whole step over a cache of latents and a paged cache with rotated keys: captured, against the
same step run eagerly; on two streams at once; and a cache of latents through its life."""

import pytest
import torch

from test_spec_gpu import DEV, _i32, _sgg

pytestmark = pytest.mark.gpu

L, PAGES, PS, ROWS, V, T, BS = 2, 70, 8, 7, 3001, 6, 3
H, HKV, D, LATENT, ROPE, DN, DV = 16, 2, 64, 128, 32, 64, 64
LENS = [13, 40, 3]
BF16, FP16, E4M3 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


def _raw(x):
    return x.view(torch.uint8)


def _state(c):
    return [getattr(c, n) for n in ("data", "k", "v", "page_table", "page_counts", "kv_lens",
                                    "ref_counts") if hasattr(c, n)]


class Step:
    """Inputs in memory of their own, two caches, and the calls of a step on them."""

    def __init__(self, cache, seed=0):
        sgg = _sgg()
        self.lat = sgg.PagedLatentCache(L, PAGES, PS, LATENT, ROPE, ROWS, 12, cache, DEV)
        self.kv = sgg.PagedKVCache(L, PAGES, PS, HKV, D, ROWS, 12, cache, DEV)
        gen = torch.Generator(DEV).manual_seed(seed)
        self.rows = _i32([4, 0, 2])
        for c in (self.lat, self.kv):
            c.commit(self.rows, _i32(LENS))
            for x in _state(c)[:1 if c is self.lat else 2]:
                x.copy_(torch.randn(x.shape, generator=gen, device=DEV))
        n, dev = BS * T, {"device": DEV}
        self.grown, self.ind = _i32([x + T for x in LENS]), _i32([0, T, 2 * T, 3 * T])
        self.kind = _i32([0, LENS[0] + T, LENS[0] + LENS[1] + 2 * T, sum(LENS) + 3 * T])
        self.parents, self.tokens = _i32([-1, 0, 0, 1, 2, 4] * BS), _i32([0] * n)
        self.inv = torch.rand(ROPE // 2, generator=gen, **dev)
        self.inv_kv = torch.rand(D // 2, generator=gen, **dev)
        zeros = lambda *shape: torch.zeros(shape, dtype=BF16, **dev)
        self.q, self.k, self.v = zeros(n, H, D), zeros(n, HKV, D), zeros(n, HKV, D)
        self.qa, self.latent, self.k_pe = zeros(n, H, LATENT + ROPE), zeros(n, LATENT), zeros(n, ROPE)
        self.qe, m = zeros(n, H, DN + ROPE), sum(LENS) + n
        self.kn, self.vn = zeros(m, H, DN), zeros(m, H, DV)
        self.logits, self.heat = zeros(n, V), torch.zeros(BS, **dev)
        self.history, self.hist_lens = _i32([[0] * 50] * ROWS), _i32([20, 0, 50, 0, 7, 0, 0])
        self.rep, self.pres = torch.full((BS,), 1.5, **dev), torch.full((BS,), 0.25, **dev)
        self.u, self.uf = torch.zeros(n, **dev), torch.zeros(BS, **dev)

    def fill(self, seed):
        gen = torch.Generator(DEV).manual_seed(seed)
        for x in (self.q, self.k, self.v, self.qa, self.latent, self.k_pe, self.qe, self.kn, self.vn,
                  self.logits):
            x.copy_(torch.randn(x.shape, generator=gen, device=DEV))
        for x in (self.tokens, self.history):
            x.copy_(torch.randint(0, V, x.shape, generator=gen, device=DEV))
        for x in (self.u, self.uf, self.heat):
            x.copy_(torch.rand(x.shape, generator=gen, device=DEV))
        self.heat[seed % BS] = 0.0

    def run(self):
        sgg, out, rows, ind = _sgg(), [], self.rows, self.ind
        for c in (self.lat, self.kv):
            out.append(c.reserve(rows, self.grown))
        mask, pos = sgg.spec_tree_mask(self.parents, ind, self.kv.kv_lens, 1, rows)
        for layer in range(L):
            q = self.kv.rope_write(layer, self.q, self.k, self.v, self.inv_kv, ind, rows, pos)
            out += [q, self.kv.attention(layer, q, ind, T, 60, mask, rows)]
            qa = self.qa.clone()
            qa[..., LATENT:] = self.lat.write(layer, self.qa[..., LATENT:], self.latent, self.k_pe,
                                              self.inv, ind, rows, pos)
            out += [qa, self.lat.attention(layer, qa, ind, T, 60, 0.1, mask, rows)]
            held, k_pe = self.lat.gather(layer, self.kind, self.kn.shape[0], rows, BF16)
            out += [held, k_pe, sgg.spec_latent_prefill(self.qe, self.kn, self.vn, k_pe, ind,
                                                        self.kind, T, 60)]
        p = sgg.spec_target_probs(self.logits, ind, T, self.heat, self.tokens, self.parents,
                                  self.history, self.hist_lens, rows=rows, repetition=self.rep,
                                  presence=self.pres)
        path, accept, nxt = sgg.spec_verify(self.tokens, self.parents, ind, p, self.u, self.uf, T)
        out += [p, path, accept, nxt]
        for c in (self.lat, self.kv):
            lens = c.compact(path, accept, rows)
            out += [lens, c.commit(rows, lens)]
        return out

    def everything(self, out):
        return [_raw(x.contiguous()).clone() for x in out + _state(self.lat) + _state(self.kv)]


def _same(a, b):
    assert len(a) == len(b)
    for i, (x, y) in enumerate(zip(a, b)):
        assert torch.equal(x, y), i


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_a_step_in_two_graphs(cache):
    """Two captured steps of their own inputs, replayed in turn with eager work between."""
    steps = [Step(cache, s) for s in (1, 2)]
    start = [[x.clone() for x in map(_raw, _state(s.lat) + _state(s.kv))] for s in steps]

    def restore(i):
        for x, y in zip(_state(steps[i].lat) + _state(steps[i].kv), start[i]):
            _raw(x).copy_(y)
    graphs, outs = [], []
    for i, s in enumerate(steps):
        s.fill(i)
        s.run()
        restore(i)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(s.run())
        graphs.append(g)
    for turn in range(4):
        for i, s in enumerate(steps):
            s.fill(10 * turn + i)
            restore(i)
            want = s.everything(s.run())
            restore(i)
            torch.cuda.synchronize()
            graphs[i].replay()
            _same(s.everything(outs[i]), want)
            assert all(torch.isfinite(x.float()).all() for x in outs[i] if x.is_floating_point())


def test_steps_on_two_streams():
    steps, want = [Step(BF16, s) for s in (3, 4)], []
    start = [[x.clone() for x in map(_raw, _state(s.lat) + _state(s.kv))] for s in steps]
    for s, kept in zip(steps, start):
        s.fill(5)
        want.append(s.everything(s.run()))
        for x, y in zip(_state(s.lat) + _state(s.kv), kept):
            _raw(x).copy_(y)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in steps], []
    for s, stream in zip(steps, streams):
        with torch.cuda.stream(stream):
            got.append(s.run())
    torch.cuda.synchronize()
    for s, out, w in zip(steps, got, want):
        _same(s.everything(out), w)


@pytest.mark.parametrize("cache", [BF16, FP16, E4M3])
def test_a_cache_of_latents_through_its_life(cache):
    """Rows written, forked, written apart, compacted, released: what is gathered is what was
    written, in the cache's type."""
    sgg, gen = _sgg(), torch.Generator().manual_seed(7)
    c = sgg.PagedLatentCache(L, 20, 4, 32, 32, 4, 8, cache, DEV)
    if cache is E4M3:
        c.scale[:] = torch.tensor([[0.5], [2.0]])
    wide = FP16 if cache is FP16 else BF16
    inv = torch.zeros(16, device=DEV)           # no angles: the rows go in as they are
    host = {}

    def grow(row, n):
        x = (torch.randn((L, n, 64), generator=gen) * 3).to(wide)
        assert not c.reserve(_i32([row]), _i32([len(host[row][0]) + n])).any()
        for layer in range(L):
            y = x[layer].to(DEV)
            assert c.write(layer, None, y[:, :32], y[:, 32:], inv, _i32([0, n]), _i32([row])) is None
            if cache is E4M3:
                unit = float(c.scale[layer])
                y = ((y.float() / unit).clamp(-448, 448).to(E4M3).float() * unit).to(wide)
            host[row][layer] += list(y.cpu())

    def commit(row, n=None):
        host[row] = [x[:n] for x in host[row]]
        assert not c.commit(_i32([row]), _i32([len(host[row][0])])).any()

    def check():
        rows = sorted(host)
        ind = [0]
        for r in rows:
            ind.append(ind[-1] + len(host[r][0]))
        for layer in range(L):
            a, b = c.gather(layer, _i32(ind), ind[-1], _i32(rows), None if cache is wide else wide)
            got = torch.cat([a, b], 1).cpu()
            want = [x for r in rows for x in host[r][layer]]
            assert torch.equal(got, torch.stack(want) if want else got[:0])
    host[1] = [[], []]
    grow(1, 10)
    commit(1)
    check()
    assert not c.fork(_i32([1]), _i32([3])).any()
    host[3] = [list(x) for x in host[1]]
    check()
    for row, n in ((1, 3), (3, 6)):             # apart, the page of both among them
        grow(row, n)
        commit(row)
    check()
    grow(3, 4)                                  # of four drafts the first and the third stay
    lens = c.compact(_i32([[0, 2, -1, -1]]), _i32([2]), _i32([3]))
    host[3] = [x[:17] + [x[18]] for x in host[3]]
    assert lens.tolist() == [18]
    assert not c.commit(_i32([3]), lens).any()
    check()
    src, dst = c.page_table[3, :2].clone(), _i32([18, 19])
    c.copy_pages(src, dst)
    assert torch.equal(_raw(c.data[:, 18:]), _raw(c.data[:, src.long()]))
    commit(1, 0)
    commit(3, 0)
    assert not c.ref_counts.any() and not c.kv_lens.any()
