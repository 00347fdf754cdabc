"""A whole speculative decoding step, captured: every replay against the same step run eagerly."""

import pytest
import torch

from test_spec_gpu import DEV, _i32, _sgg

pytestmark = pytest.mark.gpu

L, PAGES, PS, H, HQ, D, ROWS, V, T, BS = 2, 60, 8, 2, 8, 64, 7, 3001, 6, 3
STATE = ("k", "v", "page_table", "page_counts", "kv_lens", "ref_counts")


def _raw(x):
    return x.view(torch.uint8)


def _step(c, x):
    """All calls of a step on cache c with the inputs x, and the tensors that they return."""
    sgg = _sgg()
    out = [c.reserve(x["rows"], x["grown"])]
    mask, pos = sgg.spec_tree_mask(x["parents"], x["ind"], c.kv_lens, 1, x["rows"])
    out += [mask, pos]
    for layer in range(L):
        c.write(layer, x["new"][0], x["new"][1], x["ind"], x["rows"])
        out.append(c.attention(layer, x["q"], x["ind"], T, 400, tree_mask=mask, rows=x["rows"]))
    path, accept, nxt = sgg.spec_verify(x["tokens"], x["parents"], x["ind"], x["p"], x["u"], x["uf"],
                                        T, draft_probs=x["d"])
    lens = c.compact(path, accept, x["rows"])
    out += [path, accept, nxt, lens, c.commit(x["rows"], lens)]
    out.append(c.fork(x["src"], x["dst"]))
    c.copy_pages(x["from"], x["to"])
    out.append(c.commit(x["dst"], x["zeros"]))
    return out


def _fill(x, seed):
    """New values in the inputs' own memory."""
    gen = torch.Generator(DEV).manual_seed(seed)
    for key in ("q", "new"):
        for t in (x[key] if key == "new" else [x[key]]):
            t.copy_(torch.randn(t.shape, generator=gen, device=DEV))
    logits = torch.randn((BS * T, V), generator=gen, device=DEV) * 3
    x["p"].copy_(torch.softmax(logits, -1))
    x["d"].copy_(torch.softmax(logits + torch.randn((BS * T, V), generator=gen, device=DEV), -1))
    x["tokens"].copy_(torch.multinomial(x["d"], 1, generator=gen)[:, 0])
    x["u"].copy_(torch.rand(BS * T, generator=gen, device=DEV) * (0.5 if seed % 2 else 1.0))
    x["uf"].copy_(torch.rand(BS, generator=gen, device=DEV))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_a_step_in_a_graph(dtype):
    sgg = _sgg()
    c = sgg.PagedKVCache(L, PAGES, PS, H, D, ROWS, 12, dtype=dtype, device=DEV)
    gen = torch.Generator(DEV).manual_seed(9)
    for x in (c.k, c.v):
        x.copy_(torch.randn(x.shape, generator=gen, device=DEV))
    rows = _i32([4, 0, 2])
    c.commit(rows, _i32([13, 40, 3]))
    x = dict(rows=rows, grown=_i32([13 + T, 40 + T, 3 + T]), ind=_i32([0, T, 2 * T, 3 * T]),
             parents=_i32([-1, 0, 0, 1, 2, 4] * BS), src=_i32([4, 0]), dst=_i32([1, 6]),
             zeros=_i32([0, 0]), to=_i32([PAGES - 1, PAGES - 2]),
             tokens=_i32([0] * (BS * T)), u=torch.zeros(BS * T, device=DEV),
             uf=torch.zeros(BS, device=DEV), p=torch.zeros((BS * T, V), device=DEV),
             d=torch.zeros((BS * T, V), device=DEV),
             q=torch.zeros((BS * T, HQ, D), dtype=torch.bfloat16, device=DEV),
             new=[torch.zeros((BS * T, H, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)])
    x["from"] = _i32([0, 3])
    start = {name: _raw(getattr(c, name)).clone() for name in STATE}

    def restore():
        for name in STATE:
            _raw(getattr(c, name)).copy_(start[name])
    _fill(x, 0)
    _step(c, x)
    restore()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _step(c, x)
    accepted = set()
    for seed in range(5):
        _fill(x, seed)
        restore()
        want = [t.clone() for t in _step(c, x)]
        after = {name: _raw(getattr(c, name)).clone() for name in STATE}
        restore()
        for t in got:
            t.fill_(-3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (seed, i)
        for name in STATE:
            assert torch.equal(_raw(getattr(c, name)), after[name]), (seed, name)
        accepted.update(want[6].tolist())
        assert want[0].tolist() == [0, 0] and not want[3].isnan().any()
    assert len(accepted) > 1
