"""Writes into the paged cache stay within the pages that a row holds."""

import numpy as np
import pytest
import torch

from test_spec_gpu import DEV, TYPES, _i32, _pool, _sgg

pytestmark = pytest.mark.gpu


def _new(n, H, D):
    return [torch.full((n, H, D), float(i + 7), dtype=torch.bfloat16, device=DEV) for i in (0, 1)]


@pytest.mark.parametrize("trimmed", [False, True])
def test_full_pool_leaves_other_rows_alone(trimmed):
    """A row whose growth found no page, behind a fresh table entry (page 0) or one that names a
    page given back and since handed to the other row."""
    sgg = _sgg()
    H, D, ps = 2, 64, 4
    c = sgg.PagedKVCache(2, 6, ps, H, D, 2, 6, device=DEV)
    both = _i32([0, 1])
    if trimmed:                              # row 1 held pages 2 .. 5 and gave back the last two
        c.commit(both, _i32([8, 16]))
        c.commit(both, _i32([8, 8]))
        assert c.reserve(both, _i32([16, 8])).tolist() == [0, 0]
        c.commit(both, _i32([16, 8]))
    else:
        c.commit(both, _i32([20, 4]))
    table = c.page_table.tolist()
    counts, lens = c.page_counts.tolist(), c.kv_lens.tolist()
    assert table[1][counts[1]] in table[0][:counts[0]] and sum(counts) == 6
    ind = _i32([0, 0, 6])
    assert c.reserve(both, _i32([lens[0], lens[1] + 6])).tolist()[0] > 0
    before = c.k.clone(), c.v.clone()
    for layer in range(2):
        c.write(layer, *_new(6, H, D), ind, both)
    new = c.compact(_i32([[-1] * 4, [0, 2, 4, 5]]), _i32([0, 4]), both)
    assert new.tolist() == [lens[0], lens[1] + 4]
    for x, y in zip((c.k, c.v), before):
        assert torch.equal(x, y)             # (row 1 ends at a page's border: none of it has room)


@pytest.mark.parametrize("dtype,cache", [("bf16", None), ("fp16", "e4m3")])
@pytest.mark.parametrize("counts", [[0, 1, 3, 9], [-4, 2, 100, 3]])
def test_write_and_compact_stop_at_the_count(dtype, cache, counts):
    sgg = _sgg()
    rng = np.random.default_rng(len(counts) + counts[1])
    ps, P, H, D, L = 4, 30, 2, 64, 2
    lens, ql, rows = [3, 2, 5, 9], [6, 5, 12, 4], [2, 0, 3, 1]
    table = _pool(4, 6, P, ps, rng, [24, 20, 28 - 4, 24])[0]
    ct = TYPES[cache or dtype]
    k, v = ((torch.randn((L, P, ps, H, D), device=DEV) * 9).to(ct) for _ in range(2))
    want = [x.clone() for x in (k, v)]
    x = [torch.randn((sum(ql), H, D), device=DEV).to(TYPES[dtype]) for _ in range(2)]
    one = torch.ones(H, device=DEV) if cache else None
    ptr = np.concatenate([[0], np.cumsum([ql[r] for r in rows])])
    sgg.spec_kv_write(x[0], x[1], k[0], v[0], _i32(table), _i32(lens), _i32(ptr), rows=_i32(rows),
                      k_scale=one, v_scale=one, page_counts=_i32(counts))
    slots = [max(0, min(c, 6)) for c in counts]

    def place(row, pos):
        return (int(table[row, pos // ps]), pos % ps) if pos // ps < slots[row] else None
    for w, y in zip(want, x):
        for r, row in enumerate(rows):
            for i in range(ql[row]):
                at = place(row, lens[row] + i)
                if at:
                    w[0, at[0], at[1]] = y[int(ptr[r]) + i].to(ct)
    for a, w in zip((k, v), want):
        assert torch.equal(a.view(torch.uint8), w.view(torch.uint8))
    path = [[0, 2, 3, 5], [0, 1, 4, -1], [1, 2, 8, 11], [0, 3, -1, -1]]
    n = [4, 3, 4, 2]
    new = sgg.spec_kv_compact(k, v, _i32(table), _i32(lens), _i32(path), _i32(n), rows=_i32(rows),
                              page_counts=_i32(counts))
    assert new.tolist() == [lens[row] + m for row, m in zip(rows, n)]
    for w in want:
        for row, way, m in zip(rows, path, n):
            for j, i in enumerate(way[:m]):
                a, b = place(row, lens[row] + i), place(row, lens[row] + j)
                if a and b:
                    w[:, b[0], b[1]] = w[:, a[0], a[1]].clone()
    for a, w in zip((k, v), want):
        assert torch.equal(a.view(torch.uint8), w.view(torch.uint8))
