"""Latent attention: a paged cache that holds one latent vector a token for all heads.

A token's row in the cache is its latent c (``latent_dim`` columns) and the rotated key part kr
that all heads share (``rope_dim`` columns).  A head's keys and values are projections of the
latent, and there are two forms of the same attention:

- absorbed (``spec_latent_attention``): the key projection is multiplied into the queries and the
  value projection into what follows, so that every head attends over the rows as they lie in the
  cache: drafted tokens, single tokens, short chunks;
- expanded (``spec_latent_prefill``): keys and values of every head are made from the latents
  (gathered out of the pages by ``spec_latent_gather``) by the caller's projection: prompts.

Arrays, rows and streams are those of ``speculative``; include/sgg_spec.h says what each call
computes.
"""

import torch

from ._lib import check, spec_calls, tensor_args
from .speculative import (_CODES, _batch, _given_workspace, _positions, _queries, _workspace,
                          spec_kv_compact, spec_kv_copy_pages, spec_kv_fork, spec_kv_resize)
from .binding import _stream

_args = tensor_args()
_i32, _f32, _table, _heads = _args.i32, _args.f32, _args.table, _args.heads
_latents, _rows2 = _args.latents, _args.rows


def spec_latent_write(q_pe, latent, k_pe, inv_freq, cache, page_table, kv_lens, q_indptr,
                      rows=None, positions=None, interleaved=True, factor=1.0, cache_scale=None,
                      page_counts=None, q_out=None):
    """New rows of one layer's cache (pages, page_size, columns): ``latent`` (tokens, latent_dim) as
    it is and ``k_pe`` (tokens, rope_dim) rotated by its position; token i of request r at position
    kv_lens[row] + i.  The queries' parts ``q_pe`` (tokens, heads, rope_dim) are rotated alike, into
    ``q_out``, which is returned (None: a new tensor; it may be q_pe itself, or the last columns of
    the absorbed queries); q_pe None: nothing is returned.  A float8_e4m3fn cache takes
    x / ``cache_scale`` (float32 (1)).  All else as in spec_rope_write."""
    dev = cache.get_device()
    n, dim = k_pe.shape if k_pe.dim() == 2 else (0, 0)
    lp, lt = _rows2("latent", latent)
    kp, kt = _rows2("k_pe", k_pe)
    c, wide = _latents(cache, dim)
    if latent.shape != (n, wide - dim) or latent.dtype is not k_pe.dtype:
        raise ValueError(f"latent {tuple(latent.shape)} {latent.dtype} and k_pe {tuple(k_pe.shape)} "
                         f"{k_pe.dtype} must be (tokens, columns) of one type that fill the cache's "
                         f"{wide} columns")
    if latent.get_device() != dev or k_pe.get_device() != dev:
        raise ValueError("latent and k_pe must be on the cache's device")
    if 2 * inv_freq.numel() != dim:
        raise ValueError(f"inv_freq must hold {dim // 2} entries, got {inv_freq.numel()}")
    queries, q_out = _queries(q_pe, q_out, k_pe, dim, "q_pe")
    t, ld, width, num_rows = _table(page_table, dev)
    bs, ind, rp = _batch(q_indptr, rows, dev)
    check(spec_calls().spec_latent_write(
        *queries, lp, lt, kp, kt, _CODES[k_pe.dtype], _f32("inv_freq", inv_freq, dev),
        bool(interleaved), factor, _positions(positions, dev, n), c, t, ld, width, num_rows,
        0 if page_counts is None else _i32("page_counts", page_counts, dev, num_rows),
        _i32("kv_lens", kv_lens, dev, num_rows), rp, ind, bs, n,
        0 if cache_scale is None else _f32("cache_scale", cache_scale, dev, 1), _stream(cache)))
    return q_out


def spec_latent_gather(cache, page_table, kv_indptr, num_tokens, rows=None, cache_scale=None,
                       dtype=None, page_counts=None, out=None):
    """Rows of one layer's cache next to each other: the first kv_indptr[r + 1] - kv_indptr[r]
    positions of request r in rows kv_indptr[r] .. of the result (``num_tokens``, columns).  Of a
    float8_e4m3fn cache they are times ``cache_scale`` in ``dtype`` (bfloat16 unless given).
    Positions without a page (with ``page_counts``: past those that the row holds) are zeros."""
    dev = cache.get_device()
    # (rows are copied whole: where the key part begins does not matter)
    c, wide = _latents(cache, min(cache.shape[-1] - 1, 64 if cache.shape[-1] > 512 else
                                  16 // cache.element_size()))
    n = int(num_tokens)
    if out is None:
        if dtype is None:
            dtype = torch.bfloat16 if cache.dtype is torch.float8_e4m3fn else cache.dtype
        if dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"dtype must be bfloat16 or float16, got {dtype}")
        out = torch.empty((n, wide), dtype=dtype, device=cache.device)
    elif out.shape != (n, wide) or out.get_device() != dev or dtype not in (None, out.dtype):
        raise ValueError(f"out must be ({n}, {wide}) on the cache's device, got "
                         f"{tuple(out.shape)} {out.dtype}")
    op, ot = _rows2("out", out)
    t, ld, width, num_rows = _table(page_table, dev)
    bs, ind, rp = _batch(kv_indptr, rows, dev)
    check(spec_calls().spec_latent_gather(
        c, t, ld, width, num_rows,
        0 if page_counts is None else _i32("page_counts", page_counts, dev, num_rows), rp, ind, bs,
        n, op, ot, _CODES[out.dtype],
        0 if cache_scale is None else _f32("cache_scale", cache_scale, dev, 1), _stream(cache)))
    return out


def spec_latent_attention(q, cache, page_table, kv_lens, q_indptr, max_q_len, max_kv_len,
                          latent_dim, scale, tree_mask=None, rows=None, cache_scale=None, out=None,
                          workspace=None):
    """Attention over one layer's cache of latents, which holds the tokens' own rows already:
    every head's keys are the rows, its values their first ``latent_dim`` columns.  ``q`` (tokens,
    heads, columns) are the absorbed queries with their rotated parts behind them, ``scale`` that of
    the heads as the model has them.  Visibility, ``max_q_len``, ``max_kv_len`` and roundings as in
    spec_attention.  ``workspace``: a contiguous tensor on q's device for calls that follow one
    another (None: scratch of the stream's own).  Returns ``out`` (tokens, heads, latent_dim)."""
    dev = q.get_device()
    qp, qt, qh = _heads("q", q)
    n, H, wide = q.shape
    c, columns = _latents(cache, wide - latent_dim)
    if columns != wide or cache.get_device() != dev:
        raise ValueError(f"q {tuple(q.shape)} does not match the cache {tuple(cache.shape)} on its "
                         f"device")
    if out is None:
        out = torch.empty((n, H, latent_dim), dtype=q.dtype, device=q.device)
    elif out.shape != (n, H, latent_dim) or out.dtype is not q.dtype or out.get_device() != dev:
        raise ValueError(f"out {tuple(out.shape)} {out.dtype} must be ({n}, {H}, {latent_dim}) "
                         f"like q")
    op, ot, oh = _heads("out", out)
    t, ld, width, num_rows = _table(page_table, dev)
    bs, ind, rp = _batch(q_indptr, rows, dev)
    mp, words = 0, 0
    if tree_mask is not None:
        if tree_mask.dtype is not torch.int64 or tree_mask.get_device() != dev \
                or tree_mask.dim() != 2 or tree_mask.shape[0] != n \
                or not tree_mask.is_contiguous() or (n > 0 and tree_mask.shape[1] == 0):
            raise ValueError(f"tree_mask must be a contiguous int64 (tokens, words) tensor, got "
                             f"{tuple(tree_mask.shape)} {tree_mask.dtype}")
        mp, words = tree_mask.data_ptr(), tree_mask.shape[1]
    calls = spec_calls()
    if workspace is None:
        need = calls.spec_latent_attention_workspace_bytes(bs, H, latent_dim, _CODES[cache.dtype],
                                                           max_q_len, max_kv_len)
        wp, wn, _held = _workspace(q, need, False)
    else:
        wp, wn = _given_workspace(workspace, dev)
    check(calls.spec_latent_attention(
        qp, qt, qh, op, ot, oh, _CODES[q.dtype], H, c, t, ld, width, num_rows,
        _i32("kv_lens", kv_lens, dev, num_rows), rp, ind, bs, n, mp, words, scale,
        0 if cache_scale is None else _f32("cache_scale", cache_scale, dev, 1), max_q_len,
        max_kv_len, wp, wn, _stream(q)))
    return out


def spec_latent_prefill(q, k, v, k_pe, q_indptr, kv_indptr, max_q_len, max_kv_len=None,
                        scale=None, out=None):
    """Causal attention over expanded latents: the queries of request r, rows q_indptr[r] .. of
    ``q`` (tokens, heads, nope + rope), are the last of its tokens, whose keys and values are rows
    kv_indptr[r] .. of ``k`` (.., heads, nope), ``v`` (.., heads, v_dim) and ``k_pe`` (.., rope), the
    rotated key part of all heads.  ``max_q_len`` bounds a request's queries; it shapes the launch,
    not the result.  ``max_kv_len`` is not used: a row block takes all of its keys, and nothing is
    divided over them.  ``scale`` defaults to (nope + rope) ** -0.5.  Returns ``out`` (tokens,
    heads, v_dim)."""
    dev = q.get_device()
    qp, qt, qh = _heads("q", q)
    kp, kt, kh = _heads("k", k)
    vp, vt, vh = _heads("v", v)
    rp, rt = _rows2("k_pe", k_pe)
    n, H, d = q.shape
    m, dn, dr, dv = k.shape[0], k.shape[2], k_pe.shape[1], v.shape[2]
    if dev < 0 or any(x.get_device() != dev or x.dtype is not q.dtype for x in (k, v, k_pe)):
        raise ValueError("q, k, v and k_pe must be of one type on one ROCm device")
    if k.shape[1] != H or v.shape[:2] != (m, H) or k_pe.shape[0] != m or d != dn + dr:
        raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)} and k_pe "
                         f"{tuple(k_pe.shape)} do not match")
    if max_kv_len is not None and max_kv_len < 0:
        raise ValueError(f"max_kv_len={max_kv_len} is negative")
    if out is None:
        out = torch.empty((n, H, dv), dtype=q.dtype, device=q.device)
    elif out.shape != (n, H, dv) or out.dtype is not q.dtype or out.get_device() != dev:
        raise ValueError(f"out {tuple(out.shape)} {out.dtype} must be ({n}, {H}, {dv}) like q")
    op, ot, oh = _heads("out", out)
    bs, ind, _ = _batch(q_indptr, None, dev)
    check(spec_calls().spec_latent_prefill(
        qp, qt, qh, kp, kt, kh, vp, vt, vh, rp, rt, op, ot, oh, _CODES[q.dtype], H, dn, dr, dv,
        ind, _i32("kv_indptr", kv_indptr, dev, bs + 1), bs, n, m,
        d ** -0.5 if scale is None else scale, max_q_len, _stream(q)))
    return out


class PagedLatentCache:
    """Latents of ``num_layers`` layers in pages, with the page tables of ``max_rows`` sequences,
    all on the device; the counterpart of PagedKVCache, whose notes on pages that run out hold
    here too.

    ``data`` is (layers, pages, page_size, latent_dim + rope_dim); ``page_table``, ``page_counts``,
    ``kv_lens`` and ``ref_counts`` are as there.  The float8_e4m3fn cache has ``scale`` (layers, 1),
    one unless set.
    """

    def __init__(self, num_layers, num_pages, page_size, latent_dim, rope_dim, max_rows,
                 max_pages_per_row, dtype=torch.bfloat16, device="cuda"):
        if dtype not in _CODES:
            raise TypeError(f"dtype must be bfloat16, float16 or float8_e4m3fn, got {dtype}")
        if (latent_dim + rope_dim) * dtype.itemsize % 32:
            raise ValueError(f"latent_dim={latent_dim} and rope_dim={rope_dim} together must be a "
                             f"multiple of 32 bytes")
        self.page_size, self.latent_dim, self.rope_dim = int(page_size), latent_dim, rope_dim
        self.data = torch.zeros((num_layers, num_pages, page_size, latent_dim + rope_dim),
                                dtype=dtype, device=device)
        i32 = {"dtype": torch.int32, "device": device}
        self.page_table = torch.zeros((max_rows, max_pages_per_row), **i32)
        self.page_counts = torch.zeros(max_rows, **i32)
        self.kv_lens = torch.zeros(max_rows, **i32)
        self.ref_counts = torch.zeros(num_pages, **i32)
        self.scale = None
        if dtype == torch.float8_e4m3fn:
            self.scale = torch.ones((num_layers, 1), device=device)

    def _scale(self, layer):
        return None if self.scale is None else self.scale[layer]

    def _halves(self):
        """The rows as keys and values for the calls that move whole rows."""
        x = self.data.unsqueeze(3)
        half = x.shape[-1] // 2
        return x[..., :half], x[..., half:]

    def reserve(self, rows, lens):
        """Pages for ``lens`` tokens in ``rows`` (the tokens held stay as they are)."""
        return spec_kv_resize(self.page_table, self.page_counts, self.ref_counts, rows, lens,
                              self.page_size)

    def commit(self, rows, lens):
        """``rows`` hold ``lens`` tokens: their lengths are set and the pages past them given
        back (0: the row is released)."""
        return spec_kv_resize(self.page_table, self.page_counts, self.ref_counts, rows, lens,
                              self.page_size, kv_lens=self.kv_lens)

    def fork(self, src_rows, dst_rows):
        return spec_kv_fork(*self._halves(), self.page_table, self.page_counts, self.ref_counts,
                            self.kv_lens, src_rows, dst_rows)

    def copy_pages(self, src_pages, dst_pages):
        spec_kv_copy_pages(*self._halves(), src_pages, dst_pages)

    def write(self, layer, q_pe, latent, k_pe, inv_freq, q_indptr, rows=None, positions=None,
              interleaved=True, factor=1.0, q_out=None):
        """New rows, with the rotation on the way; returns the queries' rotated parts."""
        return spec_latent_write(q_pe, latent, k_pe, inv_freq, self.data[layer], self.page_table,
                                 self.kv_lens, q_indptr, rows, positions, interleaved, factor,
                                 self._scale(layer), self.page_counts, q_out)

    def attention(self, layer, q, q_indptr, max_q_len, max_kv_len, scale, tree_mask=None,
                  rows=None, out=None):
        return spec_latent_attention(q, self.data[layer], self.page_table, self.kv_lens, q_indptr,
                                     max_q_len, max_kv_len, self.latent_dim, scale, tree_mask,
                                     rows, self._scale(layer), out)

    def gather(self, layer, kv_indptr, num_tokens, rows=None, dtype=None, out=None):
        """(latents, rotated key parts) of the requests' rows, next to each other."""
        x = spec_latent_gather(self.data[layer], self.page_table, kv_indptr, num_tokens, rows,
                               self._scale(layer), dtype, self.page_counts, out)
        return x[:, :self.latent_dim], x[:, self.latent_dim:]

    def compact(self, path, accept_lens, rows=None):
        """Moves the accepted rows together; returns the lengths to ``commit``."""
        return spec_kv_compact(*self._halves(), self.page_table, self.kv_lens, path, accept_lens,
                               rows, page_counts=self.page_counts)


__all__ = ["PagedLatentCache", "spec_latent_attention", "spec_latent_gather",
           "spec_latent_prefill", "spec_latent_write"]
