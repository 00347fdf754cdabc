"""The speculative decoding step over a paged key/value cache.

Each ``spec_*`` function has the name of the C entry point it calls
(include/sgg_spec.h, which says what it computes) and only checks and marshals
its arguments; the work is enqueued on torch's current stream of the tensors'
device.  ``PagedKVCache`` holds the state of a cache and calls them on it.

Ragged arrays hold the tokens of a batch request by request, request r in rows
``q_indptr[r]`` to ``q_indptr[r + 1]``.  ``rows`` names the cache row of each
request (None: request r is row r).  Index arrays are contiguous int32 tensors
on the device; the host never reads them.
"""

import torch

from ._lib import check, spec_calls, tensor_args
from .binding import _stream

_CODES = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 2}

# the checks of one tensor argument each (csrc/tensorargs.cpp)
_args = tensor_args()
_i32, _f32, _table, _cache, _heads = _args.i32, _args.f32, _args.table, _args.cache, _args.heads
_new_i32 = _args.new_i32


_workspaces = {}
_outgrown = []


def _workspace(t, nbytes):
    """Scratch of ``nbytes`` for a call on tensor ``t``'s current stream: (address, bytes).

    Zero when it is made; every call leaves its counters at zero.  One grow-only buffer per
    stream, so calls on different streams never share one; an outgrown buffer is kept, for a
    kernel under way may still use it.  While a graph is captured the call gets a buffer of its
    own, cleared in the graph: the graph's memory is not the streams'.
    """
    if nbytes <= 0:
        return 0, 0, None
    stream = _stream(t)
    if torch._C._cuda_isCurrentStreamCapturing():
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=t.device)
        return ws.data_ptr(), nbytes, ws
    key = (t.get_device(), stream)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        size = max(int(nbytes), 1 << 22)
        if ws is not None:
            size = max(size, 2 * ws.numel())
            _outgrown.append(ws)
        ws = _workspaces[key] = torch.zeros(size, dtype=torch.uint8, device=t.device)
    return ws.data_ptr(), ws.numel(), ws


def _given_workspace(workspace, dev):
    """(address, bytes) of a caller's workspace; the library checks its size and alignment."""
    if not isinstance(workspace, torch.Tensor):
        raise TypeError(f"workspace must be a tensor, got {type(workspace).__name__}")
    if dev < 0 or workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the call's ROCm device")
    return workspace.data_ptr(), workspace.nbytes


def _batch(q_indptr, rows, dev):
    """Requests of the batch, addresses of q_indptr and rows."""
    p = _i32("q_indptr", q_indptr, dev)
    bs = q_indptr.numel() - 1
    if bs < 0 or q_indptr.dim() != 1:
        raise ValueError("q_indptr must hold bs + 1 entries")
    return bs, p, 0 if rows is None else _i32("rows", rows, dev, bs)


def spec_kv_resize(page_table, page_counts, ref_counts, rows, new_lens, page_size, kv_lens=None,
                   status=None):
    """Hold exactly the pages that ``new_lens`` (n) tokens need in cache rows ``rows`` (None:
    0 .. n - 1): give up the pages past them, then take the missing ones (lowest free page
    first).  ``kv_lens`` (rows of the table), if given, gets the new lengths.  Returns
    ``status`` (int32 [2]): pages missing (not 0: no row has grown), rows left alone."""
    dev = page_table.get_device()
    t, ld, width, num_rows = _table(page_table, dev)
    n = new_lens.numel()
    if status is None:
        status = _new_i32(page_table, 2)
    check(spec_calls().spec_kv_resize(
        t, ld, width, num_rows, _i32("page_counts", page_counts, dev, num_rows),
        _i32("ref_counts", ref_counts, dev), ref_counts.numel(),
        0 if rows is None else _i32("rows", rows, dev, n),
        _i32("new_lens", new_lens, dev, n), n, int(page_size),
        0 if kv_lens is None else _i32("kv_lens", kv_lens, dev, num_rows),
        _i32("status", status, dev, 2), _stream(page_table)))
    return status


def spec_kv_fork(k_cache, v_cache, page_table, page_counts, ref_counts, kv_lens, src_rows,
                 dst_rows, status=None):
    """Row dst_rows[i], which holds no page, goes on from row src_rows[i]: full pages are shared,
    the partial last page is copied into a fresh one in every layer.  A row that is cut back into a
    shared page is not to be written there: fork it then, and release it.  Returns ``status``
    (int32 [2]): pages missing (not 0: nothing was done), pairs left alone."""
    dev = page_table.get_device()
    c, (_, P, _, _, _) = _cache(k_cache, v_cache)
    if k_cache.get_device() != dev:
        raise ValueError("the cache must be on the page table's device")
    t, ld, width, num_rows = _table(page_table, dev)
    n = src_rows.numel()
    if status is None:
        status = _new_i32(page_table, 2)
    ws = _new_i32(page_table, 3 * n)
    check(spec_calls().spec_kv_fork(
        c, t, ld, width, num_rows, _i32("page_counts", page_counts, dev, num_rows),
        _i32("ref_counts", ref_counts, dev, P), _i32("kv_lens", kv_lens, dev, num_rows),
        _i32("src_rows", src_rows, dev, n), _i32("dst_rows", dst_rows, dev, n), n,
        _i32("status", status, dev, 2), ws.data_ptr(), 12 * n, _stream(page_table)))
    return status


def spec_kv_copy_pages(k_cache, v_cache, src_pages, dst_pages):
    """Page dst_pages[i] becomes a copy of page src_pages[i] in every layer."""
    dev = k_cache.get_device()
    c, _ = _cache(k_cache, v_cache)
    n = src_pages.numel()
    check(spec_calls().spec_kv_copy_pages(
        c, _i32("src_pages", src_pages, dev, n), _i32("dst_pages", dst_pages, dev, n), n,
        _stream(k_cache)))


def spec_kv_write(k, v, k_cache, v_cache, page_table, kv_lens, q_indptr, rows=None, k_scale=None,
                  v_scale=None, page_counts=None):
    """Keys and values (tokens, kv heads, head_dim) of one layer into that layer's cache, token i
    of request r at position kv_lens[row] + i.  A float8_e4m3fn cache takes x / scale[head].
    With ``page_counts`` (rows of the table) tokens past the pages that their row holds are
    skipped; without it every position has to have a page, for table entries past a row's count
    may name other rows' pages."""
    dev = k_cache.get_device()
    c, (L, _, _, H, D) = _cache(k_cache, v_cache)
    if L != 1:
        raise ValueError(f"k and v belong to one layer, the cache has {L}: "
                         f"{tuple(k_cache.shape)}")
    kp, kt, kh = _heads("k", k)
    vp, vt, vh = _heads("v", v)
    n = k.shape[0]
    if k.shape != (n, H, D) or v.shape != (n, H, D) or v.dtype is not k.dtype:
        raise ValueError(f"k {tuple(k.shape)} {k.dtype} and v {tuple(v.shape)} {v.dtype} must be "
                         f"(tokens, {H}, {D}) of one type")
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError("k and v must be on the cache's device")
    t, ld, width, num_rows = _table(page_table, dev)
    bs, ind, rp = _batch(q_indptr, rows, dev)
    new = (kp, kt, kh, vp, vt, vh, _CODES[k.dtype], c, t, ld, width, num_rows)
    batch = (_i32("kv_lens", kv_lens, dev, num_rows), rp, ind, bs, n,
             0 if k_scale is None else _f32("k_scale", k_scale, dev, H),
             0 if v_scale is None else _f32("v_scale", v_scale, dev, H), _stream(k_cache))
    if page_counts is None:
        check(spec_calls().spec_kv_write(*new, *batch))
    else:
        check(spec_calls().spec_kv_write_held(
            *new, _i32("page_counts", page_counts, dev, num_rows), *batch))


def spec_kv_compact(k_cache, v_cache, page_table, kv_lens, path, accept_lens, rows=None,
                    new_lens=None, page_counts=None):
    """After a verification, in every layer, the accepted tokens' rows move together: position
    kv_len + path[r, j] to kv_len + j.  ``page_counts`` as in spec_kv_write.  Returns the requests'
    new lengths (bs)."""
    dev = k_cache.get_device()
    c, _ = _cache(k_cache, v_cache)
    t, ld, width, num_rows = _table(page_table, dev)
    if path.dim() != 2:
        raise ValueError(f"path must be (requests, width), got {tuple(path.shape)}")
    bs, w = path.shape
    if new_lens is None:
        new_lens = _new_i32(k_cache, bs)
    table = (c, t, ld, width, num_rows)
    batch = (_i32("kv_lens", kv_lens, dev, num_rows),
             0 if rows is None else _i32("rows", rows, dev, bs), _i32("path", path, dev), w, w,
             _i32("accept_lens", accept_lens, dev, bs), _i32("new_lens", new_lens, dev, bs), bs,
             _stream(k_cache))
    if page_counts is None:
        check(spec_calls().spec_kv_compact(*table, *batch))
    else:
        check(spec_calls().spec_kv_compact_held(
            *table, _i32("page_counts", page_counts, dev, num_rows), *batch))
    return new_lens


def spec_tree_mask(parents, q_indptr, kv_lens, mask_words, rows=None):
    """Visibility and positions of trees of drafted tokens from their parents (local indexes, -1
    for none): (mask (tokens, mask_words) int64, bit j of a row for the token itself and its
    ancestors j; positions (tokens) int32)."""
    dev = parents.get_device()
    p = _i32("parents", parents, dev)
    bs, ind, rp = _batch(q_indptr, rows, dev)
    n = parents.numel()
    mask = torch.empty((n, int(mask_words)), dtype=torch.int64, device=parents.device)
    positions = _new_i32(parents, n)
    check(spec_calls().spec_tree_mask(p, ind, bs, n, _i32("kv_lens", kv_lens, dev), rp,
                                      kv_lens.numel(), mask.data_ptr(), int(mask_words),
                                      positions.data_ptr(), _stream(parents)))
    return mask, positions


def spec_attention(q, k_cache, v_cache, page_table, kv_lens, q_indptr, max_q_len, max_kv_len,
                   tree_mask=None, rows=None, scale=None, k_scale=None, v_scale=None, out=None,
                   workspace=None):
    """Attention of the drafted tokens q (tokens, heads, head_dim) over one layer's cache, which
    holds their own keys and values already (spec_kv_write).  Token i of a request sees its
    context and the drafted tokens of its row of ``tree_mask`` (spec_tree_mask; None: those up to
    itself).  ``max_q_len`` / ``max_kv_len`` bound the batch's tokens per request and keys per
    request (context and drafts); they shape the launch, not the result.  The softmax's weights are
    rounded to q's type for the product with the values, all else is float32.  ``scale`` defaults to
    head_dim ** -0.5.  ``workspace``: a contiguous tensor on q's device that is zero on first use,
    for calls that follow one another (None: scratch of the stream's own).  Returns ``out``
    (like q)."""
    dev = q.get_device()
    c, (L, _, _, H, D) = _cache(k_cache, v_cache)
    qp, qt, qh = _heads("q", q)
    n, hq, d = q.shape
    if L != 1 or d != D or k_cache.get_device() != dev:
        raise ValueError(f"q {tuple(q.shape)} does not match one layer's cache "
                         f"{tuple(k_cache.shape)} on its device")
    if out is None:
        out = torch.empty((n, hq, d), dtype=q.dtype, device=q.device)
    elif out.shape != q.shape or out.dtype is not q.dtype or out.get_device() != dev:
        raise ValueError(f"out {tuple(out.shape)} {out.dtype} does not match q")
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
    calls, code = spec_calls(), _CODES[k_cache.dtype]
    if workspace is None:
        need = calls.spec_attention_workspace_bytes(bs, hq, H, D, code, max_q_len, max_kv_len)
        wp, wn, _held = _workspace(q, need)
    else:
        wp, wn = _given_workspace(workspace, dev)
    check(calls.spec_attention(
        qp, qt, qh, op, ot, oh, _CODES[q.dtype], hq, c, t, ld, width, num_rows,
        _i32("kv_lens", kv_lens, dev, num_rows), rp, ind, bs, n, mp, words,
        D ** -0.5 if scale is None else scale,
        0 if k_scale is None else _f32("k_scale", k_scale, dev, H),
        0 if v_scale is None else _f32("v_scale", v_scale, dev, H), max_q_len, max_kv_len, wp, wn,
        _stream(q)))
    return out


def spec_verify(tokens, parents, q_indptr, target_probs, uniforms, final_uniforms, max_q_len,
                draft_probs=None, workspace=None):
    """Which drafted tokens the target accepts, and its next token, from given random numbers:
    (path (bs, max_q_len): accepted nodes' local indexes, node 0 first, then -1; accept_lens
    (bs); next_tokens (bs)).  Row n of ``target_probs`` (tokens, vocab) float32 is the target's
    distribution after node n; row n of ``draft_probs`` the one its children were drawn from
    (None: the candidates were chosen, not drawn).  ``workspace`` as in spec_attention."""
    dev = target_probs.get_device()
    bs, ind, _ = _batch(q_indptr, None, dev)
    n = tokens.numel()
    for name, x in (("target_probs", target_probs), ("draft_probs", draft_probs)):
        if x is not None and (x.dtype is not torch.float32 or x.dim() != 2
                              or x.get_device() != dev or x.shape[0] != n
                              or x.shape[1] != target_probs.shape[1] or x.stride(1) != 1):
            raise ValueError(f"{name} must be float32 (tokens, vocab) rows, got "
                             f"{tuple(x.shape)} {x.dtype}")
    V = target_probs.shape[1]
    path = _new_i32(target_probs, bs, int(max_q_len))
    accept, nxt = _new_i32(target_probs, bs), _new_i32(target_probs, bs)
    calls = spec_calls()
    if workspace is None:
        wp, wn, _held = _workspace(target_probs, calls.spec_verify_workspace_bytes(bs, V))
    else:
        wp, wn = _given_workspace(workspace, dev)
    check(calls.spec_verify(
        _i32("tokens", tokens, dev, n), _i32("parents", parents, dev, n), ind, bs, n,
        target_probs.data_ptr(), target_probs.stride(0) if n > 1 else V,
        0 if draft_probs is None else draft_probs.data_ptr(),
        0 if draft_probs is None else (draft_probs.stride(0) if n > 1 else V), V,
        _f32("uniforms", uniforms, dev, n), _f32("final_uniforms", final_uniforms, dev, bs),
        path.data_ptr(), int(max_q_len), int(max_q_len), accept.data_ptr(), nxt.data_ptr(), wp, wn,
        _stream(target_probs)))
    return path, accept, nxt


def spec_set_option(name, value):
    """Process-wide setting ("verify_spin_limit": polls); returns the previous value."""
    old = spec_calls().spec_set_option(name.encode() + b"\0", int(value))
    if old < 0:
        raise ValueError(f"unknown option {name!r} or negative value {value}")
    return old


class PagedKVCache:
    """Keys and values of ``num_layers`` layers in pages, with the page tables of ``max_rows``
    sequences, all on the device.

    ``k`` / ``v`` are (layers, pages, page_size, kv heads, head_dim); ``page_table``
    (max_rows, max_pages_per_row), ``page_counts``, ``kv_lens`` (max_rows) and ``ref_counts``
    (pages) are int32.  The float8_e4m3fn cache has ``k_scale`` / ``v_scale`` (layers, kv heads),
    one unless set.

    Pages can run out: ``status[0]`` of ``reserve`` then counts the missing ones, and no row has
    grown.  Nothing is written past the pages that a row holds, so the other rows keep their
    contents; the results of the rows that needed pages are worthless, and the step is not to be
    committed for them: look at the status before ``commit``, make room and reserve again.
    """

    def __init__(self, num_layers, num_pages, page_size, num_kv_heads, head_dim, max_rows,
                 max_pages_per_row, dtype=torch.bfloat16, device="cuda"):
        if dtype not in _CODES:
            raise TypeError(f"dtype must be bfloat16, float16 or float8_e4m3fn, got {dtype}")
        shape = (num_layers, num_pages, page_size, num_kv_heads, head_dim)
        self.page_size = int(page_size)
        self.k = torch.zeros(shape, dtype=dtype, device=device)
        self.v = torch.zeros(shape, dtype=dtype, device=device)
        i32 = {"dtype": torch.int32, "device": device}
        self.page_table = torch.zeros((max_rows, max_pages_per_row), **i32)
        self.page_counts = torch.zeros(max_rows, **i32)
        self.kv_lens = torch.zeros(max_rows, **i32)
        self.ref_counts = torch.zeros(num_pages, **i32)
        self.k_scale = self.v_scale = None
        if dtype == torch.float8_e4m3fn:
            self.k_scale = torch.ones((num_layers, num_kv_heads), device=device)
            self.v_scale = torch.ones((num_layers, num_kv_heads), device=device)

    def _scales(self, layer):
        if self.k_scale is None:
            return {}
        return {"k_scale": self.k_scale[layer], "v_scale": self.v_scale[layer]}

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
        return spec_kv_fork(self.k, self.v, self.page_table, self.page_counts, self.ref_counts,
                            self.kv_lens, src_rows, dst_rows)

    def copy_pages(self, src_pages, dst_pages):
        spec_kv_copy_pages(self.k, self.v, src_pages, dst_pages)

    def write(self, layer, k, v, q_indptr, rows=None):
        spec_kv_write(k, v, self.k[layer], self.v[layer], self.page_table, self.kv_lens,
                      q_indptr, rows, page_counts=self.page_counts, **self._scales(layer))

    def attention(self, layer, q, q_indptr, max_q_len, max_kv_len, tree_mask=None, rows=None,
                  scale=None, out=None):
        return spec_attention(q, self.k[layer], self.v[layer], self.page_table, self.kv_lens,
                              q_indptr, max_q_len, max_kv_len, tree_mask, rows, scale, out=out,
                              **self._scales(layer))

    def compact(self, path, accept_lens, rows=None):
        """Moves the accepted rows together; returns the lengths to ``commit``."""
        return spec_kv_compact(self.k, self.v, self.page_table, self.kv_lens, path, accept_lens,
                               rows, page_counts=self.page_counts)


__all__ = ["PagedKVCache", "spec_attention", "spec_kv_compact", "spec_kv_copy_pages",
           "spec_kv_fork", "spec_kv_resize", "spec_kv_write", "spec_set_option", "spec_tree_mask",
           "spec_verify"]
