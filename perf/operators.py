"""Cases of the speculative decoding operators: attention for drafted tokens over a paged cache,
verification of drafted tokens, and the upkeep of the cache's pages.

``run`` computes a case either in plain torch operations (``own`` false) or through this
repository's operators (``own`` true); ``exact`` computes it from the definitions in 64 bits.
"""

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "fp16": 2, "e4m3": 1}
E4M3_MAX = 448.0


# ------------------------------------------------------------------- the cases

def _attention(name, bs, q_len, ctx, tree, hq=32, hkv=8, d=128, page=16, dtype="bf16",
               cache="same", heads_first=False):
    return {"name": name, "op": "attention", "bs": bs, "q_len": q_len, "ctx": ctx, "tree": tree,
            "hq": hq, "hkv": hkv, "d": d, "page": page, "dtype": dtype, "cache": cache,
            "heads_first": heads_first}


def _verify(name, bs, q_len, vocab, drawn, chain):
    return {"name": name, "op": "verify", "bs": bs, "q_len": q_len, "vocab": vocab,
            "drawn": drawn, "chain": chain}


def _draft(name, bs, q_len, ctx, layers, hkv=8, d=128, page=16, dtype="bf16", cache="same",
           heads_first=False):
    return {"name": name, "op": "draft", "bs": bs, "q_len": q_len, "ctx": ctx, "layers": layers,
            "hkv": hkv, "d": d, "page": page, "dtype": dtype, "cache": cache,
            "heads_first": heads_first}


def _fork(name, bs, copies, ctx, layers, hkv=8, d=128, page=16, cache="bf16", heads_first=False):
    return {"name": name, "op": "fork", "bs": bs, "copies": copies, "ctx": ctx, "layers": layers,
            "hkv": hkv, "d": d, "page": page, "cache": cache, "heads_first": heads_first}


def listed():
    return [
        # one user waiting for one token early in a conversation: latency alone
        _attention("attn_one", 1, 1, 500, False),
        # the decode batch of 256 one-token requests, at middling contexts
        _attention("attn_decode", 256, 1, 2048, False),
        # a verification step: 16 drafted tokens in a tree for each of 64 requests
        _attention("attn_tree", 64, 16, 4096, True, heads_first=True),
        # two long documents in an 8-bit cache with a short draft each, a ragged length
        _attention("attn_long_e4m3", 2, 8, 100003, True, page=64, cache="e4m3"),
        # prompts taken in chunks: 8 requests of 512 tokens behind an earlier context, causal
        _attention("attn_chunk", 8, 512, 1536, False, dtype="fp16"),
        # a single user's chain of drafts sampled from a draft model, a small vocabulary
        _verify("verify_one", 1, 5, 32000, True, True),
        # trees of candidates without draft probabilities, the batch of attn_tree
        _verify("verify_tree", 64, 16, 128256, False, False),
        # trees sampled from a draft model: rejections need the residual's mass over the vocabulary
        _verify("verify_drawn", 48, 9, 128256, True, False),
        # pages, mask, new rows and accepted rows of one user's step, an 8-bit cache
        _draft("draft_one", 1, 5, 300, 2, cache="e4m3"),
        # the same for the batch of attn_tree over a 32-layer model
        _draft("draft_step", 64, 16, 200, 32),
        # one prompt forked into 4 samples, then released
        _fork("fork_one", 1, 4, 301, 2),
        # parallel sampling: 64 prompts forked into 4 samples each over 32 layers, then released
        _fork("fork_samples", 64, 4, 200, 32, heads_first=True),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["attention", "attention", "verify", "draft", "fork"])
    hkv, d = rng.choice([(8, 128), (8, 128), (4, 128), (2, 64), (8, 64), (1, 256), (4, 96)])
    page = rng.choice([8, 16, 16, 32, 64])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    cache = rng.choice(["same", "same", "e4m3"])
    first = rng.random() < 0.5
    if op == "attention":
        tree = rng.random() < 0.6
        q_len = _log(rng, 2, 64) if tree else rng.choice([1, 1, _log(rng, 2, 300)])
        bs = _log(rng, 1, 200) if q_len <= 64 else _log(rng, 1, 8)
        group = rng.choice([1, 2, 4, 4, 7, 8])
        ctx = _log(rng, 1, 100000)
        while bs * (ctx + q_len) * hkv * d > 250 * 1000 * 1024 \
                or bs * (ctx + q_len) * q_len * hkv * group > 150 * 1000 * 1000:
            bs, ctx = max(1, bs * 2 // 3), max(1, ctx * 2 // 3)
        return dict(_attention("", bs, q_len, ctx, tree, hkv * group, hkv, d, page, dtype, cache,
                               first), name="drawn")
    if op == "verify":
        bs, q_len, vocab = _log(rng, 1, 64), _log(rng, 2, 24), _log(rng, 1000, 150000)
        drawn = rng.random() < 0.5
        while bs * q_len * vocab * (2 if drawn else 1) > 100 * 1000 * 1000:
            bs, q_len = max(1, bs * 2 // 3), max(2, q_len * 3 // 4)
        return dict(_verify("", bs, q_len, vocab, drawn, rng.random() < 0.4), name="drawn")
    layers = _log(rng, 1, 32)
    bs, ctx = _log(rng, 1, 64), _log(rng, 1, 200)
    if op == "draft":
        q_len = _log(rng, 2, 32)
        while bs * (ctx + q_len + 2 * page) * layers * hkv * d > 450 * 1000 * 1000:
            layers = max(1, layers // 2)
            bs = max(1, bs * 3 // 4)
        return dict(_draft("", bs, q_len, ctx, layers, hkv, d, page, dtype, cache, first),
                    name="drawn")
    copies = rng.choice([1, 2, 3, 4, 8])
    while bs * (ctx + (copies + 1) * page) * layers * hkv * d > 450 * 1000 * 1000:
        layers = max(1, layers // 2)
        bs = max(1, bs * 3 // 4)
    return dict(_fork("", bs, copies, ctx, layers, hkv, d, page,
                      dtype if cache == "same" else cache, first), name="drawn")


# ------------------------------------------------------------------ the inputs

def _lens(bs, top, low, rs):
    """Lengths spread evenly over [low, top], in an order of the seed's."""
    return rs.permutation(np.linspace(top, low, bs).round().astype(np.int64))


def _parents(lens, chain, rs):
    """Trees of drafted tokens: node 0 the last accepted token, at most 4 children a node."""
    out = []
    for n in lens:
        kids = [0] * int(n)
        par = [-1]
        for i in range(1, int(n)):
            p = i - 1
            if not chain:
                near = [j for j in range(max(0, i - 6), i) if kids[j] < 4] or [i - 1]
                p = int(near[rs.randint(len(near))])
            kids[p] += 1
            par.append(p)
        out.append(par)
    return out


def _ancestors(par):
    """(n, n) truth values: column j is row i itself or one of its ancestors."""
    m = np.zeros((len(par), len(par)), bool)
    for i, p in enumerate(par):
        if p >= 0:
            m[i] = m[p]
        m[i, i] = True
    return m


def _words(trees, words):
    rows = [np.packbits(np.pad(_ancestors(p), ((0, 0), (0, 64 * words - len(p)))), axis=1,
                        bitorder="little").view(np.int64) for p in trees]
    return np.concatenate(rows, axis=0)


def _dev(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=dtype, device="cuda")


def _indptr(lens):
    return np.concatenate([[0], np.cumsum(lens)])


def _random(gen, shape, dtype, scale=1.0):
    if dtype == "e4m3":
        x = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
        flat, step = x.view(torch.uint8).view(-1), 1 << 26
        for i in range(0, flat.numel(), step):
            n = min(step, flat.numel() - i)
            y = torch.randn(n, generator=gen, device="cuda") * (scale * 16.0)
            flat[i:i + n] = y.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        return x
    return torch.randn(shape, generator=gen, device="cuda", dtype=DTYPES[dtype]).mul_(scale)


def _cache(gen, case, layers, pages, dtype):
    """Keys and values as (layers, pages, page, heads, d), in memory token by token or head by head."""
    shape = (layers, pages, case["page"], case["hkv"], case["d"])
    got = []
    for _ in range(2):
        if case["heads_first"]:
            got.append(_random(gen, (shape[0], shape[1], shape[3], shape[2], shape[4]),
                               dtype).transpose(2, 3))
        else:
            got.append(_random(gen, shape, dtype))
    return got


def _scales(case, gen):
    """Scales of an 8-bit cache, one for each kv head (None: the cache holds the values)."""
    if case.get("cache") != "e4m3" or case["op"] == "fork":
        return None, None
    s = torch.rand((2, case["hkv"]), generator=gen, device="cuda") * 0.02 + 0.05
    return s[0].contiguous(), s[1].contiguous()


def _prepare_attention(case, seed):
    rs, gen = np.random.RandomState(seed % (1 << 31)), torch.Generator("cuda").manual_seed(seed)
    bs, ps = case["bs"], case["page"]
    kv = _lens(bs, case["ctx"], case["ctx"] // 2, rs)
    ql = _lens(bs, case["q_len"], max(1, case["q_len"] * 3 // 4), rs)
    trees = _parents(ql, False, rs) if case["tree"] else None
    words = (case["q_len"] + 63) // 64
    counts = (kv + ql + ps - 1) // ps
    width, pages = int(counts.max()), int(counts.sum())
    table = np.zeros((bs, width), np.int64)
    order, at = rs.permutation(pages), 0
    for r, c in enumerate(counts):
        table[r, :c] = order[at:at + c]
        at += c
    cache = case["dtype"] if case["cache"] == "same" else case["cache"]
    k, v = (x[0] for x in _cache(gen, case, 1, pages, cache))
    ks, vs = _scales(case, gen)
    q = _random(gen, (int(ql.sum()), case["hq"], case["d"]), case["dtype"], 1.5)
    return {"case": case, "q": q, "k_cache": k, "v_cache": v, "page_table": _dev(table),
            "kv_lens": _dev(kv), "q_indptr": _dev(_indptr(ql)), "k_scale": ks, "v_scale": vs,
            "tree_mask": _dev(_words(trees, words), torch.int64) if trees else None,
            "scale": case["d"] ** -0.5, "max_q_len": int(ql.max()),
            "max_kv_len": int((kv + ql).max()), "trees": trees}


def _prepare_verify(case, seed):
    rs, gen = np.random.RandomState(seed % (1 << 31)), torch.Generator("cuda").manual_seed(seed)
    bs, V = case["bs"], case["vocab"]
    ql = _lens(bs, case["q_len"], max(1, case["q_len"] * 3 // 4), rs)
    trees = _parents(ql, case["chain"], rs)
    ptr = _indptr(ql)
    n = int(ptr[-1])
    # spread as widely as a language model's logits: a few tokens hold most of the mass
    logits = torch.randn((n, V), generator=gen, device="cuda") * 5.0
    guess = logits + torch.randn((n, V), generator=gen, device="cuda") * 0.7
    target = torch.softmax(logits, -1)
    draft = torch.softmax(guess, -1)
    kids = max(1, max((np.bincount([p for p in t if p >= 0]).max() for t in trees if len(t) > 1),
                      default=1))
    # the k-th child of a node: drawn from the draft's row, or the k-th likeliest in it
    if case["drawn"]:
        pick = torch.multinomial(draft, int(kids), replacement=True, generator=gen)
    else:
        pick = torch.topk(guess, int(kids), -1).indices
    parent = np.concatenate([np.asarray(t) for t in trees])
    up, rank = np.zeros(n, np.int64), np.zeros(n, np.int64)
    for r, t in enumerate(trees):
        seen = {}
        for i, p in enumerate(t):
            if p >= 0:
                up[ptr[r] + i], rank[ptr[r] + i] = ptr[r] + p, seen.get(p, 0)
                seen[p] = seen.get(p, 0) + 1
    tokens = pick[_dev(up, torch.int64), _dev(rank, torch.int64)].to(torch.int32)
    return {"case": case, "tokens": tokens, "parents": _dev(parent), "q_indptr": _dev(ptr),
            "target_probs": target, "draft_probs": draft if case["drawn"] else None,
            "uniforms": torch.rand(n, generator=gen, device="cuda"),
            "final_uniforms": torch.rand(bs, generator=gen, device="cuda"),
            "max_q_len": int(ql.max()), "max_children": int(kids), "trees": trees}


def _prepare_pages(case, seed):
    rs, gen = np.random.RandomState(seed % (1 << 31)), torch.Generator("cuda").manual_seed(seed)
    bs, ps = case["bs"], case["page"]
    fork = case["op"] == "fork"
    kv = _lens(bs, case["ctx"], max(1, case["ctx"] // 4), rs)
    ql = None if fork else _lens(bs, case["q_len"], max(1, case["q_len"] * 3 // 4), rs)
    counts = (kv + ps - 1) // ps
    extra = bs * case["copies"] if fork else bs * ((case["q_len"] + ps - 1) // ps)
    rows_n = bs * (1 + case["copies"]) if fork else bs + 3
    pages = int(counts.sum()) + extra + 5
    width = (case["ctx"] + (0 if fork else case["q_len"]) + ps - 1) // ps + 1
    table = rs.randint(0, pages, (rows_n, width))
    order, at = rs.permutation(pages), 0
    rows = rs.permutation(rows_n)
    page_counts, lens, refs = np.zeros(rows_n), np.zeros(rows_n), np.zeros(pages)
    for r, c in zip(rows, counts):
        table[r, :c] = order[at:at + c]
        refs[order[at:at + c]] = 1
        page_counts[r] = c
        at += c
    lens[rows[:bs]] = kv
    cache = case["cache"] if fork or case["cache"] != "same" else case["dtype"]
    k, v = _cache(gen, case, case["layers"], pages, cache)
    s = {"case": case, "k_cache": k, "v_cache": v, "page_table": _dev(table),
         "page_counts": _dev(page_counts), "kv_lens": _dev(lens), "ref_counts": _dev(refs)}
    if fork:
        s.update(src_rows=_dev(np.repeat(rows[:bs], case["copies"])), dst_rows=_dev(rows[bs:]),
                 zeros=_dev(np.zeros(rows_n - bs)))
        return s
    trees = _parents(ql, False, rs)
    path, accept = -np.ones((bs, int(ql.max())), np.int64), np.zeros(bs)
    for r, t in enumerate(trees):
        i, way = int(rs.randint(len(t))), []
        while i >= 0:
            way.append(i)
            i = t[i]
        path[r, :len(way)], accept[r] = way[::-1], len(way)
    shape = (int(ql.sum()), case["hkv"], case["d"])
    ks, vs = _scales(case, gen)
    s.update(rows=_dev(rows[:bs]), q_indptr=_dev(_indptr(ql)), grown=_dev(kv + ql), old=_dev(kv),
             parents=_dev(np.concatenate([np.asarray(t) for t in trees])), path=_dev(path),
             accept_lens=_dev(accept), k_new=_random(gen, shape, case["dtype"]),
             v_new=_random(gen, shape, case["dtype"]), k_scale=ks, v_scale=vs,
             max_q_len=int(ql.max()), mask_words=(case["q_len"] + 63) // 64, trees=trees)
    return s


def prepare(case, seed):
    if case["op"] == "attention":
        return _prepare_attention(case, seed)
    return _prepare_verify(case, seed) if case["op"] == "verify" else _prepare_pages(case, seed)


# ------------------------------------------------------ the operators' own calls

_package = None


def _sgg():
    global _package
    if _package is None:
        import segmented_gather_gemm_amd
        _package = segmented_gather_gemm_amd
    return _package


def _own_attention(s):
    return _sgg().spec_attention(
        s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_lens"], s["q_indptr"],
        s["max_q_len"], s["max_kv_len"], tree_mask=s["tree_mask"], scale=s["scale"],
        k_scale=s["k_scale"], v_scale=s["v_scale"])


def _own_verify(s):
    return _sgg().spec_verify(s["tokens"], s["parents"], s["q_indptr"], s["target_probs"],
                              s["uniforms"], s["final_uniforms"], s["max_q_len"],
                              draft_probs=s["draft_probs"])


def _own_draft(s):
    sgg, table, counts, refs = _sgg(), s["page_table"], s["page_counts"], s["ref_counts"]
    ps = s["case"]["page"]
    grow = sgg.spec_kv_resize(table, counts, refs, s["rows"], s["grown"], ps)
    mask, pos = sgg.spec_tree_mask(s["parents"], s["q_indptr"], s["kv_lens"], s["mask_words"],
                                   rows=s["rows"])
    sgg.spec_kv_write(s["k_new"], s["v_new"], s["k_cache"][0], s["v_cache"][0], table,
                      s["kv_lens"], s["q_indptr"], rows=s["rows"], k_scale=s["k_scale"],
                      v_scale=s["v_scale"])
    lens = sgg.spec_kv_compact(s["k_cache"], s["v_cache"], table, s["kv_lens"], s["path"],
                               s["accept_lens"], rows=s["rows"])
    trim = sgg.spec_kv_resize(table, counts, refs, s["rows"], s["old"], ps)
    return (s["k_cache"], s["v_cache"], table, counts, refs, mask, pos, lens, grow, trim)


def _own_fork(s):
    sgg, table, counts, refs = _sgg(), s["page_table"], s["page_counts"], s["ref_counts"]
    ps = s["case"]["page"]
    got = sgg.spec_kv_fork(s["k_cache"], s["v_cache"], table, counts, refs, s["kv_lens"],
                           s["src_rows"], s["dst_rows"])
    back = sgg.spec_kv_resize(table, counts, refs, s["dst_rows"], s["zeros"], ps,
                              kv_lens=s["kv_lens"])
    return (s["k_cache"], s["v_cache"], table, counts, refs, s["kv_lens"], got, back)


# ---------------------------------------------------------------- the plain forms

def _bits(x):
    """8-bit values as bytes, for indexing."""
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _owner(ptr, n):
    """Request of each of n tokens and its place in the request."""
    t = torch.arange(n, device=ptr.device)
    r = torch.searchsorted(ptr.long(), t, right=True) - 1
    return r, t - ptr.long()[r]


def _plain_attention(s):
    c, q, ptr = s["case"], s["q"], s["q_indptr"].long()
    bs, hq, hkv, d, ps = c["bs"], c["hq"], c["hkv"], c["d"], c["page"]
    n, T, S, dev = q.shape[0], s["max_q_len"], s["max_kv_len"], q.device
    kv, ql = s["kv_lens"].long(), ptr[1:] - ptr[:-1]
    r, t = _owner(ptr, n)
    pos = torch.arange(S, device=dev).expand(bs, S)
    here = pos < (kv + ql)[:, None]
    spot = torch.where(here, pos, 0)
    page = torch.gather(s["page_table"].long(), 1, spot // ps)

    def rows(cache, scale):  # (bs, hkv, S, d) in 32 bits
        x = _bits(cache)[page, spot % ps].view(cache.dtype).float()
        if scale is not None:
            x = x * scale[:, None]
        return torch.where(here[:, :, None, None], x, 0.0).transpose(1, 2).contiguous()

    # visible keys (bs, T, S): the context, and of the drafted tokens the row's own path
    j = pos - kv[:, None]
    if s["tree_mask"] is None:
        seen = j[:, None, :] <= torch.arange(T, device=dev)[None, :, None]
    else:
        at = (ptr[:-1, None] + torch.arange(T, device=dev)).clamp(max=n - 1)
        jd = j.clamp(min=0)
        word = torch.gather(s["tree_mask"][at], 2,
                            (jd // 64).clamp(max=s["tree_mask"].shape[1] - 1)
                            [:, None, :].expand(bs, T, S))
        seen = ((word >> (jd % 64)[:, None, :]) & 1).bool() | (j < 0)[:, None, :]
    seen = seen & here[:, None, :]
    qp = torch.zeros((bs, T, hq, d), device=dev)
    qp[r, t] = q.float()
    g = hq // hkv
    qp = qp.view(bs, T, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(bs, hkv, T * g, d)
    sc = torch.matmul(qp, rows(s["k_cache"], s["k_scale"]).transpose(2, 3).contiguous())
    sc = sc.view(bs, hkv, T, g, S).mul_(s["scale"])
    sc = sc.masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    top = sc.amax(-1, keepdim=True)
    w = torch.exp(sc - torch.where(top == float("-inf"), 0.0, top))
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.view(bs, hkv, T * g, S), rows(s["v_cache"], s["v_scale"]))
    o = o.view(bs, hkv, T, g, d) / torch.where(total > 0, total, 1.0)
    return o.permute(0, 2, 1, 3, 4).reshape(bs, T, hq, d)[r, t].to(q.dtype)


def _plain_verify(s):
    tokens, ptr = s["tokens"].long(), s["q_indptr"].long()
    bs, T, n, dev = ptr.numel() - 1, s["max_q_len"], tokens.numel(), tokens.device
    r, t = _owner(ptr, n)
    P, Q, u = s["target_probs"], s["draft_probs"], s["uniforms"].double()
    parent = s["parents"].long()
    up = torch.where(parent >= 0, ptr[r] + parent, torch.arange(n, device=dev))
    px = P[up, tokens].double()
    child = parent >= 0
    sib = (up[:, None] == up[None, :]) & child[:, None] & child[None, :]
    earlier = sib & torch.tril(torch.ones((n, n), dtype=torch.bool, device=dev), -1)
    same = earlier & (tokens[:, None] == tokens[None, :])
    if Q is None:
        fresh = torch.where(same.any(1), 0.0, px)      # a token already rejected is spent
        rem = 1.0 - torch.matmul(earlier.double(), fresh[:, None])[:, 0]
        ok = child & (u * rem < fresh)
        Pl = a = None
    else:
        # the residual after k rejections is max(p - a q, 0) / b, one more child rank a turn
        qx, rank = Q[up, tokens].double(), earlier.sum(1)
        a = torch.zeros(n, dtype=torch.float64, device=dev)
        b = torch.ones(n, dtype=torch.float64, device=dev)
        ok = torch.zeros(n, dtype=torch.bool, device=dev)
        kids = torch.zeros(n, dtype=torch.long, device=dev).index_add_(0, up, child.long())
        Pl, Ql = P.double(), Q.double()
        for k in range(s["max_children"]):
            left = (px - a[up] * qx).clamp(min=0)
            ok = ok | (child & (rank == k) & (u * qx * b[up] < left))
            a = torch.where(kids > k, a + b, a)
            b = torch.where(kids > k, (Pl - a[:, None] * Ql).clamp_(min=0).sum(1), b)
    ok = ok & ~(earlier & ok[None, :]).any(1)          # the first accepted child of its parent
    # on the path: the root, and nodes whose ancestors were all accepted
    reach = (t == 0) | ok
    hop, on = up, reach
    for _ in range(max(1, (T - 1).bit_length())):
        on = on & on[hop]
        hop = hop[hop]
    slot = torch.where(on, (torch.cumsum(on, 0) - 1) - (torch.cumsum(on, 0) - 1)[ptr[r]], T)
    path = torch.full((bs, T + 1), -1, dtype=torch.int32, device=dev)
    path[r, slot] = t.int()
    path = path[:, :T].contiguous()
    count = torch.zeros(bs, dtype=torch.int32, device=dev).index_add_(0, r, on.int())
    cur = ptr[:-1] + torch.gather(path, 1, (count[:, None] - 1).long())[:, 0]
    if Q is None:
        w = P[cur].double()
        drop = child & (up == cur[r])
        keep = torch.ones_like(w)
        keep[r, torch.where(drop, tokens, tokens[cur[r]])] = 0.0
        # the place used for tokens that are no child of `cur` is restored unless a child holds it
        own_tok = tokens[cur]
        held = torch.zeros(bs, device=dev).index_add_(
            0, r, (drop & (tokens == own_tok[r])).float()) > 0
        keep[torch.arange(bs, device=dev), own_tok] = (~held).double()
        w = w * keep
    else:
        w = (Pl[cur] - a[cur][:, None] * Ql[cur]).clamp_(min=0)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, P[cur].double())
    cum = torch.cumsum(w, 1)
    total = w.sum(1)
    first = (cum <= (s["final_uniforms"].double() * total)[:, None]).sum(1)
    V = P.shape[1]
    last = torch.where(w > 0, torch.arange(V, device=dev), -1).amax(1)
    return path, count, torch.minimum(first, last).int()


def _lowest_free(refs):
    """Page ids in ascending order of the free ones, and how many there are."""
    free = refs == 0
    ids = torch.zeros(refs.numel() + 1, dtype=torch.long, device=refs.device)
    rank = torch.where(free, torch.cumsum(free, 0) - 1, refs.numel())
    ids[rank] = torch.arange(refs.numel(), device=refs.device)
    return ids, free.sum()


def _plain_resize(s, rows, new_lens, commit=False):
    table, counts, refs, ps = s["page_table"], s["page_counts"], s["ref_counts"], s["case"]["page"]
    rows = rows.long()
    have, need = counts[rows].long(), (new_lens.long() + ps - 1) // ps
    slot = torch.arange(table.shape[1], device=table.device)[None, :]
    mine = table[rows].long()
    drop = (slot >= need[:, None]) & (slot < have[:, None])
    refs.index_add_(0, mine.reshape(-1), -drop.reshape(-1).int())
    ids, free = _lowest_free(refs)
    more = (need - have).clamp(min=0)
    missing = (more.sum() - free).clamp(min=0)
    want = (slot >= have[:, None]) & (slot < need[:, None]) & (missing == 0)
    rank = (torch.cumsum(more, 0) - more)[:, None] + slot - have[:, None]
    got = ids[rank.clamp(0, refs.numel())]
    refs.index_add_(0, got.reshape(-1), want.reshape(-1).int())
    table[rows] = torch.where(want, got, mine).int()
    counts[rows] = torch.where((more > 0) & (missing > 0), have, need).int()
    if commit:
        s["kv_lens"][rows] = torch.where((more > 0) & (missing > 0),
                                         s["kv_lens"][rows], new_lens)
    return torch.stack([missing, torch.zeros_like(missing)]).int()


def _put(cache, page, off, values):
    _bits(cache)[:, page, off] = _bits(values)


def _plain_draft(s):
    c, ps, rows, table = s["case"], s["case"]["page"], s["rows"].long(), s["page_table"]
    grow = _plain_resize(s, rows, s["grown"])
    ptr, parent = s["q_indptr"].long(), s["parents"].long()
    n, W = parent.numel(), s["mask_words"]
    r, t = _owner(ptr, n)
    kv = s["kv_lens"][rows].long()
    # ancestors by doubling: each turn joins a node's set with its ancestor's, twice as far up
    at = torch.arange(64 * W, device=table.device)
    has = at[None, :] == t[:, None]
    hop = torch.where(parent >= 0, ptr[r] + parent, torch.arange(n, device=table.device))
    for _ in range(max(1, (s["max_q_len"] - 1).bit_length())):
        has = has | has[hop]
        hop = hop[hop]
    mask = (has.view(n, W, 64).long() << torch.arange(64, device=table.device)).sum(-1)
    pos = (kv[r] + has.sum(1) - 1).int()
    where = kv[r] + t
    page = table[rows[r], where // ps].long()
    for cache, new, scale in ((s["k_cache"], s["k_new"], s["k_scale"]),
                              (s["v_cache"], s["v_new"], s["v_scale"])):
        x = new
        if scale is not None:
            x = (new.float() / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(cache.dtype)
        _put(cache[:1], page, where % ps, x[None])
    # accepted rows move up; a place past the path moves the root onto itself
    path, acc = s["path"].long(), s["accept_lens"].long()
    j = torch.arange(path.shape[1], device=table.device)[None, :].expand_as(path)
    real = j < acc[:, None]
    src = kv[:, None] + torch.where(real, path, 0)
    dst = kv[:, None] + torch.where(real, j, 0)
    row = rows[:, None].expand_as(path)
    for cache in (s["k_cache"], s["v_cache"]):
        moved = _bits(cache)[:, table[row, src // ps].long(), src % ps]
        _bits(cache)[:, table[row, dst // ps].long(), dst % ps] = moved
    lens = (kv + acc).int()
    trim = _plain_resize(s, rows, s["old"])
    return (s["k_cache"], s["v_cache"], table, s["page_counts"], s["ref_counts"], mask, pos, lens,
            grow, trim)


def _plain_fork(s):
    ps, table, refs = s["case"]["page"], s["page_table"], s["ref_counts"]
    src, dst = s["src_rows"].long(), s["dst_rows"].long()
    kv = s["kv_lens"][src].long()
    full, part = kv // ps, kv % ps
    ids, free = _lowest_free(refs)
    more = (part > 0).long()
    missing = (more.sum() - free).clamp(min=0)
    page = ids[(torch.cumsum(more, 0) - more).clamp(max=refs.numel())]
    slot = torch.arange(table.shape[1], device=table.device)[None, :]
    theirs, mine = table[src].long(), table[dst].long()
    new = torch.where(slot < full[:, None], theirs, mine)
    new = torch.where((slot == full[:, None]) & (more > 0)[:, None], page[:, None], new)
    table[dst] = new.int()
    refs.index_add_(0, theirs.reshape(-1), (slot < full[:, None]).reshape(-1).int())
    refs.index_add_(0, page, more.int())
    s["page_counts"][dst] = (full + more).int()
    s["kv_lens"][dst] = kv.int()
    # the partial last page; a pair without one writes its first page onto itself
    old = torch.gather(theirs, 1, torch.where(more > 0, full, 0)[:, None])[:, 0]
    to = torch.where(more > 0, page, old)
    held = (torch.arange(ps, device=table.device)[None, :] < part[:, None]) | (more == 0)[:, None]
    for cache in (s["k_cache"], s["v_cache"]):
        x = _bits(cache)
        x[:, to] = torch.where(held[None, :, :, None, None], x[:, old], x[:, to])
    got = torch.stack([missing, torch.zeros_like(missing)]).int()
    back = _plain_resize(s, dst, s["zeros"], commit=True)
    return (s["k_cache"], s["v_cache"], table, s["page_counts"], refs, s["kv_lens"], got, back)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"attention": _own_attention, "verify": _own_verify, "draft": _own_draft,
                "fork": _own_fork}[op](state)
    return {"attention": _plain_attention, "verify": _plain_verify, "draft": _plain_draft,
            "fork": _plain_fork}[op](state)


# ----------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "verify":
        n = c["bs"] * c["q_len"]
        rows = c["bs"] * c["vocab"] * 4 * (2 if c["drawn"] else 1)
        return {"bytes": rows + n * (12 + 4 * (2 if c["drawn"] else 1)) + 4 * c["bs"] * c["q_len"],
                "flops": c["bs"] * c["vocab"] * (4 if c["drawn"] else 2)}
    mean_kv = (c["ctx"] + c["ctx"] // 2) / 2 if c["op"] == "attention" else \
        (c["ctx"] + max(1, c["ctx"] // 4)) / 2
    if c["op"] != "fork":
        mean_q = (c["q_len"] + max(1, c["q_len"] * 3 // 4)) / 2 if c["bs"] > 1 else c["q_len"]
    if c["bs"] == 1:
        mean_kv = c["ctx"]
    if c["op"] == "attention":
        kb = BYTES[c["dtype"] if c["cache"] == "same" else c["cache"]]
        tok = c["bs"] * mean_q
        seen = mean_kv + (min(mean_q, 8) if c["tree"] else (mean_q + 1) / 2)
        return {"bytes": c["bs"] * (mean_kv + mean_q) * (2 * c["hkv"] * c["d"] * kb + 4 / c["page"])
                + 4 * tok * c["hq"] * c["d"], "flops": 4 * tok * c["hq"] * c["d"] * seen}
    row = 2 * c["hkv"] * c["d"]                # values of a token's key and value in a layer
    kb = BYTES[c["cache"] if c["cache"] != "same" else c["dtype"]]
    if c["op"] == "draft":
        moved = c["bs"] * min(3, c["q_len"])   # rows of a path that change their place, about
        written = c["bs"] * mean_q
        return {"bytes": moved * row * kb * c["layers"] * 2 + written * row * (2 + kb)
                + c["bs"] * (mean_kv / c["page"] + c["q_len"]) * 8, "flops": 0}
    pairs = c["bs"] * c["copies"]
    # one reading of each source's last page, half full, and one writing for each copy
    half = c["page"] / 2 * row * kb * c["layers"]
    return {"bytes": (pairs + c["bs"]) * half + pairs * mean_kv / c["page"] * 16, "flops": 0}


# ------------------------------------------------------------ the definitions, in 64 bits

def _exact_attention(s):
    c, ptr, kv = s["case"], s["q_indptr"].tolist(), s["kv_lens"].tolist()
    ps, g, out = c["page"], c["hq"] // c["hkv"], []
    for r in range(c["bs"]):
        n, total = ptr[r + 1] - ptr[r], kv[r] + ptr[r + 1] - ptr[r]
        pages = s["page_table"][r, :(total + ps - 1) // ps].long()
        seen = torch.ones((n, total), dtype=torch.bool, device="cuda")
        tail = _ancestors(s["trees"][r]) if s["trees"] else np.tril(np.ones((n, n), bool))
        seen[:, kv[r]:] = torch.from_numpy(tail).cuda()
        q = s["q"][ptr[r]:ptr[r + 1]].double()
        o = torch.empty((n, c["hq"], c["d"]), dtype=torch.float64, device="cuda")
        for h in range(c["hkv"]):
            k, v = (_bits(x)[pages, :, h].reshape(-1, c["d"])[:total].contiguous()
                    .view(x.dtype).double() for x in (s["k_cache"], s["v_cache"]))
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            for e in range(h * g, h * g + g):
                x = (q[:, e] @ k.T * s["scale"]).masked_fill(~seen, float("-inf"))
                o[:, e] = torch.softmax(x, -1) @ v
        out.append(o)
    return torch.cat(out)


def _exact_verify(s):
    ptr = s["q_indptr"].tolist()
    tokens, u = s["tokens"].tolist(), s["uniforms"].double().tolist()
    last = s["final_uniforms"].double().tolist()
    paths, counts, nexts = [], [], []
    for r, par in enumerate(s["trees"]):
        cur, path = 0, [0]
        while True:
            p = s["target_probs"][ptr[r] + cur].double().cpu().numpy()
            q = None if s["draft_probs"] is None else \
                s["draft_probs"][ptr[r] + cur].double().cpu().numpy()
            w, mass, a, nxt = p.copy(), 1.0, 0.0, -1
            for i in (i for i, x in enumerate(par) if x == cur):
                x, coin = tokens[ptr[r] + i], u[ptr[r] + i]
                if coin * mass * (1.0 if q is None else q[x]) < w[x]:
                    nxt = i
                    break
                if q is None:
                    mass -= w[x]
                    w[x] = 0.0
                else:
                    a += mass
                    w = np.maximum(p - a * q, 0.0)
                    mass = float(w.sum())
            if nxt < 0:
                break
            cur = nxt
            path.append(cur)
        w = w if w.sum() > 0 else p
        cum = np.cumsum(w)
        v = int((cum <= last[r] * w.sum()).sum())
        nexts.append(min(v, int(np.nonzero(w > 0)[0].max())))
        counts.append(len(path))
        paths.append(path + [-1] * (s["max_q_len"] - len(path)))
    return tuple(torch.tensor(x, dtype=torch.int32) for x in (paths, counts, nexts))


def _exact_pages(s):
    """The caches that the cycle leaves, followed page by page on the host; whole numbers apart."""
    ps, table = s["case"]["page"], s["page_table"].cpu().numpy().copy()
    refs, counts = s["ref_counts"].cpu().numpy().copy(), s["page_counts"].cpu().numpy()
    free = iter(np.nonzero(refs == 0)[0].tolist())
    k, v = s["k_cache"].double(), s["v_cache"].double()
    lens = s["kv_lens"].cpu().numpy()
    if s["case"]["op"] == "fork":
        for a in s["src_rows"].tolist():
            n = int(lens[a])
            if n % ps:
                old, new = int(table[a, n // ps]), next(free)
                for x in (k, v):
                    x[:, new, :n % ps] = x[:, old, :n % ps]
        return (k, v) + (None,) * 6
    rows, ptr = s["rows"].tolist(), s["q_indptr"].tolist()
    accept, path = s["accept_lens"].tolist(), s["path"].tolist()
    for r, row in enumerate(rows):
        for j in range(int(counts[row]), -(-(int(lens[row]) + ptr[r + 1] - ptr[r]) // ps)):
            table[row, j] = next(free)

    def place(row, at):
        return int(table[row, at // ps]), at % ps

    for x, new, scale in ((k, s["k_new"], s["k_scale"]), (v, s["v_new"], s["v_scale"])):
        y = new.double()
        if scale is not None:
            y = (y / scale.double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
            y = y.float().to(torch.float8_e4m3fn).double()
        for r, row in enumerate(rows):
            at = [place(row, int(lens[row]) + i) for i in range(ptr[r + 1] - ptr[r])]
            x[0][[p for p, _ in at], [o for _, o in at]] = y[ptr[r]:ptr[r + 1]]
            way = path[r][:int(accept[r])]
            a = [at[i] for i in way]
            b = at[:len(way)]
            x[:, [p for p, _ in b], [o for _, o in b]] = x[:, [p for p, _ in a], [o for _, o in a]]
    return (k, v) + (None,) * 8


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(s)
    return _exact_verify(s) if case["op"] == "verify" else _exact_pages(s)
