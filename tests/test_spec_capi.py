"""CPU tests of the speculative decoding entry points: the header is what the library
exports and the call module passes on, bad arguments are refused on the host before
anything reaches a GPU, and the oracle agrees with itself on hand-made cases."""

import ctypes
import os
import re
import struct

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sgg_spec.h")

import segmented_gather_gemm_amd as sgg  # noqa: E402
from oracle import spec as osp  # noqa: E402
from segmented_gather_gemm_amd import _lib  # noqa: E402

F = 0x10000        # a well-aligned address that no refused call follows
C = _lib.spec_calls()
BF16, FP16, E4M3 = 0, 1, 2


def _err():
    return _lib.lib().lora_last_error().decode()


def _declarations():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return dict(re.findall(r"\b(spec_\w+)\s*\(([^)]*)\)\s*;", text))


def test_header_exported_and_in_call_module():
    decl = _declarations()
    assert set(decl) == set(C.SIGNATURES)
    handle = ctypes.CDLL(_lib.LIB)
    for name, params in decl.items():
        assert hasattr(handle, name), name
        sig = ""
        for p in (x.strip() for x in params.split(",")):
            sig += "p" if "*" in p else {"int64_t": "l", "int32_t": "i", "float": "f"}[p.split()[0]]
        assert sig == C.SIGNATURES[name], name
        with pytest.raises(TypeError, match=f"takes {len(sig)} arguments"):
            getattr(C, name)(*([0] * (len(sig) + 1)))
    with pytest.raises(TypeError):
        C.spec_attention_workspace_bytes(1, 32, 8, 128, 0, 1, "many")


def cache(k=F, v=F, ks=(0, 16384, 1024, 128), vs=None, pages=64, layers=1, ps=16, heads=8,
          dim=128, dtype=BF16):
    return struct.pack("=QQ4q4qq6i", k, v, *ks, *(vs or ks), pages, layers, ps, heads, dim, dtype,
                       0)


CACHE_FAULTS = [
    (dict(k=0), -1, "k or v"), (dict(dtype=3), -1, "dtype"), (dict(pages=0), -1, "positive"),
    (dict(layers=0), -1, "positive"), (dict(heads=0), -1, "positive"),
    (dict(pages=1 << 31), -1, "num_pages"), (dict(ps=0), -1, "page_size"),
    (dict(ps=12), -2, "power of two"), (dict(dim=100), -2, "multiple of 16"),
    (dict(dim=8, dtype=E4M3), -2, "multiple of 16"), (dict(ks=(0, -16, 16, 16)), -1, "negative"),
    (dict(ks=(0, 16384, 1023, 128)), -2, "multiples of 16"),
    (dict(ks=(0, 1 << 32, 1024, 128)), -2, "4 GiB"), (dict(v=F + 8), -2, "aligned"),
    (dict(ps=1 << 20, heads=64), -2, "2 GiB"),
]


@pytest.mark.parametrize("kw,code,text", CACHE_FAULTS)
def test_cache_refused_by_every_call(kw, code, text):
    c = cache(**kw)
    for rc in (C.spec_kv_copy_pages(c, F, F, 1, 0), fork(cache=c), write(cache=c),
               compact(cache=c), attention(cache=c)):
        assert rc == code and text in _err()


def resize(table=F, ld=8, width=8, rows_n=4, counts=F, refs=F, pages=64, rows=F, lens=F, n=4,
           ps=16, kv=F, status=F):
    return C.spec_kv_resize(table, ld, width, rows_n, counts, refs, pages, rows, lens, n, ps, kv,
                            status, 0)


TABLE_FAULTS = [(dict(table=0), -1, "page_table"), (dict(width=0), -1, "max_pages"),
                (dict(rows_n=0), -1, "num_rows"), (dict(ld=7), -1, "ld_table")]


@pytest.mark.parametrize("kw,code,text", TABLE_FAULTS + [
    (dict(n=-1), -1, "negative"), (dict(n=4097), -2, "4096"), (dict(ps=0), -1, "page_size"),
    (dict(ps=24), -2, "power of two"), (dict(counts=0), -1, "page_counts"),
    (dict(lens=0), -1, "new_lens"), (dict(status=0), -1, "status"), (dict(pages=0), -1, "num_pages"),
    (dict(n=4096, width=1 << 20, ld=1 << 20), -2, "2^31")])
def test_resize_refused(kw, code, text):
    assert resize(**kw) == code and text in _err()


def fork(cache=cache(), table=F, ld=8, width=8, rows_n=4, counts=F, refs=F, kv=F, src=F, dst=F,
         n=2, status=F, ws=F, wsb=24):
    return C.spec_kv_fork(cache, table, ld, width, rows_n, counts, refs, kv, src, dst, n, status,
                          ws, wsb, 0)


@pytest.mark.parametrize("kw,code,text", TABLE_FAULTS + [
    (dict(cache=0), -1, "cache"), (dict(kv=0), -1, "kv_lens"), (dict(src=0), -1, "src_rows"),
    (dict(n=-1), -1, "negative"), (dict(n=5000), -2, "4096"), (dict(wsb=23), -3, "workspace"),
    (dict(ws=0), -1, "workspace")])
def test_fork_refused(kw, code, text):
    assert fork(**kw) == code and text in _err()


def write(k=F, kt=1024, kh=128, v=F, vt=1024, vh=128, dtype=BF16, cache=cache(), table=F, ld=8,
          width=8, rows_n=4, kv=F, rows=F, ind=F, bs=2, n=4, ks=0, vs=0):
    return C.spec_kv_write(k, kt, kh, v, vt, vh, dtype, cache, table, ld, width, rows_n, kv, rows,
                           ind, bs, n, ks, vs, 0)


@pytest.mark.parametrize("kw,code,text", TABLE_FAULTS + [
    (dict(dtype=E4M3), -1, "bf16 or fp16"), (dict(dtype=FP16), -1, "differs"),
    (dict(cache=cache(dtype=E4M3), ks=F), -1, "k_scale and v_scale"), (dict(k=0), -1, "k is NULL"),
    (dict(v=F + 2), -2, "aligned"), (dict(kt=1020), -2, "multiples of 8"), (dict(vh=-8), -1, "neg"),
    (dict(bs=-1), -1, "negative"), (dict(n=-1), -1, "num_tokens"), (dict(ind=0), -1, "q_indptr")])
def test_write_refused(kw, code, text):
    assert write(**kw) == code and text in _err()


def compact(cache=cache(), table=F, ld=8, width=8, rows_n=4, kv=F, rows=F, path=F, ldp=4, w=4,
            acc=F, new=F, bs=2):
    return C.spec_kv_compact(cache, table, ld, width, rows_n, kv, rows, path, ldp, w, acc, new, bs,
                             0)


@pytest.mark.parametrize("kw,code,text", TABLE_FAULTS + [
    (dict(w=5), -1, "path_width"), (dict(path=0), -1, "path"), (dict(acc=0), -1, "accept_lens"),
    (dict(new=0), -1, "new_lens"), (dict(bs=-2), -1, "negative")])
def test_compact_refused(kw, code, text):
    assert compact(**kw) == code and text in _err()


@pytest.mark.parametrize("kw,code,text", [
    (dict(words=0), -1, "mask_words"), (dict(rows_n=0), -1, "num_rows"),
    (dict(parents=0), -1, "parents"), (dict(mask=F + 4), -2, "aligned"), (dict(bs=-1), -1, "neg")])
def test_tree_mask_refused(kw, code, text):
    a = dict(parents=F, ind=F, bs=2, n=6, kv=F, rows=F, rows_n=4, mask=F, words=1, pos=F)
    a.update(kw)
    assert C.spec_tree_mask(*a.values(), 0) == code and text in _err()


def attention(q=F, qt=4096, qh=128, out=F, ot=4096, oh=128, dtype=BF16, hq=32, cache=cache(),
              table=F, ld=8, width=8, rows_n=4, kv=F, rows=F, ind=F, bs=2, n=8, mask=F, words=1,
              scale=0.1, ks=0, vs=0, mq=4, mkv=100, ws=F, wsb=1 << 30):
    return C.spec_attention(q, qt, qh, out, ot, oh, dtype, hq, cache, table, ld, width, rows_n, kv,
                            rows, ind, bs, n, mask, words, scale, ks, vs, mq, mkv, ws, wsb, 0)


@pytest.mark.parametrize("kw,code,text", TABLE_FAULTS + [
    (dict(dtype=E4M3), -1, "bf16 or fp16"), (dict(dtype=FP16), -1, "differs"),
    (dict(hq=12), -1, "multiple"), (dict(hq=0), -1, "multiple"),
    (dict(cache=cache(dim=264)), -2, "head_dim"), (dict(ks=F), -1, "e4m3"),
    (dict(scale=float("nan")), -1, "finite"), (dict(scale=float("inf")), -1, "finite"),
    (dict(words=0), -1, "mask_words"), (dict(mask=F + 4), -2, "aligned"),
    (dict(q=0), -1, "q is NULL"), (dict(q=F + 8), -2, "aligned"), (dict(qh=100), -2, "multiples"),
    (dict(out=0), -1, "out is NULL"), (dict(kv=0), -1, "kv_lens"), (dict(ind=0), -1, "q_indptr"),
    (dict(bs=4097), -2, "4096"), (dict(n=1 << 31), -1, "num_tokens"), (dict(mq=-1), -1, "max_q_len"),
    (dict(mkv=1 << 31), -1, "max_kv_len"), (dict(mq=1 << 30), -2, "max_q_len"),
    (dict(n=1 << 28), -2, "2^30"),
    (dict(mkv=5000, wsb=16), -3, "workspace"), (dict(mkv=5000, ws=0), -1, "workspace"),
    (dict(mkv=5000, ws=F + 8), -2, "aligned")])
def test_attention_refused(kw, code, text):
    assert attention(**kw) == code and text in _err()


def verify(tokens=F, parents=F, ind=F, bs=2, n=8, p=F, ldp=100, q=F, ldq=100, V=100, u=F, uf=F,
           path=F, ldpath=4, w=4, acc=F, nxt=F, ws=F, wsb=1 << 30):
    return C.spec_verify(tokens, parents, ind, bs, n, p, ldp, q, ldq, V, u, uf, path, ldpath, w,
                         acc, nxt, ws, wsb, 0)


@pytest.mark.parametrize("kw,code,text", [
    (dict(bs=-1), -1, "negative"), (dict(bs=4097), -2, "4096"), (dict(n=-1), -1, "num_tokens"),
    (dict(V=0), -2, "vocab"), (dict(V=(1 << 22) + 1, ldp=1 << 23, ldq=1 << 23), -2, "vocab"),
    (dict(ldp=99), -1, "ld_target"), (dict(ldq=99), -1, "ld_draft"), (dict(w=0), -1, "path_width"),
    (dict(w=5), -1, "path_width"), (dict(ind=0), -1, "q_indptr"), (dict(path=0), -1, "path"),
    (dict(p=0), -1, "target_probs"), (dict(u=0), -1, "uniforms"), (dict(uf=0), -1, "final"),
    (dict(V=50000, ldp=50000, ldq=50000, ws=0), -1, "workspace"),
    (dict(V=50000, ldp=50000, ldq=50000, wsb=16), -3, "workspace"),
    (dict(V=50000, ldp=50000, ldq=50000, ws=F + 8), -2, "aligned")])
def test_verify_refused(kw, code, text):
    assert verify(**kw) == code and text in _err()


def test_set_option():
    old = sgg.spec_set_option("verify_spin_limit", 7)
    assert sgg.spec_set_option("verify_spin_limit", old) == 7
    for name, value in (("spin", 1), ("verify_spin_limit", -1)):
        with pytest.raises(ValueError):
            sgg.spec_set_option(name, value)


def test_empty_batches_are_nothing_to_do():
    assert write(bs=0) == 0 and write(n=0) == 0 and compact(bs=0) == 0
    assert attention(bs=0) == 0 and attention(n=0) == 0 and verify(bs=0) == 0
    assert C.spec_kv_copy_pages(cache(), 0, 0, 0, 0) == 0


ZERO_BYTES = 4 * 2 * 32768 + 4 * 4096 + 8 * 3 * 1024


def test_ranges_cover_every_tile_and_fit_the_workspace():
    """The kernel's division, followed on the host: every tile of every unit belongs to one
    range, the pieces of a unit are its consecutive chunks, and no two pieces share a slot."""
    rng = np.random.default_rng(3)
    split = whole = 0
    for _ in range(300):
        bs = int(rng.integers(1, 70))
        hkv = int(rng.integers(1, 20))
        hq = hkv * int(rng.integers(1, 9))
        dim = int(rng.choice([64, 128, 256]))
        T = int(rng.choice([1, 3, 16, 61, 300]))
        kv = int(10 ** rng.uniform(0, 5.3))
        need = C.spec_attention_workspace_bytes(bs, hq, hkv, dim, BF16, T, kv)
        s = _shape(bs, hq, hkv, dim, T, kv)
        assert need == (s["slots"] > 0) * ZERO_BYTES + s["slots"] * s["rows"] * (
            -(-dim // 64) * 64 * 4 + 8)
        assert s["slots"] <= 32768
        # the batch may exceed the bounds that shaped the launch
        over = int(rng.integers(1, 3))
        lens = rng.integers(1, over * kv + 1, bs)
        ts = rng.integers(0, over * T + 1, bs)
        blocks = -(-ts * (hq // hkv) // s["rows"])
        units = [-(-int(n + t) // s["keys"]) for n, t, b in zip(lens, ts, blocks)
                 for _ in range(b)]
        total = sum(units)
        if total == 0:
            continue
        if s["ranges"] == 0:
            assert s["grid"] % hkv == 0 and s["slots"] == 0
            whole += 1
            continue
        size = max(-(-total // s["ranges"]), s["min_tiles"])
        N = -(-total // size)
        assert s["grid"] >= s["ranges"] * hkv and N <= s["ranges"]
        used, starts = set(), np.concatenate([[0], np.cumsum(units)])
        pieces = {}
        for i in range(N):
            pos, stop = i * size, min((i + 1) * size, total)
            while pos < stop:
                u = int(np.searchsorted(starts, pos, side="right")) - 1
                at, n = int(starts[u]), units[u]
                t0, t1 = pos - at, min(n, stop - at)
                r0 = at // size
                chunks = (at + n - 1) // size - r0 + 1
                pieces.setdefault(u, []).append((i - r0, chunks, t0, t1))
                if chunks > 1:
                    slot = 2 * i + (1 if i == r0 else 0)
                    assert slot not in used and slot * hkv + hkv - 1 < s["slots"]
                    used.add(slot)
                    split += 1
                pos = at + t1
        assert len(pieces) == len(units)
        for u, got in pieces.items():
            assert [c for c, *_ in got] == list(range(got[0][1])) and len(got) == got[0][1]
            assert got[0][2] == 0 and got[-1][3] == units[u]
            assert all(a[3] == b[2] for a, b in zip(got, got[1:]))
    assert split > 1000 and whole > 10
    assert C.spec_attention_workspace_bytes(1, 30, 8, 128, 0, 1, 100) == -1


def _shape(bs, hq, hkv, dim, T, kv):
    """The launch's division, as the host computes it (read through the library)."""
    out = (ctypes.c_int64 * 6)()
    fn = ctypes.CDLL(_lib.LIB).sgg_spec_attention_shape
    fn.argtypes = [ctypes.c_int32] * 6 + [ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)]
    fn(bs, hq, hkv, dim, 2, T, kv, out)
    return dict(zip(("rows", "keys", "min_tiles", "ranges", "slots", "grid"), out))


# ------------------------------------------------------------ the oracle, by hand

def test_oracle_masks():
    m = osp.ancestors([-1, 0, 0, 2, 1])
    assert m.astype(int).tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0],
                                      [1, 0, 1, 1, 0], [1, 1, 0, 0, 1]]
    assert osp.mask_words(m, 1)[:, 0].tolist() == [1, 3, 5, 13, 19]


def test_oracle_verify_by_hand():
    p = np.array([[0.5, 0.3, 0.2], [0.1, 0.1, 0.8], [0.2, 0.2, 0.6]], np.float32)
    par = [-1, 0, 0]
    # candidates 1 then 0 after the root: 0.3 is refused by 0.4, then 0.5 / 0.7 taken by 0.6
    assert osp.verify([9, 1, 0], par, p, None, [0, 0.4, 0.6], 0.5, 3) == ([0, 2], 2)
    # both refused: what is left is token 2
    assert osp.verify([9, 1, 0], par, p, None, [0, 0.4, 0.8], 0.0, 3) == ([0], 2)
    # drawn from q: token 0 refused (0.5 / 0.8 < 0.7), the residual is (0, 0.2, 0.1)
    q = np.array([[0.8, 0.1, 0.1]] * 3, np.float32)
    path, nxt = osp.verify([9, 0], [-1, 0], p[:2], q[:2], [0, 0.7], 0.6, 2)
    assert (path, nxt) == ([0], 1)
    path, nxt = osp.verify([9, 0], [-1, 0], p[:2], q[:2], [0, 0.7], 0.7, 2)
    assert (path, nxt) == ([0], 2)


def test_oracle_draft_rejection_keeps_the_target():
    """Over all outcomes of two independent draws and their coins, the first token that comes
    out has the target's distribution: the recurrence on (a, mass) is lossless."""
    p = np.array([0.5, 0.2, 0.3])
    q = np.array([0.2, 0.7, 0.1])
    got = np.zeros(3)

    def step(prob, a, mass, left):
        w = np.maximum(p - a * q, 0)
        if left == 0:
            got[:] += prob * w / w.sum()
            return
        for x in range(3):
            take = min(1.0, w[x] / (mass * q[x])) if q[x] > 0 else 0.0
            got[x] += prob * q[x] * take
            if take < 1.0:
                a2 = a + mass
                step(prob * q[x] * (1 - take), a2, np.maximum(p - a2 * q, 0).sum(), left - 1)
    step(1.0, 0.0, 1.0, 2)
    np.testing.assert_allclose(got, p, rtol=0, atol=1e-15)


def test_python_refusals():
    import torch
    z = torch.zeros(2, dtype=torch.int32)
    with pytest.raises((TypeError, ValueError)):
        sgg.spec_kv_resize(torch.zeros((2, 2)), z, z, None, z, 16)
    with pytest.raises(ValueError):
        sgg.spec_kv_resize(torch.zeros((2, 2), dtype=torch.int32), z, z, None, z, 16)
    k = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="ROCm"):
        sgg.spec_kv_copy_pages(k, k, z, z)
    with pytest.raises(TypeError, match="float8_e4m3fn"):
        sgg.spec_kv_copy_pages(k.float(), k.float(), z, z)
    with pytest.raises(ValueError, match="differ"):
        sgg.spec_kv_copy_pages(k, k.half(), z, z)
    with pytest.raises(TypeError, match="float8_e4m3fn"):
        sgg.PagedKVCache(1, 4, 16, 2, 64, 2, 2, dtype=torch.float32, device="cpu")
