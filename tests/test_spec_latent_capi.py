"""CPU tests of the entry points around a speculative decoding step: bad arguments are refused on
the host before anything reaches a GPU, and the oracle agrees with itself on hand-made cases."""

import struct

import numpy as np
import pytest
import torch

import segmented_gather_gemm_amd as sgg
from oracle import latent as ola
from test_spec_capi import BF16, C, CACHE_FAULTS, E4M3, F, FP16, _err, cache

FP32 = 3
INF = float("inf")


def refused(rc, code, text):
    assert rc == code and text in _err(), (rc, _err())


def latents(data=F, page=9216, token=576, pages=64, ps=16, latent=512, rope=64, dtype=BF16):
    return struct.pack("=Qqqq4i", data, page, token, pages, ps, latent, rope, dtype)


def rope(q=F, qt=4096, qh=128, out=F, ot=4096, oh=128, hq=32, k=F, kt=1024, kh=128, v=F, vt=1024,
         vh=128, dtype=BF16, freq=F, rot=128, start=0, inter=0, factor=1.0, pos=0, cache=cache(),
         table=F, ld=8, width=8, rows_n=4, held=0, kv=F, rows=F, ind=F, bs=4, n=9, ks=0, vs=0):
    return C.spec_rope_write(q, qt, qh, out, ot, oh, hq, k, kt, kh, v, vt, vh, dtype, freq, rot,
                             start, inter, factor, pos, cache, table, ld, width, rows_n, held, kv,
                             rows, ind, bs, n, ks, vs, 0)


@pytest.mark.parametrize("kw,code,text", CACHE_FAULTS)
def test_rope_refuses_bad_caches(kw, code, text):
    refused(rope(cache=cache(**kw)), code, text)


TABLE_FAULTS = [(dict(table=0), -1, "page_table is NULL"), (dict(width=0), -1, "positive"),
                (dict(rows_n=0), -1, "positive"), (dict(ld=7), -1, "ld_table"),
                (dict(bs=-1), -1, "negative"), (dict(bs=4097), -2, "above 4096"),
                (dict(n=-1), -1, "num_tokens"), (dict(n=1 << 31), -1, "num_tokens")]


@pytest.mark.parametrize("kw,code,text", TABLE_FAULTS + [
    (dict(dtype=E4M3), -1, "bf16 or fp16"), (dict(dtype=FP16), -1, "differs"),
    (dict(cache=cache(dtype=E4M3), ks=F), -1, "k_scale and v_scale"), (dict(hq=-1), -1, "negative"),
    (dict(hq=1 << 20), -2, "2^24"), (dict(rot=0), -2, "rotary_dim"), (dict(rot=7), -2, "rotary_dim"),
    (dict(rot=258, cache=cache(dim=512)), -2, "rotary_dim"), (dict(start=1), -1, "rotated"),
    (dict(start=-1), -1, "rotated"), (dict(rot=64, start=65), -1, "rotated"),
    (dict(factor=INF), -1, "finite"), (dict(factor=float("nan")), -1, "finite"),
    (dict(freq=0), -1, "inv_freq"), (dict(q=0), -1, "q is NULL"), (dict(out=0), -1, "q_out is NULL"),
    (dict(qt=4095), -2, "multiples of 8"), (dict(out=F + 2), -2, "aligned"),
    (dict(k=0), -1, "k is NULL"), (dict(kt=-8), -1, "negative"), (dict(v=0), -1, "v is NULL"),
    (dict(vh=4), -2, "multiples of 8"), (dict(kv=0), -1, "kv_lens"), (dict(ind=0), -1, "q_indptr"),
])
def test_rope_refused(kw, code, text):
    refused(rope(**kw), code, text)


def lwrite(q=F, qt=4096, qh=64, out=F, ot=4096, oh=64, hq=16, lat=F, lt=512, kpe=F, kt=64,
           dtype=BF16, freq=F, inter=1, factor=1.0, pos=0, cache=latents(), table=F, ld=8, width=8,
           rows_n=4, held=0, kv=F, rows=F, ind=F, bs=4, n=9, scale=0):
    return C.spec_latent_write(q, qt, qh, out, ot, oh, hq, lat, lt, kpe, kt, dtype, freq, inter,
                               factor, pos, cache, table, ld, width, rows_n, held, kv, rows, ind, bs,
                               n, scale, 0)


def gather(cache=latents(), table=F, ld=8, width=8, rows_n=4, held=0, rows=F, ind=F, bs=4, n=9,
           out=F, ot=576, dtype=BF16, scale=0):
    return C.spec_latent_gather(cache, table, ld, width, rows_n, held, rows, ind, bs, n, out, ot,
                                dtype, scale, 0)


def attention(q=F, qt=9216, qh=576, out=F, ot=8192, oh=512, dtype=BF16, heads=16, cache=latents(),
              table=F, ld=8, width=8, rows_n=4, kv=F, rows=F, ind=F, bs=4, n=9, mask=0, words=0,
              scale=0.1, cs=0, mq=4, mkv=100, ws=F, wsn=1 << 40):
    return C.spec_latent_attention(q, qt, qh, out, ot, oh, dtype, heads, cache, table, ld, width,
                                   rows_n, kv, rows, ind, bs, n, mask, words, scale, cs, mq, mkv, ws,
                                   wsn, 0)


@pytest.mark.parametrize("kw,code,text", [
    (dict(data=0), -1, "data is NULL"), (dict(dtype=3), -1, "dtype"), (dict(pages=0), -1, "num_pages"),
    (dict(pages=1 << 31), -1, "num_pages"), (dict(ps=0), -1, "page_size"),
    (dict(ps=12), -2, "power of two"), (dict(latent=0), -2, "latent_dim"),
    (dict(latent=520), -2, "latent_dim"), (dict(latent=500), -2, "latent_dim"),
    (dict(latent=504, dtype=E4M3), -2, "latent_dim"), (dict(rope=0), -2, "rope_dim"),
    (dict(rope=72), -2, "rope_dim"), (dict(rope=8, dtype=E4M3), -2, "rope_dim"),
    (dict(page=-8), -1, "negative"), (dict(token=-8), -1, "negative"),
    (dict(token=577), -2, "multiples of 16"), (dict(page=4), -2, "multiples of 16"),
    (dict(data=F + 8), -2, "aligned"), (dict(token=1 << 27), -2, "2 GiB"),
])
def test_bad_latent_caches_refused_by_every_call(kw, code, text):
    c = latents(**kw)
    for rc in (lwrite(cache=c), gather(cache=c), attention(cache=c)):
        refused(rc, code, text)


@pytest.mark.parametrize("call", [lwrite, gather, attention, rope])
@pytest.mark.parametrize("kw,code,text", TABLE_FAULTS)
def test_bad_tables_refused_by_every_call(call, kw, code, text):
    refused(call(**kw), code, text)


@pytest.mark.parametrize("kw,code,text", [
    (dict(dtype=FP32), -1, "bf16 or fp16"), (dict(dtype=FP16), -1, "differs"),
    (dict(cache=latents(dtype=E4M3)), -1, "cache_scale"), (dict(hq=-1), -1, "num_q_heads"),
    (dict(hq=1 << 17), -1, "num_q_heads"), (dict(factor=INF), -1, "finite"),
    (dict(freq=0), -1, "inv_freq"), (dict(q=0), -1, "q_pe is NULL"), (dict(qh=4), -2, "multiples of 8"),
    (dict(out=0), -1, "q_out is NULL"), (dict(lat=0), -1, "latent is NULL"),
    (dict(lt=4), -2, "multiples of 8"), (dict(kpe=0), -1, "k_pe is NULL"),
    (dict(kpe=F + 2), -2, "aligned"), (dict(kv=0), -1, "kv_lens"), (dict(ind=0), -1, "q_indptr"),
])
def test_latent_write_refused(kw, code, text):
    refused(lwrite(**kw), code, text)


@pytest.mark.parametrize("kw,code,text", [
    (dict(dtype=E4M3), -1, "bf16 or fp16"), (dict(dtype=FP16), -1, "differs"),
    (dict(scale=F), -1, "belongs to"), (dict(out=0), -1, "out is NULL"),
    (dict(ot=4), -2, "multiples of 8"), (dict(out=F + 8), -2, "aligned"),
    (dict(ind=0), -1, "kv_indptr"),
])
def test_gather_refused(kw, code, text):
    refused(gather(**kw), code, text)


@pytest.mark.parametrize("kw,code,text", [
    (dict(dtype=E4M3), -1, "bf16 or fp16"), (dict(dtype=FP16), -1, "differs"),
    (dict(cs=F), -1, "belongs to"), (dict(heads=0), -1, "num_heads"),
    (dict(heads=1 << 17), -1, "num_heads"), (dict(mq=-1), -1, "max_q_len"),
    (dict(mkv=-1), -1, "max_kv_len"), (dict(mkv=1 << 31), -1, "max_kv_len"),
    (dict(mq=1 << 28), -2, "2^30"), (dict(n=1 << 27), -2, "2^30"), (dict(scale=INF), -1, "finite"),
    (dict(scale=float("nan")), -1, "finite"), (dict(mask=F), -1, "mask_words"),
    (dict(mask=F + 4, words=1), -2, "8-byte"), (dict(q=0), -1, "q is NULL"),
    (dict(qh=4), -2, "multiples of 8"), (dict(out=0), -1, "out is NULL"), (dict(oh=4), -2, "multiples"),
    (dict(kv=0), -1, "kv_lens"), (dict(ind=0), -1, "q_indptr"), (dict(ws=0, mkv=9000), -1, "workspace"),
    (dict(wsn=1000, mkv=9000), -3, "workspace"), (dict(ws=F + 8, mkv=9000), -2, "aligned"),
])
def test_latent_attention_refused(kw, code, text):
    refused(attention(**kw), code, text)


def prefill(q=F, qt=2048, qh=192, k=F, kt=4096, kh=256, v=F, vt=4096, vh=256, kpe=F, kpt=64,
            out=F, ot=2048, oh=128, dtype=BF16, heads=16, dn=128, dr=64, dv=128, ind=F, kind=F, bs=4,
            n=9, m=20, scale=0.1, mq=4):
    return C.spec_latent_prefill(q, qt, qh, k, kt, kh, v, vt, vh, kpe, kpt, out, ot, oh, dtype, heads,
                                 dn, dr, dv, ind, kind, bs, n, m, scale, mq, 0)


@pytest.mark.parametrize("kw,code,text", [
    (dict(bs=-1), -1, "negative"), (dict(bs=4097), -2, "4096"), (dict(n=-1), -1, "num_tokens"),
    (dict(n=1 << 30), -2, "2^30"), (dict(m=-1), -2, "2^30"), (dict(m=1 << 30), -2, "2^30"),
    (dict(dtype=E4M3), -1, "bf16 or fp16"), (dict(heads=0), -1, "num_heads"),
    (dict(dn=0), -2, "nope_dim"), (dict(dn=136), -2, "nope_dim"), (dict(dv=4), -2, "v_dim"),
    (dict(dv=192), -2, "v_dim"), (dict(dr=0), -2, "rope_dim"), (dict(dr=72), -2, "rope_dim"),
    (dict(scale=INF), -1, "finite"), (dict(mq=-1), -1, "max_q_len"), (dict(q=0), -1, "q is NULL"),
    (dict(qt=7), -2, "multiples of 8"), (dict(k=0), -1, "k is NULL"), (dict(v=0), -1, "v is NULL"),
    (dict(vt=-8), -1, "negative"), (dict(kpe=0), -1, "k_pe is NULL"), (dict(out=F + 8), -2, "aligned"),
    (dict(ind=0), -1, "indptr"), (dict(kind=0), -1, "indptr"),
    (dict(heads=1 << 20, bs=4096), -2, "grid"), (dict(mq=1 << 29, heads=1 << 10), -2, "grid"),
])
def test_prefill_refused(kw, code, text):
    refused(prefill(**kw), code, text)


@pytest.mark.parametrize("kw", [dict(kt=1 << 26), dict(vt=1 << 26), dict(kpt=1 << 26)])
def test_prefill_refuses_keys_far_apart(kw):
    refused(prefill(**kw), -2, "2^26")


def probs(x=F, ldx=1000, dtype=FP32, V=1000, ind=F, bs=4, n=9, mq=4, tokens=F, parents=F, hist=F,
          ldh=50, width=50, rows_n=6, hl=F, pl=F, rows=F, temp=F, rep=F, pres=F, freq=F, bp=F, bi=F,
          bv=F, nb=7, allowed=F, lda=32, out=F, ldo=1000, ws=F, wsn=1 << 30):
    return C.spec_target_probs(x, ldx, dtype, V, ind, bs, n, mq, tokens, parents, hist, ldh, width,
                               rows_n, hl, pl, rows, temp, rep, pres, freq, bp, bi, bv, nb, allowed,
                               lda, out, ldo, ws, wsn, 0)


@pytest.mark.parametrize("kw,code,text", [
    (dict(bs=-1), -1, "negative"), (dict(bs=4097), -2, "4096"), (dict(n=-1), -1, "num_tokens"),
    (dict(dtype=E4M3), -1, "dtype"), (dict(V=0), -2, "vocab"), (dict(V=(1 << 22) + 1), -2, "vocab"),
    (dict(ldx=999), -1, "ld_logits"), (dict(ldo=999), -1, "ld_out"), (dict(mq=-1), -1, "max_q_len"),
    (dict(hl=0), -1, "history_lens"), (dict(rows_n=0), -1, "num_rows"), (dict(ldh=49), -1, "ld_history"),
    (dict(width=-1), -1, "history_width"), (dict(width=1 << 29, ldh=1 << 29), -1, "2^29"),
    (dict(nb=-1), -1, "num_bias"), (dict(bi=0), -1, "bias_ids"), (dict(bv=0), -1, "bias_values"),
    (dict(lda=31), -1, "ld_allowed"), (dict(tokens=0), -1, "parents need tokens"),
    (dict(x=0), -1, "logits"), (dict(ind=0), -1, "q_indptr"), (dict(out=0), -1, "out is NULL"),
    (dict(ws=0), -1, "workspace"), (dict(wsn=10), -3, "workspace"), (dict(ws=F + 8), -2, "aligned"),
])
def test_probs_refused(kw, code, text):
    refused(probs(**kw), code, text)


def test_empty_batches_are_nothing_to_do():
    for call in (rope, lwrite, gather, attention, prefill, probs):
        assert call(bs=0) == 0 and call(n=0) == 0


def test_workspace_sizes():
    size = C.spec_latent_attention_workspace_bytes
    assert size(1, 16, 512, BF16, 1, 32) == 0                    # nothing to divide
    assert size(-1, 16, 512, BF16, 1, 32) == -1 and size(1, 16, 520, BF16, 1, 32) == -1
    for bs, heads, latent, mq, mkv in ((1, 16, 512, 1, 100000), (64, 128, 512, 8, 9000),
                                       (4096, 8, 256, 1, 100), (3, 128, 64, 40, 1 << 30)):
        assert 0 <= size(bs, heads, latent, BF16, mq, mkv) < 1 << 28
    size = C.spec_target_probs_workspace_bytes
    assert size(-1, 10) == size(1, 0) == size(1, (1 << 22) + 1) == -1 and size(0, 10) == 0
    assert size(1000, 128256) >= 1000 * 63 * 12


def test_python_refusals():
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    i, f = torch.zeros(2, dtype=torch.int32), torch.zeros(32)
    c5, c3 = torch.zeros((2, 4, 2, 64), dtype=torch.bfloat16), torch.zeros((2, 4, 576))
    with pytest.raises(ValueError, match="device"):
        sgg.spec_rope_write(x, x, x, f, c5, c5, i[None], i, i)
    with pytest.raises(TypeError, match="cache"):
        sgg.spec_latent_attention(x, c3, i[None], i, i, 1, 1, 32, 0.1)
    with pytest.raises(ValueError, match="device"):
        sgg.spec_latent_attention(x, c3.bfloat16(), i[None], i, i, 1, 1, 32, 0.1)
    with pytest.raises(TypeError, match="q must be"):
        sgg.spec_latent_prefill(x.float(), x, x, x[0], i, i, 1, 1)
    with pytest.raises(ValueError, match="ROCm"):
        sgg.spec_latent_prefill(x, x, x, x[0], i, i, 1, 1)
    with pytest.raises(ValueError, match="device"):
        sgg.spec_target_probs(torch.zeros((2, 9)), i, 1)
    with pytest.raises(TypeError, match="dtype"):
        sgg.PagedLatentCache(1, 2, 4, 64, 32, 1, 2, dtype=torch.float32)
    with pytest.raises(ValueError, match="32 bytes"):
        sgg.PagedLatentCache(1, 2, 4, 64, 8, 1, 2, device="cpu")


# ----------------------------------------------------------------------- the oracle

def test_oracle_rotation():
    """A rotation keeps each pair's length and turns it by the angle; half a turn negates it, and
    both layouts are the same pairs in another order."""
    x = np.random.default_rng(0).normal(size=(3, 8))
    y = ola.rotate(x, 3, [np.pi / 3, 0.25], 2, True, 1.0)
    assert np.allclose(y[:, 2:4], -x[:, 2:4]) and np.array_equal(y[:, [0, 1, 6, 7]], x[:, [0, 1, 6, 7]])
    assert np.allclose(np.hypot(y[:, 4], y[:, 5]), np.hypot(x[:, 4], x[:, 5]))
    back = ola.rotate(y, -3, [np.pi / 3, 0.25], 2, True, 1.0)
    assert np.allclose(back, x)
    order = [0, 1, 2, 4, 3, 5, 6, 7]
    z = ola.rotate(x[:, order], 3, [np.pi / 3, 0.25], 2, False, 2.0)
    want = y[:, order].copy()
    want[:, 2:6] *= 2
    assert np.allclose(z, want)


def test_oracle_probs_by_hand():
    x = np.array([[2.0, -1.0, 0.0, 4.0]])
    p, y = ola.target_probs(x, [1], [-1], [3, 0, 0], 1, 1.0, 2.0, 0.5, 0.25, [(2, 1.0), (2, 0.5)],
                            np.array([[True, True, True, False]]))
    # 0: twice since the prompt; 1: the node; 2: biased; 3: in the prompt, and not allowed
    assert y[0].tolist() == [1.0 - 0.5 - 0.5, -2.0 - 0.25 - 0.5, 1.5, -np.inf]
    assert np.allclose(p[0], np.exp(y[0]) / np.exp(y[0]).sum())
    p, y = ola.target_probs(x, None, None, [3], 1, 0.0, 2.0)
    assert y[0].tolist() == [2.0, -1.0, 0.0, 2.0] and p[0].tolist() == [1, 0, 0, 0]


