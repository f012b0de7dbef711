"""Refusals of the cache and attention entry points: every bad argument is named on the host, before any launch (no GPU needed)."""

import pytest

import quantized_routed_expert_03_gb300 as qre
from quantized_routed_expert_03_gb300 import build as qbuild

A, MIS = 0x10000, 0x10008            # never dereferenced: the checks fail first


@pytest.fixture(scope="module", autouse=True)
def lib():
    qbuild.build()
    return qre.load_library()


def cache(**kw):
    d = dict(k=A, v=A, page_table=A, seq_len=A, ref_count=A, k_scale=None, v_scale=None, n_layers=2, n_pages=100,
             n_kv_heads=4, page_size=32, head_dim=128, max_seqs=8, max_pages=10, dtype=qre.QRE_BF16)
    d.update(kw)
    return qre.qre_kv_cache(**d)


def attn(**kw):
    d = dict(n_heads=8, n_kv_heads=4, head_dim=128, dtype=qre.QRE_BF16, scale=0.1, causal=1, window=0, reserved=0,
             q_token=1024, q_head=128, k_token=512, k_head=128, v_token=512, v_head=128, o_token=1024, o_head=128)
    d.update(kw)
    return qre.qre_attn(**d)


def rows(**kw):
    d = dict(k_token=512, k_head=128, v_token=512, v_head=128, dtype=qre.QRE_BF16, reserved=0)
    d.update(kw)
    return qre.qre_kv_rows(**d)


def refused(code, word, fn, *args, **kw):
    with pytest.raises(qre.QreError) as e:
        fn(*args, stream=0, **kw)
    assert e.value.status == code and word in str(e.value), str(e.value)


INV, UNS, MISA, WS = (qre.QRE_ERR_INVALID_ARG, qre.QRE_ERR_UNSUPPORTED, qre.QRE_ERR_MISALIGNED, qre.QRE_ERR_WORKSPACE)


@pytest.mark.parametrize("kw,code,word", [
    (dict(n_pages=0), INV, "pages 0"), (dict(max_pages=-1), INV, "positive"), (dict(dtype=3), INV, "dtype"),
    (dict(head_dim=96), UNS, "head_dim"), (dict(page_size=8), UNS, "page_size"), (dict(page_size=48), UNS, "page_size"),
    (dict(page_size=512), UNS, "page_size"), (dict(n_kv_heads=257), UNS, "n_kv_heads"),
    (dict(n_pages=1 << 24), UNS, "2^24"), (dict(page_size=256, max_pages=1 << 23), UNS, "31 bits"),
    (dict(k=None), INV, "k is NULL"), (dict(seq_len=MIS), MISA, "seq_len"), (dict(ref_count=None), INV, "ref_count"),
])
def test_bad_caches(kw, code, word):
    refused(code, word, qre.qre_kv_free, cache(**kw), 1, A)
    refused(code, word, qre.qre_kv_compact, cache(**kw), A, A, A, A, 1 << 20)


@pytest.mark.parametrize("kw,code,word", [
    (dict(n_heads=0), INV, "positive"), (dict(n_heads=6), INV, "multiple"), (dict(dtype=qre.QRE_E4M3), UNS, "dtype"),
    (dict(dtype=9), INV, "dtype"), (dict(head_dim=80), UNS, "head_dim"), (dict(n_heads=1028), UNS, "1024"),
    (dict(scale=0.0), INV, "scale"), (dict(scale=float("nan")), INV, "scale"), (dict(scale=float("inf")), INV, "scale"),
    (dict(window=-1), INV, "window"), (dict(window=4, causal=0), INV, "window"), (dict(reserved=1), INV, "reserved"),
    (dict(q_token=100), INV, "q_token"), (dict(o_head=-8), INV, "o_head"), (dict(q_head=1 << 40), UNS, "q_head"),
])
def test_bad_attentions(kw, code, word):
    refused(code, word, qre.qre_attn_prefill, attn(**kw), 1, 4, 4, A, A, A, A, A, A, A)
    refused(code, word, qre.qre_attn_decode, attn(**kw), cache(), 0, 1, A, 0, A, A, A, A, 1 << 24)


def test_prefill_arguments():
    f = qre.qre_attn_prefill
    refused(INV, "k_token", f, attn(k_token=12), 1, 4, 4, A, A, A, A, A, A)
    refused(INV, "v_head", f, attn(v_head=-16), 1, 4, 4, A, A, A, A, A, A)
    refused(INV, "n_seqs", f, attn(), -1, 4, 4, A, A, A, A, A, A)
    refused(UNS, "n_seqs", f, attn(), 4097, 4, 4, A, A, A, A, A, A)
    refused(INV, "negative", f, attn(), 1, -4, 4, A, A, A, A, A, A)
    refused(UNS, "2^24", f, attn(), 1, 4, 1 << 24, A, A, A, A, A, A)
    for i, name in enumerate(("cu_q", "cu_k", "q", "k", "v", "o")):
        p = [A] * 6
        p[i] = None
        refused(INV, name + " is NULL", f, attn(), 1, 4, 4, *p)
        p[i] = MIS
        refused(MISA, name, f, attn(), 1, 4, 4, *p)
    refused(MISA, "lse", f, attn(), 1, 4, 4, A, A, A, A, A, A, MIS)
    f(attn(), 0, 0, 0, None, None, None, None, None, None, stream=0)      # nothing to do, nothing launched
    f(attn(), 3, 0, 9, None, None, None, None, None, None, stream=0)


def test_decode_arguments():
    f = qre.qre_attn_decode
    need = qre.qre_attn_decode_workspace_size(attn(), cache(), 4)
    refused(INV, "differ", f, attn(n_kv_heads=8), cache(), 0, 1, A, 0, A, A, A, A, need)
    refused(INV, "differ", f, attn(head_dim=64), cache(), 0, 1, A, 0, A, A, A, A, need)
    refused(UNS, "cache of dtype", f, attn(), cache(dtype=qre.QRE_FP16), 0, 1, A, 0, A, A, A, A, need)
    refused(INV, "k_scale", f, attn(), cache(k_scale=A), 0, 1, A, 0, A, A, A, A, need)
    refused(MISA, "v_scale", f, attn(), cache(dtype=qre.QRE_E4M3, v_scale=A + 2), 0, 1, A, 0, A, A, A, A, need)
    refused(INV, "layer", f, attn(), cache(), 2, 1, A, 0, A, A, A, A, need)
    refused(INV, "layer", f, attn(), cache(), -1, 1, A, 0, A, A, A, A, need)
    refused(INV, "causal", f, attn(causal=0), cache(), 0, 1, A, 0, A, A, A, A, need)
    refused(INV, "max_len", f, attn(), cache(), 0, 1, A, -1, A, A, A, A, need)
    refused(INV, "without seqs", f, attn(), cache(), 0, 9, None, 0, A, A, A, A, 1 << 26)
    refused(UNS, "4097", f, attn(), cache(), 0, 4097, A, 0, A, A, A, A, 1 << 26)
    refused(INV, "q is NULL", f, attn(), cache(), 0, 4, A, 0, None, A, A, A, need)
    refused(MISA, "o is", f, attn(), cache(), 0, 4, A, 0, A, MIS, A, A, need)
    refused(WS, "needs", f, attn(), cache(), 0, 4, A, 0, A, A, A, A, 16)
    refused(INV, "workspace", f, attn(), cache(), 0, 4, A, 0, A, A, A, None, 0)
    f(attn(), cache(), 0, 0, None, 0, None, None, None, None, 0, stream=0)


def test_cache_call_arguments():
    c, need = cache(), qre.qre_kv_workspace_size(cache())
    refused(INV, "n_new", qre.qre_kv_reserve, c, 1, A, None, A, need)
    refused(WS, "needs", qre.qre_kv_reserve, c, 1, A, A, A, need - 1)
    refused(UNS, "4096", qre.qre_kv_reserve, c, 5000, A, A, A, need)
    refused(INV, "n = -1", qre.qre_kv_free, c, -1, A)
    refused(MISA, "dst", qre.qre_kv_fork, c, 1, A, MIS, A, need)
    refused(INV, "n_live", qre.qre_kv_compact, c, A, A, None, A, need)
    refused(MISA, "workspace", qre.qre_kv_compact, c, A, A, A, MIS, need)
    w = qre.qre_kv_write
    refused(UNS, "cache of dtype", w, c, 0, rows(dtype=qre.QRE_FP16), 1, A, A, A, A)
    refused(INV, "rows dtype", w, c, 0, rows(dtype=qre.QRE_E4M3), 1, A, A, A, A)
    refused(INV, "k_head", w, c, 0, rows(k_head=4), 1, A, A, A, A)
    refused(INV, "layer", w, c, 7, rows(), 1, A, A, A, A)
    refused(INV, "n_tokens", w, c, 0, rows(), -1, A, A, A, A)
    refused(INV, "token_pos", w, c, 0, rows(), 1, A, None, A, A)
    refused(INV, "reserved", w, c, 0, rows(reserved=2), 1, A, A, A, A)
    w(c, 0, rows(), 0, None, None, None, None, stream=0)


def test_workspace_sizes():
    sizes = [qre.qre_kv_workspace_size(cache(n_pages=n)) for n in (1, 100, 100000)]
    assert sizes == sorted(sizes) and sizes[-1] >= 8 * 100000 and all(s % 256 == 0 for s in sizes)
    assert qre.qre_attn_decode_workspace_size(attn(), cache(), 0) >= 0
