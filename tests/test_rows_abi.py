"""Refusals of the calls that norm, turn, write and read rows, and of shared prefixes: every bad argument is named on the
host, before any launch (no GPU needed); the formulas' oracle against plain restatements."""

import ctypes

import numpy as np
import pytest

import quantized_routed_expert_03_gb300 as qre
from oracle import attention as oatt
from test_attention_abi import A, INV, MIS, MISA, UNS, WS, attn, cache, lib, refused, rows  # noqa: F401


def rope(**kw):
    d = dict(inv_freq=A, q_norm=A, k_norm=A, n_heads=8, n_kv_heads=4, head_dim=128, dtype=qre.QRE_BF16, rot_dim=128,
             interleaved=0, eps=1e-6, reserved=0, q_token=1024, q_head=128, k_token=512, k_head=128, v_token=512,
             v_head=128, qo_token=1024, qo_head=128, ko_token=512, ko_head=128)
    d.update(kw)
    return qre.qre_rope(**d)


@pytest.mark.parametrize("kw,code,word", [
    (dict(n_heads=0), INV, "positive"), (dict(dtype=qre.QRE_E4M3), UNS, "dtype"), (dict(dtype=qre.QRE_E2M1), UNS, "dtype"),
    (dict(dtype=3), INV, "dtype"), (dict(head_dim=96), UNS, "head_dim"), (dict(n_heads=1025), UNS, "1024"),
    (dict(n_kv_heads=257), UNS, "n_kv_heads"), (dict(rot_dim=130), INV, "rot_dim"), (dict(rot_dim=-16), INV, "rot_dim"),
    (dict(rot_dim=24), UNS, "multiple of 16"), (dict(eps=-1.0), INV, "eps"), (dict(eps=float("nan")), INV, "eps"),
    (dict(eps=float("inf")), INV, "eps"), (dict(reserved=1), INV, "reserved"), (dict(inv_freq=None), INV, "inv_freq"),
    (dict(inv_freq=MIS), MISA, "inv_freq"), (dict(q_norm=MIS), MISA, "q_norm"), (dict(k_norm=MIS), MISA, "k_norm"),
    (dict(q_token=12), INV, "q_token"), (dict(k_head=-8), INV, "k_head"), (dict(qo_head=1 << 38), UNS, "qo_head"),
    (dict(qo_token=0), INV, "q_out"), (dict(qo_head=0), INV, "q_out"), (dict(ko_token=0), INV, "k_out"),
    (dict(ko_head=0), INV, "k_out"),
])
def test_bad_ropes(kw, code, word):
    refused(code, word, qre.qre_qk_norm_rope, rope(**kw), 2, A, A, A, A, A)
    refused(code, word, qre.qre_kv_write_rope, cache(), 0, rope(**kw), 2, A, A, A, A, A, A, A)


def test_bad_rope_calls():
    f, g = qre.qre_qk_norm_rope, qre.qre_kv_write_rope
    refused(INV, "n_tokens", f, rope(), -1, A, A, A, A, A)
    refused(UNS, "n_tokens", f, rope(), 1 << 24, A, A, A, A, A)
    refused(INV, "token_pos", f, rope(), 1, None, A, A, A, A)
    refused(MISA, "q_out", f, rope(), 1, A, A, A, MIS, A)
    refused(INV, "k_out", f, rope(), 1, A, A, A, A, None)
    refused(INV, "differ", g, cache(), 0, rope(n_kv_heads=2), 1, A, A, A, A, A, A)
    refused(INV, "differ", g, cache(), 0, rope(head_dim=64, rot_dim=64), 1, A, A, A, A, A, A)
    refused(UNS, "cache of dtype", g, cache(dtype=qre.QRE_FP16), 0, rope(), 1, A, A, A, A, A, A)
    refused(INV, "layer", g, cache(), 2, rope(), 1, A, A, A, A, A, A)
    refused(INV, "v_token", g, cache(), 0, rope(v_token=4), 1, A, A, A, A, A, A)
    refused(INV, "token_seq", g, cache(), 0, rope(), 1, None, A, A, A, A, A)
    refused(INV, "v is NULL", g, cache(), 0, rope(), 1, A, A, A, A, None, A)
    refused(MISA, "k_out", g, cache(), 0, rope(), 1, A, A, A, A, A, A, MIS)
    # without tokens nothing is launched; without k_out its strides do not matter
    f(rope(rot_dim=0, inv_freq=None), 0, None, None, None, None, None, stream=0)
    g(cache(), 0, rope(ko_token=0, ko_head=0), 0, None, None, None, None, None, None, stream=0)


def test_bad_reads():
    f = qre.qre_kv_read
    raw, c = qre.load_library().qre_kv_read, cache()
    refused(INV, "rows is NULL", lambda **k: qre._check(raw(ctypes.addressof(c), 0, None, 1, A, None, A, 1, A, A, 0), "qre_kv_read"))
    for bad in (None, attn(), A):
        with pytest.raises(TypeError, match="qre_kv_rows"):
            f(cache(), 0, bad, 1, A, None, A, 1, A, A, stream=0)
    refused(INV, "rows dtype", f, cache(), 0, rows(dtype=qre.QRE_E2M1), 1, A, None, A, 1, A, A)
    refused(UNS, "cache of dtype", f, cache(), 0, rows(dtype=qre.QRE_FP16), 1, A, None, A, 1, A, A)
    refused(INV, "n = -1", f, cache(), 0, rows(), -1, A, None, A, 1, A, A)
    refused(UNS, "n = 4097", f, cache(), 0, rows(), 4097, A, None, A, 1, A, A)
    refused(INV, "total", f, cache(), 0, rows(), 1, A, None, A, -1, A, A)
    refused(UNS, "total", f, cache(), 0, rows(), 1, A, None, A, 1 << 24, A, A)
    refused(INV, "k lie", f, cache(), 0, rows(k_token=0), 1, A, None, A, 2, A, A)
    refused(INV, "v lie", f, cache(), 0, rows(v_head=0), 1, A, None, A, 2, A, A)
    refused(INV, "without seqs", f, cache(), 0, rows(), 9, None, None, A, 1, A, A)
    refused(MISA, "first", f, cache(), 0, rows(), 1, A, MIS, A, 1, A, A)
    refused(INV, "cu is NULL", f, cache(), 0, rows(), 1, A, None, None, 1, A, A)
    refused(INV, "v is NULL", f, cache(), 0, rows(), 1, A, None, A, 1, A, None)
    f(cache(), 0, rows(), 0, None, None, None, 5, None, None, stream=0)
    f(cache(), 0, rows(), 3, A, None, A, 0, None, None, stream=0)


def test_bad_groups():
    f = qre.qre_kv_common_len
    refused(INV, "n = -1", f, cache(), -1, A, 1, A, A)
    refused(UNS, "n_groups", f, cache(), 1, A, 4097, A, A)
    refused(INV, "without seqs", f, cache(), 9, None, 1, A, A)
    refused(INV, "cu_group", f, cache(), 1, A, 1, None, A)
    refused(MISA, "common_len", f, cache(), 1, A, 1, A, MIS)
    f(cache(), 0, None, 0, None, None, stream=0)
    size = qre.qre_attn_decode_shared_workspace_size
    assert size(attn(), cache(), 64, 8) >= qre.qre_attn_decode_workspace_size(attn(), cache(), 64)
    g = qre.qre_attn_decode_shared
    need = size(attn(), cache(), 2, 1)
    refused(INV, "causal", g, attn(causal=0), cache(), 0, 2, A, 1, A, A, 0, A, A, A, A, need)
    refused(INV, "differ", g, attn(n_kv_heads=2), cache(), 0, 2, A, 1, A, A, 0, A, A, A, A, need)
    refused(INV, "max_len", g, attn(), cache(), 0, 2, A, 1, A, A, -1, A, A, A, A, need)
    refused(INV, "common_len", g, attn(), cache(), 0, 2, A, 1, A, None, 0, A, A, A, A, need)
    refused(MISA, "cu_group", g, attn(), cache(), 0, 2, A, 1, MIS, A, 0, A, A, A, A, need)
    refused(UNS, "n_groups", g, attn(), cache(), 0, 2, A, 5000, A, A, 0, A, A, A, A, need)
    refused(WS, "workspace", g, attn(), cache(), 0, 2, A, 1, A, A, 0, A, A, A, A, need - 1)
    g(attn(), cache(), 0, 0, None, 0, None, None, 0, None, None, None, None, 0, stream=0)


def test_4_bit_caches_take_scales_and_have_no_16_bit_rows():
    c = cache(dtype=qre.QRE_E2M1, k_scale=A + 4, v_scale=A)
    qre.qre_kv_write(c, 0, rows(), 0, None, None, None, None, stream=0)
    qre.qre_kv_write(c, 0, rows(dtype=qre.QRE_FP16), 0, None, None, None, None, stream=0)
    refused(MISA, "v_scale", qre.qre_kv_write, cache(dtype=qre.QRE_E2M1, v_scale=A + 2), 0, rows(), 1, A, A, A, A)
    refused(INV, "k_scale", qre.qre_kv_write, cache(k_scale=A), 0, rows(), 1, A, A, A, A)
    refused(INV, "rows dtype", qre.qre_kv_write, c, 0, rows(dtype=qre.QRE_E2M1), 1, A, A, A, A)
    refused(UNS, "attention dtype", qre.qre_attn_decode, attn(dtype=qre.QRE_E2M1), c, 0, 1, A, 0, A, A, A, A, 1 << 30)
    assert qre.qre_attn_decode_workspace_size(attn(), c, 5) > 0


def test_the_4_bit_codes_of_the_oracle():
    x = np.array([0.0, 0.25, 0.2500001, 0.75, 0.7499, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 3.49, 5.0, 5.01, 6.0, 7.0])
    want = [0, 0, 1, 2, 1, 2, 3, 4, 4, 5, 6, 5, 6, 7, 7, 7]
    assert oatt.e2m1_code(x).tolist() == want
    assert oatt.e2m1_code(-x).tolist() == [w | 8 for w in want]
    r = np.random.default_rng(0).normal(size=(3, 2, 64)) * 3
    code, s, worth = oatt.e2m1_blocks(r)
    assert (np.abs(worth - r).reshape(3, 2, 4, 16) <= np.maximum(1.0 * s, np.abs(r).reshape(3, 2, 4, 16).max(-1) / 6 * 2 ** -3)[..., None] + 1e-12).all()
    for b in range(256):                       # bytes of every E4M3 value that is a scale
        e, f = b >> 3, b & 7
        if b < 0x7f:
            assert oatt.e4m3_bytes((1 + f / 8) * 2.0 ** (e - 7) if e else f / 8 * 2.0 ** -6) == b
    assert oatt.e4m3_bytes(np.nan) == 0x7f


def test_the_rotation_of_the_oracle():
    rng = np.random.default_rng(1)
    x, pos, f = rng.normal(size=(4, 2, 64)), np.array([0, 1, 7, 1000]), 10.0 ** -rng.random(16)
    for inter in (False, True):
        y, size, angle = oatt.turn(x, pos, f, inter)
        z = (x[..., :32].reshape(4, 2, 16, 2) if inter else np.moveaxis(x[..., :32].reshape(4, 2, 2, 16), 2, 3))
        z = (z[..., 0] + 1j * z[..., 1]) * np.exp(1j * pos[:, None] * f)[:, None]
        a, b = (y[..., 0:32:2], y[..., 1:32:2]) if inter else (y[..., :16], y[..., 16:32])
        assert np.allclose(a, z.real) and np.allclose(b, z.imag) and np.array_equal(y[..., 32:], x[..., 32:])
        assert (np.abs(y) <= size + 1e-12).all()
    y, _, _ = oatt.turn(x, pos, [], False, np.full(64, 2.0), 0.0)
    assert np.allclose((y * y).mean(-1), 4.0)
