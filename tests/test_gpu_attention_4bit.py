"""Decode attention over a 4-bit cache against fp64 on what its pages are worth, within oracle.attention.tolerance."""

import math

import numpy as np
import pytest
import torch

import quantized_routed_expert_03_gb300 as qre
from oracle import attention as oatt
from quantized_routed_expert_03_gb300.attention import Attention
from test_gpu_rows import DEV, TYPE, UNIT, Pool, clean_status, i32, npy, randn, stored   # noqa: F401

pytestmark = pytest.mark.gpu


def filled(lens, page, Hk, D, kind, scaled, seed=0, k_scale=2.0):
    """A 4-bit cache whose rows were written from 16-bit ones, and what layer 1 is worth in fp64 [K or V][tokens, Hk, D]."""
    p = Pool("e2m1", lens, page, Hk, D, scaled=scaled, seed=seed)
    T = len(p.tokens)
    k, v = randn((T, Hk, D), seed + 1, kind, k_scale), randn((T, Hk, D), seed + 2, kind)
    if T:
        seq, pos = p.ids()
        p.c.write(1, seq, pos, k, v)
    worth = []
    for x, rows in ((0, k), (1, v)):
        f = p.scale(x, 1)
        _, _, w = oatt.e2m1_blocks(npy(rows), None if f is None else f.cpu().numpy())
        worth.append(w if f is None else w * f.cpu().numpy().astype(np.float64)[:, None])
    return p, worth


def reference(p, worth, q, seqs, window=0):
    n, H, D = q.shape
    first = np.concatenate([[0], np.cumsum(p.lens)])
    out = [np.zeros((n, H, D)), np.full((n, H), -np.inf), np.zeros((n, H, D)), np.zeros((n, H))]
    qs = npy(q)
    for i, s in enumerate(seqs):
        L = p.lens[s]
        lo = max(0, L - window) if window else 0
        for h in range(H):
            hk = h // (H // p.Hk)
            k, v = (w[first[s]:first[s + 1], hk] for w in worth)
            for dst, x in zip(out, oatt.attend(qs[i, h:h + 1], k, v, 1 / math.sqrt(D), [lo], [L])):
                dst[i, h] = x[0]
    return out


def check(o, lse, ref, kind, n_keys, v_max):
    """tolerance counts weights that an fp16 product loses for fp16 outputs; here all products are fp16's: with a reference
    2^10 below the maximum, what is lost is below 2^-35 of it."""
    ro, rl, ra, rb = ref
    tol = oatt.tolerance(ro, ra, rb, n_keys, ro.shape[-1], UNIT[kind], v_max) + n_keys * 2.0 ** -35 * v_max
    got = npy(o)
    assert np.isfinite(got).all() and (np.abs(got - ro) <= tol).all(), (np.abs(got - ro) - tol).max()
    gl, fin = npy(lse), np.isfinite(rl)
    assert np.array_equal(np.isneginf(gl), ~fin)
    assert (np.abs(gl - rl)[fin] <= oatt.lse_tolerance(rl, rb, n_keys, ro.shape[-1])[fin]).all()


DECODE = [
    # lens, H, Hk, D, page, kind, window, scaled
    ([1], 1, 1, 64, 16, "bf16", 0, False),
    ([0, 1, 15, 16, 17, 63, 64, 65], 4, 2, 64, 16, "bf16", 0, True),
    ([0, 1, 15, 16, 17, 63, 64, 65], 4, 2, 128, 16, "fp16", 0, False),
    ([1000, 3, 0, 513], 8, 1, 128, 64, "fp16", 0, True),
    ([777], 32, 8, 128, 16, "bf16", 0, False),
    ([700, 90], 14, 2, 64, 32, "fp16", 0, True),                 # 7 heads per KV head
    ([260, 1], 40, 2, 128, 256, "bf16", 0, False),               # 20
    ([400, 33], 64, 1, 64, 16, "fp16", 0, False),                # 64 heads on one
    ([2100, 64, 63], 6, 2, 128, 64, "bf16", 100, True),          # window
    ([500, 20], 4, 4, 64, 16, "fp16", 1, False),
    ([5003], 8, 1, 128, 16, "fp16", 0, True),
    ([300] * 40 + [7] * 60, 16, 8, 64, 128, "bf16", 0, False),   # more units than warps
]


@pytest.mark.parametrize("max_len", [0, -1])
@pytest.mark.parametrize("case", range(len(DECODE)))
def test_decode_over_4_bits(case, max_len):
    lens, H, Hk, D, page, kind, window, scaled = DECODE[case]
    p, worth = filled(lens, page, Hk, D, kind, scaled, seed=case)
    seqs = np.random.default_rng(case).permutation(len(lens))
    q = randn((len(lens), H, D), 50 + case, kind, 1.5)
    att = Attention(p.c, 1, H, len(lens), TYPE[kind], window=window)
    lse = torch.full((len(lens), H), float("nan"), device=DEV)
    o = att.decode(q, i32(seqs), lse=lse, max_len=max(lens) if max_len else 0)
    assert qre.qre_read_device_status() == 0
    v_max = float(np.abs(worth[1]).max()) if worth[1].size else 0.0
    check(o, lse, reference(p, worth, q, seqs, window), kind, max(lens), v_max)


def test_what_is_not_seen_does_not_reach_the_result():
    """Codes and scales behind the end of a sequence, before a window, and on missing pages, NaN among them."""
    p, worth = filled([50, 200], 16, 2, 64, "bf16", False)
    q = randn((2, 4, 64), 1, "bf16")
    ref = reference(p, worth, q, [0, 1], 70)
    att = Attention(p.c, 1, 4, 2, window=70)
    first = att.decode(q, None).clone()
    for byte in (0x7f, 0xff, 0x00, 0x7e):
        # behind position 50 of sequence 0 (page 3), and before the window of sequence 1 (position 129 and down, page 8)
        for pool in (p.c.k, p.c.v):
            for s, page, rows in ((0, 3, slice(2, 16)), (1, 8, slice(0, 2)), (1, 7, slice(0, 16))):
                flat = pool[1, int(p.c.page_table[s, page])].reshape(2, -1)
                flat[:, :16 * 32].view(2, 16, 32)[:, rows] = byte
                flat[:, 16 * 32:].view(2, 16, 4)[:, rows] = byte
        assert torch.equal(att.decode(q, None), first)
    lse = torch.empty((2, 4), device=DEV)
    check(att.decode(q, None, lse=lse), lse, ref, "bf16", 200, float(np.abs(worth[1]).max()))
    p.c.page_table[1, 9] = -1                                  # a page that is missing counts as not seen
    att.decode(q, None, lse=lse)
    assert qre.qre_read_device_status() == qre.QRE_DEV_BAD_INDEX and torch.isfinite(lse).all()


def test_large_values_and_queries():
    """Scales at the ends of their range, queries that fp16 does not hold."""
    for mag, qm in ((2000.0, 1e-4), (1e-3, 1e4), (2000.0, 1e20)):
        p, worth = filled([90], 16, 1, 128, "bf16", False, seed=5, k_scale=mag)
        q = randn((1, 2, 128), 9, "bf16", qm)
        att = Attention(p.c, 1, 2, 1, scale=1 / (math.sqrt(128) * qm * mag * 4))
        lse = torch.empty((1, 2), device=DEV)
        o = att.decode(q, None, lse=lse)
        ref = [np.zeros((1, 2, 128)), np.zeros((1, 2)), np.zeros((1, 2, 128)), np.zeros((1, 2))]
        for h in range(2):
            scale = float(np.float32(att.scale))
            for dst, x in zip(ref, oatt.attend(npy(q)[0, h:h + 1], worth[0][:, 0], worth[1][:, 0], scale, [0], [90])):
                dst[0, h] = x[0]
        check(o, lse, ref, "bf16", 90, float(np.abs(worth[1]).max()))


def test_chunked_prefill_behind_a_4_bit_prefix():
    """A prompt in two chunks: the second attends to the first as its pages give it back, turned keys among them; then
    one token by decode.  Graphs of the decode step replay with longer sequences."""
    from quantized_routed_expert_03_gb300.attention import KVCache, Rotary
    H, Hk, D, n1, n2 = 4, 2, 64, 37, 20
    c = KVCache(1, 12, Hk, 16, D, 2, 6, TYPE["e2m1"], device=DEV)
    rotary = Rotary(H, Hk, D, q_norm=torch.ones(D, device=DEV), k_norm=torch.ones(D, device=DEV), device=DEV)
    att = Attention(c, 0, H, 2)
    seq = i32([1])
    q, k, v = (randn((n1 + n2 + 3, h, D), i, "bf16", 1.5) for i, h in enumerate((H, Hk, Hk)))
    pos = torch.arange(n1 + n2 + 3, dtype=torch.int32, device=DEV)
    ids = torch.ones_like(pos)
    kept = []
    for a, b in ((0, n1), (n1, n1 + n2)):
        c.reserve(seq, i32([b - a]))
        qa, ka = c.write_rope(0, rotary, ids[a:b].clone(), pos[a:b].clone(), q[a:b], k[a:b], v[a:b])
        kc, vc = c.read(0, seq, i32([0, b]), b)
        kc[a:], vc[a:] = ka, v[a:b]                             # the chunk's own rows as they were
        o = att.prefill(qa, kc, vc, i32([0, b - a]), i32([0, b]))
        ref = oatt.prefill(npy(qa), npy(kc), npy(vc), [b - a], [b], D ** -0.5)
        tol = oatt.tolerance(ref[0], ref[2], ref[3], b, D, 2.0 ** -8, float(vc.abs().max()))
        assert (np.abs(npy(o) - ref[0]) <= tol).all()
        kept.append(npy(ka))
    one = i32([1])
    step_q, step_k, step_v, step_pos = q[:1].clone(), k[:1].clone(), v[:1].clone(), i32([0])
    out = torch.empty_like(step_q)

    def step():
        c.reserve(seq, one)
        qa, _ = c.write_rope(0, rotary, seq, step_pos, step_q, step_k, step_v, keep=False)
        att.decode(qa, seq, o=out)

    graph = None
    for t in range(n1 + n2, n1 + n2 + 3):
        for dst, x in ((step_q, q), (step_k, k), (step_v, v)):
            dst.copy_(x[t:t + 1])
        step_pos.fill_(t)
        if graph is None:
            step()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        qa, _ = rotary.apply(step_q, step_k, step_pos)
        kc, vc = (npy(x)[:, :, :] for x in c.read(0, seq, i32([0, t + 1]), t + 1))
        ref = [np.zeros((1, H, D)), np.zeros((1, H)), np.zeros((1, H, D)), np.zeros((1, H))]
        for h in range(H):
            for dst, x in zip(ref, oatt.attend(npy(qa)[0, h:h + 1], kc[:, h // 2], vc[:, h // 2], D ** -0.5, [0], [t + 1])):
                dst[0, h] = x[0]
        tol = oatt.tolerance(ref[0], ref[2], ref[3], t + 1, D, 2.0 ** -8, np.abs(vc).max()) + (t + 1) * 2.0 ** -35 * np.abs(vc).max()
        assert (np.abs(npy(out) - ref[0]) <= tol).all()
    assert qre.qre_read_device_status() == 0
