"""Decode attention with shared prefixes where its launches, its plan and its numbers are at an edge."""

import math

import numpy as np
import pytest
import torch

import quantized_routed_expert_03_gb300 as qre
from oracle import attention as oatt
from quantized_routed_expert_03_gb300.attention import Attention, KVCache
from test_gpu_rows import DEV, TYPE, clean_status, i32, npy, randn   # noqa: F401
from test_gpu_shared import Shared, check, run

pytestmark = pytest.mark.gpu


def test_own_positions_whose_places_pass_31_bits():
    """128 sequences that share nothing, 2^20 positions each on the same eight pages again and again, 256 KV heads: more
    than 2^31 places.  A softmax over 2^13 times the same 128 keys is the softmax over those keys, its log-sum log 2^13
    larger."""
    n, H, D, page, pages = 128, 256, 128, 16, 8
    cols = 2 ** 20 // page
    c = KVCache(1, pages, H, page, D, n, cols, device=DEV)
    c.k.copy_(randn(c.k.shape, 1, "bf16"))
    c.v.copy_(randn(c.v.shape, 2, "bf16"))
    c.page_table.copy_((torch.arange(cols, device=DEV) % pages).int().expand(n, cols))
    q = randn((n, H, D), 3, "bf16")
    c.seq_len.fill_(pages * page)
    short = torch.empty((n, H), device=DEV)
    want = Attention(c, 0, H, n).decode(q, None, lse=short)
    c.seq_len.fill_(page * cols)
    att = Attention(c, 0, H, n, max_groups=n)
    lse = torch.full((n, H), float("nan"), device=DEV)
    o = att.decode_shared(q, None, torch.arange(n + 1, dtype=torch.int32, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV), lse=lse)
    assert qre.qre_read_device_status() == 0
    # Sums of up to 2^16 chunks one after the other, each step off by at most 2^-23 of the sum (a sum that is cut off, not
    # rounded): 2^-7, of the sum and of O; bf16 weights and results on both sides, 2^-8 each time
    assert float((lse - short - math.log(2 ** 13)).abs().max()) <= 2.0 ** -7 + 1e-4
    size = float(c.v.float().abs().max())
    assert float((o.float() - want.float()).abs().max()) <= size * (2 * 2.0 ** -7 + 4 * 2.0 ** -8)


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "e2m1"])
def test_queries_without_any_group(cache):
    """No groups are bounds that do not run from 0 to n: each query by itself, and a note."""
    w = Shared([900, 600], [[5, 70], [3, 4]], 4, 2, 64, 16, "bf16", cache, seed=2)
    q = randn((4, 4, 64), 1, "bf16")
    ref, v_max = w.reference(q)
    att = Attention(w.c, 1, 4, 4, max_groups=1)
    lse = torch.empty((4, 4), device=DEV)
    o = att.decode_shared(q, i32(w.seqs), i32([0]), w.c.common_len(i32(w.seqs), i32([0])), lse=lse)
    assert qre.qre_read_device_status() == qre.QRE_DEV_BAD_INDEX
    qre.qre_clear_device_status()
    check(o, lse, ref, "bf16", 970, v_max)
    # the call itself: no arrays of groups at all
    size = qre.qre_attn_decode_shared_workspace_size(att._desc(), w.c.desc, 4, 0)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    o.fill_(float("nan"))
    lse.fill_(float("nan"))
    qre.qre_attn_decode_shared(att._desc(q, o=o), w.c.desc, 1, 4, i32(w.seqs), 0, None, None, 0, q, o, lse, ws)
    assert qre.qre_read_device_status() == qre.QRE_DEV_BAD_INDEX
    qre.qre_clear_device_status()
    check(o, lse, ref, "bf16", 970, v_max)


@pytest.mark.parametrize("cache", ["bf16", "e2m1"])
def test_plans_that_change_from_call_to_call_on_one_workspace(cache):
    """The own positions' kernel takes each call's plan (what is shared, how many CTAs it has) and no older one: calls one
    behind the other, with nothing between them, whose holes and splits differ; then as two graphs, replayed in turn."""
    w = Shared([6000, 900], [[700, 30, 1, 2000], [5, 70]], 8, 2, 128, 64, "bf16", cache, seed=12)
    seqs, n, H, D = i32(w.seqs), 6, 8, 128
    att = Attention(w.c, 1, H, n, max_groups=n)
    att.workspace.fill_(0xFF)
    # groups and common lengths: all, none, some, one group alone, the other alone, groups of one, the first in part
    plans = [([0, 4, 6], [5952, 896]), ([0, 4, 6], [0, 0]), ([0, 4, 6], [2048, 896]), ([0, 4, 6], [5952, 0]),
             ([0, 4, 6], [0, 896]), ([0, 1, 2, 3, 4, 5, 6], [0] * 6), ([0, 2, 4, 6], [5952, 5952, 896]),
             ([0, 2, 6], [128, 0])]
    plans = [(i32(cu), i32(common)) for cu, common in plans]
    q = [randn((n, H, D), 20 + i, "bf16") for i in range(len(plans))]
    want = []
    for (cu, common), x in zip(plans, q):
        lse = torch.empty((n, H), device=DEV)
        want.append((att.decode_shared(x, seqs, cu, common, lse=lse).clone(), lse))
        torch.cuda.synchronize()
    assert qre.qre_read_device_status() == 0
    for i in range(len(plans)):
        ref, v_max = w.reference(q[i])
        check(*want[i], ref, "bf16", max(w.lens), v_max)
    order = torch.randperm(20 * len(plans), generator=torch.Generator().manual_seed(1)) % len(plans)
    got = []
    for i in order.tolist():
        lse = torch.empty((n, H), device=DEV)
        got.append((att.decode_shared(q[i], seqs, *plans[i], lse=lse), lse))
    torch.cuda.synchronize()
    for i, (o, lse) in zip(order.tolist(), got):
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])

    out = [(torch.empty_like(q[0]), torch.empty((n, H), device=DEV)) for _ in plans]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for half, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            for i in range(half, len(plans), 2):
                att.decode_shared(q[i], seqs, *plans[i], o=out[i][0], lse=out[i][1])
    for step in range(20):
        for o, lse in out:
            o.fill_(float("nan"))
            lse.fill_(float("nan"))
        graphs[step & 1].replay()
        graphs[1 - (step & 1)].replay()
        torch.cuda.synchronize()
        for (o, lse), (wo, wl) in zip(out, want):
            assert torch.equal(o, wo) and torch.equal(lse, wl)
    assert qre.qre_read_device_status() == 0


def attend(c, n, H, q, o, lse, v_max, kind, only):
    """Queries `only` of a decode of sequences 0 .. n - 1 on an unscaled cache of one layer against fp64."""
    H, Hk, D = q.shape[1], c.n_kv_heads, c.head_dim
    lens = c.seq_len.tolist()
    k, v = (x.double() for x in c.read(0, i32(only), i32(np.cumsum([0] + [lens[s] for s in only])), sum(lens[s] for s in only), dtype=TYPE[kind]))
    ref = [np.zeros((n, H, D)), np.zeros((n, H)), np.zeros((n, H, D)), np.zeros((n, H))]
    at = 0
    for s in only:
        kk, vv = (x[at:at + lens[s]].cpu().numpy() for x in (k, v))
        at += lens[s]
        for h in range(H):
            j = h // (H // Hk)
            for dst, x in zip(ref, oatt.attend(npy(q)[s, h:h + 1], kk[:, j], vv[:, j], D ** -0.5, [0], [lens[s]])):
                dst[s, h] = x[0]
    check(o, lse, ref, kind, max(lens), v_max, set(only))


# both sides of the numbers of queries from which an SM holds a CTA less
@pytest.mark.parametrize("n,shared", [(232, False), (234, False), (3476, False), (3478, False), (116, True), (118, True), (1026, True)])
def test_4_bit_calls_of_many_queries(n, shared):
    H, Hk, D, page, prefix = 16, 2, 128, 16, 512
    own_pages = 4
    c = KVCache(1, prefix // page + 40 * own_pages, Hk, page, D, n, prefix // page + own_pages, TYPE["e2m1"], device=DEV)
    T = c.k.shape[1] * page                                  # rows for every page, one sequence's after the other's
    fill = KVCache(1, 1, Hk, page, D, 1, c.k.shape[1], TYPE["e2m1"], device=DEV)
    fill.desc.k, fill.desc.v, fill.desc.n_pages = c.desc.k, c.desc.v, c.desc.n_pages
    fill.page_table.copy_(torch.arange(c.k.shape[1], device=DEV)[None])
    k, v = randn((T, Hk, D), 1, "bf16", 1.5), randn((T, Hk, D), 2, "bf16")
    fill.write(0, torch.zeros(T, dtype=torch.int32, device=DEV), torch.arange(T, dtype=torch.int32, device=DEV), k, v)
    rows = torch.arange(n, device=DEV)
    c.page_table[:, :prefix // page] = torch.arange(prefix // page, dtype=torch.int32, device=DEV)
    c.page_table[:, prefix // page:] = (prefix // page + rows[:, None] % 40 * own_pages + torch.arange(own_pages, device=DEV)).int()
    c.seq_len[:] = (prefix + 1 + rows * 7 % (own_pages * page)).int()
    q = randn((n, H, D), 3, "bf16")
    lse = torch.full((n, H), float("nan"), device=DEV)
    only = sorted({0, 1, n // 2, n - 2, n - 1})
    v_max = float(v.abs().max()) * 1.2
    if shared:
        cu = i32([0, n // 2, n])
        common = c.common_len(torch.arange(n, dtype=torch.int32, device=DEV), cu)
        assert common.tolist() == [prefix, prefix]
        att = Attention(c, 0, H, n, max_groups=2)
        o = att.decode_shared(q, None, cu, common, lse=lse)
        again = att.decode_shared(q, None, cu, common)
    else:
        att = Attention(c, 0, H, n)
        o = att.decode(q, None, lse=lse)
        again = att.decode(q, None)
    assert qre.qre_read_device_status() == 0
    attend(c, n, H, q, o, lse, v_max, "bf16", only)
    assert torch.equal(o, again) and torch.isfinite(o).all()


# 6 and 240 rows of a KV head: the chains take tiles in turn, or each has rows of its own
@pytest.mark.parametrize("cache", ["bf16", "fp16", "e4m3", "e2m1"])
@pytest.mark.parametrize("D,members", [(128, 3), (64, 3), (128, 120)])
def test_a_wait_that_runs_out_and_the_next_call(cache, D, members):
    """The first CTA's loads come 20 ms late: the waits for them run out after 2 ms; the loads are issued behind that all the
    same, and the kernel waits for them, says so and ends.  The calls behind it have the same bits as the one before."""
    kind = "fp16" if cache == "fp16" else "bf16"
    w = Shared([9000], [[3, 7, 20] * (members // 3)], 4, 2, D, 64, kind, cache, seed=4)
    q = randn((members, 4, D), 1, kind)
    want = run(w, q)
    assert qre.qre_read_device_status() == 0
    try:
        qre.qre_debug_wait_test(2_000_000, 20_000_000)
        run(w, q)
        status = qre.qre_read_device_status()
    finally:
        qre.qre_debug_wait_test(0, 0)
    assert status == qre.QRE_DEV_TIMEOUT
    qre.qre_clear_device_status()
    for _ in range(3):                                       # (the tensor memory is free again)
        got = run(w, q)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert qre.qre_read_device_status() == 0


def test_sequences_in_order_need_no_ids():
    """seqs None: the same common lengths and the same attention as with 0, 1, and so on."""
    w = Shared([300, 700], [[5, 9, 1], [30, 2]], 4, 2, 64, 16, "bf16", "bf16")
    assert w.seqs == list(range(5))
    cu = i32(w.cu)
    common = w.c.common_len(None, cu)
    assert common.tolist() == [288, 688] == w.common().tolist()
    q = randn((5, 4, 64), 1, "bf16")
    o, lse = run(w, q)
    att, l2 = Attention(w.c, 1, 4, 5, max_groups=2), torch.empty_like(lse)
    assert torch.equal(att.decode_shared(q, None, cu, common, lse=l2), o) and torch.equal(l2, lse)
    assert qre.qre_read_device_status() == 0


@pytest.mark.parametrize("kind,cache,rows", [("bf16", "bf16", 6), ("fp16", "fp16", 6), ("bf16", "bf16", 160), ("bf16", "e4m3", 6),
                                             ("fp16", "e2m1", 6), ("bf16", "e2m1", 160)])
def test_a_nan_in_a_shared_prefix(kind, cache, rows):
    """One in the values of KV head 0 is that dimension of its heads (in 4 bits its block's 16), one in the keys of KV head 1
    all of its heads; KV head 2, and the other dimensions of the first, do not know."""
    H, Hk, D, page, n = 6, 3, 64, 16, rows // 2
    w = Shared([1000], [[1 + i % 7 for i in range(n)]], H, Hk, D, page, kind, cache, seed=5)
    q = randn((n, H, D), 7, kind, 1.5)
    ref, v_max = w.reference(q)
    at, row = int(w.c.page_table[0, 500 // page]), 500 % page

    def poison(pool, head, d):
        if cache == "e4m3":
            pool.view(torch.uint8)[1, at, head, row, d] = 0x7f
        elif cache == "e2m1":
            pool[1].flatten(-2)[at, head, page * D // 2 + row * (D // 16) + d // 16] = 0x7f
        else:
            pool[1, at, head, row, d] = float("nan")
    poison(w.c.v, 0, 21)
    poison(w.c.k, 1, 3)
    o, lse = run(w, q)
    assert qre.qre_read_device_status() == 0
    hit = torch.zeros((n, H, D), dtype=torch.bool, device=DEV)
    hit[:, :2, 16 if cache == "e2m1" else 21:32 if cache == "e2m1" else 22] = True
    hit[:, 2:4] = True
    assert torch.equal(torch.isnan(o), hit)
    assert torch.isnan(lse[:, 2:4]).all() and not torch.isnan(lse[:, :2]).any() and not torch.isnan(lse[:, 4:]).any()
    mask = hit.cpu().numpy()
    clean = [x.copy() for x in ref]
    clean[0][mask], clean[1][:, 2:4] = 0, 0
    got, gl = torch.where(hit, torch.zeros_like(o), o), lse.clone()
    gl[:, 2:4] = 0
    check(got, gl, clean, kind, max(w.lens), v_max)


@pytest.mark.parametrize("kind,rows", [("bf16", 6), ("fp16", 6), ("bf16", 160)])
def test_an_infinite_key_in_a_shared_prefix(kind, rows):
    """A key that scores -infinity counts nothing; one that scores +infinity leaves no softmax."""
    H, Hk, D, page, n = 6, 3, 64, 16, rows // 2
    w = Shared([1000], [[1 + i % 7 for i in range(n)]], H, Hk, D, page, kind, kind, seed=5)
    q = randn((n, H, D), 7, kind, 1.5)
    q[..., 9] = -q[..., 9].abs() - 0.125
    q[1, 4, 9] = 0.5
    (_, _, ra, rb), v_max = w.reference(q)
    for pos in (0, 127, 128, 500, 991):
        w.c.k[1, int(w.c.page_table[0, pos // page]), 2, pos % page, 9] = float("inf")
    ref, _ = w.reference(q)
    assert np.isnan(ref[0][1, 4]).all() and np.isnan(ref[0]).sum() == D
    o, lse = run(w, q)
    assert qre.qre_read_device_status() == 0
    assert torch.isnan(o[1, 4]).all() and int(torch.isnan(o).sum()) == D
    got = torch.nan_to_num(o, nan=0.0)
    gl, wl = torch.where(torch.isnan(o[..., 0]), torch.zeros_like(lse), lse), np.where(np.isnan(ref[0][..., 0]), 0, ref[1])
    # (weights that five keys leave grow by less than a part in 100, which the scores' own term covers)
    check(got, gl, (np.nan_to_num(ref[0]), wl, np.maximum(ra, np.nan_to_num(ref[2])), rb), kind, max(w.lens), v_max)
