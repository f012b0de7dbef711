"""Prefill and decode attention against fp64, within bounds derived from the roundings (oracle.attention.tolerance)."""

import math

import numpy as np
import pytest
import torch

import quantized_routed_expert_03_gb300 as qre
from oracle import attention as oatt

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": (qre.QRE_BF16, torch.bfloat16), "fp16": (qre.QRE_FP16, torch.float16),
      "e4m3": (qre.QRE_E4M3, torch.float8_e4m3fn)}
UNIT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


@pytest.fixture(autouse=True)
def clean_status():
    qre.qre_clear_device_status()
    yield
    qre.qre_clear_device_status()


def i32(a):
    return torch.tensor([int(x) for x in a], dtype=torch.int32, device=DEV)


def npy(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def randn(shape, seed, kind, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(DT[kind][1])


def layout(x, how):
    """The same values under other strides."""
    T, H, D = x.shape
    if how == "packed":
        return x
    if how == "head_major":
        return x.transpose(0, 1).contiguous().transpose(0, 1)
    pad = torch.full((T, H + 3, D + 8), float("nan"), dtype=x.dtype, device=x.device)   # what lies between is never read
    pad[:, 1:H + 1, :D] = x
    return pad[:, 1:H + 1, :D]


def check(o, lse, ref, kind, n_keys, v_max):
    ro, rl, ra, rb = ref
    D = ro.shape[-1]
    got = npy(o)
    err = np.abs(got - ro)
    tol = oatt.tolerance(ro, ra, rb, n_keys, D, UNIT[kind], v_max)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), (err - tol).max()
    if lse is not None:
        gl = npy(lse)
        assert np.array_equal(np.isneginf(gl), np.isneginf(rl))
        fin = np.isfinite(rl)
        lt = oatt.lse_tolerance(rl, rb, n_keys, D)
        assert (np.abs(gl[fin] - rl[fin]) <= lt[fin]).all()


def run_prefill(q, k, v, q_lens, k_lens, kind, causal=True, window=0, scale=None, how="packed", stream=None, lse=True):
    H, Hk, D = q.shape[1], k.shape[1], q.shape[2]
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    o = layout(torch.full(q.shape, float("nan"), dtype=q.dtype, device=DEV), how)
    l = torch.full(q.shape[:2], float("nan"), dtype=torch.float32, device=DEV) if lse else None
    a = qre.make_attn(H, Hk, D, DT[kind][0], scale, causal=causal, window=window, q=q, k=k, v=v, o=o)
    cq, ck = i32(np.concatenate([[0], np.cumsum(q_lens)])), i32(np.concatenate([[0], np.cumsum(k_lens)]))
    qre.qre_attn_prefill(a, len(q_lens), q.shape[0], k.shape[0], cq, ck, q, k, v, o, l, stream=stream)
    return o, l


CASES = [
    # q_lens, k_lens, H, Hk, D, kind, causal, window
    ([1], [1], 1, 1, 64, "bf16", True, 0),
    ([5, 1, 0, 17], [5, 1, 0, 17], 4, 2, 64, "bf16", True, 0),
    ([127, 128, 129], [127, 128, 129], 2, 1, 128, "bf16", True, 0),
    ([300], [300], 8, 1, 128, "fp16", True, 0),
    ([33, 257], [33, 257], 6, 2, 128, "bf16", True, 0),          # 3 heads per KV head
    ([64, 200], [64, 200], 7, 1, 64, "fp16", True, 0),           # 7
    ([64, 3], [600, 1000], 16, 1, 64, "bf16", True, 0),          # a prefix stands before
    ([40, 300], [40, 300], 4, 4, 64, "bf16", True, 33),          # window
    ([50, 260], [700, 400], 8, 2, 128, "fp16", True, 130),
    ([10, 200], [4, 70], 4, 1, 128, "bf16", True, 0),            # fewer keys than queries: empty rows
    ([10, 3], [0, 5], 2, 2, 64, "fp16", True, 1),                # no keys at all
    ([70, 130], [200, 31], 4, 2, 128, "bf16", False, 0),         # not causal
    ([513], [513], 32, 1, 128, "bf16", True, 0),                 # 32 heads on one
    ([9, 8], [9, 8], 20, 4, 128, "fp16", True, 0),               # 5
]


@pytest.mark.parametrize("how", ["packed", "head_major", "padded"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_prefill(case, how):
    q_lens, k_lens, H, Hk, D, kind, causal, window = CASES[case]
    q = randn((sum(q_lens), H, D), 1, kind, 1.5)
    k, v = (randn((sum(k_lens), Hk, D), 2 + i, kind) for i in range(2))
    ref = oatt.prefill(npy(q), npy(k), npy(v), q_lens, k_lens, 1.0 / math.sqrt(D), causal, window)
    o, l = run_prefill(layout(q, how), layout(k, how), layout(v, how), q_lens, k_lens, kind, causal, window, how=how)
    assert qre.qre_read_device_status() == 0
    check(o, l, ref, kind, max(k_lens), float(v.abs().max()) if v.numel() else 0.0)


@pytest.mark.parametrize("H,Hk,D,kind", [(8, 2, 64, "bf16"), (32, 8, 128, "fp16"), (3, 1, 128, "bf16")])
@pytest.mark.parametrize("q_lens,k_lens", [([1], [1]), ([16], [16]), ([17], [17]), ([1, 0, 3], [33, 5, 40]), ([30, 9, 24], [30, 9, 24]),
                                           ([0, 7, 0, 12], [4, 2, 0, 50]), ([64], [64]), ([65], [65]), ([1] * 40, [3] * 40),
                                           ([1, 0, 2] * 140, [1, 0, 2] * 140), ([1] * 256, [2] * 256), ([1] * 257, [2] * 257)])
def test_prefill_a_handful_of_keys(H, Hk, D, kind, q_lens, k_lens):
    """Around the sizes at which the work goes by rows, not by tiles; what is not seen is NaN."""
    q = randn((sum(q_lens), H, D), 1, kind, 1.5)
    k, v = (randn((sum(k_lens), Hk, D), 2 + i, kind) for i in range(2))
    for window in (0, 5):
        ref = oatt.prefill(npy(q), npy(k), npy(v), q_lens, k_lens, 1.0 / math.sqrt(D), True, window)
        kk, vv = k.clone(), v.clone()
        y = 0
        for nq, nk in zip(q_lens, k_lens):
            lo, hi = oatt.visible(nq, nk, True, window)
            seen = np.zeros(nk, bool)
            for a, b in zip(lo, hi):
                seen[a:b] = True
            for j in np.flatnonzero(~seen):
                kk[y + j] = vv[y + j] = float("nan")
            y += nk
        o, l = run_prefill(layout(q, "padded"), layout(kk, "padded"), layout(vv, "head_major"), q_lens, k_lens, kind,
                           window=window, how="padded")
        assert qre.qre_read_device_status() == 0
        check(o, l, ref, kind, max(k_lens), float(v.abs().max()))


def test_prefill_large_scores_and_scale():
    """Scores of hundreds, growing along the keys, so the running maximum moves again and again."""
    n, D = 700, 128
    q, k, v = randn((n, 4, D), 1, "bf16", 4), randn((n, 2, D), 2, "bf16"), randn((n, 2, D), 3, "bf16")
    k = (k.float() * torch.linspace(0.1, 12, n, device=DEV)[:, None, None]).to(torch.bfloat16)
    ref = oatt.prefill(npy(q), npy(k), npy(v), [n], [n], 0.5)
    o, l = run_prefill(q, k, v, [n], [n], "bf16", scale=0.5)
    check(o, l, ref, "bf16", n, float(v.abs().max()))


def test_prefill_query_tiles_at_their_own_pace():
    """Several hundred short pieces of work whose later tokens see scores that grow sharply, so that of a piece's two
    query tiles one is held up again and again while the other could go on; some first tokens see nothing."""
    rng = np.random.default_rng(5)
    q_lens = [int(x) for x in rng.integers(20, 65, 300)]
    k_lens = [int(n + x) for n, x in zip(q_lens, rng.integers(-30, 200, 300))]
    k_lens = [max(x, 0) for x in k_lens]
    H, Hk, D = 8, 2, 64
    q, k, v = (randn((sum(n), h, D), 1 + i, "bf16") for i, (n, h) in enumerate(((q_lens, H), (k_lens, Hk), (k_lens, Hk))))
    grow = torch.cat([torch.linspace(0.05, 6, 300)[:n].flip(0) if i % 3 == 0 else torch.logspace(-1, 1, max(n, 1))[:n]
                      for i, n in enumerate(k_lens)]).to(DEV)
    k = (k.float() * grow[:, None, None]).to(torch.bfloat16)
    ref = oatt.prefill(npy(q), npy(k), npy(v), q_lens, k_lens, 0.5)
    o, l = run_prefill(q, k, v, q_lens, k_lens, "bf16", scale=0.5)
    assert qre.qre_read_device_status() == 0
    check(o, l, ref, "bf16", max(k_lens), float(v.abs().max()))


def test_prefill_equal_keys_average_the_values():
    n, D = 300, 64
    q, v = randn((n, 2, D), 1, "fp16"), randn((n, 1, D), 2, "fp16")
    k = randn((1, 1, D), 3, "fp16").expand(n, 1, D)          # one key for every position: token stride 0
    ref = oatt.prefill(npy(q), npy(k), npy(v), [n], [n], 0.125)
    o, l = run_prefill(q, k, v, [n], [n], "fp16", scale=0.125)
    check(o, l, ref, "fp16", n, float(v.abs().max()))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("D,window", [(64, 0), (128, 0), (128, 50)])
def test_prefill_what_is_not_seen_does_not_count(bad, D, window):
    """One token's key and value are not finite: only the queries that see it change."""
    lens, kind = [150, 40, 260], "bf16"
    n = sum(lens)
    q, k, v = (randn((n, h, D), i, kind) for i, h in ((1, 4), (2, 2), (3, 2)))
    ref = oatt.prefill(npy(q), npy(k), npy(v), lens, lens, 1.0 / math.sqrt(D), True, window)
    for where in (100, 150, 189, 190 + 77, n - 1):           # inside, first of a sequence, last of one
        kk, vv = k.clone(), v.clone()
        vv[where, 1, 5] = bad
        o, l = run_prefill(q, kk, vv, lens, lens, kind, window=window)
        ends = np.cumsum(lens)
        s = int(np.searchsorted(ends, where, side="right"))
        last = min(int(ends[s]), where + window if window else n)
        rows = np.ones(n, bool)
        rows[where:last] = False
        part = tuple(r[rows] for r in ref)
        check(o[torch.from_numpy(rows).to(DEV)], l[torch.from_numpy(rows).to(DEV)], part, kind, 260,
              float(v.abs().max()))
        # the queries that see it: that element is not finite, their other elements are as before
        hit = o[where:last, 2:, 5].float()
        assert (torch.isnan(hit) if math.isnan(bad) else ~torch.isfinite(hit)).all()
        rest = npy(o[where:last])
        keep = np.ones((1, 4, D), bool)
        keep[:, 2:, 5] = False
        tol = oatt.tolerance(ref[0], ref[2], ref[3], 260, D, UNIT[kind], 0)[where:last]
        assert (np.abs(rest - ref[0][where:last]) <= tol)[np.broadcast_to(keep, rest.shape)].all()
        kk[where, 0, 3] = bad                                # and the key: the whole rows that see it may change
        o, l = run_prefill(q, kk, vv, lens, lens, kind, window=window)
        check(o[torch.from_numpy(rows).to(DEV)], l[torch.from_numpy(rows).to(DEV)], part, kind, 260,
              float(v.abs().max()))


def test_prefill_rows_outside_the_sequences_are_left_alone():
    """Totals beyond the last sequence (padding of the arrays): neither read as keys nor written."""
    q_lens, k_lens, H, D = [40, 100], [40, 100], 2, 64
    q, k, v = (randn((200, h, D), i, "bf16") for i, h in ((1, H), (2, 1), (3, 1)))
    k[140:], v[140:] = float("nan"), float("nan")
    ref = oatt.prefill(npy(q[:140]), npy(k[:140]), npy(v[:140]), q_lens, k_lens, 0.125)
    o, l = run_prefill(q, k, v, q_lens, k_lens, "bf16", scale=0.125)
    check(o[:140], l[:140], ref, "bf16", 100, float(v[:140].abs().max()))
    assert torch.isnan(o[140:]).all() and torch.isnan(l[140:]).all()


def test_prefill_bad_bounds_are_skipped():
    q, k, v = (randn((100, 2, 64), i, "bf16") for i in (1, 2, 3))
    o = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    a = qre.make_attn(2, 2, 64, qre.QRE_BF16, 0.125, q=q, k=k, v=v, o=o)
    qre.qre_attn_prefill(a, 3, 100, 100, i32([0, 30, 60, 90]), i32([0, 30, 200, 90]), q, k, v, o)
    assert qre.qre_read_device_status() == qre.QRE_DEV_BAD_INDEX
    assert (o[30:] == 7).all() and not (o[:30] == 7).all()
    good = o[:30].clone()
    qre.qre_clear_device_status()
    o.fill_(7.0)
    qre.qre_attn_prefill(a, 3, 100, 100, i32([0, 30, 20, 400]), i32([0, 30, 60, 90]), q, k, v, o)
    assert qre.qre_read_device_status() == qre.QRE_DEV_BAD_INDEX
    assert torch.equal(o[:30], good) and (o[30:] == 7).all()


@pytest.mark.parametrize("H,D,scale_up", [(2, 64, 1), (16, 128, 8)])
def test_prefill_padding_and_bad_bounds_by_rows_and_by_tiles(H, D, scale_up):
    """The same calls at a size that goes by rows and at one that goes by tiles: totals beyond the last sequence, bounds
    that descend or leave the arrays, a bad sequence without tokens."""
    lens, T = [40 * scale_up, 100 * scale_up], 150 * scale_up
    n = sum(lens)
    q, k, v = (randn((T, h, D), i, "bf16") for i, h in ((1, H), (2, 1), (3, 1)))
    k[n:], v[n:] = float("nan"), float("nan")
    ref = oatt.prefill(npy(q[:n]), npy(k[:n]), npy(v[:n]), lens, lens, 0.125)
    o, l = run_prefill(q, k, v, lens, lens, "bf16", scale=0.125)
    assert qre.qre_read_device_status() == 0
    check(o[:n], l[:n], ref, "bf16", lens[1], float(v[:n].abs().max()))
    assert torch.isnan(o[n:]).all() and torch.isnan(l[n:]).all()
    for cq, ck in (([0, lens[0], n, n, n - 5], [0, lens[0], n, n, n]), ([0, lens[0], n, n, n], [0, lens[0], n, n, T + 1]),
                   ([0, lens[0], n, n, T + 1], [0, lens[0], n, n, n]), ([0, lens[0], n, n, n], [0, lens[0], n, n, -4])):
        o2 = torch.full_like(o, float("nan"))
        a = qre.make_attn(H, 1, D, qre.QRE_BF16, 0.125, q=q, k=k, v=v, o=o2)
        qre.qre_attn_prefill(a, 4, T, T, i32(cq), i32(ck), q, k, v, o2)
        assert qre.qre_read_device_status() == qre.QRE_DEV_BAD_INDEX
        qre.qre_clear_device_status()
        assert torch.equal(o2[:n], o[:n]) and torch.isnan(o2[n:]).all()


def test_prefill_many_sequences_and_repeatability():
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 12, 700).tolist() + [400, 0, 3]
    n = sum(lens)
    q, k, v = (randn((n, h, 64), i, "fp16") for i, h in ((1, 4), (2, 2), (3, 2)))
    ref = oatt.prefill(npy(q), npy(k), npy(v), lens, lens, 0.125)
    o, l = run_prefill(q, k, v, lens, lens, "fp16", scale=0.125)
    check(o, l, ref, "fp16", 400, float(v.abs().max()))
    for _ in range(3):
        o2, l2 = run_prefill(q, k, v, lens, lens, "fp16", scale=0.125)
        assert torch.equal(o, o2) and torch.equal(l, l2)
    o3, _ = run_prefill(q, k, v, lens, lens, "fp16", scale=0.125, lse=False)
    assert torch.equal(o, o3)


def test_prefill_offsets_beyond_32_bits():
    n, D, stride = 600, 64, 1 << 22                          # 2.5e9 elements between first and last token
    base = torch.empty(n * stride, dtype=torch.bfloat16, device=DEV)
    q, k, v = (randn((n, 1, D), i, "bf16") for i in (1, 2, 3))
    big = [torch.as_strided(base, (n, 1, D), (stride, D, 1), i * 4096) for i in range(4)]
    for b, x in zip(big, (q, k, v)):
        b.copy_(x)
    a = qre.make_attn(1, 1, D, qre.QRE_BF16, 0.125, q=big[0], k=big[1], v=big[2], o=big[3])
    qre.qre_attn_prefill(a, 1, n, n, i32([0, n]), i32([0, n]), big[0], big[1], big[2], big[3])
    o, _ = run_prefill(q, k, v, [n], [n], "bf16", scale=0.125)
    assert torch.equal(big[3], o)


def test_prefill_on_another_stream_and_in_a_graph():
    lens = [200, 70]
    q, k, v = (randn((270, h, 128), i, "bf16") for i, h in ((1, 8), (2, 2), (3, 2)))
    o, l = run_prefill(q, k, v, lens, lens, "bf16")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o2, l2 = run_prefill(q, k, v, lens, lens, "bf16", stream=side)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(l, l2)
    a = qre.make_attn(8, 2, 128, qre.QRE_BF16, 1 / math.sqrt(128), q=q, k=k, v=v, o=o2)
    cu = i32([0, 200, 270])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qre.qre_attn_prefill(a, 2, 270, 270, cu, cu, q, k, v, o2, l2)
    for _ in range(2):
        o2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, o2)


# ---------------------------------------------------------------- decode

class Paged:
    def __init__(self, lens, Hk, D, page, kind, seed=0, layers=2, spare=3, rows=None):
        rng = np.random.default_rng(seed)
        need = [-(-l // page) for l in lens]
        n_pages, cols = sum(need) + spare, max(need + [1]) + 1
        S = (rows or len(lens)) + 1
        self.seqs = rng.permutation(S)[:len(lens)]
        order, at = rng.permutation(n_pages), 0
        table = np.full((S, cols), -1, np.int32)
        ln = np.zeros(S, np.int32)
        for i, s in enumerate(self.seqs):
            table[s, :need[i]] = order[at:at + need[i]]
            at, ln[s] = at + need[i], lens[i]
        self.lens, self.page, self.kind, self.tab = lens, page, kind, table
        shape = (layers, n_pages, Hk, page, D)
        src = "bf16" if kind == "e4m3" else kind
        self.k, self.v = (randn(shape, seed + 5 + i, src, 8 if kind == "e4m3" else 1).to(DT[kind][1]) for i in (0, 1))
        self.scales = (torch.rand((2, layers, Hk), device=DEV, generator=torch.Generator(device=DEV).manual_seed(9)) * 0.1
                       + 0.08) if kind == "e4m3" else None
        self.table, self.len = torch.from_numpy(table).to(DEV), torch.from_numpy(ln).to(DEV)
        self.ref = torch.ones(n_pages, dtype=torch.int32, device=DEV)
        sc = (None, None) if self.scales is None else (self.scales[0].contiguous(), self.scales[1].contiguous())
        self.sc = sc
        self.c = qre.make_kv_cache(self.k, self.v, self.table, self.len, self.ref, DT[kind][0], *sc)

    def rows(self, i, layer):
        """K and V of sequence i: [len, Hk, D] in fp64."""
        L = self.lens[i]
        at = self.tab[self.seqs[i], :-(-L // self.page)].tolist()
        out = []
        for pool, sc in ((self.k, self.sc[0]), (self.v, self.sc[1])):
            x = pool[layer].float()[at] if at else torch.zeros((0,) + pool.shape[2:], device=DEV)
            x = npy(x).transpose(0, 2, 1, 3).reshape(-1, pool.shape[2], pool.shape[4])[:L]
            out.append(x if sc is None else x * npy(sc[layer])[None, :, None])
        return out


def run_decode(pg, q, kind, layer=1, window=0, max_len=0, how="packed", scale=None, seqs="list", stream=None):
    n, H, D = q.shape
    Hk = pg.k.shape[2]
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    o = layout(torch.full(q.shape, float("nan"), dtype=q.dtype, device=DEV), how)
    l = torch.full((n, H), float("nan"), dtype=torch.float32, device=DEV)
    a = qre.make_attn(H, Hk, D, DT[kind][0], scale, window=window, q=q, o=o)
    ws = torch.full((qre.qre_attn_decode_workspace_size(a, pg.c, n),), 0xA5, dtype=torch.uint8, device=DEV)
    qre.qre_attn_decode(a, pg.c, layer, n, i32(pg.seqs) if seqs == "list" else None, max_len, q, o, l, ws,
                        stream=stream)
    return o, l


def decode_ref(pg, q, layer=1, window=0, scale=None):
    n, H, D = q.shape
    Hk = pg.k.shape[2]
    qs = npy(q)
    out = [np.zeros((n, H, D)), np.full((n, H), -np.inf), np.zeros((n, H, D)), np.zeros((n, H))]
    for i in range(n):
        k, v = pg.rows(i, layer)
        L = pg.lens[i]
        lo = max(0, L - window) if window else 0
        for h in range(H):
            hk = h // (H // Hk)
            r = oatt.attend(qs[i, h:h + 1], k[:, hk], v[:, hk], 1.0 / math.sqrt(D) if scale is None else scale,
                            [lo], [L])
            for dst, x in zip(out, r):
                dst[i, h] = x[0]
    return out


DECODE = [
    # lens, H, Hk, D, page, q, cache, window
    ([1], 1, 1, 64, 16, "bf16", "bf16", 0),
    ([0, 1, 15, 16, 17, 127, 128, 129], 4, 2, 64, 16, "bf16", "bf16", 0),
    ([1000, 3, 0, 513], 8, 1, 128, 64, "fp16", "fp16", 0),
    ([777], 32, 8, 128, 16, "bf16", "bf16", 0),
    ([300, 5000], 16, 1, 128, 32, "bf16", "bf16", 0),
    ([700, 90], 14, 2, 64, 32, "fp16", "fp16", 0),               # 7 heads per KV head
    ([260, 1], 40, 2, 128, 256, "bf16", "bf16", 0),              # 20
    ([400, 33], 64, 1, 64, 16, "fp16", "fp16", 0),               # 64 heads on one
    ([2100, 64, 63], 6, 2, 128, 64, "bf16", "bf16", 100),        # window
    ([500, 20], 4, 4, 64, 16, "fp16", "fp16", 1),
    ([1, 300, 2047, 0], 8, 2, 128, 128, "bf16", "e4m3", 0),
    ([900, 31], 24, 8, 64, 16, "fp16", "e4m3", 70),
    ([5003], 8, 1, 128, 16, "fp16", "e4m3", 0),
    ([140] * 40, 2, 2, 64, 64, "bf16", "e4m3", 0),
    (list(range(0, 1300, 10)), 8, 2, 64, 16, "bf16", "bf16", 0),
]


@pytest.mark.parametrize("hint", ["none", "max"])
@pytest.mark.parametrize("case", range(len(DECODE)))
def test_decode(case, hint):
    lens, H, Hk, D, page, kind, cache, window = DECODE[case]
    pg = Paged(lens, Hk, D, page, cache, seed=case)
    q = randn((len(lens), H, D), 3, kind, 1.5)
    ref = decode_ref(pg, q, window=window)
    how = ["packed", "head_major", "padded"][case % 3]
    o, l = run_decode(pg, layout(q, how), kind, window=window, max_len=max(lens) if hint == "max" else 0, how=how)
    assert qre.qre_read_device_status() == 0
    check(o, l, ref, kind, max(lens), float(pg.v.float().abs().max()) * 0.2)


def test_decode_without_ids_and_repeatability():
    pg = Paged([200, 70, 900], 2, 64, 16, "bf16", rows=3)
    pg.seqs = np.argsort(pg.seqs) * 0 + np.arange(3)          # rows 0, 1, 2
    pg.lens = [int(x) for x in pg.len[:3].cpu()]
    q = randn((3, 4, 64), 1, "bf16")
    ref = decode_ref(pg, q)
    o, l = run_decode(pg, q, "bf16", seqs=None)
    check(o, l, ref, "bf16", 900, float(pg.v.float().abs().max()))
    for _ in range(3):
        o2, l2 = run_decode(pg, q, "bf16", seqs=None)
        assert torch.equal(o, o2) and torch.equal(l, l2)


def test_decode_result_does_not_depend_on_the_other_sequences():
    lens = [700, 31, 4000]
    pg = Paged(lens, 2, 128, 32, "bf16")
    q = randn((3, 8, 128), 1, "bf16")
    ref = decode_ref(pg, q)
    o, l = run_decode(pg, q, "bf16")
    check(o, l, ref, "bf16", 4000, float(pg.v.float().abs().max()))
    # garbage in every page that the sequences do not hold, and behind their ends
    for i, s in enumerate(pg.seqs):
        last, r = lens[i] // 32, lens[i] % 32
        if r:
            pg.k[:, pg.tab[s, last], :, r:] = float("nan")
            pg.v[:, pg.tab[s, last], :, r:] = float("inf")
    free = sorted(set(range(pg.k.shape[1])) - set(pg.tab[pg.tab >= 0].tolist()))
    pg.k[:, free], pg.v[:, free] = float("nan"), float("nan")
    o2, l2 = run_decode(pg, q, "bf16")
    assert torch.equal(o, o2) and torch.equal(l, l2)


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("kind,cache,D", [("bf16", "bf16", 128), ("fp16", "fp16", 64), ("bf16", "e4m3", 64)])
def test_decode_short_sequences_left_whole(kind, cache, D, window):
    """A bound of the lengths (or a window) under which units are not cut, true or not; and with more units than warps."""
    rng = np.random.default_rng(D + window)
    lens = [0, 1, 7, 64, 700] + [int(x) for x in rng.integers(1, 60, 395)]
    pg = Paged(lens, 8, D, 16, cache)
    q = randn((len(lens), 16, D), 4, kind)
    cut, lc = run_decode(pg, q, kind, window=window)
    whole, lw = run_decode(pg, q, kind, window=window, max_len=60)
    assert qre.qre_read_device_status() == 0
    ref = decode_ref(pg, q, window=window)
    check(cut, lc, ref, kind, 700, float(pg.v.float().abs().max()))
    check(whole, lw, ref, kind, 700, float(pg.v.float().abs().max()))


@pytest.mark.parametrize("cache,kind", [("bf16", "bf16"), ("e4m3", "fp16")])
def test_decode_window_hides_what_is_before_it(cache, kind):
    pg = Paged([1000], 1, 64, 16, cache)
    q = randn((1, 4, 64), 1, kind)
    o, l = run_decode(pg, q, kind, window=77)
    head = pg.tab[pg.seqs[0], :(1000 - 77) // 16].tolist()
    raw = (lambda t: t.view(torch.uint8)) if cache == "e4m3" else (lambda t: t)
    raw(pg.k)[:, head], raw(pg.v)[:, head] = (0x7f, 0x7f) if cache == "e4m3" else (float("nan"), float("inf"))
    edge = pg.tab[pg.seqs[0], (1000 - 77) // 16]
    raw(pg.v)[:, int(edge), :, :(1000 - 77) % 16] = 0x7f if cache == "e4m3" else float("nan")
    o2, l2 = run_decode(pg, q, kind, window=77)
    assert torch.equal(o, o2) and torch.equal(l, l2)


def test_decode_nan_in_a_seen_position_shows():
    pg = Paged([300, 300], 2, 64, 16, "e4m3")
    q = randn((2, 4, 64), 1, "bf16")
    o, _ = run_decode(pg, q, "bf16")
    p = int(pg.tab[pg.seqs[1], 4])
    pg.v.view(torch.uint8)[1, p, 1, 3, 7] = 0x7f              # NaN
    o2, _ = run_decode(pg, q, "bf16")
    bad = torch.isnan(o2)
    assert bad[1, 2:, 7].all() and int(bad.sum()) == 2
    assert torch.equal(o[~bad], o2[~bad])


def test_decode_large_scores():
    pg = Paged([3000], 1, 128, 64, "bf16")
    pg.k.copy_((pg.k.float() * 3).to(torch.bfloat16))
    q = randn((1, 8, 128), 1, "bf16", 8)
    ref = decode_ref(pg, q, scale=0.7)
    o, l = run_decode(pg, q, "bf16", scale=0.7)
    check(o, l, ref, "bf16", 3000, float(pg.v.float().abs().max()))


def test_decode_bad_ids_lengths_and_missing_pages():
    pg = Paged([40, 50, 60, 70], 1, 64, 16, "bf16")
    q = randn((4, 2, 64), 1, "bf16")
    want, wl = run_decode(pg, q, "bf16")
    keep = pg.seqs.copy()
    pg.seqs = np.array([-1, keep[1], 99, keep[3]])
    o, l = run_decode(pg, q, "bf16")
    assert qre.qre_read_device_status() == qre.QRE_DEV_BAD_INDEX
    assert (o[[0, 2]] == 0).all() and torch.isneginf(l[[0, 2]]).all()
    assert torch.equal(o[[1, 3]], want[[1, 3]])
    qre.qre_clear_device_status()
    pg.seqs = keep
    pg.len[int(keep[0])] = 1 << 20                            # more than the table holds
    o, l = run_decode(pg, q, "bf16")
    assert qre.qre_read_device_status() == qre.QRE_DEV_BAD_INDEX
    assert (o[0] == 0).all() and torch.equal(o[1:], want[1:])
    qre.qre_clear_device_status()
    pg.len[int(keep[0])] = 40
    pg.table[int(keep[2]), 1] = -1                            # positions 16 .. 31 of 60 missing
    o, l = run_decode(pg, q, "bf16")
    assert qre.qre_read_device_status() == qre.QRE_DEV_BAD_INDEX
    k, v = pg.rows(2, 1)
    seen = np.r_[0:16, 32:60]
    r = oatt.attend(npy(q)[2], k[seen, 0], v[seen, 0], 0.125, [0, 0], [44, 44])
    check(o[2], l[2], r, "bf16", 60, float(pg.v.float().abs().max()))
    assert torch.equal(o[[0, 1, 3]], want[[0, 1, 3]])


@pytest.mark.parametrize("H,Hk,D,kind,cache", [(32, 8, 128, "bf16", "bf16"), (40, 2, 64, "fp16", "fp16"), (6, 2, 128, "fp16", "e4m3")])
@pytest.mark.parametrize("bound", [40, 150, 400, 900, 2000])
def test_decode_shared_by_a_cluster(H, Hk, D, kind, cache, bound):
    """Few units under a bound: 4 to 32 warps share each.  Lengths of 0 and 1, the bound itself and (a wrong bound) far
    more, a page that is missing, a bad id, another stream."""
    lens = [bound, 0, 1, bound // 2, 3 * bound, 97]
    pg = Paged(lens, Hk, D, 16, cache)
    q = randn((len(lens), H, D), 7, kind)
    v_max = float(pg.v.float().abs().max())
    ref = decode_ref(pg, q)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    o, l = run_decode(pg, q, kind, max_len=bound, stream=stream)
    stream.synchronize()
    assert qre.qre_read_device_status() == 0
    check(o, l, ref, kind, 3 * bound, v_max)
    again, _ = run_decode(pg, q, kind, max_len=bound)
    assert torch.equal(o, again)
    one, l1 = run_decode(pg, q, kind, max_len=bound, window=1)      # the last position's values themselves
    check(one, l1, decode_ref(pg, q, window=1), kind, 1, v_max)

    pg.table[int(pg.seqs[5]), 2] = -1                               # positions 32 .. 47 of 97 missing
    pg.seqs[0] = 10 ** 6
    o, l = run_decode(pg, q, kind, max_len=bound)
    assert qre.qre_read_device_status() == qre.QRE_DEV_BAD_INDEX
    assert (o[0] == 0).all() and torch.isneginf(l[0]).all()
    assert torch.equal(o[1:5], again[1:5])
    k, v = pg.rows(5, 1)
    seen = np.r_[0:32, 48:97]
    for h in range(H):
        r = oatt.attend(npy(q)[5, h:h + 1], k[seen, h // (H // Hk)], v[seen, h // (H // Hk)], D ** -0.5, [0], [len(seen)])
        check(o[5, h:h + 1], l[5, h:h + 1], r, kind, 97, v_max)


def test_decode_pool_beyond_32_bits():
    heads, page, dim, n_pages = 8, 64, 128, 40000             # 2.6e9 elements
    k = torch.empty((1, n_pages, heads, page, dim), dtype=torch.bfloat16, device=DEV)
    rows = randn((2, heads, page, dim), 4, "bf16")
    k[0, -1], k[0, 5] = rows[0], rows[1]
    table, ln = i32([n_pages - 1, 5]).view(1, 2), i32([page + 20])
    c = qre.make_kv_cache(k, k, table, ln, torch.ones(n_pages, dtype=torch.int32, device=DEV), qre.QRE_BF16)
    q = randn((1, 16, dim), 1, "bf16")
    o = torch.empty_like(q)
    a = qre.make_attn(16, heads, dim, qre.QRE_BF16, 0.1, q=q, o=o)
    ws = torch.empty(qre.qre_attn_decode_workspace_size(a, c, 1), dtype=torch.uint8, device=DEV)
    qre.qre_attn_decode(a, c, 0, 1, None, 0, q, o, None, ws)
    x = npy(rows).transpose(1, 0, 2, 3).reshape(heads, 2 * page, dim)[:, :page + 20]
    ref = [oatt.attend(npy(q)[0, 2 * h:2 * h + 2], x[h], x[h], 0.1, [0, 0], [84, 84]) for h in range(heads)]
    ref = [np.concatenate([r[j] for r in ref]) for j in range(4)]
    check(o[0], None, ref, "bf16", 84, float(rows.abs().max()))


def test_decode_in_a_graph_follows_the_lengths():
    pg = Paged([500, 900], 2, 64, 16, "bf16")
    q = randn((2, 4, 64), 1, "bf16")
    a_o = torch.empty_like(q)
    a = qre.make_attn(4, 2, 64, qre.QRE_BF16, 0.125, q=q, o=a_o)
    ws = torch.empty(qre.qre_attn_decode_workspace_size(a, pg.c, 2), dtype=torch.uint8, device=DEV)
    ids = i32(pg.seqs)
    run_decode(pg, q, "bf16", scale=0.125)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qre.qre_attn_decode(a, pg.c, 1, 2, ids, 0, q, a_o, None, ws)
    for lens in ([500, 900], [17, 600], [0, 1]):
        pg.lens = lens
        for s, L in zip(pg.seqs, lens):
            pg.len[int(s)] = L
        graph.replay()
        torch.cuda.synchronize()
        check(a_o, None, decode_ref(pg, q, scale=0.125), "bf16", 900, float(pg.v.float().abs().max()))
