"""Decode attention of sequences that share the pages of a prefix, against fp64 on what the pages are worth and within
oracle.attention.tolerance; and the common lengths that it goes by."""

import math

import numpy as np
import pytest
import torch

import quantized_routed_expert_03_gb300 as qre
from oracle import attention as oatt
from quantized_routed_expert_03_gb300.attention import Attention, KVCache
from test_gpu_rows import DEV, TYPE, UNIT, clean_status, i32, npy, randn   # noqa: F401

pytestmark = pytest.mark.gpu


class Shared:
    """Groups of sequences made by forks: group i has prompts[i] positions, sequence j of it owns[i][j] more.  Layer 1 of
    a two-layer cache; what nobody wrote is NaN."""

    def __init__(self, prompts, owns, H, Hk, D, page, kind, cache, scaled=False, seed=0, order=None, grow=0.0):
        self.H, self.Hk, self.D, self.kind = H, Hk, D, kind
        n = sum(len(o) for o in owns)
        lens = [p + x for p, o in zip(prompts, owns) for x in o]
        pages = sum(-(-p // page) for p in prompts) + sum(-(-(p % page + x) // page) + 1 for p, o in zip(prompts, owns) for x in o) + 4
        scale = (None, None)
        if scaled:
            scale = tuple((torch.rand((2, Hk), generator=torch.Generator().manual_seed(seed + i)) * 0.5 + 0.3).to(DEV) for i in range(2))
        self.c = KVCache(2, pages, Hk, page, D, n + len(prompts), -(-max(lens + [1]) // page) + 1, TYPE[cache], *scale, device=DEV)
        self.c.k.view(torch.uint8).fill_(0x7f if cache != "fp16" else 0xff)
        self.c.v.view(torch.uint8).fill_(0x7f if cache != "fp16" else 0xff)
        self.seqs, self.groups, at = [], [], 0
        for i, (p, o) in enumerate(zip(prompts, owns)):
            parent = n + i
            self._grow(parent, 0, p, seed + 17 * i, grow)
            mine = list(range(at, at + len(o)))
            at += len(o)
            if mine:
                self.c.fork(i32([parent] * len(mine)), i32(mine))
                for j, (s, x) in enumerate(zip(mine, o)):
                    self._grow(s, p, x, seed + 1000 + 31 * s, grow)
            self.c.free(i32([parent]))
            self.groups.append(mine)
        assert qre.qre_read_device_status() == 0
        self.lens = lens
        order = range(len(self.groups)) if order is None else order
        self.seqs = [s for i in order for s in self.groups[i]]
        self.cu = np.concatenate([[0], np.cumsum([len(self.groups[i]) for i in order])])

    def _grow(self, s, at, n, seed, grow):
        if not n:
            return
        self.c.reserve(i32([s]), i32([n]))
        k, v = randn((n, self.Hk, self.D), seed, self.kind, 1.5), randn((n, self.Hk, self.D), seed + 1, self.kind)
        if grow:                                             # keys that score more and more: references move
            k = (k.float() * (1 + grow * torch.arange(at, at + n, device=DEV)[:, None, None])).to(k.dtype)
        self.c.write(1, torch.full((n,), s, dtype=torch.int32, device=DEV), torch.arange(at, at + n, dtype=torch.int32, device=DEV), k, v)

    def common(self):
        return self.c.common_len(i32(self.seqs), i32(self.cu))

    def worth(self, s):
        """Keys and values of sequence s in fp64 [len, Hk, D], as the pages hold them."""
        L, page, kind = self.lens[s], self.c.page_table.shape, self.c.k.dtype
        S = self.c.k.shape[3] if kind != torch.uint8 else self.c.k.shape[3]
        out = []
        table = self.c.page_table[s, :-(-L // S)].long()
        for pool, scale in ((self.c.k, self.c.k_scale), (self.c.v, self.c.v_scale)):
            raw = pool[1].view(torch.uint8)[table] if kind == torch.float8_e4m3fn else pool[1][table]
            if kind == torch.float8_e4m3fn:
                raw = raw.view(torch.float8_e4m3fn)
            if kind == torch.uint8:
                flat = raw.flatten(-2)                        # pages, heads, bytes
                code, sb = flat[..., :S * self.D // 2].cpu().numpy(), flat[..., S * self.D // 2:].contiguous()
                nib = np.stack([code & 15, code >> 4], -1).reshape(len(table), self.Hk, S, self.D)
                sc = sb.view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64).reshape(len(table), self.Hk, S, self.D // 16)
                x = np.where(nib & 8, -1.0, 1.0) * oatt.E2M1[nib & 7] * np.repeat(sc, 16, -1)
            else:
                x = npy(raw)
            x = np.moveaxis(x, 1, 2).reshape(-1, self.Hk, self.D)[:L]
            out.append(x if scale is None else x * npy(scale)[1][:, None])
        return out

    def reference(self, q, window=0, only=None):
        """fp64 on the device: o, lse, absolute attention, largest absolute score sum; of queries `only` (None: all)."""
        n, g = len(self.seqs), self.H // self.Hk
        out = [np.zeros((n, self.H, self.D)), np.full((n, self.H), -np.inf), np.zeros((n, self.H, self.D)), np.zeros((n, self.H))]
        kept, v_max = {}, 0.0
        for i, s in enumerate(self.seqs):
            L = self.lens[s]
            if L == 0 or (only is not None and i not in only):
                continue
            lo = max(0, L - window) if window else 0
            k, v = (torch.from_numpy(x[lo:]).to(DEV) for x in self.worth(s))
            v_max = max(v_max, float(v.abs().max()))
            qq = q[i].double().view(self.Hk, g, self.D)
            sc = torch.einsum("hgd,jhd->hgj", qq, k) / math.sqrt(self.D)
            p = torch.softmax(sc, -1)
            out[0][i] = torch.einsum("hgj,jhd->hgd", p, v).reshape(self.H, self.D).cpu().numpy()
            out[1][i] = torch.logsumexp(sc, -1).reshape(self.H).cpu().numpy()
            out[2][i] = torch.einsum("hgj,jhd->hgd", p, v.abs()).reshape(self.H, self.D).cpu().numpy()
            out[3][i] = (torch.einsum("hgd,jhd->hgj", qq.abs(), k.abs()).amax(-1) / math.sqrt(self.D)).reshape(self.H).cpu().numpy()
        return out, v_max


def check(o, lse, ref, kind, n_keys, v_max, only=None):
    """Beside tolerance's steps: fp16 weights are lost below 2^-33 of the largest, and the parts are joined in fp32 (a few
    roundings of 2^-24 and of the exponential, which its own term of 2^-20 covers)."""
    sel = slice(None) if only is None else sorted(only)
    ro, rl, ra, rb = (x[sel] for x in ref)
    got, gl = npy(o)[sel], npy(lse)[sel]
    tol = oatt.tolerance(ro, ra, rb, n_keys, ro.shape[-1], UNIT[kind], v_max) + n_keys * 2.0 ** -33 * v_max
    assert np.isfinite(got).all() and (np.abs(got - ro) <= tol).all(), (np.abs(got - ro) - tol).max()
    fin = np.isfinite(rl)
    assert np.array_equal(np.isneginf(gl), ~fin)
    d = np.abs(np.where(fin, gl, 0) - np.where(fin, rl, 0))
    assert (d <= np.where(fin, oatt.lse_tolerance(np.where(fin, rl, 0), rb, n_keys, ro.shape[-1]), 0)).all()


def run(w, q, window=0, max_len=0, common=None, stream=None):
    att = Attention(w.c, 1, w.H, len(w.seqs), TYPE[w.kind], window=window, max_groups=len(w.cu) - 1)
    att.workspace.fill_(0xA5)
    lse = torch.full((len(w.seqs), w.H), float("nan"), device=DEV)
    o = torch.full_like(q, float("nan"))
    att.decode_shared(q, i32(w.seqs), i32(w.cu), w.common() if common is None else common, o=o, lse=lse, max_len=max_len, stream=stream)
    return o, lse


CASES = [
    # prompts, own positions of each sequence, H, Hk, D, page, kind, cache, window, scaled, order
    ([300], [[1, 5, 40]], 4, 2, 64, 16, "bf16", "bf16", 0, False, None),
    ([128], [[1, 1]], 1, 1, 128, 128, "fp16", "fp16", 0, False, None),
    ([1000], [[3, 1, 200, 17]], 8, 2, 128, 64, "bf16", "bf16", 0, False, None),              # one chain: 16 rows
    ([2000], [[7] * 40], 32, 8, 128, 64, "bf16", "bf16", 0, False, None),                    # 160 rows: two chains
    ([1555], [list(range(1, 61))], 8, 1, 64, 32, "fp16", "fp16", 0, False, None),            # 480 rows: two blocks
    ([900, 10, 0, 500, 2000], [[5, 5], [3, 4, 5], [9, 1], [30], [1] * 9], 10, 2, 64, 16, "bf16", "bf16", 0, False, [3, 1, 4, 0, 2]),
    ([700, 650], [[40, 3, 90], [1, 2]], 4, 2, 64, 256, "fp16", "fp16", 0, False, None),
    ([3000], [[300, 1, 700]], 8, 2, 128, 32, "bf16", "bf16", 1200, False, None),             # the window begins in the prefix
    ([3000], [[300, 1, 700]], 8, 2, 128, 32, "bf16", "bf16", 250, False, None),              # for some behind it
    ([1500, 1500], [[2] * 6, [800] * 3], 12, 4, 64, 16, "fp16", "fp16", 900, False, None),
    ([1000], [[3, 1, 200, 17]], 8, 2, 128, 64, "bf16", "e4m3", 0, True, None),
    ([1300, 400], [[1] * 30, [5, 6]], 24, 3, 64, 16, "fp16", "e4m3", 0, False, None),        # 240 rows
    ([2100], [[9] * 20], 8, 1, 128, 128, "bf16", "e4m3", 1500, True, None),
    ([1000], [[3, 1, 200, 17]], 8, 2, 128, 64, "bf16", "e2m1", 0, True, None),
    ([1300, 400], [[1] * 30, [5, 6]], 24, 3, 64, 16, "fp16", "e2m1", 0, False, None),
    ([2500], [[9] * 40], 8, 1, 128, 256, "bf16", "e2m1", 0, True, None),                     # 320 rows
    ([600] * 24, [[2, 3, 4]] * 24, 16, 8, 64, 16, "bf16", "bf16", 0, False, None),           # several units to a CTA
    ([250] * 70, [[1, 2]] * 70, 8, 8, 64, 16, "fp16", "e2m1", 0, False, None),
    ([1100, 300], [[30, 900, 2], [60, 1]], 40, 2, 128, 32, "bf16", "bf16", 0, False, None),   # 20 heads per KV head
    ([700], [[600, 3]], 24, 2, 64, 16, "fp16", "fp16", 300, False, None),                    # 12
    ([1100], [[30, 900, 2]], 48, 3, 128, 32, "bf16", "e4m3", 0, True, None),                  # 16
    ([1100], [[30, 900, 2]], 32, 2, 128, 32, "fp16", "e2m1", 0, True, None),                  # 16
    ([900], [[30, 2000, 2, 5]], 36, 2, 64, 16, "bf16", "e2m1", 1500, False, None),            # 18
    ([512], [[4000, 1]], 6, 2, 128, 64, "bf16", "e2m1", 0, True, None),                       # own positions cut over the ranges
    ([512], [[4000, 1, 0]], 4, 1, 64, 64, "fp16", "e4m3", 0, False, None),
]


# 0: not known; -1: as it is (so short that each sequence reads for itself); 10 ** 8: a hint by which sharing always pays
@pytest.mark.parametrize("max_len", [0, -1, 10 ** 8])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_shared_prefixes(case, max_len):
    prompts, owns, H, Hk, D, page, kind, cache, window, scaled, order = CASES[case]
    w = Shared(prompts, owns, H, Hk, D, page, kind, cache, scaled, seed=100 * case, order=order)
    q = randn((len(w.seqs), H, D), 5 + case, kind, 1.5)
    max_len = max(w.lens) if max_len == -1 else max_len
    o, lse = run(w, q, window, max_len)
    assert qre.qre_read_device_status() == 0
    ref, v_max = w.reference(q, window)
    check(o, lse, ref, kind, max(w.lens), v_max)
    for _ in range(3):                                       # results do not depend on timing
        o2, lse2 = run(w, q, window, max_len)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kind,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"), ("fp16", "e2m1")])
def test_keys_that_score_more_and_more(kind, cache):
    """References that move in many tiles, in both chains and across the ranges."""
    w = Shared([6000], [[10] * 3], 4, 1, 64, 64, kind, cache, seed=3, grow=3e-3 if cache != "e4m3" else 1e-3)
    q = randn((3, 4, 64), 8, kind, 2.0)
    o, lse = run(w, q)
    ref, v_max = w.reference(q)
    check(o, lse, ref, kind, 6010, v_max)


def test_long_prefix_and_many_queries():
    w = Shared([16384 + 100], [[1 + i % 50 for i in range(64)]], 32, 4, 128, 128, "bf16", "bf16", seed=9)
    q = randn((64, 32, 128), 8, "bf16")
    o, lse = run(w, q, max_len=17000)
    only = {0, 1, 31, 32, 63}
    ref, v_max = w.reference(q, only=only)
    check(o, lse, ref, "bf16", 16600, v_max, only)
    plain = Attention(w.c, 1, 32, 64).decode(q, i32(w.seqs), max_len=17000)
    d = (plain.float() - o.float()).abs()                    # two roundings of the result, and of its weights
    assert float((d / (plain.float().abs() + 0.02)).max()) < 2.0 ** -5


# one KV head's prefix lies in 76 ranges of CTAs, two parts of each: several warps of the join for a query head
@pytest.mark.parametrize("prompts,owns,H,Hk,D,kind,cache,window", [
    ([30000], [[1, 70, 9]], 3, 1, 64, "bf16", "bf16", 0),                  # 8 warps, some for two rounds
    ([29000], [[5, 400]], 2, 2, 128, "fp16", "fp16", 0),
    ([9000, 9100], [[1, 2, 900], [33, 4]], 5, 5, 128, "bf16", "e2m1", 0),    # 2 warps; heads that fill no CTA
    ([30000], [[3] * 50], 4, 1, 64, "bf16", "e4m3", 0),                    # 200 rows
    ([20000], [[3, 1000, 60]], 7, 1, 128, "fp16", "e2m1", 12000),
    ([20000], [[3, 5000, 60]], 6, 2, 64, "bf16", "bf16", 4000),              # one sequence sees no shared position
])
def test_long_prefixes_of_few_heads(prompts, owns, H, Hk, D, kind, cache, window):
    w = Shared(prompts, owns, H, Hk, D, 64, kind, cache, cache in ("e4m3", "e2m1"), 77)
    q = randn((len(w.seqs), H, D), 78, kind, 1.5)
    ref, v_max = w.reference(q, window)
    o, lse = run(w, q, window)
    check(o, lse, ref, kind, max(w.lens), v_max)
    o2, lse2 = run(w, q, window)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_common_lengths():
    w = Shared([300, 64, 0, 130, 500], [[1, 5, 40], [1, 1], [7, 8], [3], [1] * 70], 2, 1, 64, 16, "bf16", "bf16")
    assert w.common().tolist() == [288, 64, 0, 0, 496]
    assert w.common().dtype == torch.int32
    # any two sequences, the same one twice, across groups; at most the shortest length
    c = w.c
    f = lambda seqs, cu: c.common_len(i32(seqs), i32(cu)).tolist()        # noqa: E731
    assert f([0, 3, 1, 1], [0, 2, 4]) == [0, 305] and f([5, 5, 5], [0, 3]) == [7] and f([], [0, 0]) == [0]
    assert f([0, 1, 3, 4], [0, 2, 2, 4]) == [288, 0, 64]
    assert qre.qre_read_device_status() == 0
    for seqs, cu, want in (([0, 99], [0, 2], [0]), ([0, -1, 0, 1], [0, 2, 4], [0, 288]), ([0, 1], [0, 3], [0]), ([0, 1], [2, 0], [0]),
                           ([0, 1, 0, 1], [-1, 2, 4], [0, 288])):
        assert f(seqs, cu) == want
        assert qre.qre_read_device_status() == qre.QRE_DEV_BAD_INDEX
        qre.qre_clear_device_status()
    c.page_table[1, 3] = -1
    c.page_table[0, 3] = -1
    assert f([0, 1], [0, 2]) == [48]
    for cols in (255, 256, 257, 600):                        # tables of many columns
        big = KVCache(1, 700, 1, 16, 64, 9, 700, device=DEV)
        big.page_table[:, :cols] = torch.arange(cols, dtype=torch.int32, device=DEV)
        big.seq_len[:] = 16 * cols - 5
        assert big.common_len(i32(range(9)), i32([0, 9])).tolist() == [16 * cols - 5]
        big.page_table[8, cols - 1] += 1
        assert big.common_len(i32(range(9)), i32([0, 9])).tolist() == [16 * (cols - 1)]


def test_groups_and_lengths_that_are_not_so():
    """Whatever is claimed, no fault, a note, and the attention of each sequence by itself."""
    w = Shared([900, 600], [[5, 70], [3, 4]], 4, 2, 64, 16, "bf16", "bf16", seed=2)
    q = randn((4, 4, 64), 1, "bf16")
    ref, v_max = w.reference(q)
    good = w.common()
    assert good.tolist() == [896, 592]
    for cu, common in (([0, 2, 4], [-1, 592]), ([0, 2, 4], [896, 10 ** 6]), ([0, 2, 4], [2 ** 31 - 1, -2 ** 31]), ([0, 4, 2], [896, 592]),
                       ([1, 2, 4], [896, 592]), ([0, 2, 3], [896, 592]), ([0, 2, 5], [896, 592]), ([-4, 2, 4], [0, 592])):
        w.cu = np.array(cu)
        o, lse = run(w, q, common=i32(common))
        assert qre.qre_read_device_status() == qre.QRE_DEV_BAD_INDEX
        qre.qre_clear_device_status()
        check(o, lse, ref, "bf16", 970, v_max)
    w.cu = np.array([0, 2, 4])
    o, lse = run(w, q, common=i32([512, 0]))                 # less than there is: right as well
    assert qre.qre_read_device_status() == 0
    check(o, lse, ref, "bf16", 970, v_max)
    w.seqs[1] = 77                                           # a bad id: the empty result, the others as they are
    o, lse = run(w, q, common=good)
    assert qre.qre_read_device_status() == qre.QRE_DEV_BAD_INDEX
    assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()
    qre.qre_clear_device_status()
    check(o, lse, ref, "bf16", 970, v_max, {0, 2, 3})


def test_a_missing_page_in_the_prefix():
    w = Shared([900], [[5, 70, 1]], 4, 2, 64, 16, "bf16", "bf16", seed=2)
    common = w.common()
    w.c.page_table[:3, 20] = -1
    q = randn((3, 4, 64), 1, "bf16")
    o, lse = run(w, q, common=common)
    assert qre.qre_read_device_status() == qre.QRE_DEV_BAD_INDEX
    plain_lse = torch.empty_like(lse)
    plain = Attention(w.c, 1, 4, 3).decode(q, i32(w.seqs), lse=plain_lse)
    assert torch.isfinite(o).all()
    assert float((lse - plain_lse).abs().max()) < 1e-4 and float((o.float() - plain.float()).abs().max()) < 2.0 ** -6


def test_streams_strides_and_graphs():
    w = Shared([700], [[4, 9, 30, 2]], 8, 2, 64, 16, "bf16", "e2m1", seed=6)
    seqs, cu = i32(w.seqs), i32(w.cu)
    att = Attention(w.c, 1, 8, 4, max_groups=1)
    big = torch.full((4, 11, 72), float("nan"), dtype=torch.bfloat16, device=DEV)
    q, o = big[:, 1:9, :64], torch.full_like(big, 5.0)[:, 1:9, :64]
    q.copy_(randn((4, 8, 64), 1, "bf16"))
    common = w.common()
    lse = torch.empty((4, 8), device=DEV)
    att.decode_shared(q, seqs, cu, common, o=o, lse=lse)     # as it is
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.c.common_len(seqs, cu, out=common)
        att.decode_shared(q, seqs, cu, common, o=o, lse=lse)
    for step in range(3):                                    # replayed with other queries and longer sequences
        q.copy_(randn((4, 8, 64), 30 + step, "bf16"))
        for s in range(4):
            w._grow(s, w.lens[s], 7, 500 + 9 * step + s, 0.0)
            w.lens[s] += 7
        graph.replay()
        torch.cuda.synchronize()
        ref, v_max = w.reference(q)
        check(o, lse, ref, "bf16", max(w.lens), v_max)
    assert (o._base[:, 0] == 5.0).all() and (o._base[:, 9:] == 5.0).all()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = att.decode_shared(q, seqs, cu, common, stream=s)
    s.synchronize()
    assert torch.equal(again, o)
    assert qre.qre_read_device_status() == 0


def test_most_queries_of_a_call():
    """4096 queries in 2048 pairs: launches of the sequences' own positions in parts."""
    H, Hk, D, page, pairs = 2, 1, 64, 16, 2048
    c = KVCache(1, 9 * 4, Hk, page, D, 2 * pairs, 10, device=DEV)
    c.k.copy_(randn(c.k.shape, 1, "bf16"))
    c.v.copy_(randn(c.v.shape, 2, "bf16"))
    rows = torch.arange(2 * pairs, device=DEV)
    c.page_table[:, :8] = ((rows // 2 % 4) * 9)[:, None].int() + torch.arange(8, dtype=torch.int32, device=DEV)
    c.page_table[:, 8] = (rows % 4 * 9 + 8).int()
    c.seq_len[:] = (129 + rows % 16).int()
    att = Attention(c, 0, H, 2 * pairs, max_groups=pairs)
    q = randn((2 * pairs, H, D), 3, "bf16")
    cu = torch.arange(0, 2 * pairs + 1, 2, dtype=torch.int32, device=DEV)
    common = c.common_len(rows.int(), cu)
    assert (common == 128).all()
    l0, l1 = (torch.empty((2 * pairs, H), device=DEV) for _ in range(2))
    a = att.decode(q, None, lse=l0)
    b = att.decode_shared(q, None, cu, common, lse=l1)
    assert qre.qre_read_device_status() == 0
    assert float((l0 - l1).abs().max()) < 1e-4 and float((a.float() - b.float()).abs().max()) < 2.0 ** -6


def test_a_wait_that_gives_up():
    """With a limit of a microsecond waits of the pipeline run out: a status, and the next call is as it was."""
    w = Shared([5000], [[3, 7, 20]], 8, 2, 128, 64, "bf16", "e4m3", seed=4)
    q = randn((3, 8, 128), 1, "bf16")
    want = run(w, q)
    assert qre.qre_read_device_status() == 0
    try:
        qre.qre_debug_wait_test(1000, 0)
        run(w, q)
        assert qre.qre_read_device_status() & ~qre.QRE_DEV_TIMEOUT == 0
    finally:
        qre.qre_debug_wait_test(0, 0)
    qre.qre_clear_device_status()
    for _ in range(2):
        got = run(w, q)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert qre.qre_read_device_status() == 0


@pytest.mark.parametrize("cache,pages", [("e2m1", 40000), ("bf16", 16000), ("e4m3", 24000)])
def test_pools_beyond_32_bits(cache, pages):
    """Pages whose bytes lie 4 GB and more behind the pool's begin, in the second layer: turned rows written and read
    back, decode by itself and shared."""
    H, Hk, D, page, shared = 16, 8, 128, 256, 512
    lens = [shared + 3, shared + 90, shared + 256]
    c = KVCache(2, pages, Hk, page, D, 3, 4, TYPE[cache], device=DEV)       # (not initialised: NaN and what not)
    last = pages - 1
    c.page_table[:, :2] = i32([last, last - 7])
    c.page_table[:, 2] = i32([last - 1, last - 2, last - 3])
    c.seq_len[:] = i32(lens)
    seq = i32([0] * shared + [s for s, n in enumerate(lens) for _ in range(n - shared)])
    pos = i32(list(range(shared)) + [p for n in lens for p in range(shared, n)])
    T = seq.numel()
    q, k, v = (randn((T, h, D), i, "bf16") for i, h in enumerate((H, Hk, Hk)))
    from quantized_routed_expert_03_gb300.attention import Rotary
    _, ko = c.write_rope(1, Rotary(H, Hk, D, 0, q_norm=None, k_norm=None, device=DEV), seq, pos, q, k, v)
    assert torch.equal(ko, k)
    cu = np.concatenate([[0], np.cumsum(lens)])
    kr, vr = c.read(1, None, i32(cu), int(cu[-1]))
    own = {s: (torch.cat([k[:shared], k[seq == s][shared if s == 0 else 0:]]), torch.cat([v[:shared], v[seq == s][shared if s == 0 else 0:]])) for s in range(3)}
    for s in range(3):
        for got, rows in ((kr, own[s][0]), (vr, own[s][1])):
            want = npy(rows)
            if cache == "e2m1":
                want = oatt.e2m1_blocks(want)[2]
            elif cache == "e4m3":
                want = oatt.e4m3_round(want)
            assert np.array_equal(npy(got[cu[s]:cu[s + 1]]), want)
    qq = randn((3, H, D), 9, "bf16")
    att = Attention(c, 1, H, 3, max_groups=1)
    ref = [np.zeros((3, H, D)), np.zeros((3, H)), np.zeros((3, H, D)), np.zeros((3, H))]
    for s in range(3):
        kk, vv = npy(kr[cu[s]:cu[s + 1]]), npy(vr[cu[s]:cu[s + 1]])
        for h in range(H):
            for dst, x in zip(ref, oatt.attend(npy(qq)[s, h:h + 1], kk[:, h // 2], vv[:, h // 2], D ** -0.5, [0], [lens[s]])):
                dst[s, h] = x[0]
    lse = torch.empty((3, H), device=DEV)
    check(att.decode(qq, None, lse=lse), lse, ref, "bf16", max(lens), float(vr.float().abs().max()))
    groups = i32([0, 3])
    common = c.common_len(i32([0, 1, 2]), groups)
    assert common.tolist() == [shared]
    check(att.decode_shared(qq, None, groups, common, lse=lse), lse, ref, "bf16", max(lens), float(vr.float().abs().max()))
    assert qre.qre_read_device_status() == 0
