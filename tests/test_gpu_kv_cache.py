"""The paged cache's pages (reserve, fork, free, compact) and writes against the fp64 / one-request-at-a-time oracle."""

import numpy as np
import pytest
import torch

import quantized_routed_expert_03_gb300 as qre
from oracle import attention as oatt

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": (qre.QRE_BF16, torch.bfloat16), "fp16": (qre.QRE_FP16, torch.float16),
      "e4m3": (qre.QRE_E4M3, torch.float8_e4m3fn)}


@pytest.fixture(autouse=True)
def clean_status():
    qre.qre_clear_device_status()
    yield
    qre.qre_clear_device_status()


class Cache:
    """A device cache whose page p holds the number p everywhere, beside the oracle's Pages."""

    def __init__(self, n_pages, page, max_seqs, max_pages, layers=2, heads=2, dim=64, kind="bf16"):
        self.model = oatt.Pages(n_pages, page, max_seqs, max_pages)
        shape = (layers, n_pages, heads, page, dim)
        base = torch.arange(n_pages, device=DEV, dtype=torch.int32).view(1, -1, 1, 1, 1)
        self.k = ((base + torch.arange(layers, device=DEV, dtype=torch.int32).view(-1, 1, 1, 1, 1) * 7)
                  .expand(shape).to(torch.int16).view(torch.bfloat16).contiguous())
        self.v = (base + 3).expand(shape).to(torch.int16).view(torch.bfloat16).contiguous()
        self.layers = layers
        self.table = torch.full((max_seqs, max_pages), -1, dtype=torch.int32, device=DEV)
        self.len = torch.zeros(max_seqs, dtype=torch.int32, device=DEV)
        self.ref = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
        self.c = qre.make_kv_cache(self.k, self.v, self.table, self.len, self.ref, qre.QRE_BF16)
        self.ws = torch.full((qre.qre_kv_workspace_size(self.c),), 0xA5, dtype=torch.uint8, device=DEV)

    def reserve(self, seqs, new):
        qre.qre_kv_reserve(self.c, len(seqs), i32(seqs), i32(new), self.ws)
        return self.model.reserve(seqs, new)

    def fork(self, src, dst):
        qre.qre_kv_fork(self.c, len(src), i32(src), i32(dst), self.ws)
        return self.model.fork(src, dst)

    def free(self, seqs):
        qre.qre_kv_free(self.c, len(seqs), i32(seqs))
        self.model.free(seqs)

    def compact(self):
        live = torch.full((4,), -1, dtype=torch.int32, device=DEV)
        qre.qre_kv_compact(self.c, self.table, self.ref, live, self.ws)
        assert int(live[0]) == self.model.compact()

    def check(self):
        m = self.model
        np.testing.assert_array_equal(self.len.cpu().numpy(), m.length)
        np.testing.assert_array_equal(self.table.cpu().numpy(), m.table)
        np.testing.assert_array_equal(self.ref.cpu().numpy(), m.ref)
        used = np.flatnonzero(m.ref > 0)
        k, v = (t.view(torch.int16).cpu().numpy().astype(np.int64) for t in (self.k, self.v))
        for l in range(self.layers):
            assert (k[l, used] == (m.content[used] + 7 * l)[:, None, None, None]).all()
            assert (v[l, used] == (m.content[used] + 3)[:, None, None, None]).all()


def i32(a):
    return torch.tensor(list(a), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("n_pages,page,max_pages", [(37, 16, 6), (5000, 32, 64), (9001, 256, 40)])
def test_random_life_of_a_cache(n_pages, page, max_pages):
    rng = np.random.default_rng(n_pages)
    S = 24
    c = Cache(n_pages, page, S, max_pages, heads=1)
    for step in range(40):
        m = c.model
        empty, full = np.flatnonzero(m.length == 0), np.flatnonzero(m.length > 0)
        what = rng.integers(5)
        if what <= 1:
            seqs = rng.permutation(S)[:rng.integers(1, S + 1)]
            c.reserve(seqs, rng.integers(0, page * max_pages // 3 + 1, len(seqs)))
        elif what == 2 and len(full) and len(empty):
            n = rng.integers(1, len(empty) + 1)
            c.fork(rng.choice(full, n), rng.permutation(empty)[:n])
        elif what == 3 and len(full):
            c.free(rng.permutation(full)[:rng.integers(1, len(full) + 1)])
        else:
            c.compact()
        c.check()
    assert qre.qre_read_device_status() & ~qre.QRE_DEV_NO_PAGE == 0


def test_requests_that_do_not_fit():
    c = Cache(10, 16, 6, 8)
    assert c.reserve([0, 1], [16 * 4, 16 * 3]) == []
    assert c.reserve([2, 3, 4, 0], [16 * 4, 16, 0, 0]) == [0, 1]        # 3 pages left: not served, nor what follows it
    c.check()
    assert qre.qre_read_device_status() == qre.QRE_DEV_NO_PAGE
    qre.qre_clear_device_status()
    assert c.reserve([1], [16 * 6]) == [0]                              # beyond max_pages
    assert qre.qre_read_device_status() == qre.QRE_DEV_NO_PAGE
    c.check()
    assert c.reserve([2, 3], [16 * 2 + 1, 0]) == []
    assert c.fork([2], [5]) == [0]                                      # no page for the copy
    c.check()


def test_positions_inside_a_page_take_no_page():
    c = Cache(4, 16, 2, 4)
    for n in (1, 1, 14, 1, 15, 1):
        c.reserve([1], [n])
        c.check()


def test_bad_ids_are_dropped():
    c = Cache(8, 16, 3, 4)
    c.reserve([0], [20])
    for call in (lambda: qre.qre_kv_reserve(c.c, 3, i32([-1, 3, 1]), i32([5, 5, -2]), c.ws),
                 lambda: qre.qre_kv_fork(c.c, 4, i32([0, 9, 0, 0]), i32([0, 1, -7, 3]), c.ws),
                 lambda: qre.qre_kv_free(c.c, 2, i32([-1, 3]))):
        call()
        assert qre.qre_read_device_status() == qre.QRE_DEV_BAD_INDEX
        qre.qre_clear_device_status()
        c.check()
    qre.qre_kv_free(c.c, 2, i32([0, 0]))                                # twice in one call: given back once
    c.model.free([0])
    c.check()
    assert qre.qre_read_device_status() == 0


def test_empty_calls_and_empty_sequences():
    c = Cache(8, 16, 3, 4)
    c.free([0, 1])
    c.fork([0], [1])
    c.compact()
    c.check()
    qre.qre_kv_reserve(c.c, 0, None, None, None, 0)
    qre.qre_kv_fork(c.c, 0, None, None, None, 0)
    qre.qre_kv_free(c.c, 0, None)


def test_compact_into_other_arrays_leaves_the_cache():
    c = Cache(300, 16, 10, 30)
    c.reserve(range(10), [16 * 25 + i for i in range(10)])
    c.free([0, 3, 4, 8])
    before = (c.table.clone(), c.ref.clone())
    table, ref, live = torch.zeros_like(c.table), torch.full_like(c.ref, -9), i32([0, 0, 0, 0])
    qre.qre_kv_compact(c.c, table, ref, live, c.ws)
    assert torch.equal(before[0], c.table) and torch.equal(before[1], c.ref)
    assert int(live[0]) == c.model.compact()
    c.table, c.ref = table, ref
    c.check()


@pytest.mark.parametrize("row,kind", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"), ("fp16", "e4m3")])
@pytest.mark.parametrize("dim,heads,page,fused", [(64, 3, 16, False), (128, 8, 64, True)])
def test_write(row, kind, dim, heads, page, fused):
    rng = np.random.default_rng(3)
    n, layers, n_pages, S, cols = 77, 2, 40, 5, 6
    g = torch.Generator(device=DEV).manual_seed(1)
    x = (torch.randn((n, 2 * heads + 2, dim), generator=g, device=DEV) * 30).to(DT[row][1])
    x[0, 0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 0.0]).to(DT[row][1])
    k, v = x[:, :heads], x[:, heads:2 * heads]
    if not fused:                                        # head-major
        k = k.transpose(0, 1).contiguous().transpose(0, 1)
    shape = (layers, n_pages, heads, page, dim)
    pool_k = torch.randn(shape, generator=g, device=DEV).to(DT[kind][1])
    pool_v = torch.randn(shape, generator=g, device=DEV).to(DT[kind][1])
    table = torch.from_numpy(rng.permutation(n_pages)[:S * cols].astype(np.int32).reshape(S, cols)).to(DEV)
    at = rng.permutation(S * cols * page)[:n]            # distinct places
    seq, pos = (at // (cols * page)).astype(np.int32), (at % (cols * page)).astype(np.int32)
    pos[5] = -1                                          # padding
    scales = torch.rand((2, layers, heads), generator=g, device=DEV) + 0.25 if kind == "e4m3" else (None, None)
    cache = qre.make_kv_cache(pool_k, pool_v, table, i32([0] * S), i32([1] * n_pages), DT[kind][0],
                              *(s if s is None else s.contiguous() for s in scales))
    want_k, want_v = (t.view(torch.uint8).clone() if kind == "e4m3" else t.clone() for t in (pool_k, pool_v))
    qre.qre_kv_write(cache, 1, qre.make_kv_rows(DT[row][0], k, v), n, torch.from_numpy(seq).to(DEV),
                     torch.from_numpy(pos).to(DEV), k, v)
    assert qre.qre_read_device_status() == 0
    page_of = table.cpu().numpy()[seq, np.maximum(pos, 0) // page]
    for want, got, new, sc in ((want_k, pool_k, k, scales[0]), (want_v, pool_v, v, scales[1])):
        for t in range(n):
            if pos[t] < 0:
                continue
            r = new[t]
            if kind == "e4m3":
                # the product with the reciprocal, in fp32, is what is rounded; rounding by the oracle
                vals = torch.from_numpy(oatt.e4m3_round((r.float() * (1.0 / sc[1])[:, None]).cpu().numpy())).float()
                r = vals.to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
            want[1, page_of[t], :, pos[t] % page] = r
        if kind == "e4m3":
            a, b = got.float(), want.view(torch.float8_e4m3fn).float()
        else:
            a, b = got.float(), want.float()
        assert torch.equal(torch.isnan(a), torch.isnan(b))
        assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


@pytest.mark.parametrize("heads,dim,n,kind", [(3, 64, 100003, "bf16"), (64, 128, 40000, "e4m3"), (256, 64, 2501, "bf16")])
def test_write_many_tokens(heads, dim, n, kind):
    """Several tokens for each CTA, up to the most that one takes; an odd number of tokens."""
    page, cols = 64, 500
    g = torch.Generator(device=DEV).manual_seed(2)
    n_pages = -(-n // page) + 7
    S = -(-n_pages // cols)
    k, v = (torch.randn((n, heads, dim), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    pool_k, pool_v = (torch.zeros((2, n_pages, heads, page, dim), dtype=torch.uint8 if kind == "e4m3" else torch.bfloat16,
                                  device=DEV).view(DT[kind][1]) for _ in range(2))
    table = torch.full((S, cols), -1, dtype=torch.int32, device=DEV)
    table.view(-1)[:n_pages] = torch.randperm(n_pages, generator=g, device=DEV).int()
    at = torch.randperm(n_pages * page, generator=g, device=DEV)[:n]
    seq, pos = (at // (cols * page)).int(), (at % (cols * page)).int()
    scales = torch.rand((2, 2, heads), generator=g, device=DEV) + 0.25 if kind == "e4m3" else (None, None)
    cache = qre.make_kv_cache(pool_k, pool_v, table, i32([0] * S), i32([1] * n_pages), DT[kind][0],
                              *(s if s is None else s.contiguous() for s in scales))
    qre.qre_kv_write(cache, 1, qre.make_kv_rows(qre.QRE_BF16, k, v), n, seq, pos, k, v)
    assert qre.qre_read_device_status() == 0
    bits = torch.uint8 if kind == "e4m3" else torch.int16
    where = table.view(-1)[at // page].long(), (at % page)
    for pool, new, sc in ((pool_k, k, scales[0]), (pool_v, v, scales[1])):
        r = new if kind == "bf16" else (new.float() * (1.0 / sc[1])[:, None]).to(torch.float8_e4m3fn)
        assert torch.equal(pool.view(bits)[1][where[0], :, where[1]], r.view(bits))
        pool.view(bits)[1][where[0], :, where[1]] = 0
        assert int(torch.count_nonzero(pool.view(bits))) == 0       # and nowhere else


def test_write_without_a_page():
    pool = torch.zeros((1, 4, 1, 16, 64), dtype=torch.bfloat16, device=DEV)
    table = i32([0, -1, 9, 1]).view(2, 2)
    c = qre.make_kv_cache(pool, pool.clone(), table, i32([0, 0]), i32([1] * 4), qre.QRE_BF16)
    rows = torch.ones((6, 1, 64), dtype=torch.bfloat16, device=DEV)
    qre.qre_kv_write(c, 0, qre.make_kv_rows(qre.QRE_BF16, rows, rows), 6, i32([0, 0, 1, 2, -1, 1]),
                     i32([3, 16, 3, 0, 0, 99]), rows, rows)
    assert qre.qre_read_device_status() == qre.QRE_DEV_BAD_INDEX
    want = torch.zeros_like(pool)
    want[0, 0, 0, 3] = 1
    assert torch.equal(pool, want)


def test_a_pool_whose_offsets_pass_32_bits():
    heads, page, dim, n_pages = 8, 64, 128, 40000          # 2.6e9 elements
    k = torch.empty((1, n_pages, heads, page, dim), dtype=torch.bfloat16, device=DEV)
    k[0, -3:] = 5.0
    k[0, :4] = 0.0
    table, ln, ref = i32([n_pages - 2, -1]).view(1, 2), i32([page]), torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    ref[n_pages - 2] = 1
    c = qre.make_kv_cache(k, k, table, ln, ref, qre.QRE_BF16)      # k and v the same memory: both copies write the same
    ws = torch.empty(qre.qre_kv_workspace_size(c), dtype=torch.uint8, device=DEV)
    rows = torch.full((1, heads, dim), 3.0, dtype=torch.bfloat16, device=DEV)
    qre.qre_kv_write(c, 0, qre.make_kv_rows(qre.QRE_BF16, rows, rows), 1, i32([0]), i32([7]), rows, rows)
    assert (k[0, n_pages - 2, :, 7] == 3).all() and (k[0, n_pages - 2, :, 8] == 5).all()
    live = i32([0, 0, 0, 0])
    qre.qre_kv_compact(c, table, ref, live, ws)
    assert int(live[0]) == 1 and table.tolist() == [[0, -1]] and int(ref[0]) == 1 and int(ref.sum()) == 1
    assert (k[0, 0, :, 7] == 3).all() and (k[0, 0, :, 9] == 5).all() and (k[0, 1] == 0).all()
    assert qre.qre_read_device_status() == 0
