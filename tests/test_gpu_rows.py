"""Rows on their way into the paged cache and out of it: norms and rotation against fp64 within bounds derived from the
roundings (oracle.attention.turn_tolerance); 4-bit rows and what is read back bit for bit."""

import numpy as np
import pytest
import torch

import quantized_routed_expert_03_gb300 as qre
from oracle import attention as oatt
from quantized_routed_expert_03_gb300.attention import KVCache, Rotary

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn, "e2m1": torch.float4_e2m1fn_x2}
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
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(TYPE[kind])


def spread(x):
    """The same values with other strides; what lies between is NaN."""
    T, H, D = x.shape
    pad = torch.full((T, H + 3, D + 8), float("nan"), dtype=x.dtype, device=x.device)
    pad[:, 1:H + 1, :D] = x
    return pad[:, 1:H + 1, :D]


def within(got, y, size, angle, kind, D):
    tol = oatt.turn_tolerance(y, size, angle, UNIT[kind], D)
    assert np.isfinite(got).all() and (np.abs(got - y) <= tol).all(), (np.abs(got - y) - tol).max()


ROPE = [
    # heads, kv_heads, D, rot_dim, interleaved, norm, kind, positions
    (1, 1, 64, 64, False, True, "bf16", [0]),
    (8, 2, 128, 128, False, True, "bf16", range(7)),
    (8, 2, 128, 128, True, True, "fp16", [3, 0, 131071, 5]),
    (6, 3, 64, 48, False, False, "fp16", [1000000, 2 ** 31 - 1, 17]),       # three lanes turn, one passes its elements on
    (28, 4, 64, 16, True, True, "bf16", [5, -1, 9, -7, 100]),               # padding
    (40, 8, 128, 96, False, True, "bf16", range(513)),
    (5, 5, 128, 0, False, True, "fp16", range(33)),                         # a norm alone
    (64, 1, 128, 32, True, False, "bf16", range(50)),
]


@pytest.mark.parametrize("how", ["packed", "spread", "inplace"])
@pytest.mark.parametrize("case", range(len(ROPE)))
def test_norm_and_rotation(case, how):
    H, Hk, D, rot, inter, norm, kind, pos = ROPE[case]
    pos = list(pos)
    q, k = (randn((len(pos), h, D), 3 + i, kind, 2.0) for i, h in enumerate((H, Hk)))
    w = torch.rand((2, D), device=DEV, generator=torch.Generator(device=DEV).manual_seed(9)) + 0.5
    rotary = Rotary(H, Hk, D, rot, interleaved=inter, q_norm=w[0].contiguous() if norm else None,
                    k_norm=w[1].contiguous() if norm else None, eps=1e-3, dtype=TYPE[kind], device=DEV)
    freq = [] if rotary.inv_freq is None else npy(rotary.inv_freq)
    ref = [oatt.turn(npy(x), pos, freq, inter, npy(w[i]) if norm else None, float(np.float32(1e-3))) for i, x in enumerate((q, k))]
    if how == "packed":
        qo, ko = (torch.full_like(x, 77.0) for x in (q, k))
    elif how == "spread":
        q, k = spread(q), spread(k)
        qo, ko = (spread(torch.full_like(x, 77.0)) for x in (q, k))
    else:
        qo, ko = q, k
    before = [x.clone() for x in (qo, ko)]
    rotary.apply(q, k, i32(pos), qo, ko)
    assert qre.qre_read_device_status() == 0
    live = np.array(pos) >= 0
    for out, was, (y, size, angle) in zip((qo, ko), before, ref):
        within(npy(out)[live], y[live], size[live], angle[live], kind, D)
        assert torch.equal(out[torch.from_numpy(~live).to(DEV)], was[torch.from_numpy(~live).to(DEV)])
    if how == "spread":
        base = qo._base if qo._base is not None else qo
        assert torch.isnan(base[:, 0]).all() and torch.isnan(base[:, H + 1:]).all() and torch.isnan(base[:, :, D:]).all()


def test_one_of_the_two_is_normed():
    q, k = randn((3, 2, 64), 1, "bf16"), randn((3, 2, 64), 2, "bf16")
    w = torch.full((64,), 1.5, device=DEV)
    for qn, kn in ((w, None), (None, w)):
        qo, ko = Rotary(2, 2, 64, 0, q_norm=qn, k_norm=kn, device=DEV).apply(q, k, i32([0, 1, 2]))
        for out, x, n in ((qo, q, qn), (ko, k, kn)):
            if n is None:
                assert torch.equal(out, x)
            else:
                within(npy(out), *oatt.turn(npy(x), [0, 1, 2], [], False, npy(w), 1e-6), "bf16", 64)


class Pool:
    """A cache of two layers with sequences of some lengths on pages in random order, and what its rows are worth."""

    def __init__(self, kind, lens, page=16, Hk=2, D=64, rows_kind="bf16", scaled=False, seed=0, extra=3, layers=2):
        rng = np.random.default_rng(seed)
        self.kind, self.page, self.D, self.Hk, self.lens = kind, page, D, Hk, list(lens)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + extra
        scale = (None, None)
        if scaled:
            scale = tuple((torch.rand((layers, Hk), generator=torch.Generator().manual_seed(seed + i)) + 0.3).to(DEV) for i in range(2))
        self.c = KVCache(layers, pages, Hk, page, D, len(lens) + 1, max(need) + 1, TYPE[kind], *scale, device=DEV)
        order, at = rng.permutation(pages), 0
        for s, n in enumerate(need):
            self.c.page_table[s, :n] = i32(order[at:at + n])
            at += n
        self.c.seq_len[:len(lens)] = i32(lens)
        self.c.ref_count[:] = i32(np.isin(np.arange(pages), order[:at]))
        self.c.k.view(torch.uint8).fill_(0x7f)                # what nobody wrote is NaN
        self.c.v.view(torch.uint8).fill_(0x7f)
        self.tokens = [(s, p) for s, n in enumerate(lens) for p in range(n)]

    def ids(self):
        return i32([s for s, _ in self.tokens]), i32([p for _, p in self.tokens])

    def raw(self, x, layer, s, pos):
        """The stored bytes of one row: 16- or 8-bit elements, or codes and scale bytes."""
        pool = (self.c.k if x == 0 else self.c.v)[layer, int(self.c.page_table[s, pos // self.page])]
        row = pos % self.page
        if self.kind != "e2m1":
            return pool[:, row]
        flat = pool.reshape(self.Hk, -1)
        n = self.page * self.D // 2
        return (flat[:, :n].view(self.Hk, self.page, -1)[:, row], flat[:, n:].view(self.Hk, self.page, -1)[:, row])

    def scale(self, x, layer):
        s = self.c.k_scale if x == 0 else self.c.v_scale
        return None if s is None else s[layer]


def stored(pool, x, layer, rows):
    """(codes and scales or bytes, values in fp32 with the head's factor) that rows [tokens, Hk, D] become."""
    f = pool.scale(x, layer)
    f = None if f is None else f.cpu().numpy()
    if pool.kind == "e2m1":
        code, s, worth = oatt.e2m1_blocks(rows, f)
        value = worth.astype(np.float32)
        raw = (code[..., 0::2] | code[..., 1::2] << 4, oatt.e4m3_bytes(s))
    elif pool.kind == "e4m3":
        y = rows if f is None else (rows * (np.float32(1) / f).astype(np.float64)[:, None]).astype(np.float32)
        value = oatt.e4m3_round(y).astype(np.float32)
        raw = None
    else:
        value, raw = rows.astype(np.float32), None
    return raw, value if f is None else value * f[:, None]


def rounded(value, kind):
    return torch.from_numpy(value.astype(np.float32)).to(TYPE[kind])


@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("kind,rows_kind,D,page,Hk", [("e2m1", "bf16", 64, 16, 2), ("e2m1", "fp16", 128, 64, 3), ("e2m1", "bf16", 128, 256, 1),
                                                      ("e4m3", "fp16", 64, 32, 2), ("e4m3", "bf16", 128, 16, 8), ("bf16", "bf16", 128, 16, 2),
                                                      ("fp16", "fp16", 64, 128, 5)])
def test_rows_written_and_read_back(kind, rows_kind, D, page, Hk, scaled):
    """Codes and scales bit for bit, and each value read back its product rounded once."""
    if scaled and kind not in ("e4m3", "e2m1"):
        pytest.skip("no scales")
    p = Pool(kind, [1, 40, 16, 0, 259, 17], page, Hk, D, scaled=scaled)
    T = len(p.tokens)
    k, v = randn((T, Hk, D), 5, rows_kind, 3.0), randn((T, Hk, D), 6, rows_kind, 0.02)
    v[3] = 0                                                  # a row of zeros
    k[5] = k[5].sign() * torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], device=DEV).to(k.dtype).repeat(D // 8)   # ties
    k[7] *= 1000.0                                            # beyond the largest scale
    seq, pos = p.ids()
    p.c.write(1, seq, pos, spread(k), v)
    assert qre.qre_read_device_status() == 0
    rng = np.random.default_rng(1)
    order = rng.permutation(6)
    cu = np.concatenate([[0], np.cumsum([p.lens[s] for s in order])])
    out = torch.full((2, T + 2, Hk, D), 55.0, dtype=TYPE[rows_kind], device=DEV)
    p.c.read(1, i32(order), i32(cu), T, k=out[0, :T], v=out[1, :T])
    assert qre.qre_read_device_status() == 0
    first = np.concatenate([[0], np.cumsum(p.lens)])
    back = np.concatenate([np.arange(first[s], first[s + 1]) for s in order]).astype(int)
    for x, rows in ((0, k), (1, v)):
        raw, value = stored(p, x, 1, npy(rows))
        assert torch.equal(out[x, :T].cpu(), rounded(value[back], rows_kind))
        assert (out[x, T:] == 55.0).all()
        if raw is not None:
            for t in range(0, T, 7):
                code, s = p.raw(x, 1, *p.tokens[t])
                assert np.array_equal(code.cpu().numpy(), raw[0][t]) and np.array_equal(s.cpu().numpy(), raw[1][t])
    assert (p.c.k[0].view(torch.uint8) == 0x7f).all() and (p.c.v[0].view(torch.uint8) == 0x7f).all()   # the other layer


def test_4_bit_rows_that_are_not_finite():
    """A NaN makes its 16 NaN and nothing else; an infinity saturates."""
    p = Pool("e2m1", [4])
    k, v = randn((4, 2, 64), 1, "bf16"), randn((4, 2, 64), 2, "bf16")
    k[1, 0, 20] = float("nan")
    k[2, 1, 5], k[2, 1, 40] = float("inf"), float("-inf")
    seq, pos = p.ids()
    p.c.write(0, seq, pos, k, v)
    ko, vo = p.c.read(0, None, i32([0, 4]), 4)
    assert torch.isnan(ko[1, 0, 16:32]).all() and int(torch.isnan(ko).sum()) == 16 and not torch.isnan(vo).any()
    assert float(ko[2, 1, 5]) == 6 * 448 and float(ko[2, 1, 40]) == -6 * 448
    code, s, worth = oatt.e2m1_blocks(npy(k))
    fin = ~np.isnan(worth)
    assert np.array_equal(npy(ko)[fin], rounded(worth, "bf16").double().numpy()[fin])


@pytest.mark.parametrize("kind", ["bf16", "e2m1"])
def test_reads_of_parts_and_of_what_is_not_there(kind):
    p = Pool(kind, [50, 20, 33], seed=4)
    T = len(p.tokens)
    k, v = randn((T, 2, 64), 1, "bf16"), randn((T, 2, 64), 2, "bf16")
    seq, pos = p.ids()
    p.c.write(0, seq, pos, k, v)
    value = rounded(stored(p, 0, 0, npy(k))[1], "bf16").to(DEV)
    # the ends of two sequences, one of them twice
    ko, _ = p.c.read(0, i32([2, 0, 2]), i32([0, 3, 13, 15]), 15, first=i32([30, 40, 0]))
    assert torch.equal(ko, torch.cat([value[100:103], value[40:50], value[70:72]]))
    assert qre.qre_read_device_status() == 0
    # beyond a sequence's end, a bad id, a negative first, a missing page: zeros
    p.c.page_table[1, 0] = -1
    for seqs, first, zero in (([1], [18], [2, 3]), ([9], [0], range(4)), ([-1], [0], range(4)), ([0], [-1], range(4)),
                              ([1], [14], [0, 1]), ([0], [2 ** 31 - 2], range(4))):
        ko, vo = p.c.read(0, i32(seqs), i32([0, 4]), 4, first=i32(first))
        zero = list(zero)
        rest = [i for i in range(4) if i not in zero]
        assert (ko[zero] == 0).all() and (vo[zero] == 0).all()
        assert all(torch.equal(ko[i], value[50 + first[0] + i]) for i in rest)
        assert qre.qre_read_device_status() == qre.QRE_DEV_BAD_INDEX
        qre.qre_clear_device_status()
    # bad bounds are skipped, rows of nobody stay
    out = torch.full((2, 10, 2, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    p.c.read(0, i32([0, 2]), i32([2, 5, 11]), 10, k=out[0], v=out[1])
    assert qre.qre_read_device_status() == qre.QRE_DEV_BAD_INDEX
    assert torch.equal(out[0, 2:5], value[:3]) and (out[0, :2] == 3.0).all() and (out[0, 5:] == 3.0).all()


@pytest.mark.parametrize("D,rot,inter,norm", [(64, 64, False, True), (128, 128, True, True), (64, 16, False, False), (64, 48, True, True),
                                              (128, 48, False, True), (128, 0, False, True)])
@pytest.mark.parametrize("kind,rows_kind", [("bf16", "bf16"), ("fp16", "fp16"), ("e4m3", "bf16"), ("e2m1", "bf16"), ("e2m1", "fp16")])
def test_rows_turned_on_their_way_into_the_pages(kind, rows_kind, D, rot, inter, norm):
    H, Hk = 6, 3
    low = kind in ("e4m3", "e2m1")
    p = Pool(kind, [1, 37, 70], 32, Hk, D, scaled=low, seed=2)
    T = len(p.tokens)
    q, k, v = (randn((T, h, D), 20 + i, rows_kind, 2.0) for i, h in enumerate((H, Hk, Hk)))
    w = torch.linspace(0.5, 1.5, D, device=DEV)
    rotary = Rotary(H, Hk, D, rot, interleaved=inter, q_norm=w if norm else None, k_norm=w if norm else None,
                    dtype=TYPE[rows_kind], device=DEV)
    seq, pos = p.ids()
    pos_n = pos.cpu().numpy()
    pad = pos.clone()
    pad[5] = -1                                              # padding in the middle
    qo = torch.full_like(q, 9.0)
    ko = torch.full_like(k, 9.0)
    p.c.write_rope(1, rotary, seq, pad, spread(q), spread(k), spread(v), qo, ko)
    assert qre.qre_read_device_status() == 0
    live = np.arange(T) != 5
    freq = [] if rotary.inv_freq is None else npy(rotary.inv_freq)
    yq, yk = (oatt.turn(npy(x), pos_n, freq, inter, npy(w) if norm else None, float(np.float32(1e-6))) for x in (q, k))
    within(npy(qo)[live], *(a[live] for a in yq), rows_kind, D)
    within(npy(ko)[live], *(a[live] for a in yk), rows_kind, D)
    assert (qo[5] == 9.0).all() and (ko[5] == 9.0).all()
    # the same bits as the arrays' call, and without k_out
    qa, ka = rotary.apply(q, k, pos)
    assert torch.equal(qa[torch.from_numpy(live).to(DEV)], qo[torch.from_numpy(live).to(DEV)])
    assert torch.equal(ka[torch.from_numpy(live).to(DEV)], ko[torch.from_numpy(live).to(DEV)])
    before = p.c.k.clone()
    q2, none = p.c.write_rope(1, rotary, seq, pad, q, k, v, keep=False)
    assert none is None and torch.equal(p.c.k.view(torch.uint8), before.view(torch.uint8))
    assert torch.equal(q2[:5], qo[:5]) and torch.equal(q2[6:], qo[6:])
    # what the pages hold
    cu = np.concatenate([[0], np.cumsum(p.lens)])
    kr, vr = (npy(x) for x in p.c.read(1, None, i32(cu), T, dtype=TYPE[rows_kind]))
    assert np.array_equal(vr[live], rounded(stored(p, 1, 1, npy(v))[1], rows_kind).double().numpy()[live])
    if not low:
        assert np.array_equal(kr[live], npy(ko)[live])
        return
    y, size, angle = (a[live] for a in yk)
    f = p.scale(0, 1).cpu().numpy().astype(np.float64)[:, None]
    near = oatt.turn_tolerance(y, size, angle, 0.0, D) / f   # of the fp32 row over the head's factor
    near += np.abs(y / f) * 2.0 ** -22
    if kind == "e4m3":                                       # a rounding by half a step of the rounded value
        step = np.maximum(np.abs(y / f) + near, 2.0 ** -6) * 2.0 ** -4
    else:                                                    # scale: amax / 6, off by half a step; then half a code step, or a saturated amax
        most = (np.abs(y / f) + near).reshape(y.shape[:-1] + (-1, 16)).max(-1)
        s = np.maximum(most / 6 * (1 + 2.0 ** -4), 2.0 ** -9)
        step = np.repeat(np.maximum(s, most - 6 * np.maximum(most / 6 * (1 - 2.0 ** -4) - 2.0 ** -10, 0)), 16, -1)
    back = np.abs(kr[live]) * UNIT[rows_kind] + 2.0 ** -25
    assert (np.abs(kr[live] - y) <= (near + step) * f + back).all()
    # nearly all of them are the very values that the fp64 row rounds to
    exact = rounded(stored(p, 0, 1, y)[1], rows_kind).double().numpy()
    assert (exact == kr[live]).mean() > 0.99


def test_tokens_without_a_page():
    p = Pool("e2m1", [20, 5])
    rotary = Rotary(2, 2, 64, device=DEV)
    q, k, v = (randn((4, 2, 64), i, "bf16") for i in range(3))
    before = p.c.k.clone()
    qo, ko = p.c.write_rope(0, rotary, i32([0, 7, -1, 1]), i32([64, 3, 3, 2 ** 30]), q, k, v)
    assert qre.qre_read_device_status() == qre.QRE_DEV_BAD_INDEX
    assert torch.equal(p.c.k, before)
    qa, ka = rotary.apply(q, k, i32([64, 3, 3, 2 ** 30]))
    assert torch.equal(qo, qa) and torch.equal(ko, ka)
    qre.qre_clear_device_status()
    p.c.write(0, i32([0, 7, -1, 1]), i32([64, 3, 3, 2 ** 30]), k, v)
    assert qre.qre_read_device_status() == qre.QRE_DEV_BAD_INDEX and torch.equal(p.c.k, before)


def test_large_calls_and_many_heads():
    """More tokens than CTAs run at once, the most KV heads that are allowed."""
    for Hk, T in ((256, 30), (1, 20000)):
        p = Pool("e2m1", [T], 256, Hk, 64, layers=1)
        k, v = randn((T, Hk, 64), 1, "fp16"), randn((T, Hk, 64), 2, "fp16")
        rotary = Rotary(Hk, Hk, 64, 0, dtype=torch.float16, device=DEV)
        seq, pos = p.ids()
        qo, ko = p.c.write_rope(0, rotary, seq, pos, k, k, v)
        assert torch.equal(qo, k) and torch.equal(ko, k)
        got = p.c.read(0, None, i32([0, T]), T, dtype=torch.float16)
        p.c.k.zero_(), p.c.v.zero_()
        p.c.write(0, seq, pos, k, v)
        again = p.c.read(0, None, i32([0, T]), T, dtype=torch.float16)
        for a, b, x in zip(got, again, (k, v)):
            assert torch.equal(a, b)
            some = slice(0, T, max(1, T // 50))
            assert torch.equal(a[some].cpu(), rounded(oatt.e2m1_blocks(npy(x[some]))[2], "fp16"))
        assert qre.qre_read_device_status() == 0


def test_4_bit_pages_are_forked_and_compacted():
    p = Pool("e2m1", [37, 5], seed=3, extra=6)
    T = len(p.tokens)
    k, v = randn((T, 2, 64), 1, "bf16"), randn((T, 2, 64), 2, "bf16")
    seq, pos = p.ids()
    for layer in range(2):
        p.c.write(layer, seq, pos, k, v)
    want = p.c.read(1, i32([0]), i32([0, 37]), 37)
    p.c.fork(i32([0]), i32([2]))
    for step in range(2):
        got = p.c.read(1, i32([2]), i32([0, 37]), 37)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        if not step:
            p.c.free(i32([0, 1]))
            live = int(p.c.compact()[0])
            assert live == 3
    assert qre.qre_read_device_status() == 0


def test_streams_and_graphs():
    """Captured and replayed with other inputs in the same buffers; on a stream of its own."""
    p = Pool("e2m1", [64, 64], seed=7)
    rotary = Rotary(4, 2, 64, q_norm=torch.ones(64, device=DEV), k_norm=torch.ones(64, device=DEV), device=DEV)
    q, k, v = (randn((2, h, 64), i, "bf16") for i, h in enumerate((4, 2, 2)))
    seq, pos, cu = i32([0, 1]), i32([3, 9]), i32([0, 64, 128])
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    kr, vr = (torch.empty((128, 2, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.c.write_rope(0, rotary, seq, pos, q, k, v, qo, ko)
        p.c.read(0, seq, cu, 128, k=kr, v=vr)
    for step in range(3):
        for i, x in enumerate((q, k, v)):
            x.copy_(randn(x.shape, 100 * step + i, "bf16"))
        pos.copy_(i32([step, 60 - step]))
        graph.replay()
        torch.cuda.synchronize()
        a, b = rotary.apply(q, k, pos)
        assert torch.equal(a, qo) and torch.equal(b, ko)
        want = rounded(oatt.e2m1_blocks(npy(v))[2], "bf16").to(DEV)
        assert torch.equal(vr[step], want[0]) and torch.equal(vr[64 + 60 - step], want[1])
    s = torch.cuda.Stream()
    with torch.cuda.stream(torch.cuda.default_stream()):
        s.wait_stream(torch.cuda.current_stream())
        out = p.c.read(0, seq, cu, 128, stream=s)
    s.synchronize()
    for a, b in ((out[0], kr), (out[1], vr)):                 # bits: rows that nobody wrote are NaN
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert qre.qre_read_device_status() == 0
