"""Prefill and decode attention where calls mix what is usually apart, or lie at the end of a range; against fp64."""

import math

import numpy as np
import pytest
import torch

import quantized_routed_expert_03_gb300 as qre
from oracle import attention as oatt
from quantized_routed_expert_03_gb300.attention import Attention, KVCache
from test_gpu_attention import (DEV, DT, UNIT, Paged, check, clean_status, decode_ref, i32, npy, randn,  # noqa: F401
                                run_decode, run_prefill)

pytestmark = pytest.mark.gpu


def prefill_ref(q, k, v, q_lens, k_lens, scale, window=0):
    """oracle.attention.prefill's four results (causal), a sequence and a KV head at a time in torch's fp64."""
    T, H, D = q.shape
    g = H // k.shape[1]
    f64 = dict(dtype=torch.float64, device=DEV)
    o, a = torch.zeros(q.shape, **f64), torch.zeros(q.shape, **f64)
    lse, big = torch.full((T, H), -math.inf, **f64), torch.zeros((T, H), **f64)
    x = y = 0
    for nq, nk in zip(q_lens, k_lens):
        lo, hi = (torch.tensor(b, device=DEV)[None, :, None] for b in oatt.visible(nq, nk, True, window))
        j = torch.arange(nk, device=DEV)[None, None]
        seen = (j >= lo) & (j < hi)                                             # [1, nq, nk]
        used = seen.any(1)[0]
        for hk in range(k.shape[1]):
            heads = slice(hk * g, hk * g + g)
            qq = q[x:x + nq, heads].double().transpose(0, 1)                      # [g, nq, D]
            kk, vv = (torch.where(used[:, None], t[y:y + nk, hk].double(), 0.0) for t in (k, v))
            s = torch.where(seen, qq @ kk.T * scale, -math.inf)
            l = torch.logsumexp(s, -1)
            p = torch.where(seen, torch.exp(s - torch.where(l.isinf(), 0.0, l)[..., None]), 0.0)
            lse[x:x + nq, heads] = l.T
            o[x:x + nq, heads], a[x:x + nq, heads] = (p @ vv).transpose(0, 1), (p @ vv.abs()).transpose(0, 1)
            b = torch.where(seen, qq.abs() @ kk.abs().T * scale, 0.0)
            big[x:x + nq, heads] = (b.amax(-1) if nk else torch.zeros((g, nq), **f64)).T
        x, y = x + nq, y + nk
    return tuple(t.cpu().numpy() for t in (o, lse, a, big))


def hide_unseen(k, v, q_lens, k_lens, window):
    """NaN in every key and value that no query sees."""
    k, v = k.clone(), v.clone()
    y = 0
    for nq, nk in zip(q_lens, k_lens):
        lo, hi = oatt.visible(nq, nk, True, window)
        seen = np.zeros(nk + 1, int)
        for a, b in zip(lo, hi):
            seen[a] += 1
            seen[b] -= 1
        gone = torch.from_numpy(y + np.flatnonzero(np.cumsum(seen)[:nk] == 0)).to(DEV)
        k[gone], v[gone] = float("nan"), float("nan")
        y += nk
    return k, v


@pytest.mark.parametrize("window", [0, 200])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("H,Hk", [(8, 8), (32, 8), (32, 4)])           # 128, 32 and 16 tokens to a query tile
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_few_new_tokens_on_long_contexts_beside_short_prompts(D, H, Hk, many, window):
    """Pieces of work without a second query tile and with many key tiles, in front of short prompts with two: the second
    tile's softmax is pieces ahead of the keys and values that are being fetched.  More pieces than SMs, and at most and more than 128 sequences
    (two orders of the work).  What is not seen is NaN."""
    rng = np.random.default_rng(D + H + Hk + many)
    tile = 128 // (H // Hk)
    n_long, n_short = (80, 60) if many else (44, 30)
    long = [(int(a), int(b)) for a, b in zip(rng.integers(1, tile + 1, n_long), rng.integers(300, 4001 if not many else 1200, n_long))]
    if tile == 128:   # two query tiles and a cut first key tile: more queries than keys
        short = [(int(a), int(b)) for a, b in zip(rng.integers(130, 250, n_short), rng.integers(20, 128, n_short))]
    else:
        short = [(int(a), int(a)) for a in rng.integers(tile + 1, 128, n_short)]
    lens = [(long + short)[i] for i in rng.permutation(n_long + n_short)]
    q_lens, k_lens = [a for a, _ in lens], [b for _, b in lens]
    kind = "bf16" if D == 128 else "fp16"
    q = randn((sum(q_lens), H, D), 1, kind, 1.5)
    k, v = (randn((sum(k_lens), Hk, D), 2 + i, kind) for i in range(2))
    ref = prefill_ref(q, k, v, q_lens, k_lens, D ** -0.5, window)
    v_max = float(v.abs().max())
    k, v = hide_unseen(k, v, q_lens, k_lens, window)
    o, l = run_prefill(q, k, v, q_lens, k_lens, kind, window=window)
    assert qre.qre_read_device_status() == 0
    check(o, l, ref, kind, max(k_lens), v_max)
    for _ in range(10):
        o2, l2 = run_prefill(q, k, v, q_lens, k_lens, kind, window=window)
        assert torch.equal(o, o2) and torch.equal(l, l2)


def test_the_fp64_reference_of_this_file():
    q_lens, k_lens = [5, 9, 3, 0], [30, 4, 3, 7]
    q, k, v = (randn((sum(n), h, 64), i, "bf16") for i, (n, h) in enumerate(((q_lens, 4), (k_lens, 2), (k_lens, 2))))
    for window in (0, 3):
        mine = prefill_ref(q, k, v, q_lens, k_lens, 0.125, window)
        for a, b in zip(mine, oatt.prefill(npy(q), npy(k), npy(v), q_lens, k_lens, 0.125, True, window)):
            assert np.array_equal(np.isneginf(a), np.isneginf(b))
            assert np.allclose(np.where(np.isneginf(a), 0, a), np.where(np.isneginf(b), 0, b), rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_infinities_that_one_query_tile_sees_whole_and_the_other_cut(D):
    """The value tile is one for both query tiles of a piece: what is taken out of it for the one that a window cuts has to
    reach the result of the one that sees all of it, whichever of the two is ahead."""
    n, seqs, H, Hk, window = 400, 60, 8, 2, 170             # 32 tokens to a query tile
    lens = [n] * seqs
    q, k, v = (randn((n * seqs, h, D), i, "bf16") for i, h in ((1, H), (2, Hk), (3, Hk)))
    scale = 0.02                                             # no weight is so small that it is rounded to zero
    want, _ = run_prefill(q, k, v, lens, lens, "bf16", window=window, scale=scale)
    bad = v.clone()
    at = torch.arange(seqs, device=DEV) * n + torch.arange(seqs, device=DEV) * 6 % n
    bad[at, 1, 3] = float("inf")
    token = torch.arange(n * seqs, device=DEV).view(seqs, n)
    sees = ((token >= at[:, None]) & (token < at[:, None] + window)).view(-1)
    for _ in range(10):
        o, _ = run_prefill(q, k, bad, lens, lens, "bf16", window=window, scale=scale)
        hit = o[:, 4:, 3]
        assert torch.isposinf(hit[sees]).all() and torch.isfinite(hit[~sees]).all()
        rest = torch.ones_like(o, dtype=torch.bool)
        rest[:, 4:, 3] = ~sees[:, None]
        assert torch.equal(o[rest], want[rest])


@pytest.mark.parametrize("n,gone", [(48, 40), (700, 300)])              # by rows, by tiles
def test_prefill_keys_that_score_minus_infinity_first(n, gone):
    """A row's first keys, more than one step of the kernel, score -infinity: they count nothing."""
    q, k, v = (randn((n, h, 64), i, "bf16") for i, h in ((1, 2), (2, 1), (3, 1)))
    q[:, :, 0] = q[:, :, 0].abs() + 0.1
    ref = [r.copy() for r in prefill_ref(q[gone:], k[gone:], v[gone:], [n - gone], [n - gone], 0.125)]
    k[:gone, :, 0] = -float("inf")
    o, l = run_prefill(q, k, v, [n], [n], "bf16", scale=0.125)
    check(o[gone:], l[gone:], ref, "bf16", n, float(v.abs().max()))


@pytest.mark.parametrize("lens,H,Hk,D,rows", [
    ([16], 8, 2, 64, True), ([8, 5, 30], 32, 8, 128, True), ([2] * 64, 32, 8, 128, True), ([2] * 128, 8, 2, 64, True),
    ([5] * 40, 8, 2, 64, True), ([128], 32, 8, 128, False), ([1] * 99 + [400], 8, 2, 64, False),
    ([1] * 60 + [300], 8, 2, 64, False), ([512] + [0] * 399, 32, 8, 128, False), ([0] * 255 + [300], 32, 8, 128, False)])
def test_prefill_which_way_a_handful_of_keys_goes(lens, H, Hk, D, rows):
    """By rows only where no sequence of an uneven or padded call can be long.  Rows keep their weights in fp32, tiles round
    them to bf16: of two keys with weights 1 and 0.999 and values 1 and -1 the one leaves 0.0005, the other nothing."""
    n = sum(lens)
    q, k, v = (torch.zeros((n, h, D), dtype=torch.bfloat16, device=DEV) for h in (H, Hk, Hk))
    q[:, :, 0], v[:] = 1.0, 1.0
    first = int(np.cumsum([0] + lens)[int(np.argmax(lens))])
    k[first + 1, :, 0], v[first + 1] = -0.001, -1.0
    o, l = run_prefill(q, k, v, lens, lens, "bf16", scale=1.0)
    check(o, l, prefill_ref(q, k, v, lens, lens, 1.0), "bf16", max(lens), 1.0)
    assert bool((o[first + 1] != 0).all()) == rows and bool((o[first + 1] == 0).all()) == (not rows)


def rising(n, heads, D, seed):
    """Queries and keys whose scores (base 2, for scale = ln 2) are some 0 for 130 keys and then rise by 50."""
    rise = torch.cat([torch.zeros(130, device=DEV), torch.linspace(20, 50, n - 130, device=DEV)])
    k = torch.randn((n, heads, D), generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV) * 0.1
    k[:, :, 0] = rise[:, None] / 8
    return k.to(torch.bfloat16)


def queries(n, heads, D, seed):
    q = torch.randn((n, heads, D), generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV) * 0.1
    q[:, :, 0] = 8.0
    return q.to(torch.bfloat16)


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_large_finite_values_under_scores_that_rise(D):
    """Values of 2^100, and weights that would be 2^50 against the row's first keys: the product has to stay finite."""
    n, scale = 600, math.log(2)
    q, k = queries(n, 4, D, 1), rising(n, 2, D, 2)
    v = (randn((n, 2, D), 3, "bf16").float() * 2.0 ** 100).to(torch.bfloat16)
    o, l = run_prefill(q, k, v, [n], [n], "bf16", scale=scale)
    check(o, l, prefill_ref(q, k, v, [n], [n], scale), "bf16", n, float(v.abs().max()))


def one_far_ahead(n, heads, D, kind, seed):
    """Keys and values: the key at 5 scores 26 (base 2, scale ln 2, queries of `ahead_queries`) and its value is zero, the
    others score 0 to 1 and together still decide the result."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    k = torch.zeros((n, heads, D), device=DEV)
    k[:, :, 0] = torch.randint(0, 5, (n, heads), generator=g, device=DEV) / 4
    k[5, :, 0] = 26.0
    v = torch.randn((n, heads, D), generator=g, device=DEV) * 4 + 64
    v[5] = 0.0
    return tuple(x.to(DT[kind][1]) for x in (k, v))


def ahead_queries(n, heads, D, kind):
    q = torch.zeros((n, heads, D), device=DEV)
    q[:, :, 0] = 1.0
    return q.to(DT[kind][1])


def check_small_weights(o, lse, ref, kind, n_keys, v_max, lost):
    """check(), but weights are rounded to fp16's steps (2^-24) `lost` powers of two lower than against the row's maximum."""
    ro, rl, ra, rb = ref
    D = ro.shape[-1]
    tol = oatt.tolerance(ro, ra, rb, n_keys, D, UNIT[kind], 0.0) + n_keys * 2.0 ** (-25 - lost) * v_max
    assert (np.abs(npy(o) - ro) <= tol).all(), (np.abs(npy(o) - ro) - tol).max()
    assert (np.abs(npy(lse) - rl) <= oatt.lse_tolerance(rl, rb, n_keys, D)).all()


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_fp16_many_small_weights_behind_one_key(D):
    """Each weight is below fp16's smallest against the row's maximum; 60,000 of them weigh 2^-10."""
    q_lens, k_lens, scale = [3, 40], [60000, 20000], math.log(2)
    k, v = (torch.cat(x) for x in zip(*(one_far_ahead(n, 1, D, "fp16", n) for n in k_lens)))
    q = ahead_queries(43, 2, D, "fp16")
    ref = prefill_ref(q, k, v, q_lens, k_lens, scale)
    o, l = run_prefill(q, k, v, q_lens, k_lens, "fp16", scale=scale)
    check_small_weights(o, l, ref, "fp16", 60000, float(v.abs().max()), 4)
    # the oracle's bound tells them apart: the keys behind the first weigh far more than it allows
    assert (np.abs(ref[0][:3]) > 4 * 60000 * 2.0 ** -29 * float(v.abs().max())).all()


# ---------------------------------------------------------------- decode

@pytest.mark.parametrize("seqs", ["list", None])
def test_decode_rows_of_a_billion_positions(seqs):
    """Table rows so long that a call's chunks are counted apart for some of its sequences; the sequences are short."""
    lens = [0, 1, 700, 33] + [int(x) for x in np.random.default_rng(1).integers(1, 300, 33)]
    pg = Paged(lens, 2, 128, 256, "bf16", rows=len(lens) - 1)
    if seqs is None:
        pg.seqs = np.arange(len(lens))
        pg.lens = [int(x) for x in pg.len.cpu()[:len(lens)]]
    wide = torch.full((pg.table.shape[0], 1 << 22), -1, dtype=torch.int32, device=DEV)
    wide[:, :pg.table.shape[1]] = pg.table
    pg.c = qre.make_kv_cache(pg.k, pg.v, wide, pg.len, pg.ref, qre.QRE_BF16)
    q = randn((len(lens), 8, 128), 3, "bf16")
    for hint, window in ((0, 0), (700, 0), (0, 50)):
        o, l = run_decode(pg, q, "bf16", max_len=hint, window=window, seqs=seqs, how="padded")
        assert qre.qre_read_device_status() == 0
        check(o, l, decode_ref(pg, q, window=window), "bf16", 700, float(pg.v.float().abs().max()))


def test_decode_more_chunks_than_32_bits_count():
    """33 sequences of 2^30 positions, every page of them the same one: 2^31 and more chunks of 16.  Keys are zero, so all
    weights are 1, and values of -1, 0 and 1 add up exactly."""
    n, cols, page, D = 33, 1 << 22, 256, 128
    k = torch.zeros((1, 1, 1, page, D), dtype=torch.bfloat16, device=DEV)
    v = (torch.arange(D, device=DEV) % 3 - 1).to(torch.bfloat16).expand(k.shape).contiguous()
    table, ln, ref = torch.zeros((n, cols), dtype=torch.int32, device=DEV), i32([cols * page] * n), i32([1])
    c = qre.make_kv_cache(k, v, table, ln, ref, qre.QRE_BF16)
    q = randn((n, 2, D), 1, "bf16")
    o, lse = torch.empty_like(q), torch.empty((n, 2), dtype=torch.float32, device=DEV)
    a = qre.make_attn(2, 1, D, qre.QRE_BF16, 0.1, q=q, o=o)
    ws = torch.empty(qre.qre_attn_decode_workspace_size(a, c, n), dtype=torch.uint8, device=DEV)
    qre.qre_attn_decode(a, c, 0, n, None, 0, q, o, lse, ws)
    assert qre.qre_read_device_status() == 0
    assert torch.equal(o, v[0, 0, 0, :1].expand(o.shape))
    assert (lse - 30 * math.log(2)).abs().max() < 2.0 ** -17


@pytest.mark.parametrize("hint", [0, 1, 900])                     # cut; one warp goes through a whole sequence; a cluster shares it
@pytest.mark.parametrize("D", [64, 128])
def test_decode_large_finite_values_under_scores_that_rise(D, hint):
    pg = Paged([900, 500, 3000], 2, D, 16, "bf16")
    pg.v.copy_((pg.v.float() * 2.0 ** 100).to(torch.bfloat16))
    for i, n in enumerate(pg.lens):
        k = rising(n, 2, D, i)
        for p in range(-(-n // 16)):
            rows = k[16 * p:16 * p + 16].transpose(0, 1)
            pg.k[1, pg.tab[pg.seqs[i], p], :, :rows.shape[1]] = rows
    q = queries(3, 8, D, 9)
    o, l = run_decode(pg, q, "bf16", scale=math.log(2), max_len=hint)
    check(o, l, decode_ref(pg, q, scale=math.log(2)), "bf16", 3000, float(pg.v.float().abs().max()))


@pytest.mark.parametrize("hint", [0, 1])                                # cut; one warp goes through a whole sequence
@pytest.mark.parametrize("kind,cache,D", [("fp16", "fp16", 64), ("fp16", "fp16", 128), ("bf16", "e4m3", 64), ("fp16", "e4m3", 128)])
def test_decode_fp16_products_many_small_weights_behind_one_key(kind, cache, D, hint):
    n, scale = 60000, math.log(2)
    pg = Paged([n, 300], 1, D, 64, cache)
    if cache == "e4m3":
        pg.scales.fill_(1.0)
        for s in pg.sc:
            s.fill_(1.0)
    k, v = one_far_ahead(n, 1, D, cache, 1)
    for pool, x in ((pg.k, k), (pg.v, v)):
        raw = (lambda t: t.view(torch.uint8)) if cache == "e4m3" else (lambda t: t)
        pages = torch.from_numpy(pg.tab[pg.seqs[0], :-(-n // 64)]).long().to(DEV)
        pad = torch.zeros((pages.numel() * 64, D), device=DEV).to(x.dtype)
        raw(pad)[:n] = raw(x)[:, 0]
        raw(pool)[1, pages, 0] = raw(pad).view(-1, 64, D)
    q = ahead_queries(2, 4, D, kind)
    ref = decode_ref(pg, q, scale=scale)
    o, l = run_decode(pg, q, kind, scale=scale, max_len=hint)
    v_max = float(v.float().abs().max())
    check_small_weights(o[:1], l[:1], [r[:1] for r in ref], kind, n, v_max, 10)
    assert (np.abs(ref[0][0]) > 100 * n * 2.0 ** -35 * v_max).all()


# ---------------------------------------------------------------- the Python classes

@pytest.mark.parametrize("on", ["stream", "handle", "default", "0"])
@pytest.mark.parametrize("what", ["prefill", "decode"])
def test_an_output_made_for_another_stream(what, on):
    """The current stream has work before it on memory that was given back to the allocator; the call on the other stream
    must not be given that memory."""
    n, H, Hk, D = 300, 8, 2, 128
    cache = KVCache(1, 40, Hk, 16, D, 4, 40)
    att = Attention(cache, 0, H, 4)
    q, k, v = (randn((n, h, D), i, "bf16") for i, h in ((1, H), (2, Hk), (3, Hk)))
    cu, seqs = i32([0, n]), i32([0])
    cache.reserve(seqs, i32([n]))
    cache.write(0, i32([0] * n), torch.arange(n, dtype=torch.int32, device=DEV), k, v)
    x = q if what == "prefill" else q[-1:].clone()
    call = (lambda **kw: att.prefill(x, k, v, cu, cu, **kw)) if what == "prefill" else (lambda **kw: att.decode(x, seqs, **kw))
    want = call()
    side = torch.cuda.Stream()
    here, there = (side, torch.cuda.default_stream()) if on in ("default", "0") else (torch.cuda.current_stream(), side)
    torch.cuda.synchronize()
    with torch.cuda.stream(here):
        for _ in range(3):
            old = torch.empty_like(x)
            torch.cuda._sleep(20_000_000)    # some 10 ms
            old.fill_(float("nan"))          # pending on this stream
            del old
            o = call(stream=there if on in ("stream", "default") else there.cuda_stream)
            torch.cuda.synchronize()
            assert torch.equal(o, want)
