"""What stands around the paged cache and its attention, as it is measured: cases, inputs and plain forms.

Four operators: norms of queries and keys for each head with the position rotation in the same pass, on arrays
(`rope`) or on the way into the cache's pages; rows rounded to 4 bits with a scale for every 16 as a cache takes them,
and a sequence's rows read back out of its pages (`chunk`); attention of one new token per sequence over a 4-bit cache
(`decode`); attention of one new token for sequences that share the pages of a long prefix (`shared`).

A case is a dict of plain values; `prepare` makes a case's inputs on the GPU, `run` takes one pass through the operator
(its plain form in torch, or the library's calls where `own` is true), `exact` gives the result by the definition in 64
bits.

A page of a 4-bit cache holds, for each KV head, its rows' codes (two to a byte, the first in the low half), then its
rows' scales, one E4M3 byte for every 16 elements.  An element is worth code * scale (* the head's own factor).  A code
is a sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6.  A block's scale is a sixth of its largest magnitude.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
BITS = {"bf16": 16.0, "fp16": 16.0, "e4m3": 8.0, "e2m1": 4.5}
CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a batch: queries and keys normed and turned, keys and values into their pages
        dict(name="rope_step", op="rope", type="bf16", heads=32, kv_heads=8, dim=128, turn=128, pairs="halves", norm=True,
             cache="bf16", seqs=64, longest=1, mix=0, far=8192, page=64, keep=False),
        # prompts admitted: views of one projection's output; the keys go on to the prompt's own attention too
        dict(name="rope_admit", op="rope", type="bf16", heads=32, kv_heads=8, dim=128, turn=128, pairs="halves", norm=True,
             cache="bf16", seqs=12, longest=2048, mix=6, far=0, page=64, keep=True),
        # no cache and no norm: half of each head turned, neighbours as pairs, far positions, an odd number of tokens
        dict(name="rope_far", op="rope", type="fp16", heads=28, kv_heads=4, dim=64, turn=32, pairs="neighbours", norm=False,
             cache="", seqs=3, longest=509, mix=5, far=1000000, page=16, keep=True),
        # chunks of a few prompts behind what is in a 4-bit cache already: the chunk written, all of it read back
        dict(name="chunk_batch", op="chunk", type="fp16", cache="e2m1", kv_heads=4, dim=64, seqs=8, longest=509, mix=5,
             before=4000, page=32, factor=True),
        # the next chunk of one very long prompt
        dict(name="chunk_long", op="chunk", type="bf16", cache="e2m1", kv_heads=8, dim=128, seqs=1, longest=2048, mix=0,
             before=129024, page=128, factor=False),
        # one user, a short context: latency
        dict(name="decode_one", op="decode", type="bf16", cache="e2m1", heads=32, kv_heads=8, dim=128, seqs=1,
             longest=777, mix=0, window=0, page=16, factor=False),
        # a serving batch of sequences of different lengths, an odd number of heads per KV head, a window
        dict(name="decode_window", op="decode", type="fp16", cache="e2m1", heads=28, kv_heads=4, dim=64, seqs=256,
             longest=2000, mix=4, window=1500, page=32, factor=True),
        # a few very long contexts
        dict(name="decode_long", op="decode", type="bf16", cache="e2m1", heads=64, kv_heads=8, dim=128, seqs=4,
             longest=131072, mix=0, window=0, page=128, factor=True),
        # four samples of one short prompt: latency
        dict(name="shared_few", op="shared", type="bf16", cache="bf16", heads=8, kv_heads=2, dim=64, groups=1, members=4,
             longest=500, mix=0, own=40, window=0, page=16, factor=False),
        # several samples of each of several prompts of different lengths
        dict(name="shared_samples", op="shared", type="bf16", cache="bf16", heads=32, kv_heads=8, dim=128, groups=8,
             members=8, longest=8192, mix=2, own=500, window=0, page=64, factor=False),
        # many users behind one system prompt
        dict(name="shared_system", op="shared", type="bf16", cache="bf16", heads=32, kv_heads=8, dim=128, groups=1,
             members=64, longest=16384, mix=3, own=1500, window=0, page=64, factor=False),
        # questions about one long document in a 4-bit cache
        dict(name="shared_document", op="shared", type="bf16", cache="e2m1", heads=64, kv_heads=8, dim=128, groups=1,
             members=32, longest=32768, mix=9, own=300, window=0, page=128, factor=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "chunk", "decode", "shared"])
    mix = rng.randrange(1, 1 << 20)
    kv = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    t = rng.choice(["bf16", "fp16"])
    if op == "rope":
        longest = _log(rng, 1, 4096)
        return dict(op=op, type=t, heads=kv * rng.choice([1, 2, 3, 4]), kv_heads=kv, dim=dim,
                    turn=rng.choice([16, 32, 48, 64, dim]), pairs=rng.choice(["halves", "neighbours"]),
                    norm=rng.choice([False, True]), cache=rng.choice(["", t, t]),
                    seqs=max(1, min(_log(rng, 1, 256), 11000 // longest)), longest=longest, mix=mix,
                    far=rng.choice([0, 0, _log(rng, 1, 8192)]), page=page, keep=rng.choice([False, True]))
    if op == "chunk":
        longest, before = _log(rng, 1, 2048), rng.choice([0, _log(rng, 1, 120000)])
        cache = rng.choice([t, "e4m3", "e2m1", "e2m1"])
        return dict(op=op, type=t, cache=cache, kv_heads=kv, dim=dim, longest=longest,
                    seqs=max(1, min(_log(rng, 1, 64), 120000 // (longest + before))), mix=mix, before=before, page=page,
                    factor=cache in ("e4m3", "e2m1") and rng.choice([False, True]))
    if op == "decode":
        longest = _log(rng, 1, 131072)
        return dict(op=op, type=t, cache="e2m1", heads=kv * rng.choice([1, 2, 3, 4, 6, 7, 8, 16]), kv_heads=kv, dim=dim,
                    seqs=max(1, min(_log(rng, 1, 256), 4 * 131072 // longest)), longest=longest, mix=mix,
                    window=rng.choice([0, 0, _log(rng, 1, 8192)]), page=page, factor=rng.choice([False, True]))
    longest, groups, members = _log(rng, 1, 16384), _log(rng, 1, 32), _log(rng, 1, 64)
    groups = max(1, min(groups, 64 // members))
    cache = rng.choice([t, t, "e4m3", "e2m1"])
    return dict(op=op, type=t, cache=cache, heads=kv * rng.choice([1, 2, 4, 5, 8]), kv_heads=kv, dim=dim, groups=groups,
                members=members, longest=longest, mix=mix, own=_log(rng, 1, 1500),
                window=rng.choice([0, 0, 0, _log(rng, 1, 16384)]), page=page,
                factor=cache in ("e4m3", "e2m1") and rng.choice([False, True]))


def lengths(n, longest, mix):
    """n lengths from 1 to longest, one of them longest; all longest for mix 0."""
    if not mix:
        return np.full(n, longest, np.int64)
    r = np.random.RandomState(mix)
    out = np.maximum(1, np.floor(longest * r.rand(n) ** 1.5)).astype(np.int64)
    out[r.randint(n)] = longest
    return out


def begins(case):
    """Position of the first new row of each sequence: up to `far`, or what a chunk finds before it."""
    most = case["far"] if case["op"] == "rope" else case["before"]
    if case["op"] == "chunk" and not case["mix"]:
        return np.full(case["seqs"], most, np.int64)
    return np.random.RandomState(case["mix"] + 1).randint(0, most + 1, case["seqs"]).astype(np.int64)


def shared_lengths(case):
    """Of each group its prefix's positions (whole pages), of each sequence all of its positions."""
    prompt = lengths(case["groups"], case["longest"], case["mix"])
    rest = np.random.RandomState(case["mix"] + 1).randint(1, case["own"] + 1, (case["groups"], case["members"]))
    return prompt // case["page"] * case["page"], (prompt[:, None] + rest).reshape(-1)


def work(case):
    row = case["kv_heads"] * case["dim"]                       # elements of a token's keys
    if case["op"] == "rope":
        n = int(lengths(case["seqs"], case["longest"], case["mix"]).sum())
        rows = 2 * case["heads"] * case["dim"] + row           # q, its result, k
        if case["cache"]:
            rows += 3 * row + (row if case["keep"] else 0)     # k to its page, v, v to its page; k beside
        else:
            rows += row
        return {"bytes": 2 * n * rows + 4 * n, "flops": 8 * n * (case["heads"] + case["kv_heads"]) * case["dim"]}
    if case["op"] == "chunk":
        n = int(lengths(case["seqs"], case["longest"], case["mix"]).sum())
        all_ = n + int(begins(case).sum())
        stored = BITS[case["cache"]] / 8
        return {"bytes": int(2 * row * (n * (2 + stored) + all_ * (2 + stored))), "flops": 0}
    stored = BITS[case["cache"]] / 8
    if case["op"] == "decode":
        n = lengths(case["seqs"], case["longest"], case["mix"])
        seen = np.minimum(n, case["window"]) if case["window"] else n
        read, pairs, seqs = int(seen.sum()), int(seen.sum()), case["seqs"]
    else:
        prefix, n = shared_lengths(case)
        lo = np.maximum(n - case["window"], 0) if case["window"] else np.zeros_like(n)
        pairs, seqs = int((n - lo).sum()), n.size
        pre = np.repeat(prefix if case["members"] > 1 else np.zeros_like(prefix), case["members"])
        first = np.minimum(lo.reshape(case["groups"], -1).min(1), pre.reshape(case["groups"], -1)[:, 0])
        read = int((n - np.maximum(lo, pre)).sum() + (pre.reshape(case["groups"], -1)[:, 0] - first).sum())
    return {"bytes": int(2 * read * row * stored + 4 * seqs * case["heads"] * case["dim"] + 4 * seqs * case["heads"]),
            "flops": 4 * pairs * case["heads"] * case["dim"]}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _to_codes(x):
    """The nearest code of each element of x (fp32, at most a little above 6 in size), ties to the even one; 8 for a sign."""
    m = x.abs()
    code = torch.zeros(x.shape, dtype=torch.uint8, device=x.device)
    code += m > 0.25
    code += m >= 0.75
    code += m > 1.25
    code += m >= 1.75
    code += m > 2.5
    code += m >= 3.5
    code += m > 5.0
    return code | (torch.signbit(x).to(torch.uint8) << 3)


def _to_blocks(x):
    """x (fp32, [..., dim]): codes, two to a byte [..., dim / 2], and the blocks' scales, E4M3 bytes [..., dim / 16]."""
    b = x.unflatten(-1, (-1, 16))
    scale = (b.abs().amax(-1) / 6.0).clamp(max=E4M3_MAX).to(torch.float8_e4m3fn)
    s = scale.float()[..., None]
    code = torch.where(s > 0, _to_codes(b / torch.where(s > 0, s, 1.0)), 0).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8)


def _pool(shape, kind, g):
    """Random page contents.  shape: pages, KV heads, page size, dim; one layer.  A 4-bit pool is bytes, 9 for 16 elements."""
    pages, heads, size, dim = shape
    if kind != "e2m1":
        x = torch.randn((1,) + shape, generator=g, device=DEV, dtype=torch.float16 if kind == "fp16" else torch.bfloat16)
        return (x * 16).to(torch.float8_e4m3fn) if kind == "e4m3" else x
    out = torch.empty((pages, heads, size * dim * 9 // 16), dtype=torch.uint8, device=DEV)
    for a in range(0, pages, 1024):
        part = out[a:a + 1024]
        code, scale = _to_blocks(torch.randn((part.shape[0],) + shape[1:], generator=g, device=DEV) * 4)
        part[..., :size * dim // 2] = code.flatten(-2)
        part[..., size * dim // 2:] = scale.flatten(-2)
    return out.view(1, pages, heads, size, dim * 9 // 16)


def _factors(case, g):
    """[1, kv_heads] factors of the keys and of the values, or None."""
    if not case.get("factor"):
        return None, None
    s = torch.rand((2, 1, case["kv_heads"]), generator=g, device=DEV) * 0.05 + 0.04
    if case["cache"] == "e2m1":
        s = s * 5
    return s[0].contiguous(), s[1].contiguous()


def _tables(length, page, seed, prefix=None, members=1):
    """Page tables of sequences on random pages: table, reference counts, number of pages; prefix: shared positions of a group."""
    n = len(length)
    need = -(-length // page)
    cols = int(need.max())
    share = np.zeros(n, np.int64) if prefix is None else np.repeat(prefix // page, members)
    pages = int((need - share).sum()) + (0 if prefix is None else int((prefix // page).sum())) + 3
    order, table, at = np.random.RandomState(seed % (1 << 31)).permutation(pages), np.full((n, cols), -1, np.int32), 0
    for s in range(n):
        if share[s]:
            if s % members == 0:
                table[s, :share[s]] = order[at:at + share[s]]
                at += share[s]
            else:
                table[s, :share[s]] = table[s - s % members, :share[s]]
        rest = need[s] - share[s]
        table[s, share[s]:need[s]] = order[at:at + rest]
        at += rest
    ref = np.bincount(table[table >= 0], minlength=pages).astype(np.int32)
    return table, ref, pages


def prepare(case, seed):
    g = _gen(seed)
    Hk, D, page = case["kv_heads"], case["dim"], case["page"]
    t = TYPES[case["type"]]
    st = dict(case=case)
    if case["op"] == "rope":
        n, start = lengths(case["seqs"], case["longest"], case["mix"]), begins(case)
        H, T = case["heads"], int(n.sum())
        x = (torch.randn((T, (H + 2 * Hk) * D), generator=g, device=DEV) * 2).to(t).view(T, H + 2 * Hk, D)
        st.update(q=x[:, :H], k=x[:, H:H + Hk], v=x[:, H + Hk:], eps=1e-6,
                  inv_freq=(10000.0 ** (-torch.arange(0, case["turn"], 2, dtype=torch.float64) / case["turn"])).float().to(DEV),
                  q_norm=None, k_norm=None, q_out=torch.empty((T, H, D), dtype=t, device=DEV),
                  k_out=torch.empty((T, Hk, D), dtype=t, device=DEV) if case["keep"] or not case["cache"] else None,
                  token_pos=_i32(np.concatenate([np.arange(a, a + b) for a, b in zip(start, n)])))
        if case["norm"]:
            w = torch.rand((2, D), generator=g, device=DEV) + 0.5
            st.update(q_norm=w[0].contiguous(), k_norm=w[1].contiguous())
        if case["cache"]:
            table, ref, pages = _tables(start + n, page, seed)
            st.update(token_seq=_i32(np.repeat(np.arange(case["seqs"]), n)), table=_i32(table), ref=_i32(ref),
                      len=_i32(start + n), k_scale=None, v_scale=None, k_pool=_pool((pages, Hk, page, D), case["cache"], g),
                      v_pool=_pool((pages, Hk, page, D), case["cache"], g))
    elif case["op"] == "chunk":
        n, start = lengths(case["seqs"], case["longest"], case["mix"]), begins(case)
        table, ref, pages = _tables(start + n, page, seed)
        T, total = int(n.sum()), int((start + n).sum())
        st.update(k=torch.randn((T, Hk, D), generator=g, device=DEV).to(t), v=torch.randn((T, Hk, D), generator=g, device=DEV).to(t),
                  token_seq=_i32(np.repeat(np.arange(case["seqs"]), n)),
                  token_pos=_i32(np.concatenate([np.arange(a, a + b) for a, b in zip(start, n)])),
                  seqs=_i32(np.arange(case["seqs"])), cu=_i32(np.concatenate([[0], np.cumsum(start + n)])), total=total,
                  table=_i32(table), ref=_i32(ref), len=_i32(start + n),
                  k_pool=_pool((pages, Hk, page, D), case["cache"], g), v_pool=_pool((pages, Hk, page, D), case["cache"], g),
                  k_out=torch.empty((total, Hk, D), dtype=t, device=DEV), v_out=torch.empty((total, Hk, D), dtype=t, device=DEV))
        st["k_scale"], st["v_scale"] = _factors(case, g)
    else:
        if case["op"] == "decode":
            n, prefix, members = lengths(case["seqs"], case["longest"], case["mix"]), None, 1
        else:
            prefix, n = shared_lengths(case)
            members = case["members"]
        table, ref, pages = _tables(n, page, seed, prefix, members)
        H = case["heads"]
        st.update(q=torch.randn((len(n), H, D), generator=g, device=DEV).to(t), seqs=_i32(np.arange(len(n))),
                  table=_i32(table), ref=_i32(ref), len=_i32(n), longest=int(n.max()), scale=1.0 / math.sqrt(D),
                  k_pool=_pool((pages, Hk, page, D), case["cache"], g), v_pool=_pool((pages, Hk, page, D), case["cache"], g),
                  o=torch.empty((len(n), H, D), dtype=t, device=DEV), lse=torch.empty((len(n), H), dtype=torch.float32, device=DEV))
        if case["op"] == "shared":
            st.update(cu=_i32(np.arange(0, len(n) + 1, members)), common=torch.empty(case["groups"], dtype=torch.int32, device=DEV))
        st["k_scale"], st["v_scale"] = _factors(case, g)
    if own:
        _handles(st)
    return st


def _handles(st):
    """What a program that uses the library keeps beside its buffers: the descriptors of its arrays, and a workspace."""
    import quantized_routed_expert_03_gb300 as qre
    case = st["case"]
    dtype = {"bf16": qre.QRE_BF16, "fp16": qre.QRE_FP16, "e4m3": qre.QRE_E4M3, "e2m1": qre.QRE_E2M1}
    if "k_pool" in st:
        st["cache"] = qre.make_kv_cache(st["k_pool"], st["v_pool"], st["table"], st["len"], st["ref"], dtype[case["cache"]],
                                        st["k_scale"], st["v_scale"])
    if case["op"] == "rope":
        st["rope"] = qre.make_rope(case["heads"], case["kv_heads"], case["dim"], dtype[case["type"]], st["inv_freq"],
                                   interleaved=case["pairs"] == "neighbours", q_norm=st["q_norm"], k_norm=st["k_norm"],
                                   eps=st["eps"], q=st["q"], k=st["k"], v=st["v"] if case["cache"] else None,
                                   q_out=st["q_out"], k_out=st["k_out"])
    elif case["op"] == "chunk":
        st["rows"] = qre.make_kv_rows(dtype[case["type"]], st["k"], st["v"])
        st["rows_out"] = qre.make_kv_rows(dtype[case["type"]], st["k_out"], st["v_out"])
    else:
        st["attn"] = qre.make_attn(case["heads"], case["kv_heads"], case["dim"], dtype[case["type"]], st["scale"],
                                   window=case["window"], q=st["q"], o=st["o"])
        n = st["q"].shape[0]
        size = qre.qre_attn_decode_workspace_size(st["attn"], st["cache"], n) if case["op"] == "decode" else \
            qre.qre_attn_decode_shared_workspace_size(st["attn"], st["cache"], n, case["groups"])
        st["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)


# ---------------------------------------------------------------- one pass

def run(st):
    case = st["case"]
    if own:
        return _run_own(st, case)
    if case["op"] == "rope":
        return plain_rope(st, case)
    if case["op"] == "chunk":
        plain_write(st, case, st["k"], st["v"])
        return plain_read(st, case)
    if case["op"] == "decode":
        return plain_decode(st, case)
    common = plain_common(st, case)
    return {**plain_decode(st, case), "common": common}


def _run_own(st, case):
    import quantized_routed_expert_03_gb300 as qre
    if case["op"] == "rope":
        if not case["cache"]:
            qre.qre_qk_norm_rope(st["rope"], st["q"].shape[0], st["token_pos"], st["q"], st["k"], st["q_out"], st["k_out"])
            return {"q": st["q_out"], "k": st["k_out"]}
        qre.qre_kv_write_rope(st["cache"], 0, st["rope"], st["q"].shape[0], st["token_seq"], st["token_pos"], st["q"],
                              st["k"], st["v"], st["q_out"], st["k_out"])
        out = {"q": st["q_out"], "k_pool": st["k_pool"], "v_pool": st["v_pool"]}
        return {**out, "k": st["k_out"]} if case["keep"] else out
    if case["op"] == "chunk":
        qre.qre_kv_write(st["cache"], 0, st["rows"], st["k"].shape[0], st["token_seq"], st["token_pos"], st["k"], st["v"])
        qre.qre_kv_read(st["cache"], 0, st["rows_out"], case["seqs"], st["seqs"], None, st["cu"], st["total"], st["k_out"],
                        st["v_out"])
        return {"k": st["k_out"], "v": st["v_out"]}
    n = st["q"].shape[0]
    if case["op"] == "decode":
        qre.qre_attn_decode(st["attn"], st["cache"], 0, n, st["seqs"], st["longest"], st["q"], st["o"], st["lse"], st["ws"])
        return {"o": st["o"], "lse": st["lse"]}
    qre.qre_kv_common_len(st["cache"], n, st["seqs"], case["groups"], st["cu"], st["common"])
    qre.qre_attn_decode_shared(st["attn"], st["cache"], 0, n, st["seqs"], case["groups"], st["cu"], st["common"],
                               st["longest"], st["q"], st["o"], st["lse"], st["ws"])
    return {"o": st["o"], "lse": st["lse"], "common": st["common"]}


def _normed(x, weight, eps):
    x = x.float()
    return x if weight is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight


def _turned(x, cos, sin, case):
    """x [tokens, heads, dim] with its first `turn` elements rotated in pairs by the tokens' angles."""
    n = case["turn"]
    out = x.clone()
    if case["pairs"] == "halves":
        a, b = slice(0, n // 2), slice(n // 2, n)
    else:
        a, b = slice(0, n, 2), slice(1, n, 2)
    out[..., a] = x[..., a] * cos - x[..., b] * sin
    out[..., b] = x[..., b] * cos + x[..., a] * sin
    return out


def plain_rope(st, case):
    angle = st["token_pos"].double()[:, None] * st["inv_freq"].double()[None]     # far positions: 32 bits would lose it
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    t = TYPES[case["type"]]
    q = _turned(_normed(st["q"], st["q_norm"], st["eps"]), cos, sin, case).to(t)
    k = _turned(_normed(st["k"], st["k_norm"], st["eps"]), cos, sin, case).to(t)
    if not case["cache"]:
        return {"q": q, "k": k}
    plain_write(st, case, k, st["v"])
    out = {"q": q, "k_pool": st["k_pool"], "v_pool": st["v_pool"]}
    return {**out, "k": k} if case["keep"] else out


def plain_write(st, case, k, v):
    page, D = case["page"], case["dim"]
    pos = st["token_pos"].long()
    at, row = st["table"][st["token_seq"].long(), pos // page].long(), pos % page
    for pool, x, scale in ((st["k_pool"], k, st["k_scale"]), (st["v_pool"], v, st["v_scale"])):
        if case["cache"] in ("bf16", "fp16"):
            pool[0][at, :, row] = x
            continue
        x = x.float() if scale is None else x.float() * (1.0 / scale[0])[None, :, None]
        if case["cache"] == "e4m3":
            pool.view(torch.uint8)[0][at, :, row] = x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
            continue
        code, scales = _to_blocks(x)
        flat = pool[0].flatten(-2)
        flat[..., :page * D // 2].unflatten(-1, (page, -1))[at, :, row] = code
        flat[..., page * D // 2:].unflatten(-1, (page, -1))[at, :, row] = scales


def _worth(pages, scale, case):
    """What the rows of some pages are worth, in fp32: pages [..., heads, page, bytes or elements] of a pool."""
    D, page = case["dim"], case["page"]
    if case["cache"] == "e2m1":
        flat = pages.flatten(-2)
        pair = torch.tensor([[(-1.0 if c & 8 else 1.0) * CODES[c & 7] for c in (b & 15, b >> 4)] for b in range(256)], device=DEV)
        code = pair[flat[..., :page * D // 2].int()].flatten(-2).unflatten(-1, (page, D // 16, 16))
        s = flat[..., page * D // 2:].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (page, D // 16))
        x = (code * s[..., None]).flatten(-2)
    elif case["cache"] == "e4m3":
        x = pages.view(torch.float8_e4m3fn).float()
    else:
        x = pages.float()
    return x if scale is None else x * scale[0][:, None, None]


def _raw(pool):
    return pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool


def plain_read(st, case):
    page, cu = case["page"], st["cu"].long()
    seq = torch.repeat_interleave(torch.arange(case["seqs"], device=DEV), cu[1:] - cu[:-1], output_size=st["total"])
    pos = torch.arange(st["total"], device=DEV) - cu[seq]
    at = st["table"][st["seqs"].long()[seq], pos // page].long()
    t, out = TYPES[case["type"]], {}
    for name, pool, scale in (("k", st["k_pool"], st["k_scale"]), ("v", st["v_pool"], st["v_scale"])):
        all_ = _worth(_raw(pool)[0], scale, case)                # pages, heads, page, dim
        out[name] = all_[at, :, pos % page].to(t)
    return out


def plain_common(st, case):
    """Leading positions on pages that all sequences of a group hold in the same place; 0 for a group of one."""
    table = st["table"].view(case["groups"], case["members"], -1)
    length = st["len"].view(case["groups"], -1).amin(1)
    same = (table == table[:, :1]).all(1) & (table[:, 0] >= 0)
    common = torch.minimum(torch.cumprod(same.int(), 1).sum(1) * case["page"], length)
    return (common if case["members"] > 1 else torch.zeros_like(common)).int()


def plain_decode(st, case):
    H, Hk, D, n = case["heads"], case["kv_heads"], case["dim"], st["q"].shape[0]
    table = st["table"].long().clamp(min=0)
    rows = []
    for pool, scale in ((st["k_pool"], st["k_scale"]), (st["v_pool"], st["v_scale"])):
        x = _worth(_raw(pool)[0], scale, case)[table]            # n, pages, heads, page, dim
        rows.append(x.transpose(1, 2).flatten(2, 3))
    q = st["q"].float().view(n, Hk, H // Hk, D)
    length = st["len"].long()[:, None]
    pos = torch.arange(rows[0].shape[2], device=DEV)[None]
    seen = pos < length
    if case["window"]:
        seen = seen & (pos >= length - case["window"])
    s = (q @ rows[0].transpose(-1, -2)) * st["scale"]
    s = torch.where(seen[:, None, None], s, torch.full((), -math.inf, device=DEV))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    o = (p @ rows[1]) / total
    return {"o": o.reshape(n, H, D).to(TYPES[case["type"]]), "lse": (m + torch.log(total)).reshape(n, H)}


# ---------------------------------------------------------------- by the definition, in 64 bits

def _stored(x, case, scale):
    """What a cache keeps of rows x [tokens, heads, dim] (float64) and gives back, before the head's factor.  The factor's
    reciprocal and the product with it are rounded to 32 bits: that is the definition."""
    if case["cache"] in ("bf16", "fp16"):
        return x
    if scale is not None:
        inv = torch.from_numpy(np.float32(1) / scale[0].cpu().numpy()).to(DEV)
        x = (x * inv.double()[None, :, None]).float().double()
    if case["cache"] == "e4m3":
        return _round_e4m3(x.clamp(-E4M3_MAX, E4M3_MAX))
    out = torch.empty_like(x)
    values = torch.tensor(CODES, dtype=torch.float64, device=DEV)
    middle = (values[1:] + values[:-1]) / 2
    for b in range(0, x.shape[-1], 16):
        y = x[..., b:b + 16]
        s = _round_e4m3((y.abs().amax(-1, keepdim=True) / 6).clamp(max=E4M3_MAX))
        m = torch.where(s > 0, y.abs() / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(y))
        low = torch.bucketize(m, middle, right=False)            # how many middles lie below m
        high = torch.bucketize(m, middle, right=True)            # and at or below it: one more on a tie
        code = torch.where((low != high) & (low % 2 == 1), high, low)
        out[..., b:b + 16] = torch.copysign(values[code], y) * s
    return out


def _round_e4m3(x):
    """x (float64, at most 448 in size) to the nearest E4M3 value, ties to even: steps of 2^(e-3), e >= -6."""
    e = torch.floor(torch.log2(torch.where(x == 0, torch.ones_like(x), x.abs()))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _head_worth(pool, h, case, scale):
    """Rows of all pages of head h in float64 [pages, page, dim], the head's factor among it."""
    D, page = case["dim"], case["page"]
    if case["cache"] == "e2m1":
        raw = pool[0, :, h].reshape(pool.shape[1], -1)
        code, byte = raw[:, :page * D // 2], raw[:, page * D // 2:]
        e, f = (byte >> 3).double(), (byte & 7).double()
        s = torch.where(e > 0, (1 + f / 8) * torch.exp2(e - 7), f / 8 * 2.0 ** -6)
        nibble = torch.stack([code & 15, code >> 4], -1).view(-1, page, D // 16, 16)
        e, f = ((nibble >> 1) & 3).double(), (nibble & 1).double()
        x = torch.where(e > 0, (1 + f / 2) * torch.exp2(e - 1), f / 2)
        x = (torch.where(nibble > 7, -x, x) * s.view(-1, page, D // 16, 1)).view(-1, page, D)
    else:
        x = pool[0, :, h].double()
    return x if scale is None else x * scale[0, h].double()


def exact(case, seed):
    global own
    mine, own = own, False                  # the inputs alone: the definition needs no descriptors
    try:
        st = prepare(case, seed)
    finally:
        own = mine
    Hk, D, page = case["kv_heads"], case["dim"], case["page"]
    table, length = st["table"].cpu().numpy() if "table" in st else None, st["len"].cpu().numpy() if "len" in st else None
    if case["op"] == "rope":
        pos = st["token_pos"].cpu().numpy().astype(np.float64)
        angle = pos[:, None] * st["inv_freq"].cpu().numpy().astype(np.float64)[None]
        c, s = (torch.from_numpy(f(angle)).to(DEV) for f in (np.cos, np.sin))
        half, out = case["turn"] // 2, {}
        for name, w in (("q", st["q_norm"]), ("k", st["k_norm"])):
            x = st[name].double().clone()
            if w is not None:
                x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D + st["eps"]) * w.double()
            y = x.clone()
            for i in range(half):
                a, b = (i, i + half) if case["pairs"] == "halves" else (2 * i, 2 * i + 1)
                y[:, :, a] = x[:, :, a] * c[:, i, None] - x[:, :, b] * s[:, i, None]
                y[:, :, b] = x[:, :, a] * s[:, i, None] + x[:, :, b] * c[:, i, None]
            out[name] = y
        if not case["cache"]:
            return out
        ts, tp = st["token_seq"].cpu().numpy(), st["token_pos"].cpu().numpy()
        where = torch.from_numpy(table[ts, tp // page].astype(np.int64)).to(DEV)
        row = torch.from_numpy((tp % page).astype(np.int64)).to(DEV)
        res = {"q": out["q"], "k_pool": st["k_pool"].double(), "v_pool": st["v_pool"].double()}
        for h in range(Hk):
            res["k_pool"][0, where, h, row] = out["k"][:, h]
            res["v_pool"][0, where, h, row] = st["v"][:, h].double()
        if case["keep"]:
            res["k"] = out["k"]
        return res
    if case["op"] == "chunk":
        cu, n, start = st["cu"].cpu().numpy(), lengths(case["seqs"], case["longest"], case["mix"]), begins(case)
        first, res = np.concatenate([[0], np.cumsum(n)]), {}
        for name, pool, scale in (("k", st["k_pool"], st["k_scale"]), ("v", st["v_pool"], st["v_scale"])):
            new = _stored(st[name].double(), case, scale)
            if scale is not None:
                new = new * scale[0].double()[None, :, None]
            x = torch.zeros((st["total"], Hk, D), dtype=torch.float64, device=DEV)
            for h in range(Hk):
                old = _head_worth(pool, h, case, scale)
                for i in range(case["seqs"]):
                    a, b, c = int(cu[i]), int(cu[i]) + int(start[i]), int(cu[i + 1])
                    pages = torch.from_numpy(table[i, :-(-(b - a) // page)].astype(np.int64)).to(DEV)
                    x[a:b, h] = old[pages].reshape(-1, D)[:b - a]
                    x[b:c, h] = new[int(first[i]):int(first[i + 1]), h]
            res[name] = x
        return res
    H, n = case["heads"], st["q"].shape[0]
    g = H // Hk
    o = torch.zeros(st["o"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device=DEV)
    for h in range(Hk):
        kv = [_head_worth(st[x + "_pool"], h, case, st[x + "_scale"]) for x in ("k", "v")]
        for i in range(n):
            L = int(length[i])
            lo = max(0, L - case["window"]) if case["window"] else 0
            at = torch.from_numpy(table[i, :-(-L // page)].astype(np.int64)).to(DEV)
            k, v = (x[at].reshape(-1, D)[lo:L] for x in kv)
            s = torch.einsum("id,jd->ij", st["q"][i, h * g:(h + 1) * g].double(), k) * st["scale"]
            lse[i, h * g:(h + 1) * g] = torch.logsumexp(s, -1)
            o[i, h * g:(h + 1) * g] = torch.softmax(s, -1) @ v
    res = {"o": o, "lse": lse}
    if case["op"] == "shared":
        common = np.zeros(case["groups"], np.int32)
        for a in range(case["groups"]):
            rows = table[a * case["members"]:(a + 1) * case["members"]]
            same = 0
            while same < rows.shape[1] and rows[0, same] >= 0 and len(set(rows[:, same].tolist())) == 1:
                same += 1
            if case["members"] > 1:
                common[a] = min(same * page, int(length[a * case["members"]:(a + 1) * case["members"]].min()))
        res["common"] = common
    return res
