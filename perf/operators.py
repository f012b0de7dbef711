"""The key-value cache and attention operators as they are measured: their cases, inputs and plain forms.

Four operators: attention over packed prompts (`prefill`), attention of one new token per sequence over a
paged key-value cache (`decode`), the write of new keys and values into the cache's pages (`write`), and the
bookkeeping of its pages (`pages`: free, reserve, fork, compact).

A case is a dict of plain values; `prepare` makes a case's inputs on the GPU, `run` takes one pass through
the operator (its plain form in torch, or the library's calls where `own` is true), `exact` gives the result
by the definition in 64 bits.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "e4m3": 1}
E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases

def listed():
    return [
        # three short prompts in one call: a chat's first turns, where latency counts
        dict(name="prefill_few", op="prefill", type="bf16", heads=8, kv_heads=2, dim=64, seqs=3, longest=40, mix=3,
             prefix=0, window=0, fused=False),
        # a batch of prompts of different lengths, q, k and v as views of one projection's output
        dict(name="prefill_packed", op="prefill", type="bf16", heads=32, kv_heads=8, dim=128, seqs=16, longest=2048,
             mix=1, prefix=0, window=0, fused=True),
        # one long prompt: the token count of the library's prefill workload
        dict(name="prefill_prompt", op="prefill", type="bf16", heads=32, kv_heads=8, dim=128, seqs=1, longest=8192,
             mix=0, prefix=0, window=0, fused=False),
        # chunks of prompts behind a prefix that is in the keys already, with a sliding window
        dict(name="prefill_chunk", op="prefill", type="fp16", heads=32, kv_heads=4, dim=64, seqs=8, longest=509, mix=5,
             prefix=4000, window=1024, fused=False),
        # one user, a short context: latency
        dict(name="decode_one", op="decode", type="bf16", cache="bf16", heads=32, kv_heads=8, dim=128, seqs=1,
             longest=777, mix=0, window=0, page=16),
        # a serving batch of sequences of different lengths
        dict(name="decode_batch", op="decode", type="bf16", cache="bf16", heads=32, kv_heads=8, dim=128, seqs=64,
             longest=8192, mix=2, window=0, page=64),
        # a few very long contexts in an 8-bit cache
        dict(name="decode_long", op="decode", type="bf16", cache="e4m3", heads=64, kv_heads=8, dim=128, seqs=4,
             longest=131072, mix=0, window=0, page=128),
        # many short sequences, an odd number of heads per KV head, a window
        dict(name="decode_many", op="decode", type="fp16", cache="fp16", heads=28, kv_heads=4, dim=64, seqs=256,
             longest=2000, mix=4, window=1500, page=32),
        # one decode step's new rows of a batch
        dict(name="write_step", op="write", type="bf16", cache="bf16", kv_heads=8, dim=128, seqs=64, longest=1, mix=0,
             page=64, admit=False),
        # prompts admitted: their old rows' pages freed, pages reserved, all rows rounded to 8 bits and written
        dict(name="write_admit", op="write", type="bf16", cache="e4m3", kv_heads=8, dim=128, seqs=12, longest=2048,
             mix=6, page=64, admit=True),
        # a beam step: the children of the last step are freed, the winners forked
        dict(name="pages_fork", op="pages", do="fork", cache="bf16", kv_heads=8, dim=128, layers=4, page=32, seqs=16,
             longest=1000, children=64, pages=768, mix=7),
        # compaction after many sequences have ended
        dict(name="pages_compact", op="pages", do="compact", cache="bf16", kv_heads=8, dim=128, layers=4, page=32,
             seqs=48, longest=800, children=0, pages=1024, mix=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "decode", "write", "pages"])
    mix = rng.randrange(1, 1 << 20)
    kv = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "prefill":
        longest = _log(rng, 1, 8192)
        prefix = rng.choice([0, 0, _log(rng, 1, 8192)])
        heads = kv * rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 16) if kv * g <= 32])
        # the plain form's score matrix stays below the largest listed case's
        room = 32 * 8192 * 8192 // (heads * longest * (longest + prefix))
        seqs = max(1, min(_log(rng, 1, 64), room, 16384 // longest))
        if room < 1:
            prefix = 0
        return dict(op=op, type=rng.choice(["bf16", "fp16"]), heads=heads, kv_heads=kv, dim=dim, seqs=seqs,
                    longest=longest, mix=mix, prefix=prefix, window=rng.choice([0, 0, _log(rng, 1, 4096)]),
                    fused=rng.choice([False, True]) and prefix == 0)
    if op == "decode":
        longest = _log(rng, 1, 131072)
        heads = kv * rng.choice([1, 2, 3, 4, 6, 7, 8, 16])
        t = rng.choice(["bf16", "fp16"])
        cache = rng.choice([t, "e4m3"])
        seqs = max(1, min(_log(rng, 1, 256), 4 * 131072 // (longest * SIZE[cache])))
        return dict(op=op, type=t, cache=cache, heads=heads, kv_heads=kv, dim=dim, seqs=seqs,
                    longest=longest, mix=mix, window=rng.choice([0, 0, _log(rng, 1, 8192)]), page=page)
    if op == "write":
        longest = _log(rng, 1, 4096)
        t = rng.choice(["bf16", "fp16"])
        return dict(op=op, type=t, cache=rng.choice([t, "e4m3"]), kv_heads=kv, dim=dim,
                    seqs=max(1, min(_log(rng, 1, 256), 16384 // longest)), longest=longest, mix=mix, page=page,
                    admit=rng.choice([False, True]))
    longest = _log(rng, 1, 2000)
    seqs = _log(rng, 1, 48)
    children = _log(rng, 1, 64)
    layers = rng.choice([1, 2, 4])
    # a pool of 0.4 GB at most
    room = (400 << 20) // (2 * layers * kv * page * dim * 2)
    seqs = max(1, min(seqs, (room - 64) // (2 * (-(-longest // page)))))
    used = seqs * -(-longest // page)
    return dict(op=op, do=rng.choice(["fork", "compact"]), cache=rng.choice(["bf16", "fp16", "e4m3"]), kv_heads=kv,
                dim=dim, layers=layers, page=page, seqs=seqs, longest=longest, children=children,
                pages=used + children + rng.randrange(1, max(2, used // 2 + 2)), mix=mix)


def lengths(n, longest, mix):
    """n lengths from 1 to longest, one of them longest; all longest for mix 0."""
    if not mix:
        return np.full(n, longest, np.int64)
    r = np.random.RandomState(mix)
    out = np.maximum(1, np.floor(longest * r.rand(n) ** 1.5)).astype(np.int64)
    out[r.randint(n)] = longest
    return out


def prefill_lengths(case):
    """(queries, keys) of each sequence."""
    q = lengths(case["seqs"], case["longest"], case["mix"])
    if not case["prefix"]:
        return q, q.copy()
    return q, q + np.random.RandomState(case["mix"] + 1).randint(0, case["prefix"] + 1, case["seqs"])


def visible_pairs(q, k, window):
    """How many (query, key) pairs the causal mask and the window leave."""
    total = 0
    for a, b in zip(q, k):
        last = np.arange(b - a, b, dtype=np.int64)          # position of each query
        seen = last + 1
        total += int((np.minimum(seen, window) if window else seen).sum())
    return total


def work(case):
    if case["op"] == "prefill":
        q, k = prefill_lengths(case)
        pairs = visible_pairs(q, k, case["window"])
        rows = 2 * int(q.sum()) * case["heads"] + 2 * int(k.sum()) * case["kv_heads"]
        return {"bytes": rows * case["dim"] * 2 + 4 * int(q.sum()) * case["heads"],
                "flops": 4 * case["dim"] * pairs * case["heads"]}
    if case["op"] == "decode":
        n = lengths(case["seqs"], case["longest"], case["mix"])
        if case["window"]:
            n = np.minimum(n, case["window"])
        rows = int(n.sum())
        return {"bytes": 2 * rows * case["kv_heads"] * case["dim"] * SIZE[case["cache"]]
                + 4 * case["seqs"] * case["heads"] * case["dim"] + 4 * case["seqs"] * case["heads"]
                + 4 * int((-(-n // case["page"])).sum()),
                "flops": 4 * rows * case["heads"] * case["dim"]}
    if case["op"] == "write":
        rows = int(lengths(case["seqs"], case["longest"], case["mix"]).sum())
        return {"bytes": 2 * rows * case["kv_heads"] * case["dim"] * (2 + SIZE[case["cache"]]) + 8 * rows, "flops": 0}
    page = 2 * case["layers"] * case["kv_heads"] * case["page"] * case["dim"] * SIZE[case["cache"]]
    plan = page_plan(case)
    if case["do"] == "fork":
        moved = int((plan["len"][plan["parents"]] % case["page"] > 0).sum())
    else:
        live = int((plan["ref"] > 0).sum())
        moved = int((plan["ref"][live:] > 0).sum())
    return {"bytes": 2 * moved * page + 8 * plan["table"].size + 8 * plan["ref"].size, "flops": 0}


# ---------------------------------------------------------------- inputs

def page_plan(case):
    """Tables of a cache in use, on the host: sequences of random lengths on random pages, some with a shared prefix."""
    r = np.random.RandomState(case["mix"])
    n, page, pages = case["seqs"], case["page"], case["pages"]
    rows = n + case["children"]
    cols = -(-case["longest"] // page)
    table = np.full((rows, cols), -1, np.int32)
    ref = np.zeros(pages, np.int32)
    length = np.zeros(rows, np.int32)
    length[:n] = lengths(n, case["longest"], case["mix"])
    order = r.permutation(pages)
    at = 0
    for s in range(n):
        need = -(-int(length[s]) // page)
        share = 0
        if s % 4 == 3:                                      # every fourth shares whole pages with the one before
            share = min(int(length[s - 1]), int(length[s])) // page // 2
            table[s, :share] = table[s - 1, :share]
        table[s, share:need] = order[at:at + need - share]
        at += need - share
        np.add.at(ref, table[s, :need], 1)
    parents = r.randint(0, n, case["children"]).astype(np.int32)
    return {"table": table, "ref": ref, "len": length, "parents": parents,
            "dst": np.arange(n, rows, dtype=np.int32)}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _pool(shape, kind, g):
    """Random page contents."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float16 if kind == "fp16" else torch.bfloat16)
    return (x * 16).to(torch.float8_e4m3fn) if kind == "e4m3" else x


def _scales(kv_heads, kind, g):
    if kind != "e4m3":
        return None, None
    s = torch.rand((2, 1, kv_heads), generator=g, device=DEV) * 0.05 + 0.04
    return s[0].contiguous(), s[1].contiguous()


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    if case["op"] == "prefill":
        q_len, k_len = prefill_lengths(case)
        H, Hk, D, t = case["heads"], case["kv_heads"], case["dim"], TYPES[case["type"]]
        nq, nk = int(q_len.sum()), int(k_len.sum())
        if case["fused"]:
            x = torch.randn((nq, (H + 2 * Hk) * D), generator=g, device=DEV).to(t)
            x = x.view(nq, H + 2 * Hk, D)
            st.update(q=x[:, :H], k=x[:, H:H + Hk], v=x[:, H + Hk:])
        else:
            st.update(q=torch.randn((nq, H, D), generator=g, device=DEV).to(t),
                      k=torch.randn((nk, Hk, D), generator=g, device=DEV).to(t),
                      v=torch.randn((nk, Hk, D), generator=g, device=DEV).to(t))
        st.update(cu_q=_i32(np.concatenate([[0], np.cumsum(q_len)])), cu_k=_i32(np.concatenate([[0], np.cumsum(k_len)])),
                  max_q=int(q_len.max()), max_k=int(k_len.max()), scale=1.0 / math.sqrt(D),
                  o=torch.empty((nq, H, D), dtype=t, device=DEV),
                  lse=torch.empty((nq, H), dtype=torch.float32, device=DEV))
    elif case["op"] == "decode":
        H, Hk, D, page, n = case["heads"], case["kv_heads"], case["dim"], case["page"], case["seqs"]
        length = lengths(n, case["longest"], case["mix"])
        need = -(-length // page)
        pages, cols = int(need.sum()) + 3, int(need.max())
        r = np.random.RandomState(seed % (1 << 31))
        order, table, at = r.permutation(pages), np.full((n + 1, cols), -1, np.int32), 0
        seqs = r.permutation(n + 1)[:n]
        row_len = np.zeros(n + 1, np.int32)
        for i, s in enumerate(seqs):
            table[s, :need[i]] = order[at:at + need[i]]
            row_len[s] = length[i]
            at += need[i]
        ref = np.zeros(pages, np.int32)
        ref[table[table >= 0]] = 1
        st.update(q=torch.randn((n, H, D), generator=g, device=DEV).to(TYPES[case["type"]]),
                  seqs=_i32(seqs), table=_i32(table), len=_i32(row_len), ref=_i32(ref), scale=1.0 / math.sqrt(D),
                  k=_pool((1, pages, Hk, page, D), case["cache"], g), v=_pool((1, pages, Hk, page, D), case["cache"], g),
                  longest=int(length.max()), o=torch.empty((n, H, D), dtype=TYPES[case["type"]], device=DEV),
                  lse=torch.empty((n, H), dtype=torch.float32, device=DEV))
        st["k_scale"], st["v_scale"] = _scales(Hk, case["cache"], g)
    elif case["op"] == "write":
        Hk, D, page, n = case["kv_heads"], case["dim"], case["page"], case["seqs"]
        length = lengths(n, case["longest"], case["mix"])
        r = np.random.RandomState(seed % (1 << 31))
        start = np.zeros(n, np.int64) if case["admit"] else np.random.RandomState(case["mix"] + 1).randint(0, 4 * page, n)
        need = -(-(start + length) // page)
        pages, cols = int(need.sum()) * 2 + 8, int(need.max())
        order, table, at = r.permutation(pages), np.full((n, cols), -1, np.int32), 0
        for s in range(n):
            table[s, :need[s]] = order[at:at + need[s]]
            at += need[s]
        ref = np.zeros(pages, np.int32)
        ref[table[table >= 0]] = 1
        if case["admit"]:                                   # pages that other sequences hold
            ref[order[at:at + int(need.sum()) // 2]] = 1
        rows = int(length.sum())
        st.update(new_k=torch.randn((rows, Hk, D), generator=g, device=DEV).to(TYPES[case["type"]]),
                  new_v=torch.randn((rows, Hk, D), generator=g, device=DEV).to(TYPES[case["type"]]),
                  token_seq=_i32(np.repeat(np.arange(n), length)),
                  token_pos=_i32(np.concatenate([np.arange(a, a + b) for a, b in zip(start, length)])),
                  seqs=_i32(np.arange(n)), n_new=_i32(length), table=_i32(table), len=_i32(start + length), ref=_i32(ref),
                  k=_pool((1, pages, Hk, page, D), case["cache"], g), v=_pool((1, pages, Hk, page, D), case["cache"], g))
        st["k_scale"], st["v_scale"] = _scales(Hk, case["cache"], g)
    else:
        plan = page_plan(case)
        shape = (case["layers"], case["pages"], case["kv_heads"], case["page"], case["dim"])
        st.update(table=_i32(plan["table"]), len=_i32(plan["len"]), ref=_i32(plan["ref"]), parents=_i32(plan["parents"]),
                  dst=_i32(plan["dst"]), k=_pool(shape, case["cache"], g), v=_pool(shape, case["cache"], g),
                  k_scale=None, v_scale=None, table_out=_i32(plan["table"]), ref_out=_i32(plan["ref"]),
                  n_live=_i32([0]))
    if own:
        _handles(st)
    return st


def _handles(st):
    """What a program that uses the library keeps beside its buffers: the descriptors of its arrays, and a workspace."""
    import quantized_routed_expert_03_gb300 as qre
    case = st["case"]
    dtype = {"bf16": qre.QRE_BF16, "fp16": qre.QRE_FP16, "e4m3": qre.QRE_E4M3}
    if case["op"] != "prefill":
        st["cache"] = qre.make_kv_cache(st["k"], st["v"], st["table"], st["len"], st["ref"],
                                        dtype[case["cache"]], st["k_scale"], st["v_scale"])
    if case["op"] == "prefill":
        st["attn"] = qre.make_attn(case["heads"], case["kv_heads"], case["dim"], dtype[case["type"]], st["scale"],
                                   window=case["window"], q=st["q"], k=st["k"], v=st["v"], o=st["o"])
    elif case["op"] == "decode":
        st["attn"] = qre.make_attn(case["heads"], case["kv_heads"], case["dim"], dtype[case["type"]], st["scale"],
                                   window=case["window"], q=st["q"], o=st["o"])
        st["ws"] = torch.empty(qre.qre_attn_decode_workspace_size(st["attn"], st["cache"], case["seqs"]),
                               dtype=torch.uint8, device=DEV)
    else:
        st["ws"] = torch.empty(qre.qre_kv_workspace_size(st["cache"]), dtype=torch.uint8, device=DEV)
        if case["op"] == "write":
            st["rows"] = qre.make_kv_rows(dtype[case["type"]], st["new_k"], st["new_v"])


# ---------------------------------------------------------------- one pass

def run(st):
    case = st["case"]
    if own:
        return _run_own(st, case)
    if case["op"] == "prefill":
        return plain_prefill(st, case)
    if case["op"] == "decode":
        return plain_decode(st, case)
    if case["op"] == "write":
        if case["admit"]:
            plain_free(st, st["seqs"])
            plain_reserve(st, st["seqs"], st["n_new"])
        plain_write(st, case)
        return {"k": st["k"], "v": st["v"], "table": st["table"], "len": st["len"], "ref": st["ref"]}
    if case["do"] == "fork":
        plain_free(st, st["dst"])
        plain_fork(st)
        return {"k": st["k"], "v": st["v"], "table": st["table"], "len": st["len"], "ref": st["ref"]}
    return plain_compact(st)


def _run_own(st, case):
    import quantized_routed_expert_03_gb300 as qre
    if case["op"] == "prefill":
        qre.qre_attn_prefill(st["attn"], case["seqs"], st["q"].shape[0], st["k"].shape[0], st["cu_q"], st["cu_k"],
                             st["q"], st["k"], st["v"], st["o"], st["lse"])
        return {"o": st["o"], "lse": st["lse"]}
    if case["op"] == "decode":
        qre.qre_attn_decode(st["attn"], st["cache"], 0, case["seqs"], st["seqs"], st["longest"], st["q"], st["o"],
                            st["lse"], st["ws"])
        return {"o": st["o"], "lse": st["lse"]}
    if case["op"] == "write":
        if case["admit"]:
            qre.qre_kv_free(st["cache"], case["seqs"], st["seqs"])
            qre.qre_kv_reserve(st["cache"], case["seqs"], st["seqs"], st["n_new"], st["ws"])
        qre.qre_kv_write(st["cache"], 0, st["rows"], st["new_k"].shape[0], st["token_seq"], st["token_pos"],
                         st["new_k"], st["new_v"])
        return {"k": st["k"], "v": st["v"], "table": st["table"], "len": st["len"], "ref": st["ref"]}
    if case["do"] == "fork":
        qre.qre_kv_free(st["cache"], case["children"], st["dst"])
        qre.qre_kv_fork(st["cache"], case["children"], st["parents"], st["dst"], st["ws"])
        return {"k": st["k"], "v": st["v"], "table": st["table"], "len": st["len"], "ref": st["ref"]}
    qre.qre_kv_compact(st["cache"], st["table_out"], st["ref_out"], st["n_live"], st["ws"])
    return {"k": st["k"], "v": st["v"], "table": st["table_out"], "ref": st["ref_out"], "live": st["n_live"]}


def _softmax_pv(s, v, seen):
    """softmax over the last axis of s where `seen`, times v; rows that see nothing give 0 and -inf."""
    s = torch.where(seen, s, torch.full((), -math.inf, device=s.device))
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    return o, (m + torch.log(total)).squeeze(-1)


def plain_prefill(st, case):
    """Every sequence padded to the longest, one masked score matrix for all."""
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    n, g = case["seqs"], H // Hk
    cq, ck = st["cu_q"].long(), st["cu_k"].long()
    ql, kl = cq[1:] - cq[:-1], ck[1:] - ck[:-1]
    i, j = torch.arange(st["max_q"], device=DEV), torch.arange(st["max_k"], device=DEV)
    iq = (cq[:-1, None] + torch.minimum(i[None], ql[:, None] - 1))
    jk = (ck[:-1, None] + torch.minimum(j[None], kl[:, None] - 1))
    q = st["q"][iq].float().view(n, -1, Hk, g, D).permute(0, 2, 3, 1, 4)        # n, Hk, g, i, D
    k = st["k"][jk].float().permute(0, 2, 3, 1).unsqueeze(2)                    # n, Hk, 1, D, j
    v = st["v"][jk].float().permute(0, 2, 1, 3).unsqueeze(2)
    pos = (i[None] + (kl - ql)[:, None])[:, :, None]
    seen = (j[None, None] <= pos) & (j[None, None] < kl[:, None, None])
    if case["window"]:
        seen = seen & (j[None, None] > pos - case["window"])
    o, lse = _softmax_pv((q @ k) * st["scale"], v, seen[:, None, None])
    valid = i[None] < ql[:, None]
    o = o.permute(0, 3, 1, 2, 4).reshape(n, -1, H, D)[valid].to(TYPES[case["type"]])
    return {"o": o, "lse": lse.permute(0, 3, 1, 2).reshape(n, -1, H)[valid]}


def _gather(pool, table, scale):
    """Rows of the listed pages in fp32: [n, heads, positions, dim]."""
    raw = pool[0]
    if raw.dtype == torch.float8_e4m3fn:
        x = raw.view(torch.uint8)[table].view(torch.float8_e4m3fn).float()
    else:
        x = raw[table].float()
    n, p, h, t, d = x.shape
    x = x.permute(0, 2, 1, 3, 4).reshape(n, h, p * t, d)
    return x if scale is None else x * scale[0][None, :, None, None]


def plain_decode(st, case):
    H, Hk, D, n = case["heads"], case["kv_heads"], case["dim"], case["seqs"]
    rows = st["seqs"].long()
    table = st["table"][rows].long().clamp(min=0)
    length = st["len"][rows].long()[:, None]
    k, v = _gather(st["k"], table, st["k_scale"]), _gather(st["v"], table, st["v_scale"])
    q = st["q"].float().view(n, Hk, H // Hk, D)
    pos = torch.arange(k.shape[2], device=DEV)[None]
    seen = pos < length
    if case["window"]:
        seen = seen & (pos >= length - case["window"])
    o, lse = _softmax_pv((q @ k.transpose(-1, -2)) * st["scale"], v, seen[:, None, None])
    return {"o": o.reshape(n, H, D).to(TYPES[case["type"]]), "lse": lse.reshape(n, H)}


def _rows_to_cache(x, scale, kind):
    if kind != "e4m3":
        return x
    return (x.float() / scale[0][None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def plain_write(st, case):
    page = case["page"]
    pos = st["token_pos"].long()
    at, row = st["table"][st["token_seq"].long(), pos // page].long(), pos % page
    raw = (lambda t: t.view(torch.uint8)) if case["cache"] == "e4m3" else (lambda t: t)
    raw(st["k"])[0][at, :, row] = _rows_to_cache(st["new_k"], st["k_scale"], case["cache"])
    raw(st["v"])[0][at, :, row] = _rows_to_cache(st["new_v"], st["v_scale"], case["cache"])


def plain_free(st, seqs):
    seqs = seqs.long()
    page = st["case"]["page"]
    table, cols = st["table"][seqs].long(), torch.arange(st["table"].shape[1], device=DEV)
    held = cols[None] < (st["len"][seqs].long()[:, None] + page - 1) // page
    st["ref"].index_add_(0, torch.where(held, table, 0).reshape(-1), -held.reshape(-1).int())
    st["table"][seqs] = -1
    st["len"][seqs] = 0


def _free_pages(ref):
    """Page numbers, the free ones first in ascending order."""
    return torch.sort((ref > 0).int(), stable=True).indices


def plain_reserve(st, seqs, n_new):
    """For sequences that hold nothing yet, as here."""
    page = st["case"]["page"]
    need = (n_new.long() + page - 1) // page
    first = torch.cumsum(need, 0) - need
    cols = torch.arange(st["table"].shape[1], device=DEV)
    held = cols[None] < need[:, None]
    pick = _free_pages(st["ref"])[torch.where(held, first[:, None] + cols[None], 0)]
    st["table"][seqs.long()] = torch.where(held, pick, -1).int()
    st["ref"].index_add_(0, pick.reshape(-1), held.reshape(-1).int())
    st["len"][seqs.long()] = n_new


def plain_fork(st):
    page = st["case"]["page"]
    src, dst = st["parents"].long(), st["dst"].long()
    length = st["len"][src].long()
    full, part = length // page, length % page > 0
    cols = torch.arange(st["table"].shape[1], device=DEV)[None]
    table = st["table"][src].long()
    whole = cols < full[:, None]
    fresh = _free_pages(st["ref"])[torch.cumsum(part.int(), 0) - part.int()]
    old = torch.gather(table, 1, torch.where(part, full, 0)[:, None]).squeeze(1)
    row = torch.where(whole, table, torch.where((cols == full[:, None]) & part[:, None], fresh[:, None], -1))
    st["ref"].index_add_(0, torch.where(row >= 0, row, 0).reshape(-1), (row >= 0).reshape(-1).int())
    st["table"][dst] = row.int()
    st["len"][dst] = length.int()
    raw = (lambda t: t.view(torch.uint8)) if st["k"].dtype == torch.float8_e4m3fn else (lambda t: t)
    raw(st["k"])[:, fresh[part]] = raw(st["k"])[:, old[part]]
    raw(st["v"])[:, fresh[part]] = raw(st["v"])[:, old[part]]


def plain_compact(st):
    """Live pages beyond the first n_live go to the free places among these, both in ascending order."""
    ref = st["ref"]
    live, at = ref > 0, torch.arange(ref.numel(), device=DEV)
    n_live = live.sum()
    moves, holes = live & (at >= n_live), ~live & (at < n_live)
    hole = torch.sort((~holes).int(), stable=True).indices
    new = torch.where(moves, hole[(torch.cumsum(moves.int(), 0) - 1).clamp(min=0)], at)
    table = st["table"].long()
    held = table >= 0
    st["table_out"].copy_(torch.where(held, new[table.clamp(min=0)], -1))
    to = new[moves]
    ref_out = torch.where(moves, 0, ref)
    ref_out[to] = ref[moves]
    st["ref_out"].copy_(ref_out)
    st["n_live"].copy_(n_live)
    raw = (lambda t: t.view(torch.uint8)) if st["k"].dtype == torch.float8_e4m3fn else (lambda t: t)
    raw(st["k"])[:, to] = raw(st["k"])[:, moves]
    raw(st["v"])[:, to] = raw(st["v"])[:, moves]
    return {"k": st["k"], "v": st["v"], "table": st["table_out"], "ref": st["ref_out"], "live": st["n_live"]}


# ---------------------------------------------------------------- by the definition, in 64 bits

def _attend(q, k, v, scale, lo, hi):
    """One head: q [i, D], k and v [j, D] in float64; query i sees keys lo[i] <= j < hi[i]."""
    s = torch.einsum("id,jd->ij", q, k) * scale
    j = torch.arange(k.shape[0], device=s.device)
    s = s.masked_fill((j[None] < lo[:, None]) | (j[None] >= hi[:, None]), -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None])
    return torch.einsum("ij,jd->id", p, v), lse


def exact(case, seed):
    global own
    mine, own = own, False                  # the inputs alone: the definition needs no descriptors
    try:
        st = prepare(case, seed)
    finally:
        own = mine
    if case["op"] == "prefill":
        q_len, k_len = prefill_lengths(case)
        H, g = case["heads"], case["heads"] // case["kv_heads"]
        o = torch.zeros(st["o"].shape, dtype=torch.float64, device=DEV)
        lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device=DEV)
        a = b = 0
        for nq, nk in zip(q_len.tolist(), k_len.tolist()):
            pos = torch.arange(nk - nq, nk, device=DEV)
            lo = (pos - case["window"] + 1).clamp(min=0) if case["window"] else torch.zeros_like(pos)
            for h in range(H):
                o[a:a + nq, h], lse[a:a + nq, h] = _attend(
                    st["q"][a:a + nq, h].double(), st["k"][b:b + nk, h // g].double(),
                    st["v"][b:b + nk, h // g].double(), st["scale"], lo, pos + 1)
            a, b = a + nq, b + nk
        return {"o": o, "lse": lse}
    if case["op"] == "decode":
        n, page, g = case["seqs"], case["page"], case["heads"] // case["kv_heads"]
        o = torch.zeros(st["o"].shape, dtype=torch.float64, device=DEV)
        lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device=DEV)
        table, length, seqs = st["table"].cpu().numpy(), st["len"].cpu().numpy(), st["seqs"].cpu().numpy()
        for i in range(n):
            L = int(length[seqs[i]])
            at = torch.from_numpy(table[seqs[i], :-(-L // page)].astype(np.int64)).to(DEV)
            hi = torch.tensor([L], device=DEV)
            lo = (hi - case["window"]).clamp(min=0) if case["window"] else torch.zeros_like(hi)
            for h in range(case["kv_heads"]):
                rows = []
                for pool, scale in ((st["k"], st["k_scale"]), (st["v"], st["v_scale"])):
                    x = torch.stack([pool[0, p, h].double() for p in at]) if pool.dtype == torch.float8_e4m3fn \
                        else pool[0, at, h].double()
                    x = x.reshape(-1, case["dim"])[:L]
                    rows.append(x if scale is None else x * scale[0, h].double())
                heads = slice(h * g, (h + 1) * g)
                o[i, heads], lse[i, heads] = _attend(st["q"][i, heads].double(), rows[0], rows[1], st["scale"],
                                                     lo.expand(g), hi.expand(g))
        return {"o": o, "lse": lse}
    table, length, ref = (st[x].cpu().numpy().copy() for x in ("table", "len", "ref"))
    page = case["page"]
    k, v = st["k"].double(), st["v"].double()
    if case["op"] == "write":
        if case["admit"]:
            for s in st["seqs"].tolist():
                for c in range(-(-int(length[s]) // page)):
                    ref[table[s, c]] -= 1
                table[s], length[s] = -1, 0
            for s, new in zip(st["seqs"].tolist(), st["n_new"].tolist()):
                for c in range(-(-new // page)):
                    p = int(np.flatnonzero(ref == 0)[0])
                    table[s, c], ref[p] = p, 1
                length[s] = new
        ts, tp = st["token_seq"].cpu().numpy(), st["token_pos"].cpu().numpy()
        where = torch.from_numpy(table[ts, tp // page].astype(np.int64)).to(DEV)
        row = torch.from_numpy((tp % page).astype(np.int64)).to(DEV)
        # the stored value is the definition's too: x, or x over the scale rounded to 8 bits
        for pool, new, scale in ((k, st["new_k"], st["k_scale"]), (v, st["new_v"], st["v_scale"])):
            x = new.double() if scale is None else \
                _round_e4m3((new.double() / scale[0].double()[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX))
            for h in range(case["kv_heads"]):
                pool[0, where, h, row] = x[:, h]
        return {"k": k, "v": v, "table": table, "len": length, "ref": ref}
    if case["do"] == "fork":
        for s, d in zip(st["parents"].tolist(), st["dst"].tolist()):
            L = int(length[s])
            for c in range(L // page):
                table[d, c] = table[s, c]
        fresh = iter(np.flatnonzero(ref == 0).tolist())
        for s, d in zip(st["parents"].tolist(), st["dst"].tolist()):
            L = int(length[s])
            for c in range(L // page):
                ref[table[s, c]] += 1
            if L % page:
                p = next(fresh)
                k[:, p], v[:, p] = k[:, int(table[s, L // page])], v[:, int(table[s, L // page])]
                table[d, L // page], ref[p] = p, 1
            length[d] = L
        return {"k": k, "v": v, "table": table, "len": length, "ref": ref}
    n_live = int((ref > 0).sum())
    holes = [p for p in range(n_live) if ref[p] == 0]
    movers = [p for p in range(n_live, len(ref)) if ref[p] > 0]
    for a, b in zip(movers, holes):
        table[table == a] = b
        ref[b], ref[a] = ref[a], 0
        k[:, b], v[:, b] = k[:, a], v[:, a]
    return {"k": k, "v": v, "table": table, "ref": ref, "live": np.array([n_live], np.int32)}


def _round_e4m3(x):
    """x (float64, at most 448 in size) to the nearest E4M3 value, ties to even: steps of 2^(e-3), e >= -6."""
    a = x.abs()
    e = torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a)))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step
