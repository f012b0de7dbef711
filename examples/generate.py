"""A small decoder with routed experts generates text from several prompts, several samples each.

Shows the paged cache, prefill and decode attention and the MoE layer as a server uses them:

  * the prompts go through the model in one packed call; keys and values are attended to as
    they come from the projection and written into pages on the way;
  * each prompt is forked into its samples, which share the prompt's full pages;
  * decode steps run in a CUDA graph: the lengths and pages live on the device, so one graph
    serves all steps;
  * all but the best sample of each prompt are freed, the pages are compacted, and the rest
    goes on.

With --rotary the heads of queries and keys are normed and turned by their positions on the way
into the pages; with --shared the samples of a prompt read the pages that they share together.

Weights are random (there is no tokenizer either: tokens are numbers).  The norms of the residual
stream, the projections and the residual stream itself are plain PyTorch.

    python examples/generate.py [--cache e4m3 | e2m1] [--rotary] [--shared] [--steps 24]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_routed_expert_03_gb300 as qre                                    # noqa: E402
from quantized_routed_expert_03_gb300.attention import Attention, KVCache, Rotary # noqa: E402
from quantized_routed_expert_03_gb300.layer import ExpertArena, MoELayer          # noqa: E402


class Decoder:
    def __init__(self, hidden=256, inter=128, experts=16, top_k=4, group=32, heads=4, kv_heads=2, head_dim=64,
                 layers=2, vocab=500, page=16, n_pages=200, max_seqs=16, max_pages=32, t_max=512,
                 cache_dtype=torch.bfloat16, seed=0, device="cuda:0", rotary=False, shared=False):
        dev = torch.device(device)
        g = torch.Generator(device=dev).manual_seed(seed)

        def rand(*shape, scale=1.0):
            return torch.randn(shape, generator=g, device=dev) * scale

        self.device, self.heads, self.kv_heads, self.head_dim = dev, heads, kv_heads, head_dim
        scales = None
        if cache_dtype == torch.float8_e4m3fn:   # E4M3 holds values up to 448; keys here are a few units large
            scales = torch.full((layers, kv_heads), 1 / 32, device=dev)
        self.shared = shared
        self.rotary = None
        if rotary:
            self.rotary = Rotary(heads, kv_heads, head_dim, q_norm=torch.ones(head_dim, device=dev),
                                 k_norm=torch.ones(head_dim, device=dev), device=dev)
        self.cache = KVCache(layers, n_pages, kv_heads, page, head_dim, max_seqs, max_pages, cache_dtype, scales,
                             scales, dev)
        self.embed = rand(vocab, hidden).bfloat16()
        self.w_out = rand(hidden, vocab, scale=hidden ** -0.5).bfloat16()
        self.layers = []
        for l in range(layers):
            arena = ExpertArena(hidden, inter, group, experts + 1, device=dev)
            for e in range(experts + 1):
                arena.quantize_into(e, rand(inter, hidden, scale=hidden ** -0.5),
                                    rand(inter, hidden, scale=hidden ** -0.5), rand(hidden, inter, scale=inter ** -0.5))
            moe = MoELayer(hidden, inter, experts, top_k, group, t_max, device=dev)
            moe.set_slots([arena.addresses(e) + (0,) for e in range(experts + 1)])
            self.layers.append(dict(
                w_qkv=rand(hidden, (heads + 2 * kv_heads) * head_dim, scale=hidden ** -0.5).bfloat16(),
                w_o=rand(heads * head_dim, hidden, scale=(heads * head_dim) ** -0.5).bfloat16(),
                w_router=rand(experts, hidden, scale=hidden ** -0.5), arena=arena, moe=moe,
                attention=Attention(self.cache, l, heads, max_seqs, max_groups=max_seqs if shared else 0)))
        self.trace = None    # a list: gets (layer, q, k, v, o) of every attention

    def _write(self, layer, token_seq, token_pos, q, k, v):
        """Keys and values into the pages; the queries and keys that attention takes."""
        if self.rotary is not None:
            return self.cache.write_rope(layer, self.rotary, token_seq, token_pos, q, k, v)
        self.cache.write(layer, token_seq, token_pos, k, v)
        return q, k

    def _forward(self, tokens, attend):
        """attend(layer's Attention, q, k, v) -> q, k, o writes the cache and attends."""
        x = self.embed[tokens]
        T, split = x.shape[0], (self.heads, self.kv_heads, self.kv_heads)
        for l, p in enumerate(self.layers):
            qkv = F.rms_norm(x, x.shape[1:]) @ p["w_qkv"]
            q, k, v = qkv.view(T, -1, self.head_dim).split(split, 1)     # strided views: nothing is copied
            q, k, o = attend(p["attention"], q, k, v)
            if self.trace is not None:
                self.trace.append((l, q.clone(), k.clone(), v.clone(), o.clone()))
            x = x + o.view(T, -1) @ p["w_o"]
            p["moe"].forward(F.rms_norm(x, x.shape[1:]), p["w_router"], None, T)
            x = x + p["moe"].y_bf16[:T]
        return x

    def _logits(self, x):
        return (F.rms_norm(x, x.shape[1:]) @ self.w_out).float()

    def prefill(self, prompts, seqs):
        """prompts: lists of tokens, for the empty sequences ``seqs``; the logits after each prompt."""
        i32 = dict(dtype=torch.int32, device=self.device)
        lens = torch.tensor([len(p) for p in prompts], **i32)
        cu = F.pad(lens.cumsum(0, dtype=torch.int32), (1, 0))
        tokens = torch.tensor(sum(prompts, []), **i32)
        token_seq = torch.repeat_interleave(seqs, lens)
        token_pos = torch.arange(tokens.numel(), **i32) - torch.repeat_interleave(cu[:-1], lens)
        self.cache.reserve(seqs, lens)

        def attend(att, q, k, v):
            q, k = self._write(att.layer, token_seq, token_pos, q, k, v)
            return q, k, att.prefill(q, k, v, cu, cu)

        return self._logits(self._forward(tokens, attend)[cu[1:] - 1])

    def step(self, tokens, seqs, ones, cu_group=None):
        """One new token for each of ``seqs`` (ones: as many int32 ones); the logits after it.  cu_group: groups of
        neighbours in ``seqs`` that share pages."""
        pos = self.cache.seq_len[seqs]
        self.cache.reserve(seqs, ones)
        common = None if cu_group is None else self.cache.common_len(seqs, cu_group)

        def attend(att, q, k, v):
            q, k = self._write(att.layer, seqs, pos, q, k, v)
            return q, k, att.decode(q, seqs) if common is None else att.decode_shared(q, seqs, cu_group, common)

        return self._logits(self._forward(tokens, attend))


class Sampler:
    """Greedy continuation of a set of sequences: tokens so far and their log-probability."""

    def __init__(self, model, seqs, tokens, score, graph=True, cu_group=None):
        self.model, self.seqs, self.use_graph, self.cu_group = model, seqs, graph, cu_group
        self.tokens, self.score = tokens.to(torch.int32).clone(), score.clone()
        self.ones = torch.ones_like(seqs)
        self.graph = None

    def _step(self):
        logp = F.log_softmax(self.model.step(self.tokens, self.seqs, self.ones, self.cu_group), -1)
        best = logp.max(-1)
        self.score += best.values
        self.tokens.copy_(best.indices)

    def run(self, steps):
        """[steps, sequences]: the tokens taken."""
        out = []
        for _ in range(steps):
            if self.graph is not None:
                self.graph.replay()
            else:
                self._step()             # the first step runs as it is (it also warms up what PyTorch loads lazily)
                if self.use_graph:
                    torch.cuda.synchronize()
                    self.graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(self.graph):
                        self._step()     # recorded, not run
            out.append(self.tokens.clone())
        return torch.stack(out)


def generate(model, prompts, samples=3, steps=24, graph=True):
    """Each prompt's best of ``samples`` continuations: tokens [prompts][2 * steps + 1], pages in use before and after."""
    n, dev, cache = len(prompts), model.device, model.cache
    seqs = torch.arange(n * samples, dtype=torch.int32, device=dev)    # prompt i's samples: i, i + n, i + 2 n, ...
    logp = F.log_softmax(model.prefill(prompts, seqs[:n]), -1)
    first = logp.topk(samples, -1)
    for s in range(1, samples):
        cache.fork(seqs[:n], seqs[s * n:(s + 1) * n].clone())    # arrays begin at 16-byte boundaries
    # the order of the batch: with shared pages read together, a prompt's samples side by side
    order, cu_group = torch.arange(n * samples, device=dev), None
    if model.shared:
        order = order.view(samples, n).t().reshape(-1)
        cu_group = torch.arange(0, n * samples + 1, samples, dtype=torch.int32, device=dev)
    back = torch.argsort(order)
    run = Sampler(model, seqs[order], first.indices.t().reshape(-1)[order], first.values.t().reshape(-1)[order], graph,
                  cu_group)
    begin = run.tokens[back].clone()
    part1 = run.run(steps)[:, back]
    live1 = cache.compact().clone()

    best = run.score[back].view(samples, n).argmax(0)
    keep = (best * n + torch.arange(n, device=dev)).to(torch.int32)
    drop = torch.ones(n * samples, dtype=torch.bool, device=dev)
    drop[keep.long()] = False
    cache.free(seqs[drop])
    live2 = cache.compact().clone()
    rest = Sampler(model, keep, run.tokens[back][keep.long()], run.score[back][keep.long()], graph)
    part2 = rest.run(steps)
    tokens = torch.cat([begin[None], part1])[:, keep.long()]
    return torch.cat([tokens, part2]).t().cpu(), int(live1), int(live2)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--cache", choices=["bf16", "e4m3", "e2m1"], default="bf16")
    ap.add_argument("--rotary", action="store_true")
    ap.add_argument("--shared", action="store_true")
    ap.add_argument("--steps", type=int, default=24)
    args = ap.parse_args()
    kinds = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e2m1": torch.float4_e2m1fn_x2}
    model = Decoder(cache_dtype=kinds[args.cache], rotary=args.rotary, shared=args.shared)
    prompts = [[(7 * i + 3 * j) % 500 for j in range(n)] for i, n in enumerate((5, 33, 70, 16))]
    tokens, live1, live2 = generate(model, prompts, steps=args.steps)
    status = qre.qre_read_device_status()
    for p, t in zip(prompts, tokens.tolist()):
        print(f"prompt of {len(p):3d} tokens ->", *t)
    print(f"pages in use: {live1} with all samples, {live2} after all but the best were freed; device status {status:#x}")
    return 1 if status else 0


if __name__ == "__main__":
    sys.exit(main())
