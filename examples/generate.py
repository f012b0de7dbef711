"""A small decoder with routed experts generates text from several prompts, several samples each.

Shows the paged cache, prefill and decode attention and the MoE layer as a server uses them:

  * the prompts go through the model in one packed call; keys and values are attended to as
    they come from the projection and written into pages on the way;
  * each prompt is forked into its samples, which share the prompt's full pages;
  * decode steps run in a CUDA graph: the lengths and pages live on the device, so one graph
    serves all steps;
  * all but the best sample of each prompt are freed, the pages are compacted, and the rest
    goes on.

Weights are random (there is no tokenizer either: tokens are numbers).  Norms, projections and
the residual stream are plain PyTorch.

    python examples/generate.py [--cache e4m3] [--steps 24]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_routed_expert_03_gb300 as qre                                    # noqa: E402
from quantized_routed_expert_03_gb300.attention import Attention, KVCache         # noqa: E402
from quantized_routed_expert_03_gb300.layer import ExpertArena, MoELayer          # noqa: E402


class Decoder:
    def __init__(self, hidden=256, inter=128, experts=16, top_k=4, group=32, heads=4, kv_heads=2, head_dim=64,
                 layers=2, vocab=500, page=16, n_pages=200, max_seqs=16, max_pages=32, t_max=512,
                 cache_dtype=torch.bfloat16, seed=0, device="cuda:0"):
        dev = torch.device(device)
        g = torch.Generator(device=dev).manual_seed(seed)

        def rand(*shape, scale=1.0):
            return torch.randn(shape, generator=g, device=dev) * scale

        self.device, self.heads, self.kv_heads, self.head_dim = dev, heads, kv_heads, head_dim
        scales = None
        if cache_dtype == torch.float8_e4m3fn:   # E4M3 holds values up to 448; keys here are a few units large
            scales = torch.full((layers, kv_heads), 1 / 32, device=dev)
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
                attention=Attention(self.cache, l, heads, max_seqs)))
        self.trace = None    # a list: gets (layer, q, k, v, o) of every attention

    def _forward(self, tokens, attend):
        """attend(layer's Attention, q, k, v) -> o writes the cache and attends."""
        x = self.embed[tokens]
        T, split = x.shape[0], (self.heads, self.kv_heads, self.kv_heads)
        for l, p in enumerate(self.layers):
            qkv = F.rms_norm(x, x.shape[1:]) @ p["w_qkv"]
            q, k, v = qkv.view(T, -1, self.head_dim).split(split, 1)     # strided views: nothing is copied
            o = attend(p["attention"], q, k, v)
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
            self.cache.write(att.layer, token_seq, token_pos, k, v)
            return att.prefill(q, k, v, cu, cu)

        return self._logits(self._forward(tokens, attend)[cu[1:] - 1])

    def step(self, tokens, seqs, ones):
        """One new token for each of ``seqs`` (ones: as many int32 ones); the logits after it."""
        pos = self.cache.seq_len[seqs]
        self.cache.reserve(seqs, ones)

        def attend(att, q, k, v):
            self.cache.write(att.layer, seqs, pos, k, v)
            return att.decode(q, seqs)

        return self._logits(self._forward(tokens, attend))


class Sampler:
    """Greedy continuation of a set of sequences: tokens so far and their log-probability."""

    def __init__(self, model, seqs, tokens, score, graph=True):
        self.model, self.seqs, self.use_graph = model, seqs, graph
        self.tokens, self.score = tokens.to(torch.int32).clone(), score.clone()
        self.ones = torch.ones_like(seqs)
        self.graph = None

    def _step(self):
        logp = F.log_softmax(self.model.step(self.tokens, self.seqs, self.ones), -1)
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
    run = Sampler(model, seqs, first.indices.t().reshape(-1), first.values.t().reshape(-1), graph)
    begin = run.tokens.clone()
    part1 = run.run(steps)
    live1 = cache.compact().clone()

    best = run.score.view(samples, n).argmax(0)
    keep = (best * n + torch.arange(n, device=dev)).to(torch.int32)
    drop = torch.ones(n * samples, dtype=torch.bool, device=dev)
    drop[keep.long()] = False
    cache.free(seqs[drop])
    live2 = cache.compact().clone()
    rest = Sampler(model, keep, run.tokens[keep.long()], run.score[keep.long()], graph)
    part2 = rest.run(steps)
    tokens = torch.cat([begin[None], part1])[:, keep.long()]
    return torch.cat([tokens, part2]).t().cpu(), int(live1), int(live2)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--cache", choices=["bf16", "e4m3"], default="bf16")
    ap.add_argument("--steps", type=int, default=24)
    args = ap.parse_args()
    model = Decoder(cache_dtype=torch.float8_e4m3fn if args.cache == "e4m3" else torch.bfloat16)
    prompts = [[(7 * i + 3 * j) % 500 for j in range(n)] for i, n in enumerate((5, 33, 70, 16))]
    tokens, live1, live2 = generate(model, prompts, steps=args.steps)
    status = qre.qre_read_device_status()
    for p, t in zip(prompts, tokens.tolist()):
        print(f"prompt of {len(p):3d} tokens ->", *t)
    print(f"pages in use: {live1} with all samples, {live2} after all but the best were freed; device status {status:#x}")
    return 1 if status else 0


if __name__ == "__main__":
    sys.exit(main())
