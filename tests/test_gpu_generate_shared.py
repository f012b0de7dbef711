"""The example decoder with turned and normed heads, pages of 4 bits and samples that read their prompt's pages together:
every decode step's attention against fp64 on the rows that the pages hold, and the same tokens from CUDA graphs."""

import numpy as np
import pytest
import torch

import quantized_routed_expert_03_gb300 as qre
from oracle import attention as oatt
from test_gpu_generate import DEV, PROMPTS, example, npy   # noqa: F401

pytestmark = pytest.mark.gpu
KINDS = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e2m1": torch.float4_e2m1fn_x2}


@pytest.mark.parametrize("kind", ["bf16", "e2m1"])
def test_steps_of_shared_samples(example, kind):   # noqa: F811
    qre.qre_clear_device_status()
    model = example.Decoder(cache_dtype=KINDS[kind], device=DEV, rotary=True, shared=True, max_seqs=20, n_pages=300)
    H, Hk, D, samples = 4, 2, 64, 3
    prompts = [[(11 * i + 5 * j) % 500 for j in range(n)] for i, n in enumerate((1, 160, 290))]
    n = len(prompts)
    i32 = dict(dtype=torch.int32, device=DEV)
    seqs = torch.arange(n * samples, **i32)
    model.trace = []
    first = model.prefill(prompts, seqs[:n]).argmax(-1)
    # the prompts' attention, on the keys as they were turned
    lens = [len(p) for p in prompts]
    for layer, q, k, v, o in model.trace:
        q, k, v, o = (npy(x) for x in (q, k, v, o))
        ref = oatt.prefill(q, k, v, lens, lens, D ** -0.5)
        tol = oatt.tolerance(ref[0], ref[2], ref[3], max(lens), D, 2.0 ** -8, np.abs(v).max())
        assert (np.abs(o - ref[0]) <= tol).all()
    for s in range(1, samples):
        model.cache.fork(seqs[:n], seqs[s * n:(s + 1) * n].clone())
    order = torch.arange(n * samples, device=DEV).view(samples, n).t().reshape(-1)
    batch, cu = seqs[order], torch.arange(0, n * samples + 1, samples, **i32)
    assert model.cache.common_len(batch, cu).tolist() == [m // 16 * 16 for m in lens]
    tokens = first.repeat(samples)[order].to(torch.int32)
    for step in range(3):
        model.trace = []
        tokens = (model.step(tokens, batch, torch.ones_like(batch), cu).argmax(-1) + torch.arange(len(batch), device=DEV)).to(torch.int32) % 500
        held = model.cache.seq_len[batch].tolist()
        assert held == [lens[int(s) % n] + step + 1 for s in batch]
        ends = np.concatenate([[0], np.cumsum(held)])
        for layer, q, k, v, o in model.trace:
            q, o = npy(q), npy(o)
            rows = [npy(x) for x in model.cache.read(layer, batch, torch.tensor(ends, **i32), int(ends[-1]))]
            for i in range(len(batch)):
                kk, vv = (x[ends[i]:ends[i + 1]] for x in rows)
                for h in range(H):
                    ro, _, ra, rb = oatt.attend(q[i, h:h + 1], kk[:, h // 2], vv[:, h // 2], D ** -0.5, [0], [len(kk)])
                    tol = oatt.tolerance(ro, ra, rb, len(kk), D, 2.0 ** -8, np.abs(vv).max()) + len(kk) * 2.0 ** -33 * np.abs(vv).max()
                    assert (np.abs(o[i, h] - ro[0]) <= tol[0]).all()
    assert qre.qre_read_device_status() == 0


@pytest.mark.parametrize("kind", ["e4m3", "e2m1"])
def test_graphs_and_shared_pages_give_tokens(example, kind):   # noqa: F811
    out = []
    for graph in (False, True):
        model = example.Decoder(cache_dtype=KINDS[kind], device=DEV, rotary=True, shared=True)
        out.append(example.generate(model, PROMPTS, samples=3, steps=12, graph=graph))
        assert qre.qre_read_device_status() == 0
    assert torch.equal(out[0][0], out[1][0]) and out[0][1:] == out[1][1:]
    assert out[0][0].shape == (3, 25) and out[0][2] == 1 + 2 + 4       # pages as without sharing the reads
