"""The example decoder: every attention it makes, over forked, freed and compacted pages, against fp64 on the rows that
its own projections gave; and the same tokens with and without CUDA graphs."""

import importlib.util
import pathlib

import numpy as np
import pytest
import torch

import quantized_routed_expert_03_gb300 as qre
from oracle import attention as oatt

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def example():
    path = pathlib.Path(__file__).resolve().parent.parent / "examples" / "generate.py"
    spec = importlib.util.spec_from_file_location("example_generate", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def npy(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def close(o, ref, n_keys, v_max):
    ro, _, ra, rb = ref
    tol = oatt.tolerance(ro, ra, rb, n_keys, ro.shape[-1], 2.0 ** -8, v_max)
    assert (np.abs(o - ro) <= tol).all(), (np.abs(o - ro) - tol).max()


PROMPTS = [[(11 * i + 5 * j) % 500 for j in range(n)] for i, n in enumerate((1, 16, 45))]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attention_of_a_generation(example, kind):
    qre.qre_clear_device_status()
    model = example.Decoder(cache_dtype=torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16, device=DEV)
    model.trace = []
    H, Hk, D, n, samples, steps = 4, 2, 64, 3, 2, 18
    example.generate(model, PROMPTS, samples=samples, steps=steps, graph=False)
    assert qre.qre_read_device_status() == 0
    scale, lens = D ** -0.5, [len(p) for p in PROMPTS]

    def stored(x):                                  # what the cache keeps of a row
        return x if kind == "bf16" else oatt.e4m3_round(x * 32.0) / 32.0

    calls = iter(model.trace)
    rows = [{} for _ in range(2)]                   # layer -> sequence -> [k rows], [v rows]
    for l in range(2):
        layer, q, k, v, o = next(calls)
        assert layer == l
        q, k, v, o = npy(q), npy(k), npy(v), npy(o)
        close(o, oatt.prefill(q, k, v, lens, lens, scale), max(lens), np.abs(v).max())
        for i, a in enumerate(np.concatenate([[0], np.cumsum(lens)])[:-1]):
            for s in range(samples):
                rows[l][i + s * n] = [stored(k[a:a + lens[i]]), stored(v[a:a + lens[i]])]
    seqs = list(range(n * samples))
    for step in range(2 * steps):
        for l in range(2):
            layer, q, k, v, o = next(calls)
            assert layer == l
            q, k, v, o = npy(q), npy(k), npy(v), npy(o)
            if step == steps and l == 0:            # the kept ones are known by their number of rows written
                seqs = [int(s) for s in np.flatnonzero(model.cache.seq_len.cpu().numpy())]
                seqs.sort(key=lambda s: s % n)
                assert len(seqs) == n
            for i, s in enumerate(seqs):
                kk, vv = rows[l][s]
                kk, vv = np.concatenate([kk, stored(k[i:i + 1])]), np.concatenate([vv, stored(v[i:i + 1])])
                rows[l][s] = [kk, vv]
                ref = [np.zeros((1, H, D)), np.zeros((1, H)), np.zeros((1, H, D)), np.zeros((1, H))]
                for h in range(H):
                    r = oatt.attend(q[i, h:h + 1], kk[:, h // 2], vv[:, h // 2], scale, [0], [len(kk)])
                    for dst, x in zip(ref, r):
                        dst[0, h] = x[0]
                close(o[i:i + 1], ref, len(kk), np.abs(vv).max())
    assert next(calls, None) is None
    # every kept sequence holds its prompt and all its tokens, on pages 0 .. live - 1 (then one more page a step)
    assert [int(model.cache.seq_len[s]) for s in seqs] == [m + 2 * steps for m in lens]


def test_graphs_give_the_same_tokens(example):
    out = []
    for graph in (False, True):
        model = example.Decoder(device=DEV)
        tokens, live1, live2 = example.generate(model, PROMPTS, samples=3, steps=12, graph=graph)
        assert qre.qre_read_device_status() == 0
        out.append(tokens)
        # full prompt pages are shared: 16 positions a page, prompts of 1, 16 and 45 tokens, 12 written behind each
        assert live1 == 3 * 1 + (1 + 3 * 1) + (2 + 3 * 2)
        assert live2 == 1 + 2 + 4
    assert torch.equal(out[0], out[1])
