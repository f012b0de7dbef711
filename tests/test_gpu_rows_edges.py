"""Rows read back out of the cache where the bounds of the sequences are not what they should be."""

import numpy as np
import pytest
import torch

import quantized_routed_expert_03_gb300 as qre
from quantized_routed_expert_03_gb300.attention import KVCache
from test_gpu_rows import DEV, TYPE, clean_status, i32, randn   # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "e2m1"])
@pytest.mark.parametrize("cu,total", [
    ([0, 100, 4, 8], 8),                      # one that ends behind the rows, one that ends before it begins, one that is right
    ([0, 5, 3, 3, 9], 9),                     # right, wrong, empty, and one that shares rows 3 and 4 with the first
    ([-7, 2, 30, 20, 25], 30),                # from below 0; right; wrong; right inside the second: rows of both
    ([9, 0, 4], 4),                           # the first begins behind all rows
    ([0, 4, -1, 6], 8),                       # a bound below 0 between two
    ([0] + [2 ** 31 - 1, 0] * 40 + [7], 7),   # many that are wrong
    ([0, 6] + [10 ** 9] * 300 + [6, 40], 40),   # more bounds than a CTA has threads
])
def test_sequences_beside_wrong_bounds_are_read(cu, total, cache):
    Hk, D, page, n = 2, 64, 16, len(cu) - 1
    c = KVCache(1, 4 * n, Hk, page, D, n, 4, TYPE[cache], device=DEV)
    seqs, lens = i32(range(n)), i32([50] * n)
    c.reserve(seqs, lens)
    pos = torch.arange(50, dtype=torch.int32, device=DEV)
    k, v = randn((n * 50, Hk, D), 1, "bf16"), randn((n * 50, Hk, D), 2, "bf16")
    c.write(0, seqs.repeat_interleave(50), pos.repeat(n), k, v)
    kr, vr = c.read(0, None, i32(np.arange(0, 50 * n + 1, 50)), 50 * n)      # what each has, by bounds that are right
    assert qre.qre_read_device_status() == 0
    ko, vo = (torch.full((total, Hk, D), 7.5, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    c.read(0, None, i32(cu), total, first=i32([1] * n), k=ko, v=vo)
    assert qre.qre_read_device_status() == qre.QRE_DEV_BAD_INDEX
    owners = [[s for s in range(n) if 0 <= cu[s] <= t < cu[s + 1] <= total] for t in range(total)]
    assert any(owners)
    for t, who in enumerate(owners):
        for got, rows in ((ko, kr), (vo, vr)):
            want = [rows[50 * s + 1 + t - cu[s]] for s in who] or [torch.full((Hk, D), 7.5, dtype=torch.bfloat16, device=DEV)]
            assert any(torch.equal(got[t], x) for x in want), (t, who)


def test_rows_that_nobody_has_stay_beside_many_sequences():
    """A padded result: right bounds, rows before the first sequence and behind the last."""
    Hk, D, n = 1, 64, 700
    c = KVCache(1, n, Hk, 16, D, n, 1, device=DEV)
    c.reserve(i32(range(n)), i32([3] * n))
    k, v = randn((3 * n, Hk, D), 1, "bf16"), randn((3 * n, Hk, D), 2, "bf16")
    c.write(0, i32(np.repeat(np.arange(n), 3)), i32(np.tile(np.arange(3), n)), k, v)
    total = 3 * n + 5000
    ko, vo = (torch.full((total, Hk, D), 7.5, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    c.read(0, None, i32(np.arange(11, 3 * n + 12, 3)), total, k=ko, v=vo)
    assert qre.qre_read_device_status() == 0
    assert torch.equal(ko[11:3 * n + 11], k) and torch.equal(vo[11:3 * n + 11], v)
    for x in (ko, vo):
        assert (x[:11] == 7.5).all() and (x[3 * n + 11:] == 7.5).all()
