"""Decode attention with shared prefixes where its launches, its plan and its numbers are at an edge."""

import math

import numpy as np
import pytest
import torch

import quantized_routed_expert_03_gb300 as qre
from oracle import attention as oatt
from quantized_routed_expert_03_gb300.attention import Attention, KVCache
from test_gpu_rows import DEV, UNIT, clean_status, i32, npy, randn   # noqa: F401
from test_gpu_shared import Shared, check, run

pytestmark = pytest.mark.gpu


def test_own_positions_whose_places_pass_31_bits():
    """128 sequences that share nothing, 2^20 positions each on the same eight pages again and again, 256 KV heads: more
    than 2^31 places.  A softmax over 2^13 times the same 128 keys is the softmax over those keys, its log-sum log 2^13
    larger."""
    n, H, D, page, pages = 128, 256, 128, 16, 8
    cols = 2 ** 20 // page
    c = KVCache(1, pages, H, page, D, n, cols, device=DEV)
    c.k.copy_(randn(c.k.shape, 1, "bf16"))
    c.v.copy_(randn(c.v.shape, 2, "bf16"))
    c.page_table.copy_((torch.arange(cols, device=DEV) % pages).int().expand(n, cols))
    q = randn((n, H, D), 3, "bf16")
    c.seq_len.fill_(pages * page)
    short = torch.empty((n, H), device=DEV)
    want = Attention(c, 0, H, n).decode(q, None, lse=short)
    c.seq_len.fill_(page * cols)
    att = Attention(c, 0, H, n, max_groups=n)
    lse = torch.full((n, H), float("nan"), device=DEV)
    o = att.decode_shared(q, None, torch.arange(n + 1, dtype=torch.int32, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV), lse=lse)
    assert qre.qre_read_device_status() == 0
    # Sums of up to 2^16 chunks one after the other, each step off by at most 2^-23 of the sum (a sum that is cut off, not
    # rounded): 2^-7, of the sum and of O; bf16 weights and results on both sides, 2^-8 each time
    assert float((lse - short - math.log(2 ** 13)).abs().max()) <= 2.0 ** -7 + 1e-4
    size = float(c.v.float().abs().max())
    assert float((o.float() - want.float()).abs().max()) <= size * (2 * 2.0 ** -7 + 4 * 2.0 ** -8)
