"""The paged cache's bookkeeping where a call asks for more than the pool has, or sums pass 32 bits."""

import numpy as np
import pytest
import torch

import quantized_routed_expert_03_gb300 as qre
from test_gpu_kv_cache import DEV, Cache, clean_status, i32  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_pages,wants", [(64, [40, 40, 40]), (16, [3, 20, 1, 0, 2]), (10, [11, 1, 0, 12]), (9, [9, 1, 1])])
def test_requests_behind_the_end_of_the_pool(n_pages, wants):
    """The sum of the wants passes the pool in the middle of the list, by more than a page: what needs a page behind that
    place stays as it was."""
    c = Cache(n_pages, 16, len(wants) + 1, 64)
    failed = c.reserve(range(len(wants)), [16 * w - 5 if w else 0 for w in wants])
    assert failed and qre.qre_read_device_status() == qre.QRE_DEV_NO_PAGE
    c.check()
    qre.qre_clear_device_status()
    # positions inside the last page need none; a further request finds what is left
    c.reserve([i for i in range(len(wants)) if i not in failed], [4] * (len(wants) - len(failed)))
    c.check()
    c.reserve(failed, [16 * n_pages] + [1] * (len(failed) - 1))
    c.check()


@pytest.mark.parametrize("n_pages,page,max_pages", [(37, 16, 30), (1500, 32, 640)])
def test_random_life_of_a_cache_that_runs_out(n_pages, page, max_pages):
    rng = np.random.default_rng(n_pages)
    S, passed = 24, 0
    c = Cache(n_pages, page, S, max_pages, heads=1)
    for step in range(60):
        m = c.model
        empty, full = np.flatnonzero(m.length == 0), np.flatnonzero(m.length > 0)
        what = rng.integers(5)
        if what <= 1:
            seqs = rng.permutation(S)[:rng.integers(1, S + 1)]
            new = rng.integers(0, page * max_pages // 2 + 1, len(seqs)) * rng.integers(0, 2, len(seqs))
            passed += int((-(-(m.length[seqs] + new) // page) - -(-m.length[seqs] // page)).sum() > n_pages + 1)
            c.reserve(seqs, new)
        elif what == 2 and len(full) and len(empty):
            n = rng.integers(1, len(empty) + 1)
            c.fork(rng.choice(full, n), rng.permutation(empty)[:n])
        elif what >= 3 and len(full):
            c.free(rng.permutation(full)[:rng.integers(1, len(full) + 1)])
        c.check()
    assert passed >= 5                                       # calls whose wants pass the whole pool
    assert qre.qre_read_device_status() & ~qre.QRE_DEV_NO_PAGE == 0


@pytest.mark.parametrize("small", [0, 3])
def test_reserve_whose_needs_pass_32_bits(small):
    """1024 requests of 2^21 pages each (2^31 in all), behind a few that fit a pool of 50."""
    S, max_pages, page, n_pages = 1024 + small, 1 << 21, 16, 50
    pool = torch.empty((1, n_pages, 1, page, 64), dtype=torch.bfloat16, device=DEV)
    table = torch.full((S, max_pages), -1, dtype=torch.int32, device=DEV)
    ln, ref = torch.zeros(S, dtype=torch.int32, device=DEV), torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    c = qre.make_kv_cache(pool, pool, table, ln, ref, qre.QRE_BF16)
    ws = torch.full((qre.qre_kv_workspace_size(c),), 0xA5, dtype=torch.uint8, device=DEV)
    qre.qre_kv_reserve(c, S, i32(range(S)), i32([page * 2] * small + [page * max_pages] * 1024), ws)
    assert qre.qre_read_device_status() == qre.QRE_DEV_NO_PAGE
    assert ln.tolist() == [page * 2] * small + [0] * 1024
    assert ref.tolist() == [1] * (2 * small) + [0] * (n_pages - 2 * small)
    assert table[:small, :2].flatten().tolist() == list(range(2 * small))
    assert int((table >= 0).sum()) == 2 * small
