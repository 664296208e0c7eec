"""pa_beam_reorder of rows that do not have blocks of their own: flagged, and nothing copied."""
import numpy as np
import pytest
import torch

from tests.test_gpu_beam_reorder import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa(cuda_device):
    from paged_kv_cache_218_gb300 import binding
    binding.pa_device_error_flags()
    return binding


@pytest.mark.parametrize("length", [37, 47, 32])
@pytest.mark.parametrize("pools", [True, False])
def test_rows_straight_from_a_fork(pa, length, pools):
    """Equal rows, the partly filled block among them: a second child would write into its
    sibling's.  At a block's end there is none yet, and nothing is wrong."""
    from paged_kv_cache_218_gb300.block_manager import BlockManager
    W = 4
    c = Case(1, 1, W, 2, 2, 64, lens=[length] * W, parents=[[0, 0, 2, 3]], width=5)
    bm = BlockManager(16, 16, prefix_caching=False)
    bm.add_sequence(0, list(range(length)))
    for w in range(1, W):
        bm.fork(0, w)
    tables, lens = bm.build_tables(list(range(W)), 5)
    tables = np.asarray(tables, np.int32)
    if length % 16 == 0:
        tables[:, 2] = 0  # (whatever the caller has there until it gives out blocks)
    c.dev[0].copy_(torch.from_numpy(tables))
    was = c.k.clone(), c.v.clone()
    c.run(pa, pools=pools)
    torch.cuda.synchronize()
    assert pa.pa_device_error_flags() == (pa.PA_DEVERR_BLOCK_ID if length % 16 else 0)
    assert torch.equal(c.bits(c.k), c.bits(was[0])) and torch.equal(c.bits(c.v), c.bits(was[1]))
    # every beam once: each keeps what it has, and nothing is wrong with that
    c.dev[2].copy_(torch.tensor([[2, 0, 3, 1]], dtype=torch.int32))
    c.run(pa, pools=pools)
    torch.cuda.synchronize()
    assert pa.pa_device_error_flags() == 0


def test_requests_of_a_padded_batch(pa):
    """Rows of nothing, all alike, without parents or each its own."""
    c = Case(2, 3, 4, 1, 2, 64, lens=[50] * 4 + [0] * 8,
             parents=[[1, 1, 0, 2], [-1] * 4, [0, 1, 2, 3]])
    c.tables[4:] = 0
    c.dev[0][4:] = 0
    c.expect()
    c.run(pa)
    c.check()
    assert pa.pa_device_error_flags() == 0


def test_two_of_many_alike(pa):
    """Only the child that would get such a block is left without its copy."""
    c = Case(3, 1, 5, 2, 2, 64, lens=[37] * 5, parents=[[0, 0, 0, 1, 1]], width=5)
    copies = c.expect()  # beams 2, 3, 4 give theirs away
    c.dev[0][3, 2] = int(c.tables[1, 2])  # old beam 3 has beam 1's
    at = [i for i, x in enumerate(copies) if x[1] == c.tables[3, 2]]
    assert len(at) == 1
    ref = [c.bits(p).clone() for p in (c.k, c.v)]
    for i, (source, target, n) in enumerate(copies):
        if i not in at:
            for p in ref:
                p[:, target, :n] = p[:, source, :n]
    c.run(pa)
    torch.cuda.synchronize()
    assert pa.pa_device_error_flags() == pa.PA_DEVERR_BLOCK_ID
    for p, r in zip((c.k, c.v), ref):
        assert torch.equal(c.bits(p), r)
