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


def test_blocks_reserved_with_the_block_manager(pa):
    """The way the header names: sequences of as many tokens as a beam may still get, their
    blocks behind the prompt's full ones; beam 0 has the prompt's partly filled one in front."""
    from paged_kv_cache_218_gb300.block_manager import BlockManager
    W, prompt, steps, own = 4, 37, 40, 3
    rng = np.random.default_rng(4)
    bm = BlockManager(32, 16, prefix_caching=False)
    bm.add_sequence(0, list(range(prompt)))
    for w in range(W):
        bm.add_sequence(1 + w, [0] * (16 * own))
    rows, _ = bm.build_tables(list(range(W + 1)), 8)
    bm.end_step()
    width, full = 8, prompt // 16
    tables = np.full((W, width), -1, np.int32)
    for w in range(W):
        line = ([int(rows[0][full])] if w == 0 else []) + [int(b) for b in rows[1 + w][:own]]
        # (beams not begun: of length 0, their own blocks from column 0 on)
        line = [int(b) for b in rows[0][:full]] + line if w == 0 else line
        tables[w, :len(line)] = line
    k = torch.zeros((1, 32, 16, 1, 64), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    for t in range(prompt):
        k[0, int(tables[0, t // 16]), t % 16] = float(t % 128)
    history = [[t % 128 for t in range(prompt)]] + [[] for _ in range(W - 1)]
    tb = torch.from_numpy(tables).cuda()
    lens = torch.tensor([prompt, 0, 0, 0], dtype=torch.int32, device="cuda")
    out_t, out_l = torch.empty_like(tb), torch.empty_like(lens)
    for step in range(steps):
        parents = [0] * W if step == 0 else rng.integers(0, W, W).tolist()
        pa.pa_beam_reorder(out_t, out_l, tb, lens,
                           torch.tensor([parents], dtype=torch.int32, device="cuda"), k, v)
        assert pa.pa_device_error_flags() == 0
        tb, out_t = out_t, tb
        lens.copy_(out_l + 1)
        history = [history[p] + [int(rng.integers(0, 128))] for p in parents]
        host = tb.cpu().numpy()
        for w in range(W):
            n = len(history[w])
            assert int(lens[w]) == n
            k[0, int(host[w, (n - 1) // 16]), (n - 1) % 16] = float(history[w][-1])
        for w in range(W):
            got = k[0, torch.from_numpy(host[w, :(n + 15) // 16].astype(np.int64)).cuda(), :, 0, 0]
            assert got.flatten()[:n].int().tolist() == history[w]
    for s in range(W + 1):
        bm.free_sequence(s)
    bm.end_step()
    assert bm.num_free_blocks() == 32
