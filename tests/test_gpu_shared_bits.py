"""pa_decode_shared against 64-bit attention with weights rounded no further than to a sum of
two bf16 numbers: the prefix pass, each sequence's own part, and the one-launch way for narrow
tables alike."""
import numpy as np
import pytest
import torch

from tests import window_ref as ref
from tests.test_gpu_shared import Case, lengths

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa(cuda_device):
    from paged_kv_cache_218_gb300 import binding
    binding.pa_device_error_flags()
    return binding


def check(c, rows=None):
    """A weight p = hi + lo: hi is off by up to 2^-8 p, so lo is no larger than that, and off by
    2^-8 of itself: 2^-16 p."""
    q, lens, tables = ref.to64(c.q), c.lens.cpu().numpy(), c.tables.cpu().numpy()
    G = c.q.shape[1] // c.kc.shape[2]
    for s in range(len(lens)) if rows is None else rows:
        n = int(lens[s])
        ids = torch.from_numpy(tables[s, :(n + 15) // 16].astype(np.int64)).cuda()
        k = ref.to64(c.kc[ids].flatten(0, 1)[:n])
        v = ref.to64(c.vc[ids].flatten(0, 1)[:n])
        for h in range(c.q.shape[1]):
            out, lse, tol, tol_l = ref.attend(q[s, h], k[:, h // G], v[:, h // G], c.scale,
                                              2.0**-16)
            ref.assert_within(c.out[s, h], out, tol, ("out", s, h))
            ref.assert_within(c.lse[s, h], np.array(lse), np.array(tol_l), ("lse", s, h))


# (small queries and keys: a score's own error, 128 additions, stays far below a bf16 step)
@pytest.mark.parametrize("members,G", [(1, 4), (4, 4), (20, 4), (32, 4), (33, 4), (60, 2), (9, 7)])
@pytest.mark.parametrize("prefix", [1, 3, 8, 21])
def test_weights_over_the_prefix(pa, members, G, prefix):
    """Lone CTAs (16 query rows, 128) and pairs; a block, part of a tile, a tile, several."""
    rng = np.random.default_rng(members * 100 + prefix)
    c = Case(members * G + prefix, [(prefix, lengths(rng, members, prefix, 3)), (prefix, [])],
             2 * G, 2, amp=0.3)
    c.run(pa)
    check(c, rows=sorted({0, members // 2, members - 1}))


def test_members_that_end_inside_the_prefix(pa):
    c = Case(6, [(9, [1, 15, 17, 127, 128, 129, 144, 150]), (20, [0, 5, 100, 33])], 8, 4, amp=0.3)
    c.run(pa)
    check(c)


@pytest.mark.parametrize("small", [False, True])
def test_own_parts(pa, small):
    """Sequences in no group, groups without a prefix, own parts longer than the prefix."""
    rng = np.random.default_rng(7)
    c = Case(7, [(0, [0, 1, 16, 40]), (2, lengths(rng, 3, 2, 200))], 8, 2, loose=5, amp=0.3,
             small=small)
    c.run(pa)
    check(c)


def test_equal_weights_in_either_width_of_table(pa):
    """Narrow and wide tables take different kernels: the same output but for the order of
    their sums, and so but for the last bit of an output next to the middle of two."""
    rng = np.random.default_rng(8)
    groups = [(12, lengths(rng, 6, 12, 40)), (5, lengths(rng, 4, 5, 90))]
    a, b = (Case(8, groups, 8, 2, amp=0.3, small=small) for small in (False, True))
    a.run(pa)
    b.run(pa)
    assert torch.equal(a.q, b.q) and torch.equal(a.lens, b.lens)
    check(a)
    check(b)
    assert (a.out != b.out).float().mean() < 0.02
