"""pa_decode_shared where a group's members do not reach its prefix, where lengths are no
lengths, and where scores are so far apart that each row is one key's."""
import numpy as np
import pytest
import torch

from tests import window_ref as ref
from tests.test_gpu_shared import Case, lengths
from tests.test_gpu_shared_bits import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa(cuda_device):
    from paged_kv_cache_218_gb300 import binding
    binding.pa_device_error_flags()
    return binding


@pytest.mark.parametrize("nothing", [-1, 2**31 - 1])
def test_prefix_entries_that_no_member_sees(pa, nothing):
    """They may name anything, as those behind a length may in pa_decode: a group whose members
    all end early, or are empty, over several key tiles and pieces."""
    groups = [(20, [0, 5, 100, 33]), (90, [140, 17]), (9, [0, 0, 0]), (200, [0]), (64, [1, 0, 512])]
    c = Case(1, groups, 8, 4)
    tables, s = c.tables.cpu().numpy(), 0
    for p, members in groups:
        seen = (max(members) + 15) // 16
        tables[s:s + len(members), seen:] = nothing
        s += len(members)
    c.tables.copy_(torch.from_numpy(tables))
    c.run(pa)
    check(c)
    assert pa.pa_device_error_flags() == 0


@pytest.mark.parametrize("length", [-1, -(2**31), -(2**31) + 1, -(2**31) + 160])
@pytest.mark.parametrize("members", [3, 40, 70])
def test_lengths_below_zero(pa, length, members):
    """Flagged, and as empty as 0: zeros and -inf, no matter which member; the others stay."""
    rng = np.random.default_rng(members)
    c = Case(members, [(20, lengths(rng, members, 20, 30)), (3, [60, 50])], 8, 2, amp=0.3)
    bad = [0, members // 2, members + 1]
    c.lens[bad] = length
    c.run(pa)
    torch.cuda.synchronize()
    assert pa.pa_device_error_flags() == pa.PA_DEVERR_SEQ_LEN
    assert (c.out[bad] == 0).all() and (c.lse[bad] == -float("inf")).all()
    check(c, rows=[s for s in (1, members - 1, members) if s not in bad])


@pytest.mark.parametrize("members,G", [(4, 4), (20, 4), (60, 4)])
@pytest.mark.parametrize("scale", [1e9, 1e30, 1e36])
def test_rows_of_one_key(pa, members, G, scale):
    """Scores of 10^9 and more in log2 units: a row's output is the value of the key with its
    largest score, and its lse that score, wherever the next one is farther below than the dot
    product's 128 roundings (2^-23 of sum |q k| each)."""
    rng = np.random.default_rng(members)
    c = Case(members, [(40, lengths(rng, members, 40, 300)), (7, lengths(rng, 3, 7, 90))], 2 * G, 2,
             scale=scale)
    c.run(pa)
    assert pa.pa_device_error_flags() == 0
    q, lens, tables = ref.to64(c.q), c.lens.cpu().numpy(), c.tables.cpu().numpy()
    checked = 0
    for s in sorted({0, 1, members // 2, members - 1, members, members + 2}):
        n = int(lens[s])
        ids = torch.from_numpy(tables[s, :(n + 15) // 16].astype(np.int64)).cuda()
        k = ref.to64(c.kc[ids].flatten(0, 1)[:n])
        v = ref.to64(c.vc[ids].flatten(0, 1)[:n])
        for h in range(2 * G):
            x = k[:, h // G] @ q[s, h]
            off = 128 * 2.0**-23 * (np.abs(k[:, h // G]) @ np.abs(q[s, h])).max()
            order = np.argsort(-x)
            lse = x[order[0]] * scale
            assert abs(float(c.lse[s, h]) - lse) <= off * scale + 2.0**-21 * abs(lse)
            # (64 log2 units apart besides: no weight of the next one's is left)
            if x[order[0]] - x[order[1]] > 2 * off + 64 / scale:
                checked += 1
                want = v[order[0], h // G]
                ref.assert_within(c.out[s, h], want, 2.0**-8 * np.abs(want), (s, h))
    assert checked >= 3 * G
