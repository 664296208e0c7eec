"""pa_decode_shared where a group's members do not reach its prefix, and where lengths are no
lengths."""
import numpy as np
import pytest
import torch

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
