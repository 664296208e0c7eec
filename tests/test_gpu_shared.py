"""pa_decode_shared against 64-bit attention over each sequence's own keys, with the
roundings of window_ref (weights over the prefix are rounded to bf16)."""
import numpy as np
import pytest
import torch

from tests import window_ref as ref

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def pa(cuda_device):
    from paged_kv_cache_218_gb300 import binding
    binding.pa_device_error_flags()
    return binding


class Case:
    """groups: (shared blocks, [lengths of the members]).  Every slot that no sequence sees is
    NaN, and table entries of blocks without one are ids outside the pool.  Tables are so
    wide that the call takes the prefix apart; small: as narrow as they can be."""

    def __init__(self, seed, groups, Hq, Hkv, loose=0, scale=None, amp=1.0, small=False):
        rng = np.random.default_rng(seed)
        lens = [n for _, m in groups for n in m] + [int(rng.integers(0, 90)) for _ in range(loose)]
        S = len(lens)
        width = max([1] + [p for p, m in groups] + [(n + 15) // 16 for n in lens]) + 1
        if not small:  # more than 96 MB
            width = max(width, (96 << 20) // (S * Hkv * 8192) + 1)
        tables = np.full((S, width), -7, dtype=np.int64)
        tables[:, 1::2] = 2**31 - 1
        seen = []  # of each block given out
        s = 0

        def block(tokens):
            seen.append(tokens)
            return len(seen) - 1

        for p, members in groups:
            longest = max(members, default=0)
            prefix = [block(min(16, max(0, longest - 16 * j))) for j in range(p)]
            for n in members:
                tables[s, :p] = prefix
                for j in range(p, (n + 15) // 16):
                    tables[s, j] = block(min(16, n - 16 * j))
                s += 1
        for n in lens[s:]:
            for j in range((n + 15) // 16):
                tables[s, j] = block(min(16, n - 16 * j))
            s += 1
        used = len(seen)
        place = rng.permutation(used + 3)[:used]
        mine = (tables >= 0) & (tables < 2**31 - 1)
        tables[mine] = place[tables[mine]]
        kc = (amp * rng.standard_normal((used + 3, 16, Hkv, D))).astype(np.float32)
        vc = rng.standard_normal((used + 3, 16, Hkv, D)).astype(np.float32)
        hidden = np.ones((used + 3, 16), dtype=bool)
        for b, n in enumerate(seen):
            hidden[place[b], :n] = False
        kc[hidden] = np.nan
        vc[hidden] = np.nan
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.kc, self.vc = dev(kc).bfloat16(), dev(vc).bfloat16()
        self.tables, self.lens = dev(tables.astype(np.int32)), dev(np.array(lens, np.int32))
        self.q = dev((amp * rng.standard_normal((S, Hq, D))).astype(np.float32)).bfloat16()
        cu = np.concatenate([[0], np.cumsum([len(m) for _, m in groups])])
        self.offsets = dev(cu.astype(np.int32))
        self.shared = dev(np.array([p for p, _ in groups], np.int32))
        self.max_group = max([1] + [len(m) for _, m in groups])
        self.scale = D**-0.5 if scale is None else scale
        self.out = torch.full_like(self.q, float("nan"))
        self.lse = torch.full((S, Hq), float("nan"), device="cuda")
        self.ws = None

    def workspace(self, pa, fill=0xFF):
        S, Hq, _ = self.q.shape
        return torch.full((pa.pa_decode_shared_workspace_size(
            S, self.shared.shape[0], self.max_group, Hq, self.kc.shape[2], D),), fill,
            dtype=torch.uint8, device="cuda")

    def run(self, pa, stream=None):
        if self.ws is None:
            self.ws = self.workspace(pa)  # (any content: NaN here)
        pa.pa_decode_shared(self.out, self.q, self.kc, self.vc, self.tables, self.lens,
                            self.offsets, self.max_group, self.shared, self.scale, self.ws,
                            out_lse=self.lse, stream=stream)

    def check(self, rows=None):
        q, lens = ref.to64(self.q), self.lens.cpu().numpy()
        tables = self.tables.cpu().numpy()
        G = self.q.shape[1] // self.kc.shape[2]
        for s in range(len(lens)) if rows is None else rows:
            n = int(lens[s])
            ids = torch.from_numpy(tables[s, :(n + 15) // 16].astype(np.int64)).cuda()
            k = ref.to64(self.kc[ids].flatten(0, 1)[:n])
            v = ref.to64(self.vc[ids].flatten(0, 1)[:n])
            for h in range(self.q.shape[1]):
                # each weight off by 2^-8 of itself: the output by at most 2^-8 sum w |v| / sum w,
                # here bounded by 2^-8 max |v|
                out, lse, tol, tol_l = ref.attend(q[s, h], k[:, h // G], v[:, h // G], self.scale,
                                                  2.0**-8)
                ref.assert_within(self.out[s, h], out, tol, ("out", s, h))
                ref.assert_within(self.lse[s, h], np.array(lse), np.array(tol_l), ("lse", s, h))


def lengths(rng, n, prefix, most):
    return [16 * prefix + int(x) for x in rng.integers(0, most + 1, n)]


@pytest.mark.parametrize("G,Hkv", [(1, 2), (2, 1), (3, 3), (4, 8), (5, 1), (6, 2), (7, 1), (8, 2)])
def test_groups_of_heads(pa, G, Hkv):
    rng = np.random.default_rng(G)
    c = Case(G, [(9, lengths(rng, 5, 9, 40)), (17, lengths(rng, 3, 17, 70))], G * Hkv, Hkv)
    c.run(pa)
    c.check()
    assert pa.pa_device_error_flags() == 0


@pytest.mark.parametrize("prefix", [0, 1, 2, 7, 8, 9, 15, 16, 17, 64])
@pytest.mark.parametrize("members", [1, 2, 33])
def test_prefix_and_group_sizes(pa, prefix, members):
    rng = np.random.default_rng(prefix * 100 + members)
    c = Case(prefix, [(prefix, lengths(rng, members, prefix, 50))], 8, 2)
    c.run(pa)
    c.check()


@pytest.mark.parametrize("members", [16, 17, 31, 32, 33, 63, 64, 65, 129, 200])
def test_groups_past_a_tile_and_a_pair(pa, members):
    """32 members of four heads fill a query tile, 64 a pair's two (16 and fewer leave half
    a tile free)."""
    rng = np.random.default_rng(members)
    c = Case(members, [(11, lengths(rng, members, 11, 30))], 8, 2)
    c.run(pa)
    c.check(rows=sorted({0, 1, min(30, members - 1), members - 1, members // 2,
                         min(31, members - 1), min(32, members - 1), min(63, members - 1),
                         min(64, members - 1)}))


@pytest.mark.parametrize("G,members", [(4, 1), (4, 4), (4, 5), (8, 2), (8, 3), (1, 16), (1, 17)])
def test_many_small_groups(pa, G, members):
    """Up to 16 query rows have the next group's queries loaded ahead: many groups of a few
    key tiles for each worker, on both sides of that."""
    rng = np.random.default_rng(50 * G + members)
    groups = [(p, lengths(rng, members, p, 20)) for p in rng.integers(1, 30, 160)]
    c = Case(G, groups, 2 * G, 2)
    c.run(pa)
    c.check(rows=sorted({int(x) for x in rng.integers(0, 160 * members, 60)}
                        | {0, 160 * members - 1}))
    assert pa.pa_device_error_flags() == 0


@pytest.mark.parametrize("G,members", [(1, 128), (1, 129), (3, 21), (3, 42), (3, 50), (5, 12),
                                       (5, 13), (5, 26), (6, 60), (7, 9), (7, 18), (7, 40)])
def test_tiles_that_heads_do_not_fill(pa, G, members):
    """floor(128 / G) members to a tile, with rows to spare; several items for a worker."""
    rng = np.random.default_rng(100 * G + members)
    groups = [(p, lengths(rng, members, p, 20)) for p in (3, 12, 20)]
    c = Case(G, groups, 2 * G, 2)
    c.run(pa)
    n = 3 * members
    c.check(rows=sorted({0, 1, members - 1, members, 128 // G - 1, min(128 // G, n - 1),
                         min(2 * (128 // G), n - 1), n - 1}))


@pytest.mark.parametrize("groups", [[(9, [150, 160, 144])], [(3, [0, 20, 48, 49]), (0, [70]), (5, [])],
                                    [(60, [1000, 961, 3])]])
def test_small_batches(pa, groups):
    """One launch, each sequence through its own row; no matter what the groups say."""
    c = Case(30, groups, 8, 2, loose=2, small=True)
    c.run(pa)
    c.check()
    c.shared.fill_(-5)
    c.offsets.fill_(10**6)
    c.out.zero_()
    c.run(pa)
    c.check()
    assert pa.pa_device_error_flags() == 0


def test_many_ragged_groups(pa):
    """More groups than a warp has lanes, some empty, some without a prefix, sequences in no
    group behind them."""
    rng = np.random.default_rng(5)
    groups = []
    for g in range(70):
        p = int(rng.choice([0, 1, 5, 8, 12, 20]))
        groups.append((p, lengths(rng, int(rng.choice([0, 1, 2, 5, 9])), p, 60)))
    c = Case(5, groups, 6, 2, loose=7)
    c.run(pa)
    c.check()
    assert pa.pa_device_error_flags() == 0


def test_members_that_end_inside_the_prefix(pa):
    """Lengths from nothing to the whole of it; a group of which no member reaches its last
    blocks; a group whose members are all empty."""
    c = Case(6, [(20, [0, 1, 15, 16, 17, 127, 128, 129, 200, 319, 320, 321, 400]),
                 (20, [0, 5, 100, 33]), (30, [140, 17]), (9, [0, 0, 0]), (12, [192, 193])], 8, 4)
    c.run(pa)
    c.check()


@pytest.mark.parametrize("Hkv", [1, 3, 8, 80])
def test_long_prefix_cut_over_the_device(pa, Hkv):
    """One prefix, cut into as many pieces as there are teams; heads beyond the pairs."""
    rng = np.random.default_rng(Hkv)
    p = 1500 if Hkv < 80 else 40
    c = Case(Hkv, [(p, lengths(rng, 3, p, 20))], Hkv, Hkv)
    c.run(pa)
    c.check()


def test_long_own_parts(pa):
    rng = np.random.default_rng(8)
    c = Case(8, [(10, lengths(rng, 4, 10, 3000)), (30, lengths(rng, 2, 30, 5))], 8, 2)
    c.run(pa)
    c.check()


def test_a_batch_behind_one_system_prompt(pa):
    rng = np.random.default_rng(9)
    c = Case(9, [(128, lengths(rng, 150, 128, 200))], 32, 8)
    c.run(pa)
    c.check(rows=[0, 1, 63, 64, 100, 127, 128, 149])


@pytest.mark.parametrize("scale,amp", [(1e-3, 1.0), (0.09, 6.0), (3.0, 3.0), (1e30, 1.0)])
def test_scores_flat_sharp_and_far(pa, scale, amp):
    """Reference maxima that move from tile to tile, and far from zero."""
    rng = np.random.default_rng(10)
    c = Case(10, [(40, lengths(rng, 5, 40, 300))], 8, 2, scale=scale, amp=amp)
    c.run(pa)
    if scale < 1e3:
        c.check()
    else:  # each row's weight lies on its largest score
        assert torch.isfinite(c.out).all()


def test_rising_scores(pa):
    """A prefix whose keys grow: every key tile moves every row's maximum."""
    c = Case(11, [(64, [1030, 1050, 1024, 1100])], 8, 2)
    flat = c.tables[0, :64].long()
    ramp = torch.linspace(0.1, 4.0, 64, device="cuda").view(64, 1, 1, 1)
    c.kc[flat] = (c.kc[flat].float().abs() * ramp).bfloat16()
    c.q = c.q.abs()
    c.run(pa)
    c.check()


def test_agrees_with_plain_decode_and_equal_bits(pa):
    rng = np.random.default_rng(12)
    c = Case(12, [(33, lengths(rng, 8, 33, 100)) for _ in range(6)], 16, 4)
    c.run(pa)
    first = c.out.clone(), c.lse.clone()
    for fill in (0, 0x7F):
        c.ws.fill_(fill)
        c.run(pa)
        assert torch.equal(first[0], c.out) and torch.equal(first[1], c.lse)
    out, lse = torch.empty_like(c.out), torch.empty_like(c.lse)
    ws = torch.zeros(pa.pa_decode_workspace_size(48, 16, 4, D, c.tables.shape[1]),
                     dtype=torch.uint8, device="cuda")
    pa.pa_decode(out, c.q, c.kc, c.vc, c.tables, c.lens, c.scale, workspace=ws, out_lse=lse)
    assert (out.float() - c.out.float()).abs().max() < 0.05
    assert (lse - c.lse).abs().max() < 1e-4


def test_offsets_past_32_bits(pa):
    """Pools of 4.8 GB each, prefixes and own blocks at their end; then the small call."""
    for small in (False, True):
        rng = np.random.default_rng(13)
        c = Case(13, [(20, lengths(rng, 5, 20, 90)), (9, lengths(rng, 40, 9, 60))], 16, 8, loose=2,
                 small=small)
        n, nb = c.kc.shape[0], 150000
        big = [torch.empty((nb, 16, 8, D), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
        for pool, part in zip(big, (c.kc, c.vc)):
            pool[nb - n:] = part
        here = (c.tables >= 0) & (c.tables < n)
        c.tables = torch.where(here, c.tables + (nb - n), c.tables).contiguous()
        c.kc, c.vc = big
        c.run(pa)
        c.check()
        assert pa.pa_device_error_flags() == 0


def test_bad_metadata_is_flagged(pa):
    """Offsets that overlap, fall or leave the batch, groups larger than said, prefixes longer
    than a row, ids outside the pool, lengths outside the row: flagged, nothing faults."""
    rng = np.random.default_rng(13)

    def fresh():
        return Case(13, [(9, lengths(rng, 6, 9, 30)), (5, lengths(rng, 4, 5, 30))], 8, 2)

    for offsets in ([0, 10, 10], [-3, 6, 10], [0, 6, 99], [6, 0, 10], [10, 0, 2**31 - 1]):
        c = fresh()
        c.offsets.copy_(torch.tensor(offsets, dtype=torch.int32))
        c.run(pa)
        torch.cuda.synchronize()
        if offsets != [0, 10, 10]:
            assert pa.pa_device_error_flags() & pa.PA_DEVERR_GROUP, offsets
        pa.pa_device_error_flags()
    # many groups that each claim the whole batch
    c = fresh()
    c.offsets = torch.tensor([0, 10] * 20, dtype=torch.int32, device="cuda")
    c.shared = torch.full((39,), 9, dtype=torch.int32, device="cuda")
    c.max_group = 10
    c.run(pa)
    torch.cuda.synchronize()
    assert pa.pa_device_error_flags() & pa.PA_DEVERR_GROUP
    c = fresh()
    c.max_group = 4  # the first group has six: two attend on their own
    c.run(pa)
    c.check()
    assert pa.pa_device_error_flags() == pa.PA_DEVERR_GROUP
    for bad in (-1, 1000):
        c = fresh()
        c.shared[1] = bad
        c.run(pa)
        c.check(rows=range(6))
        assert pa.pa_device_error_flags() & pa.PA_DEVERR_GROUP
    c = fresh()
    c.tables[0, 3], c.tables[7, 2] = -1, 2**31 - 1
    c.run(pa)
    torch.cuda.synchronize()
    assert pa.pa_device_error_flags() == pa.PA_DEVERR_BLOCK_ID
    c = fresh()
    c.lens[2] = 10**6
    c.run(pa)
    torch.cuda.synchronize()
    assert pa.pa_device_error_flags() & pa.PA_DEVERR_SEQ_LEN


def test_captured_replayed_and_on_streams(pa):
    rng = np.random.default_rng(14)
    c = Case(14, [(20, lengths(rng, 4, 20, 64)) for _ in range(5)], 8, 2)
    c.ws = c.workspace(pa)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(pa)
    for _ in range(2):
        c.q.copy_(torch.randn(c.q.shape, device="cuda"))
        c.lens.sub_(1)
        c.out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        c.check()
    cases = [Case(20 + i, [(20, lengths(rng, 6, 20, 64)) for _ in range(8)], 8, 2)
             for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for x, s in zip(cases, streams):
            x.run(pa, stream=s)
    torch.cuda.synchronize()
    for x in cases:
        x.check()


def test_lengths_and_tables_written_just_before(pa):
    """The decode's CTAs start before the prefix pass is done; what the kernels before both
    wrote must be there."""
    rng = np.random.default_rng(15)
    c = Case(15, [(20, lengths(rng, 6, 20, 64)) for _ in range(10)], 8, 2)
    lens, tables, q = c.lens.clone(), c.tables.clone(), c.q.clone()
    for _ in range(20):
        c.lens.fill_(1)
        c.tables.fill_(0)
        c.q.fill_(1.0)
        c.run(pa)
        c.lens.copy_(lens)
        c.tables.copy_(tables)
        c.q.copy_(q)
        c.run(pa)
    c.check()


def test_stalled_prefix_pass_times_out(pa):
    rng = np.random.default_rng(16)
    c = Case(16, [(20, lengths(rng, 6, 20, 64))], 8, 2)
    c.ws = c.workspace(pa)
    pa.pa_test_decode_shared_stalled(c.out, c.q, c.kc, c.vc, c.tables, c.lens, c.offsets,
                                     c.max_group, c.shared, c.scale, c.ws, wait_limit_us=2000)
    torch.cuda.synchronize()
    assert pa.pa_device_error_flags() & pa.PA_DEVERR_TIMEOUT
    c.run(pa)
    c.check()
    assert pa.pa_device_error_flags() == 0


def test_refusals_on_the_device(pa):
    c = Case(17, [(2, [40, 50])], 8, 2)
    ws = c.workspace(pa)
    for bad in (ws[:-1], ws[1:]):
        with pytest.raises(pa.PAError) as e:
            pa.pa_decode_shared(c.out, c.q, c.kc, c.vc, c.tables, c.lens, c.offsets, c.max_group,
                                c.shared, c.scale, bad)
        assert e.value.status == pa.PA_ERR_WORKSPACE
    with pytest.raises(ValueError, match="group_offsets"):
        pa.pa_decode_shared(c.out, c.q, c.kc, c.vc, c.tables, c.lens, c.offsets[:1], c.max_group,
                            c.shared, c.scale, ws)
    none = Case(18, [], 8, 2, loose=3)
    none.run(pa)
    none.check()
