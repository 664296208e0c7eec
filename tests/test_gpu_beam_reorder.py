"""pa_beam_reorder against its definition: tables and lengths equal, pools bit for bit."""
import numpy as np
import pytest
import torch

from tests import beam_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa(cuda_device):
    from paged_kv_cache_218_gb300 import binding
    binding.pa_device_error_flags()
    return binding


class Case:
    """Tables whose history is shared at random and whose own blocks are each beam's."""

    def __init__(self, seed, R, W, layers, Hkv, D, fp8=False, lens=None, parents=None, own=2,
                 width=None, max_len=200, layer_pad=0):
        rng = np.random.default_rng(seed)
        self.fp8 = fp8
        rows = R * W
        if lens is None:
            lens = np.repeat(rng.integers(0, max_len, R), W)
        self.lens = np.asarray(lens, np.int32)
        if parents is None:
            parents = rng.integers(-1, W, (R, W))
        self.parents = np.asarray(parents, np.int32)
        width = width or int(self.lens.max()) // 16 + own + 1
        blocks = rows * own + 9
        place = rng.permutation(blocks).astype(np.int32)
        self.tables = rng.choice(place[rows * own:], (rows, width)).astype(np.int32)
        for i in range(rows):
            f = int(self.lens[i]) // 16
            tail = place[i * own:(i + 1) * own][:max(0, width - f)]
            self.tables[i, f:f + len(tail)] = tail
            self.tables[i, f + len(tail):] = -1
        shape = (layers, blocks * (1 + layer_pad), 16, Hkv, D)
        self.k, self.v = (torch.randint(0, 256, shape[:-1] + (D * (1 if fp8 else 2),),
                                        dtype=torch.uint8, device="cuda") for _ in range(2))
        if not fp8:  # any bits, NaN among them
            self.k, self.v = self.k.view(torch.bfloat16), self.v.view(torch.bfloat16)
        self.k, self.v = self.k[:, :blocks], self.v[:, :blocks]
        self.dev = [torch.from_numpy(x).cuda() for x in (self.tables, self.lens, self.parents)]
        self.out_tables = torch.full_like(self.dev[0], 99)
        self.out_lens = torch.full_like(self.dev[1], 99)

    def bits(self, pool):
        return pool.view(torch.uint8 if self.fp8 else torch.int16)

    def run(self, pa, stream=None, pools=True):
        call = pa.pa_beam_reorder_fp8 if self.fp8 else pa.pa_beam_reorder
        call(self.out_tables, self.out_lens, *self.dev, self.k if pools else None,
             self.v if pools else None, stream=stream)

    def expect(self):
        self.tables_ref, self.lens_ref, copies = beam_ref.reorder(self.tables, self.lens,
                                                                  self.parents)
        self.ref = [self.bits(p).clone() for p in (self.k, self.v)]
        for source, target, n in copies:
            for p in self.ref:
                p[:, target, :n] = p[:, source, :n]
        return copies

    def check(self):
        assert np.array_equal(self.out_tables.cpu().numpy(), self.tables_ref)
        assert np.array_equal(self.out_lens.cpu().numpy(), self.lens_ref)
        for p, ref in zip((self.k, self.v), self.ref):
            assert torch.equal(self.bits(p), ref)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("R,W,layers,Hkv,D", [
    (1, 1, 1, 1, 64), (1, 4, 3, 8, 128), (7, 3, 2, 3, 64), (2, 32, 1, 2, 16), (64, 4, 5, 8, 128),
    (300, 2, 1, 1, 32), (1, 5, 40, 1, 128), (3, 8, 1, 64, 256)])
def test_sizes(pa, R, W, layers, Hkv, D, fp8):
    for seed in range(3):
        c = Case(seed, R, W, layers, Hkv, D, fp8)
        c.expect()
        c.run(pa)
        c.check()
    assert pa.pa_device_error_flags() == 0


@pytest.mark.parametrize("parents", [
    [0, 0, 0, 0], [3, 3, 3, 3], [0, 1, 2, 3], [3, 2, 1, 0], [1, 1, 2, 2], [2, -1, 2, -1],
    [-1, -1, -1, -1], [-1, 0, 0, 0]])
@pytest.mark.parametrize("length", [0, 1, 15, 16, 17, 31, 160])
def test_shapes_of_a_family(pa, parents, length):
    c = Case(length, 2, 4, 2, 2, 64, parents=[parents, parents[::-1]], lens=[length] * 8)
    c.expect()
    c.run(pa)
    c.check()


def test_lengths_that_differ_within_a_request(pa):
    """A beam that ended early, beams not begun: own blocks move to the columns behind the
    history they get."""
    for seed in range(6):
        rng = np.random.default_rng(seed)
        c = Case(seed, 5, 6, 2, 2, 64, lens=rng.integers(0, 120, 30), own=3, width=9)
        c.expect()
        c.run(pa)
        c.check()


def test_rows_full_to_the_last_slot(pa):
    """A length that fills its table: no block of its own, nothing to copy."""
    c = Case(1, 3, 4, 1, 2, 64, lens=[64] * 12, own=1, width=4)
    c.expect()
    c.run(pa)
    c.check()
    assert pa.pa_device_error_flags() == 0


def test_first_step_from_one_beam(pa):
    """The prompt lies in beam 0, the others have but blocks of their own."""
    c = Case(2, 4, 5, 2, 2, 64, lens=[90, 0, 0, 0, 0] * 4, parents=[[0] * 5] * 4, own=2, width=8)
    assert len(c.expect()) == 16
    c.run(pa)
    c.check()


@pytest.mark.parametrize("fp8", [False, True])
def test_layers_apart_one_layer_and_none(pa, fp8):
    c = Case(3, 4, 4, 3, 2, 64, fp8, layer_pad=1)
    assert not c.k.is_contiguous()
    c.expect()
    c.run(pa)
    c.check()
    one = Case(4, 4, 4, 1, 2, 64, fp8)
    one.expect()
    k, v = one.k, one.v
    one.k, one.v = k[0], v[0]
    one.run(pa)
    one.k, one.v = k, v
    one.check()
    none = Case(5, 4, 4, 1, 2, 64, fp8)
    none.expect()
    none.ref = [none.bits(p).clone() for p in (none.k, none.v)]
    none.run(pa, pools=False)
    none.check()


def test_long_tables(pa):
    c = Case(6, 2, 3, 1, 1, 64, lens=[70000] * 6, width=5000)
    c.expect()
    c.run(pa)
    c.check()


def test_offsets_past_32_bits(pa):
    """Pools of 4.8 GB each: blocks and layers beyond 2^32 bytes."""
    c = Case(7, 2, 4, 1, 8, 128)
    blocks = 73000
    k = torch.zeros((2, blocks, 16, 8, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    small, c.k, c.v = c.k.shape[1], k, v
    far = blocks - small
    k[:, far:] = torch.randn((2, small, 16, 8, 128), device="cuda")
    v[:, far:] = torch.randn((2, small, 16, 8, 128), device="cuda")
    c.tables = np.where(c.tables >= 0, c.tables + far, -1).astype(np.int32)
    c.dev[0].copy_(torch.from_numpy(c.tables))
    c.expect()
    c.run(pa)
    c.check()


def test_bad_metadata_is_flagged_and_left_out(pa):
    c = Case(8, 2, 4, 2, 2, 64, lens=[50] * 8, parents=[[1, 1, 0, 2], [3, 3, 3, 0]])
    c.dev[2][0, 3] = 4       # no such beam: as -1
    c.parents[0, 3] = -1
    c.expect()
    c.run(pa)
    c.check()
    assert pa.pa_device_error_flags() == pa.PA_DEVERR_BEAM

    c = Case(9, 1, 4, 2, 2, 64, lens=[50] * 4, parents=[[1, 1, 1, 0]])
    copies = c.expect()
    c.ref = [c.bits(p).clone() for p in (c.k, c.v)]
    bad = copies[0][1]  # the first copy's destination is out of the pool
    for p in c.ref:
        for source, target, n in copies[1:]:
            p[:, target, :n] = p[:, source, :n]
    where = c.tables == bad
    c.dev[0][torch.from_numpy(where).cuda()] = c.k.shape[1]
    c.tables_ref[c.tables_ref == bad] = c.k.shape[1]
    c.run(pa)
    c.check()
    assert pa.pa_device_error_flags() == pa.PA_DEVERR_BLOCK_ID

    c = Case(10, 1, 2, 1, 2, 64, lens=[32, 32], parents=[[0, 1]], width=4)
    c.lens[:] = [64, 0]
    c.expect()
    c.dev[1][0], c.dev[1][1] = 65, -3
    c.run(pa)
    c.check()
    assert pa.pa_device_error_flags() == pa.PA_DEVERR_SEQ_LEN


def test_captured_and_on_another_stream(pa):
    c = Case(11, 6, 4, 3, 2, 64)
    c.expect()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    c.run(pa, stream=s)
    s.synchronize()
    c.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(pa)
    for seed in (12, 13):
        new = Case(seed, 6, 4, 3, 2, 64, lens=c.lens, width=c.tables.shape[1])
        c.parents, c.tables = new.parents, new.tables
        c.dev[0].copy_(new.dev[0])
        c.dev[2].copy_(new.dev[2])
        c.expect()
        graph.replay()
        torch.cuda.synchronize()
        c.check()


def test_the_host_s_block_manager_copies_the_same(pa):
    """Fork and copy on write on the host, and this call, give beams the same tokens."""
    from paged_kv_cache_218_gb300.block_manager import BlockManager
    W, n = 4, 37
    parents = [2, 0, 2, 2]
    k = torch.randn((1, 64, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    v = torch.randn_like(k)
    bm = BlockManager(64, 16, prefix_caching=False)
    bm.add_sequence(0, list(range(n - 5)))
    for w in range(1, W):
        bm.fork(0, w)
    bm.end_step()
    for t in range(5):  # five tokens each: every beam gets a last block of its own
        for w in range(W):
            bm.append_token(w, 100 + w)
        pairs = bm.end_step()
        if len(pairs):
            pa.pa_copy_blocks(k[0], v[0], torch.from_numpy(np.asarray(pairs, np.int64)).cuda())
    for w in range(W):
        tables, lens = bm.build_tables([w], 4)
    tables, lens = bm.build_tables(list(range(W)), 4)
    tables, lens = np.asarray(tables, np.int32), np.asarray(lens, np.int32)
    assert (lens == n).all() and len(set(tables[:, 2])) == W

    def tokens(tb, row):
        return torch.cat([k[0, int(tb[row, j])] for j in range(3)])[:n]

    want = [tokens(tables, p).clone() for p in parents]
    out_t = torch.zeros((W, 4), dtype=torch.int32, device="cuda")
    out_l = torch.zeros(W, dtype=torch.int32, device="cuda")
    pa.pa_beam_reorder(out_t, out_l, torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda(),
                       torch.tensor([parents], dtype=torch.int32, device="cuda"), k, v)
    got = out_t.cpu().numpy()
    assert len(set(got[:, 2])) == W and (out_l == n).all()
    for w in range(W):
        assert torch.equal(tokens(got, w), want[w])


def test_refusals_of_the_binding(pa):
    c = Case(14, 2, 4, 2, 2, 64)
    with pytest.raises(ValueError, match="row for each"):
        pa.pa_beam_reorder(c.out_tables, c.out_lens, c.dev[0][:7], c.dev[1], c.dev[2], c.k, c.v)
    with pytest.raises(ValueError, match="layer"):
        pa.pa_beam_reorder(c.out_tables, c.out_lens, *c.dev, c.k[:, :, :, :1], c.v[:, :, :, :1])
    with pytest.raises(TypeError):
        pa.pa_beam_reorder_fp8(c.out_tables, c.out_lens, *c.dev, c.k, c.v)
    with pytest.raises(TypeError):
        pa.pa_beam_reorder(c.out_tables, c.out_lens, *c.dev, c.k, None)
    with pytest.raises(pa.PAError):
        pa.pa_beam_reorder(c.dev[0], c.out_lens, *c.dev, c.k, c.v)
