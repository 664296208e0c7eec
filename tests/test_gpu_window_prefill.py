"""pa_prefill_window against its fp64 definition (calls of few and of many
query tokens and kv heads, which take different kernels): window, sink and chunk edges
on both sides of block and tile borders, every group size, more items than CTA
pairs, ragged and empty chunks, garbage in everything that no query sees,
inconsistent metadata, the bounded waits, streams, graphs and refusals."""
import math

import numpy as np
import pytest
import torch

from tests import window_ref as R

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def pa(cuda_device):
    from paged_kv_cache_218_gb300 import binding
    return binding


class Chunks:
    """Chunks [(start, queries)], their caches holding `beyond` later keys too."""

    def __init__(self, chunks, Hq, Hkv, window, sinks, device, seed=0, beyond=0):
        self.window, self.sinks, self.scale = window, sinks, 1.0 / math.sqrt(D)
        starts, counts = [c[0] for c in chunks], [c[1] for c in chunks]
        lens = [s + n for s, n in chunks]
        self.kc, self.vc, bt = R.paged_cache(lens, window, sinks, Hkv, D, seed, device,
                                             first_query=starts)
        pad = torch.full((len(chunks), (beyond + 15) // 16), 2**30, dtype=torch.int32,
                         device=device)
        self.bt = torch.cat([bt, pad], 1).contiguous()
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=device)  # noqa: E731
        self.q = torch.randn(sum(counts), Hq, D, generator=g, device=device, dtype=torch.bfloat16)
        self.cu, self.start = i32([0] + np.cumsum(counts).tolist()), i32(starts)
        self.lens, self.max_q = i32([n + beyond for n in lens]), max(counts)

    def call(self, pa, o=None, l=None, **change):
        out = torch.full_like(self.q, float("nan")) if o is None else o
        lse = torch.full(self.q.shape[:2], float("nan"), device=self.q.device) if l is None else l
        pa.pa_prefill_window(**{**dict(
            out=out, q=self.q, k_cache=self.kc, v_cache=self.vc, block_tables=self.bt,
            cu_q_lens=self.cu, q_start_pos=self.start, seq_lens=self.lens, max_q_len=self.max_q,
            window=self.window, sinks=self.sinks, scale=self.scale, out_lse=lse), **change})
        return out, lse

    def check(self, pa):
        out, lse = self.call(pa)
        torch.cuda.synchronize()
        assert pa.pa_device_error_flags() == 0
        ro, rl, to, tl = R.prefill(self.q, self.kc, self.vc, self.bt, self.cu, self.start,
                                   self.window, self.sinks, self.scale)
        R.assert_within(lse, rl, tl, "lse")
        R.assert_within(out, ro, to, "out")


# Few (token, kv head) pairs in a call, and many: more than two for each SM.
both = pytest.mark.parametrize("hkv", [1, 8])

MIX = [(0, 1), (0, 40), (24, 72), (1000, 5), (513, 260), (300, 0), (17, 130)]


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 0), (16, 16), (17, 5), (63, 4),
                                          (64, 0), (65, 17), (128, 130), (129, 1), (200, 0),
                                          (500, 700), (5000, 9), (3, 5000),
                                          (2**31 - 1, 2**31 - 1)])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (2, 2)])
def test_window_edges(pa, cuda_device, window, sinks, Hq, Hkv):
    Chunks(MIX, Hq, Hkv, window, sinks, cuda_device, seed=window % 1000).check(pa)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (4, 1), (8, 1), (3, 3), (16, 2), (6, 3)])
def test_groups(pa, cuda_device, Hq, Hkv):
    Chunks([(70, 300), (5, 33)], Hq, Hkv, 100, 4, cuda_device, seed=Hq).check(pa)


FEW = {"one": [(1000, 1)], "first": [(0, 1)], "some": [(5, 3), (0, 0), (700, 7), (31, 2)],
       "draft": [(2047, 8)], "many": [(17 * i % 400, i % 3) for i in range(70)]}


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 5), (64, 0), (200, 16),
                                          (1500, 700), (2**31 - 1, 2**31 - 1)])
@pytest.mark.parametrize("name", FEW)
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (1, 1), (16, 2)])
def test_few_queries(pa, cuda_device, window, sinks, name, Hq, Hkv):
    Chunks(FEW[name], Hq, Hkv, window, sinks, cuda_device, seed=window % 1000).check(pa)


@pytest.mark.parametrize("Hkv", [1, 2, 3])
@pytest.mark.parametrize("times", [1, 2])
@pytest.mark.parametrize("window,sinks", [(90, 3), (400, 20)])
def test_around_the_number_of_sms(pa, cuda_device, Hkv, times, window, sinks):
    sms = times * torch.cuda.get_device_properties(cuda_device).multi_processor_count
    for tokens in (sms // Hkv - 1, sms // Hkv, sms // Hkv + 1):
        Chunks([(300, tokens - 40), (2, 40)], 4 * Hkv, Hkv, window, sinks, cuda_device).check(pa)


@pytest.mark.parametrize("window,sinks", [(300, 4), (1024, 40), (50, 0)])
def test_more_items_than_pairs(pa, cuda_device, window, sinks):
    Chunks([(2000, 2500), (0, 1000)], 16, 4, window, sinks, cuda_device).check(pa)


def test_many_ragged_chunks(pa, cuda_device):
    rng = np.random.default_rng(5)
    chunks = [(int(rng.integers(0, 400)), int(rng.integers(0, 50))) for _ in range(150)]
    Chunks(chunks, 4, 1, 37, 3, cuda_device).check(pa)


def test_dozens_of_items_per_pair(pa, cuda_device):
    """Every ring of the kernel goes around several times."""
    rng = np.random.default_rng(6)
    chunks = [(int(rng.integers(0, 300)), int(rng.integers(1, 60))) for _ in range(600)]
    Chunks(chunks, 32, 4, 150, 3, cuda_device).check(pa)


def test_a_long_window_needs_several_batches_of_block_ids(pa, cuda_device):
    Chunks([(9000, 70)], 2, 1, 10**6, 0, cuda_device).check(pa)
    Chunks([(14000, 33)], 2, 1, 8400, 700, cuda_device).check(pa)


@pytest.mark.parametrize("beyond", [1, 9, 16, 100])
@both
def test_later_keys_of_the_sequence_stay_unseen(pa, cuda_device, beyond, hkv):
    """The cache holds keys behind the chunk's: their slots are NaN here, their blocks no ids."""
    Chunks([(100, 77), (32, 16)], 4 * hkv, hkv, 60, 2, cuda_device, beyond=beyond).check(pa)


@both
def test_scores_that_climb_along_the_keys(pa, cuda_device, hkv):
    c = Chunks([(700, 130)], 4 * hkv, hkv, 600, 4, cuda_device)
    c.q = c.q.abs().clamp(min=0.5)
    for b in range(c.bt.shape[1]):
        i = int(c.bt[0, b])
        if 0 <= i < c.kc.shape[0]:
            hidden = c.kc[i].isnan()
            c.kc[i] = 0.02 * (b + 1)
            c.kc[i][hidden] = float("nan")
    c.scale = 1.0
    c.check(pa)


@both
def test_infinite_scores(pa, cuda_device, hkv):
    c = Chunks([(0, 60)], 2 * hkv, hkv, 20, 0, cuda_device)
    c.q[:] = 1.0
    i = int(c.bt[0, 1])
    c.kc[i, 3] = -float("inf")  # key 19: weight exactly 0
    out, lse = c.call(pa)
    c.kc[i, 3] = -3e4
    ref, ref_lse = c.call(pa)
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    c.kc[i, 3] = float("nan")  # seen by the queries at 19 .. 38 and by no other
    out, _ = c.call(pa)
    bad = out.isnan().flatten(1)
    assert bad[19:39].all() and not bad[:19].any() and not bad[39:].any()
    c.kc[:] = -float("inf")
    out, lse = c.call(pa)
    assert (out == 0).all() and (lse == -float("inf")).all()


def test_whole_sequence_gives_pa_prefill_chunks_result(pa, cuda_device):
    """Both within their rounding of the definition, so of each other within twice that."""
    c = Chunks([(100, 300), (0, 64)], 8, 2, 10**6, 0, cuda_device)
    out, lse = c.call(pa)
    ref, ref_lse = torch.empty_like(out), torch.empty_like(lse)
    pa.pa_prefill_chunk(ref, c.q, c.kc, c.vc, c.bt, c.cu, c.start, c.lens, c.max_q, c.scale,
                        out_lse=ref_lse)
    torch.cuda.synchronize()
    _, _, to, tl = R.prefill(c.q, c.kc, c.vc, c.bt, c.cu, c.start, c.window, c.sinks, c.scale)
    R.assert_within(out, R.to64(ref), 2 * to, "out")
    R.assert_within(lse, R.to64(ref_lse), 2 * tl, "lse")


@both
def test_inconsistent_chunks_are_skipped_and_flagged(pa, cuda_device, hkv):
    c = Chunks([(10, 40), (0, 30), (50, 20), (7, 33)], 4 * hkv, hkv, 25, 2, cuda_device)
    good, good_lse = c.call(pa)
    rows = [slice(0, 40), slice(40, 70), slice(70, 90), slice(90, 123)]
    cap = c.bt.shape[1] * 16
    for what, value in (("lens", 29), ("lens", cap + 1), ("lens", -1), ("start", -1),
                        ("start", 2**31 - 1), ("lens", 2**31 - 1)):
        t = getattr(c, what)
        old = t.clone()
        t[1] = value
        out, lse = c.call(pa)
        assert pa.pa_device_error_flags() == pa.PA_DEVERR_CHUNK, (what, value)
        t.copy_(old)
        for k in (0, 2, 3):
            assert torch.equal(out[rows[k]], good[rows[k]])
            assert torch.equal(lse[rows[k]], good_lse[rows[k]])
        assert out[rows[1]].isnan().all() and lse[rows[1]].isnan().all()
    cu = c.cu.clone()
    c.cu[4] = 124  # past the queries' rows
    out, _ = c.call(pa)
    assert pa.pa_device_error_flags() == pa.PA_DEVERR_CHUNK
    assert out[rows[3]].isnan().all() and torch.equal(out[:90], good[:90])
    c.cu.copy_(cu)
    c.cu[2] = 30  # chunk 1 runs backwards; chunk 2 takes its rows over
    c.call(pa)
    assert pa.pa_device_error_flags() == pa.PA_DEVERR_CHUNK


@pytest.mark.parametrize("bad", [-1, -2**31, 2**31 - 1])
@both
def test_bad_block_reads_as_zeros_and_is_flagged(pa, cuda_device, bad, hkv):
    c = Chunks([(40, 50)], 2 * hkv, hkv, 60, 4, cuda_device)
    zero = c.kc.shape[0] - 1
    c.kc[zero], c.vc[zero] = 0, 0
    c.bt[0, 3] = zero
    ref, ref_lse = c.call(pa)
    assert pa.pa_device_error_flags() == 0
    c.bt[0, 3] = bad
    out, lse = c.call(pa)
    assert pa.pa_device_error_flags() == pa.PA_DEVERR_BLOCK_ID
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


def test_equal_bits_on_streams_and_graph_replays(pa, cuda_device):
    c = Chunks([(900, 700), (3, 250)], 8, 2, 300, 4, cuda_device)
    want, want_lse = c.call(pa)
    got = [(torch.empty_like(want), torch.empty_like(want_lse)) for _ in range(2)]
    graphs = []
    for o, l in got:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(pa, o, l)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(4):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        eager, eager_lse = c.call(pa)
    torch.cuda.synchronize()
    for o, l in got + [(eager, eager_lse)]:
        assert torch.equal(o, want) and torch.equal(l, want_lse)
    c.q.mul_(0.5)
    want, want_lse = c.call(pa)
    graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(got[1][0], want) and torch.equal(got[1][1], want_lse)


def test_few_queries_in_a_graph_see_new_chunks(pa, cuda_device):
    """A replay reads the chunks' positions and lengths anew."""
    c = Chunks([(50, 3), (7, 2)], 8, 2, 30, 2, cuda_device)
    want, want_lse = c.call(pa)
    o, l = torch.empty_like(want), torch.empty_like(want_lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(pa, o, l)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(l, want_lse)
    c.start.sub_(1)
    c.lens.sub_(1)
    c.kc.nan_to_num_()
    c.vc.nan_to_num_()
    c.bt.clamp_(0, c.kc.shape[0] - 1)
    want, want_lse = c.call(pa)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(l, want_lse)


@both
def test_rows_outside_the_chunks_stay(pa, cuda_device, hkv):
    c = Chunks([(30, 40), (0, 20)], 4 * hkv, hkv, 25, 2, cuda_device)
    out = torch.full((70, 4 * hkv, D), 7.0, dtype=torch.bfloat16, device=cuda_device)
    lse = torch.full((70, 4 * hkv), 7.0, device=cuda_device)
    c.q = torch.cat([c.q, c.q[:10]])  # ten more query rows, of no chunk
    c.call(pa, out, lse)
    torch.cuda.synchronize()
    assert (out[60:] == 7).all() and (lse[60:] == 7).all()
    assert not (out[:60] == 7).any()
    c.call(pa, out, out_lse=None)


def test_stalled_loads_run_into_the_wait_limit(pa, cuda_device):
    c = Chunks([(300, 700)], 8, 2, 200, 4, cuda_device)
    good, good_lse = c.call(pa)
    out = torch.empty_like(good)
    pa.pa_test_prefill_window_stalled(out, c.q, c.kc, c.vc, c.bt, c.cu, c.start, c.lens, c.max_q,
                                      c.window, c.sinks, c.scale, wait_limit_us=1000)
    torch.cuda.synchronize()
    assert pa.pa_device_error_flags() == pa.PA_DEVERR_TIMEOUT
    again, again_lse = c.call(pa)
    torch.cuda.synchronize()
    assert pa.pa_device_error_flags() == 0
    assert torch.equal(again, good) and torch.equal(again_lse, good_lse)


def test_refusals(pa, cuda_device):
    c = Chunks([(10, 20), (0, 9)], 4, 2, 25, 2, cuda_device)
    out = torch.full_like(c.q, 3.0)
    lse = torch.full(c.q.shape[:2], 3.0, device=cuda_device)
    for bad in (dict(window=0), dict(sinks=-1), dict(window=2**32 + 7), dict(sinks=2**31),
                dict(max_q_len=-1), dict(out=out[:3]), dict(v_cache=c.vc[:-1]),
                dict(block_tables=c.bt[:1]), dict(seq_lens=c.lens[:1]), dict(cu_q_lens=c.cu[:2]),
                dict(out_lse=lse[:3]), dict(q=c.q.cpu()), dict(q=c.q.transpose(0, 1))):
        with pytest.raises(ValueError):
            c.call(pa, out, lse, **bad)
    for bad in (dict(q=c.q.half()), dict(cu_q_lens=c.cu.long()), dict(k_cache=None)):
        with pytest.raises(TypeError):
            c.call(pa, out, lse, **bad)
    for bad in (dict(scale=0.0), dict(scale=float("inf"))):
        with pytest.raises(pa.PAError) as e:
            c.call(pa, out, lse, **bad)
        assert e.value.status == pa.PA_ERR_INVALID
    torch.cuda.synchronize()
    assert (out == 3).all() and (lse == 3).all() and pa.pa_device_error_flags() == 0


def equal_scores(pa, device, hkv, q, k, ahead, factor=0.0):
    """300 queries of q over keys of k, 128 columns each, at scale 1; `ahead`:
    key 200 has half of k.  All partial sums are exact, so scores are equal:
    weights 1 on every visible key, from query 200 on with `ahead` on that one
    alone (the others lose by more than 2^7 in log2 units).  Out: one rounding
    to bf16, 300 fp32 additions of values, a division; and, where weights may
    differ from 1 by a common factor that the normalizer has unrounded, their
    rounding to bf16, 2^-8 (`factor`).  lse: the rounding of
    the score in base 2 and back, four steps of 2^-24."""
    c = Chunks([(0, 300)], 2 * hkv, hkv, 300, 0, device)
    c.scale = 1.0
    c.q[:] = q
    c.kc[:] = k
    if ahead:
        c.kc[int(c.bt[0, 200 // 16]), 200 % 16] = k / 2
    out, lse = c.call(pa)
    torch.cuda.synchronize()
    assert pa.pa_device_error_flags() == 0
    v = R.to64(c.vc[c.bt[0, :19].long()]).reshape(-1, hkv, D)[:300].repeat(2, 1)
    count = np.arange(1.0, 301)[:, None, None]
    ref, score = v.cumsum(0) / count, np.full((300, 2 * hkv), float(D * q * k))
    ref_lse = score + np.log(count[:, :, 0])
    if ahead:
        ref[200:], ref_lse[200:] = v[200], score[200:] / 2
    R.assert_within(lse, ref_lse, 2.0**-22 * np.abs(ref_lse), "lse")
    R.assert_within(out, ref, (2.0**-8 + factor + 2.0**-21) * np.abs(ref) +
                    300 * 2.0**-23 * np.abs(v).max(), "out")


@pytest.mark.parametrize("ahead", [0, 1])
@both
def test_scores_near_the_lowest_fp32(pa, cuda_device, ahead, hkv):
    """Scores of -2^126: lower than any reference maximum but the lowest fp32."""
    equal_scores(pa, cuda_device, hkv, 2.0**99, -2.0**20, ahead)


@pytest.mark.parametrize("q,k,ahead", [
    (1.25 * 2.0**98, 1.125 * 2.0**20, 0), (1.25 * 2.0**98, -1.125 * 2.0**20, 0),
    (1.25 * 2.0**98, -1.125 * 2.0**20, 1), (1.25 * 2.0**12, 1.125 * 2.0**12, 0),
    (1.25 * 2.0**12, -1.125 * 2.0**12, 0), (1.25 * 2.0**12, -1.125 * 2.0**12, 1),
    (1.25 * 2.0**8, 1.125 * 2.0**9, 0), (1.25 * 2.0**8, -1.125 * 2.0**9, 1)])
@both
def test_scores_whose_base_2_product_is_rounded_far(pa, cuda_device, q, k, ahead, hkv):
    """The product of such a score with log2(e) is off by 2^102, 248 and 1.9
    from the nearest fp32: the reference maximum and the score's distance from
    it may differ by no more than a factor that fp32 holds."""
    equal_scores(pa, cuda_device, hkv, q, k, ahead, factor=2.0**-8)


@pytest.mark.parametrize("scale", [1e-38, 1e-36, 1e-20])
@both
def test_scales_that_leave_every_weight_alike(pa, cuda_device, scale, hkv):
    c = Chunks([(0, 300), (900, 40)], 2 * hkv, hkv, 200, 4, cuda_device)
    c.scale = scale
    c.check(pa)


@pytest.mark.parametrize("chunks,Hq,Hkv,window,sinks", [
    # up to 72 key tiles an item: the ring of ids goes around
    ([(9000, 70), (8500, 40)], 8, 8, 10**6, 0), ([(14000, 60)], 16, 8, 8400, 700),
    # 35 key tiles, and another such item behind most
    ([(5000, 330), (4700, 320)], 64, 8, 4300, 40)])
def test_items_of_several_batches_of_block_ids(pa, cuda_device, chunks, Hq, Hkv, window, sinks):
    """More than two (token, kv head) pairs for each SM, as for `both`."""
    assert sum(n for _, n in chunks) * Hkv > 2 * torch.cuda.get_device_properties(
        cuda_device).multi_processor_count
    Chunks(chunks, Hq, Hkv, window, sinks, cuda_device).check(pa)
