"""pa_decode_window against its fp64 definition: window and sink edges on both
sides of block borders, empty and one-token sequences, every group size, the
split over a cluster, garbage in everything that no query sees, extreme
scores, streams, graphs and refusals."""
import math

import numpy as np
import pytest
import torch

from tests import window_ref as R

pytestmark = pytest.mark.gpu

LENS = [0, 1, 2, 15, 16, 17, 31, 33, 100, 257, 700]


@pytest.fixture(scope="module")
def pa(cuda_device):
    from paged_kv_cache_218_gb300 import binding
    return binding


def make(lens, Hq, Hkv, D, window, sinks, seed, device, **kw):
    kc, vc, bt = R.paged_cache(lens, window, sinks, Hkv, D, seed, device, **kw)
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    q = torch.randn(len(lens), Hq, D, generator=g, device=device, dtype=torch.bfloat16)
    return q, kc, vc, bt, torch.tensor(lens, dtype=torch.int32, device=device)


def call(pa, q, kc, vc, bt, sl, window, sinks, scale, **kw):
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), dtype=torch.float32, device=q.device)
    pa.pa_decode_window(out, q, kc, vc, bt, sl, window, sinks, scale, out_lse=lse, **kw)
    return out, lse


def check(pa, lens, Hq, Hkv, D, window, sinks, device, seed=0, scale=None, mutate=None):
    x = make(lens, Hq, Hkv, D, window, sinks, seed, device)
    if mutate:
        mutate(*x)
    scale = scale or 1.0 / math.sqrt(D)
    out, lse = call(pa, *x, window, sinks, scale)
    torch.cuda.synchronize()
    assert pa.pa_device_error_flags() == 0
    ro, rl, to, tl = R.decode(*x, window, sinks, scale)
    R.assert_within(out, ro, to, "out")
    R.assert_within(lse, rl, tl, "lse")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 0), (15, 4), (16, 16), (17, 17),
                                          (33, 1), (100, 40), (1000, 0), (5000, 9),
                                          (3, 5000), (2**31 - 1, 2**31 - 1)])
def test_window_edges(pa, cuda_device, D, window, sinks):
    check(pa, LENS, 8, 2, D, window, sinks, cuda_device, seed=window % 1000 + sinks % 100)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (3, 1), (5, 1), (8, 1), (4, 4), (12, 4), (21, 3)])
@pytest.mark.parametrize("D", [64, 128])
def test_groups(pa, cuda_device, Hq, Hkv, D):
    check(pa, [40, 0, 130, 77], Hq, Hkv, D, 50, 4, cuda_device, seed=Hq)


@pytest.mark.parametrize("lens,window,sinks", [
    ([4999], 4096, 4), ([5000, 90], 4000, 100), ([9, 3000, 0], 10**6, 0), ([1], 4096, 0),
    ([20000], 20000, 0), ([6000, 17, 2500], 300, 300)])
@pytest.mark.parametrize("D", [64, 128])
def test_split_over_a_cluster(pa, cuda_device, D, lens, window, sinks):
    check(pa, lens, 4, 1, D, window, sinks, cuda_device, seed=len(lens))


def test_many_sequences(pa, cuda_device):
    rng = np.random.default_rng(3)
    check(pa, rng.integers(0, 300, 400).tolist(), 16, 8, 128, 100, 4, cuda_device)


def test_scores_that_climb_along_the_window(pa, cuda_device):
    """The reference maximum moves at every block."""
    def climb(q, kc, vc, bt, sl):
        q.copy_(q.abs().clamp(min=0.5))
        n = int(sl[0])
        for b in range((n + 15) // 16):
            kc[bt[0, b].long()] = 0.05 * (b + 1)
    check(pa, [800], 8, 1, 128, 800, 0, cuda_device, scale=1.0, mutate=climb)


def test_scores_that_fall_far(pa, cuda_device):
    """Weights of later blocks underflow to nothing."""
    def fall(q, kc, vc, bt, sl):
        q.fill_(4.0)
        for b in range((int(sl[0]) + 15) // 16):
            kc[bt[0, b].long()] = 8.0 - b
    check(pa, [330], 2, 1, 64, 330, 0, cuda_device, scale=1.0, mutate=fall)


@pytest.mark.parametrize("ahead", [0, 1])
def test_scores_near_the_lowest_fp32(pa, cuda_device, ahead):
    """All products and sums are powers of two, so equal scores (-2^126) stay
    equal: weights 1 each, or all on the one key whose score is half as low."""
    def low(q, kc, vc, bt, sl):
        q.fill_(2.0**100)
        kc[:] = -2.0**20
        if ahead:
            kc[bt[0, 2].long(), 5] = -2.0**19
    check(pa, [64], 2, 1, 64, 64, 0, cuda_device, scale=1.0, mutate=low)


def test_infinite_keys_take_or_lose_all_weight(pa, cuda_device):
    x = make([40], 2, 1, 64, 40, 0, 1, cuda_device)
    q, kc, vc, bt, sl = x
    q.fill_(1.0)
    kc[bt[0, 0].long(), 3] = -float("inf")  # weight exactly 0
    out, lse = call(pa, *x, 40, 0, 0.125)
    kc[bt[0, 0].long(), 3] = -3e4
    ref, ref_lse = call(pa, *x, 40, 0, 0.125)
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    kc[:] = -float("inf")  # every score -inf: nothing is attended
    out, lse = call(pa, *x, 40, 0, 0.125)
    assert (out == 0).all() and (lse == -float("inf")).all()
    kc[bt[0, 1].long(), 2] = float("nan")  # a visible NaN is not hidden
    out, _ = call(pa, *x, 40, 0, 0.125)
    assert out.isnan().all()


def test_lengths_out_of_range_are_clamped_and_flagged(pa, cuda_device):
    x = make([32, 40], 2, 1, 64, 20, 4, 2, cuda_device)
    cap = x[3].shape[1] * 16
    full = make([cap, cap], 2, 1, 64, 20, 4, 2, cuda_device)
    q, kc, vc, bt, _ = full
    bt = bt[:, :cap // 16].contiguous()
    good, good_lse = call(pa, q, kc, vc, bt, torch.tensor([0, cap], dtype=torch.int32,
                                                          device=cuda_device), 20, 4, 0.125)
    assert pa.pa_device_error_flags() == 0
    out, lse = call(pa, q, kc, vc, bt, torch.tensor([-5, cap + 1], dtype=torch.int32,
                                                    device=cuda_device), 20, 4, 0.125)
    assert pa.pa_device_error_flags() == pa.PA_DEVERR_SEQ_LEN
    assert torch.equal(out, good) and torch.equal(lse, good_lse)
    assert (out[0] == 0).all()


@pytest.mark.parametrize("bad", [-1, -2**31, 2**31 - 1])
def test_bad_block_reads_as_zeros_and_is_flagged(pa, cuda_device, bad):
    q, kc, vc, bt, sl = make([48], 4, 2, 128, 48, 0, 5, cuda_device)
    zero = kc.shape[0] - 1
    kc[zero], vc[zero] = 0, 0
    bt[0, 1] = zero
    ref, ref_lse = call(pa, q, kc, vc, bt, sl, 48, 0, 0.1)
    bt[0, 1] = bad
    out, lse = call(pa, q, kc, vc, bt, sl, 48, 0, 0.1)
    assert pa.pa_device_error_flags() == pa.PA_DEVERR_BLOCK_ID
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


def test_equal_bits_on_streams_and_graph_replays(pa, cuda_device):
    """Two captured graphs and an eager call in flight at once; a replay sees
    new lengths and queries."""
    x = make([3000, 100, 2047], 8, 2, 128, 2000, 4, 6, cuda_device)
    q, kc, vc, bt, sl = x
    want, want_lse = call(pa, *x, 2000, 4, 0.09)
    outs = [(torch.empty_like(q), torch.empty_like(want_lse)) for _ in range(2)]
    graphs = []
    side = torch.cuda.Stream()
    for o, l in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            pa.pa_decode_window(o, q, kc, vc, bt, sl, 2000, 4, 0.09, out_lse=l)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        eager, eager_lse = call(pa, *x, 2000, 4, 0.09)
    torch.cuda.synchronize()
    for o, l in outs + [(eager, eager_lse)]:
        assert torch.equal(o, want) and torch.equal(l, want_lse)
    sl.copy_(torch.tensor([2999, 0, 2047], dtype=torch.int32))
    q.mul_(0.5)
    want, want_lse = call(pa, *x, 2000, 4, 0.09)
    graphs[0].replay()
    torch.cuda.synchronize()
    # one key shorter, sequence 0's window takes in a slot that holds NaN
    for got, ref in zip(outs[0], (want, want_lse)):
        assert torch.allclose(got, ref, rtol=0, atol=0, equal_nan=True)
    assert want[0].isnan().all() and not want[1:].isnan().any()


def test_rows_behind_the_last_sequence_stay(pa, cuda_device):
    q, kc, vc, bt, sl = make([40, 50, 60], 4, 2, 64, 30, 2, 7, cuda_device)
    out = torch.full((5, 4, 64), 7.0, dtype=torch.bfloat16, device=cuda_device)
    lse = torch.full((5, 4), 7.0, device=cuda_device)
    pa.pa_decode_window(out[1:4], q, kc, vc, bt, sl, 30, 2, 0.125, out_lse=lse[1:4])
    torch.cuda.synchronize()
    assert (out[[0, 4]] == 7).all() and (lse[[0, 4]] == 7).all()
    assert not (out[1:4] == 7).any()
    pa.pa_decode_window(out[1:4], q, kc, vc, bt, sl, 30, 2, 0.125)  # no lse


def test_whole_sequence_matches_pa_decode(pa, cuda_device):
    x = make([300, 17, 64], 8, 2, 128, 10**6, 0, 8, cuda_device)
    out, lse = call(pa, *x, 10**6, 0, 0.09)
    q, kc, vc, bt, sl = x
    kc, vc, bt = kc.nan_to_num(), vc.nan_to_num(), bt.clamp(0, kc.shape[0] - 1)
    ref = torch.empty_like(q)
    ref_lse = torch.empty_like(lse)
    pa.pa_decode(ref, q, kc, vc, bt, sl, 0.09, partition_tokens=-1, out_lse=ref_lse)
    torch.cuda.synchronize()
    assert torch.allclose(out.float(), ref.float(), atol=1e-2, rtol=1e-2)
    assert torch.allclose(lse, ref_lse, atol=1e-4, rtol=1e-5)


def test_argument_forms(pa, cuda_device):
    """An explicit stream, whole numbers of numpy, parameters in place of tensors."""
    x = make([100, 7], 4, 2, 64, 50, 2, 10, cuda_device)
    want, want_lse = call(pa, *x, 50, 2, 0.1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out, lse = call(pa, *x, np.int64(50), np.int32(2), np.float64(0.1), stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    q = torch.nn.Parameter(x[0])
    out, lse = call(pa, q, *x[1:], 50, 2, 0.1)
    assert torch.equal(out, want)
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        out, lse = call(pa, *x, 50, 2, 0.1)
    side.synchronize()
    assert torch.equal(out, want)
    for bad in (50.0, "50", None):
        with pytest.raises(TypeError):
            call(pa, *x, bad, 2, 0.1)


def test_no_sequence_and_no_reference_kept(pa, cuda_device):
    import sys
    q, kc, vc, bt, sl = make([40], 4, 2, 64, 30, 2, 11, cuda_device)
    pa.pa_decode_window(q[:0], q[:0], kc, vc, bt[:0], sl[:0], 30, 2, 0.1)
    before = [sys.getrefcount(t) for t in (q, kc, bt, torch.bfloat16)]
    out = torch.empty_like(q)
    for _ in range(50):
        pa.pa_decode_window(out, q, kc, vc, bt, sl, 30, 2, 0.1)
        with pytest.raises(ValueError):
            pa.pa_decode_window(out, q, kc, vc, bt, sl, 0, 2, 0.1)
    assert [sys.getrefcount(t) for t in (q, kc, bt, torch.bfloat16)] == before


def test_refusals(pa, cuda_device):
    q, kc, vc, bt, sl = make([40, 50], 4, 2, 64, 30, 2, 9, cuda_device)
    out = torch.full_like(q, 3.0)
    go = lambda **k: pa.pa_decode_window(**{**dict(  # noqa: E731
        out=out, q=q, k_cache=kc, v_cache=vc, block_tables=bt, seq_lens=sl, window=30, sinks=2,
        scale=0.1), **k})
    for bad in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(window=2**31),
                dict(sinks=2**32 + 5), dict(out=out[:1]), dict(v_cache=vc[:-1]),
                dict(seq_lens=sl[:1]), dict(block_tables=bt[:1]), dict(q=q[:, :, :32]),
                dict(out_lse=torch.empty(2, 3, device=cuda_device)),
                dict(k_cache=kc.transpose(1, 2)), dict(q=q.cpu()), dict(seq_lens=sl.cpu())):
        with pytest.raises(ValueError):
            go(**bad)
    for bad in (dict(q=q.half()), dict(seq_lens=sl.long()), dict(block_tables=None)):
        with pytest.raises(TypeError):
            go(**bad)
    for bad in (dict(scale=0.0), dict(scale=float("nan")), dict(scale=-1.0)):
        with pytest.raises(pa.PAError) as e:
            go(**bad)
        assert e.value.status == pa.PA_ERR_INVALID
    torch.cuda.synchronize()
    assert (out == 3).all()
    assert pa.pa_device_error_flags() == 0


@pytest.mark.parametrize("q,k", [(1.25 * 2.0**98, 1.125 * 2.0**20),
                                 (1.25 * 2.0**98, -1.125 * 2.0**20),
                                 (1.25 * 2.0**12, 1.125 * 2.0**12),
                                 (1.25 * 2.0**12, -1.125 * 2.0**12)])
@pytest.mark.parametrize("D", [64, 128])
def test_equal_scores_whose_base_2_product_is_rounded_far(pa, cuda_device, q, k, D):
    """All partial sums are exact, so scores are equal and every weight is 1.
    Out: one rounding to bf16, 200 fp32 additions of values, a division.  lse:
    the rounding of the score in base 2 and back, four steps of 2^-24."""
    x = make([200, 1, 3000], 2, 1, D, 200, 0, 1, cuda_device)
    x[0][:], x[1][:] = q, k
    out, lse = call(pa, *x, 200, 0, 1.0)
    torch.cuda.synchronize()
    assert pa.pa_device_error_flags() == 0
    vc, bt = R.to64(x[2]), x[3].cpu().numpy()
    for s, (first, n) in enumerate([(0, 200), (0, 1), (2800, 200)]):
        j = np.arange(first, first + n)
        v = vc[bt[s, j // 16], j % 16, 0]
        ref = np.tile(v.mean(0), (2, 1))
        ref_lse = np.full(2, D * q * k + np.log(n))
        R.assert_within(lse[s], ref_lse, 2.0**-22 * np.abs(ref_lse), "lse")
        R.assert_within(out[s], ref, (2.0**-8 + 2.0**-21) * np.abs(ref) +
                        200 * 2.0**-23 * np.abs(v).max(), "out")


@pytest.mark.parametrize("D,units,blocks", [
    # (sequence, kv head) pairs and visible blocks for which the launcher takes,
    # on 152 SMs, one warp a pair
    (128, 640, 14), (64, 2048, 8),
    # two; 34 to 36 blocks a warp, whose ids come in batches of 32
    (128, 400, 14), (64, 800, 14), (128, 2432, 70),
    # four; 32 and 33 blocks a warp
    (128, 1024, 66), (64, 1024, 66), (64, 1600, 130),
    # eight; up to 38 blocks a warp
    (128, 320, 130), (64, 400, 100), (128, 320, 300)])
def test_more_units_than_run_at_once(pa, cuda_device, D, units, blocks):
    """Sequences that share the blocks of one small pool in random orders."""
    rng = np.random.default_rng(units + blocks)
    g = torch.Generator(device=cuda_device)
    g.manual_seed(units)
    Hkv, pool = 8, 40
    S, window, sinks = units // Hkv, 16 * (blocks - 2), 4
    lens = rng.integers(0, window + 100, S)
    lens[rng.permutation(S)[:S // 2]] += window  # half of them past their window
    lens[:3] = 0, 1, window + sinks
    width = int(lens.max()) // 16 + 1
    rnd = lambda *s: torch.randn(*s, generator=g, device=cuda_device).bfloat16()  # noqa: E731
    q = rnd(S, Hkv * (1 if units * blocks > 60000 else 3), D)
    kc, vc = rnd(pool, 16, Hkv, D), rnd(pool, 16, Hkv, D)
    bt = torch.from_numpy(rng.integers(0, pool, (S, width)).astype(np.int32)).to(cuda_device)
    sl = torch.from_numpy(lens.astype(np.int32)).to(cuda_device)
    out, lse = call(pa, q, kc, vc, bt, sl, window, sinks, D**-0.5)
    torch.cuda.synchronize()
    assert pa.pa_device_error_flags() == 0
    ro, rl, to, tl = R.decode(q, kc, vc, bt, sl, window, sinks, D**-0.5)
    R.assert_within(lse, rl, tl, "lse")
    R.assert_within(out, ro, to, "out")


@pytest.mark.parametrize("D", [64, 128])
def test_a_value_that_is_not_finite_stays_in_its_column(pa, cuda_device, D):
    x = make([60, 40], 4, 2, D, 40, 3, 12, cuda_device)
    want, want_lse = call(pa, *x, 40, 3, 0.1)
    x[2][int(x[3][0, 2]), 5, 1, 7] = float("inf")  # key 37 of sequence 0, kv head 1
    out, lse = call(pa, *x, 40, 3, 0.1)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[0, 2:, 7] = True
    assert not out[hit].isfinite().any()
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse, want_lse)
