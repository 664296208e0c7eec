"""pa_beam_select against the 64-bit definition: the same candidates in the same order,
scores within the roundings of one fp32 pass."""
import math

import numpy as np
import pytest
import torch

from tests import beam_ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def pa(cuda_device):
    from paged_kv_cache_218_gb300 import binding
    return binding


class Case:
    def __init__(self, logits, scores, choices, finished=None, end=-1):
        self.logits, self.scores, self.finished, self.end = logits, scores, finished, end
        shape, dev = (logits.shape[0], choices), logits.device
        self.parents = torch.full(shape, 77, dtype=torch.int32, device=dev)
        self.tokens = torch.full(shape, 77, dtype=torch.int32, device=dev)
        self.out_scores = torch.full(shape, 77.0, device=dev)
        self.marks = torch.ones(shape, dtype=torch.bool, device=dev)

    def run(self, pa, stream=None):
        pa.pa_beam_select(self.parents, self.tokens, self.out_scores, self.logits, self.scores,
                          finished=self.finished, out_finished=self.marks, end_token=self.end,
                          stream=stream)

    def check(self):
        fin = None if self.finished is None else self.finished.cpu().numpy().astype(bool)
        par, tok, val, mark = beam_ref.select(
            self.logits.double().cpu().numpy(), self.scores.double().cpu().numpy(), fin, self.end,
            self.parents.shape[1])
        assert np.array_equal(self.parents.cpu().numpy(), par)
        assert np.array_equal(self.tokens.cpu().numpy(), tok)
        assert np.array_equal(self.marks.cpu().numpy(), mark)
        got = self.out_scores.double().cpu().numpy()
        some = par >= 0
        assert (got[~some] == -np.inf).all()
        tol = beam_ref.score_tolerance(val[some], self.logits.shape[2], self.logits.dtype == F32)
        assert (np.abs(got[some] - val[some]) <= tol).all()


def make(gen, R, W, V, K, dtype, spread=3.0, **kw):
    x = (spread * torch.randn((R, W, V), generator=gen, device="cuda")).to(dtype)
    s = -3.0 * torch.rand((R, W), generator=gen, device="cuda").cumsum(1)
    return Case(x, s, K, **kw)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R,W,V,K", [
    (1, 1, 1, 1), (1, 1, 7, 3), (2, 4, 33, 8), (3, 1, 5000, 1), (1, 4, 32000, 4), (5, 3, 50001, 5),
    (2, 32, 1000, 64), (3, 8, 4096, 31), (3, 8, 4097, 32), (2, 5, 70000, 33), (1, 32, 40000, 63),
    (40, 4, 3000, 8), (1, 2, 300000, 4), (1, 32, 290000, 16)])
def test_sizes(pa, R, W, V, K, dtype):
    c = make(gen(R * 1000 + V), R, W, V, K, dtype)
    c.run(pa)
    c.check()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R,W,V,K", [
    (8, 27, 2123, 54), (1, 32, 16705, 64), (20, 17, 65, 43), (5, 9, 131, 54), (70, 6, 50497, 57)])
def test_many_choices(pa, R, W, V, K, dtype):
    """Many choices out of few parts of the rows; the candidates of one beam, of two beams
    and of all of them far above the others'."""
    c = make(gen(V), R, W, V, K, dtype)
    c.scores[0, 1:] -= 60.0
    if R > 3:
        c.scores[1, 2:] -= 60.0
        c.scores[2, :] = c.scores[2, :1]
    c.run(pa)
    c.check()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("offset,pad", [(0, 1), (1, 0), (3, 5), (8, 8), (13, 31)])
def test_strides_and_alignment(pa, dtype, offset, pad):
    """Rows that begin anywhere, of a wider matrix, requests apart, beams in another order."""
    R, W, V = 3, 4, 777
    g = gen(offset)
    base = torch.full((offset + (R + 1) * 5 * (V + pad) + 64,), math.inf, device="cuda",
                      dtype=dtype)
    x = torch.as_strided(base, (R, W, V), (5 * (V + pad), V + pad, 1), offset)
    x.copy_(torch.randn((R, W, V), generator=g, device="cuda"))
    scores = -torch.rand((R, W), generator=g, device="cuda")
    c = Case(x, scores, 8)
    c.run(pa)
    c.check()
    t = Case(x.transpose(0, 1), scores.t().contiguous(), 6)
    t.run(pa)
    t.check()


def test_offsets_past_32_bits(pa):
    """Beams and requests beyond 2^32 bytes, and 2^32 elements, of one another."""
    base = torch.empty(((1 << 32) + (1 << 31) + 60000,), device="cuda", dtype=BF16)
    x = torch.as_strided(base, (2, 2, 50021), (1 << 32, (1 << 31) + 7, 1), 3)
    x.copy_(3 * torch.randn((2, 2, 50021), generator=gen(21), device="cuda"))
    s = -torch.rand((2, 2), generator=gen(22), device="cuda")
    c = Case(x, s, 6)
    c.run(pa)
    c.check()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ties(pa, dtype):
    """Few distinct logits, many of them equal; whole rows equal; beams equal to one another."""
    g = gen(5)
    x = torch.randint(-3, 2, (4, 3, 5000), generator=g, device="cuda").to(dtype)
    x[1] = 0.25
    x[2] = x[2, 0]
    x[3, 2] = x[3, 1]
    scores = torch.tensor([[0.0, -0.125, -0.25], [-1.0, -1.0, -1.0], [-2.0, -2.0, -2.0],
                           [-9.0, -1.0, -1.0]], device="cuda")
    for k in (1, 7, 31, 64):
        c = Case(x, scores, k)
        c.run(pa)
        c.check()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_equal_beams_at_other_alignments(pa, dtype):
    """Equal rows that begin at different places of their 32 bytes tie all the same."""
    V = 10007
    row = (2 * torch.randn(V, generator=gen(6), device="cuda")).to(dtype)
    base = torch.zeros((6 * (V + 3) + 5,), device="cuda", dtype=dtype)
    x = torch.as_strided(base, (1, 6, V), (6 * (V + 3), V + 3, 1), 5)
    x.copy_(row.expand(1, 6, V))
    c = Case(x, torch.full((1, 6), -4.0, device="cuda"), 40)
    c.run(pa)
    c.check()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("steps", [1, 2, 3])
def test_beams_a_rounding_apart(pa, dtype, steps):
    """The same logits in another order, scores some fp32 steps apart: the sums of one
    fp32 pass could not tell these beams apart."""
    V = 30011
    g = gen(steps)
    row = (2 * torch.randn(V, generator=g, device="cuda")).to(dtype)
    x = torch.stack([row[torch.randperm(V, generator=g, device="cuda")] for _ in range(8)])[None]
    s = np.full(8, np.float32(-7.0))
    order = np.random.default_rng(steps).permutation(8)
    for i, w in enumerate(order):
        for _ in range(i * steps):
            s[w] = np.nextafter(s[w], np.float32(-100.0))
    c = Case(x, torch.tensor(s, device="cuda")[None], 24)
    c.run(pa)
    c.check()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R", [1, 3, 40, 160])
@pytest.mark.parametrize("few", [True, False])
def test_sums_taken_again_by_whole_clusters(pa, dtype, R, few):
    """Beams of the same logits in another order, a rounding apart or equal, in calls large
    enough for every CTA of a cluster (of 16, 13, 7, 1) to take its share; few: candidates that
    are gathered, or so many equal ones that lists find them.  Some requests have no doubt."""
    V, K = 70001, 33
    g = gen(R)
    row = 2 * torch.randn(V, generator=g, device="cuda") if few else \
        torch.randint(-3, 2, (V,), generator=g, device="cuda").float()
    x = torch.stack([row[torch.randperm(V, generator=g, device="cuda")]
                     for _ in range(4)]).to(dtype)[None].expand(R, 4, V).contiguous()
    s = torch.full((R, 4), -7.0, device="cuda")
    s[:, 1] = torch.nextafter(s[:, 1], torch.zeros_like(s[:, 1]))
    s[::3, 1:] -= torch.tensor([20.0, 40.0, 60.0], device="cuda")
    c = Case(x, s, K)
    c.run(pa)
    # (one request of each kind, and that all of a kind are the same)
    for i in range(R):
        first = 0 if i % 3 == 0 else 1
        for t in (c.parents, c.tokens, c.out_scores):
            assert torch.equal(t[i], t[first])
    n = min(R, 2)
    c.logits, c.scores = x[:n], s[:n]
    c.parents, c.tokens, c.out_scores, c.marks = (
        t[:n] for t in (c.parents, c.tokens, c.out_scores, c.marks))
    c.check()


def test_displaced_by_the_last_choice_s_own_row(pa):
    """Beam 1's best lies a rounding above beam 0's K-th candidate, which ties with more of
    its own row: the K + 1 best of an fp32 pass may all be beam 0's."""
    V = 4096
    for step in (-1, 0, 1):
        x = torch.full((1, 2, V), -8.0, device="cuda")
        x[0, 0, 100:140] = 3.0
        x[0, 1, 7] = 3.0
        x[0, 1, 2000:2039] = 3.0  # the same sum in another order
        s = np.array([-5.0, -5.0], dtype=np.float32)
        if step:
            s[1] = np.nextafter(s[1], np.float32(100.0 * step))
        for k in (1, 3, 20):
            c = Case(x, torch.tensor(s, device="cuda")[None], k)
            c.run(pa)
            c.check()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_forbidden_tokens(pa, dtype):
    """-inf logits; rows with few or none others; the type's lowest value; NaN and +inf."""
    g = gen(8)
    x = (2 * torch.randn((6, 4, 3001), generator=g, device="cuda")).to(dtype)
    low = torch.finfo(dtype).min
    x[0, :, 5:] = -math.inf
    x[1] = -math.inf
    x[1, 2, 3000] = -7.0
    x[2, 0] = -math.inf
    x[2, 1] = low
    x[2, 2, 10:] = low
    x[3] = low
    x[4, 0, ::3] = math.nan
    x[4, 1, 1::2] = math.inf
    x[4, 2] = math.nan
    x[4, 3] = math.inf
    x[4, 3, 1234] = 0.5
    x[5, :2] = -math.inf
    x[5, 2, 17] = -math.inf
    for k in (2, 9, 40):
        c = Case(x, -torch.rand((6, 4), generator=g, device="cuda"), k)
        c.run(pa)
        c.check()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ended_and_absent_beams(pa, dtype):
    """Ended beams propose their end token once; beams at -inf (or no number) nothing,
    whatever their logits hold."""
    g = gen(9)
    x = torch.randn((5, 4, 2000), generator=g, device="cuda").to(dtype)
    scores = -5 * torch.rand((5, 4), generator=g, device="cuda")
    fin = torch.zeros((5, 4), dtype=torch.bool, device="cuda")
    fin[0, 1] = fin[1, :] = fin[2, 3] = fin[3, 0] = fin[4, 0] = True
    scores[2, :3] = -math.inf
    scores[3, 1], scores[3, 0] = math.nan, -math.inf
    scores[4] = -1.0
    x[0, 1] = math.nan
    x[2, :3] = math.nan
    for end in (0, 999, 1999):
        for k in (1, 4, 8):
            c = Case(x, scores, k, finished=fin, end=end)
            c.run(pa)
            c.check()
            c.finished = fin.to(torch.uint8)
            c.run(pa)
            c.check()


def test_nothing_at_all(pa):
    x = torch.zeros((2, 3, 100), device="cuda")
    c = Case(x, torch.full((2, 3), -math.inf, device="cuda"), 5)
    c.run(pa)
    c.check()
    assert (c.parents == -1).all()
    empty = Case(x[:0], torch.zeros((0, 3), device="cuda"), 5)
    empty.run(pa)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_orders_that_move_every_list(pa, dtype):
    """Logits that rise with the token, fall, or rise within blocks only."""
    V = 20000
    up = torch.linspace(-90, 5, V, device="cuda")
    x = torch.stack([up, up.flip(0), up.view(-1, 40).t().reshape(-1)])[None].to(dtype)
    c = Case(x, torch.tensor([[-1.0, -1.25, -1.5]], device="cuda"), 64)
    c.run(pa)
    c.check()


@pytest.mark.parametrize("scale", [1e-30, 1e3, 1e30, 3e38])
def test_far_logits(pa, scale):
    g = gen(11)
    x = torch.rand((2, 4, 3000), generator=g, device="cuda") * scale
    c = Case(x, -torch.rand((2, 4), generator=g, device="cuda"), 8)
    c.run(pa)
    c.check()


@pytest.mark.parametrize("V", [40, 3000])
def test_values_past_fp32(pa, V):
    """Logits of -3e38 behind a score of -1e38 have no value in fp32: no candidates, in few
    blocks as in lists."""
    x = torch.full((2, 2, V), -3e38, device="cuda")
    x[:, :, 5:8] = torch.tensor([1.0, 3.0, 2.0], device="cuda")
    x[1, 0] = -3e38
    s = torch.full((2, 2), -1e38, device="cuda")
    s[1, 1] = -1.0
    c = Case(x, s, 16)
    c.run(pa)
    par, tok = c.parents.cpu().tolist(), c.tokens.cpu().tolist()
    # (the logits tell -1e38 + 3 from -1e38 + 2: a value's second float holds them)
    assert par[0] == [0, 1] * 3 + [-1] * 10 and tok[0] == [6, 6, 7, 7, 5, 5] + [-1] * 10
    # (beam 0 of request 1: every logit the same, -3e38 - ln V behind the sum; beam 1's
    # -3e38 - 1 are values)
    assert par[1] == [1] * 3 + [0] * 13 and tok[1] == [6, 7, 5] + list(range(13))
    assert torch.isinf(c.out_scores[0, 6:]).all() and (c.out_scores[0, :6] < -9e37).all()


def test_scores_in_place_and_a_few_steps(pa):
    """Outputs over the inputs they replace, as a loop keeps them."""
    g = gen(12)
    scores = torch.full((6, 4), -math.inf, device="cuda")
    scores[:, 0] = 0.0
    fin = torch.zeros((6, 4), dtype=torch.bool, device="cuda")
    for step in range(4):
        x = (3 * torch.randn((6, 4, 900), generator=g, device="cuda")).to(BF16)
        x[:, :, 3] += 6.0  # the end token is likely
        c = Case(x, scores.clone(), 4, finished=fin.clone(), end=3)
        c.out_scores, c.marks = scores, fin
        pa.pa_beam_select(c.parents, c.tokens, scores, x, scores, finished=fin, out_finished=fin,
                          end_token=3)
        c.check()


def test_captured_replayed_and_on_two_streams(pa):
    g = gen(13)
    cases = [make(g, 9, 4, 8000, 8, BF16) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(cases, streams):
            c.run(pa, stream=s)
    torch.cuda.synchronize()
    for c in cases:
        c.check()
    c = make(g, 3, 5, 6000, 33, F32)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(pa)
    for _ in range(2):
        c.logits.copy_(torch.randn(c.logits.shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        c.check()


def test_first_call_of_a_variant_captured(pa):
    """(the launch sets attributes of its kernel the first time)"""
    g = gen(14)
    c = make(g, 2, 3, 5000, 64, BF16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(pa)
    graph.replay()
    torch.cuda.synchronize()
    c.check()


def test_equal_calls_give_equal_bits(pa):
    c = make(gen(15), 20, 8, 60000, 16, BF16)
    c.run(pa)
    first = [t.clone() for t in (c.parents, c.tokens, c.out_scores)]
    for _ in range(5):
        c.run(pa)
        assert all(torch.equal(x, y) for x, y in zip(first, (c.parents, c.tokens, c.out_scores)))


def test_refusals_of_the_binding(pa):
    c = make(gen(16), 2, 3, 100, 4, BF16)
    with pytest.raises(ValueError, match="contiguous"):
        pa.pa_beam_select(c.parents, c.tokens, c.out_scores, c.logits.transpose(1, 2), c.scores)
    with pytest.raises(ValueError, match="scores"):
        pa.pa_beam_select(c.parents, c.tokens, c.out_scores, c.logits, c.scores[:, :2])
    with pytest.raises(ValueError, match="tokens"):
        pa.pa_beam_select(c.parents, c.tokens[:, :3], c.out_scores, c.logits, c.scores)
    with pytest.raises(pa.PAError):
        pa.pa_beam_select(c.parents, c.tokens, c.out_scores, c.logits, c.scores, end_token=100)
    with pytest.raises(pa.PAError):
        pa.pa_beam_select(c.parents, c.parents, c.out_scores, c.logits, c.scores)
