"""pa_beam_select where beams are held back and tokens forbidden by finite numbers, and beams
have ended beside them: against the definition in exact arithmetic (a double cannot tell
-3.4e38 - 1 from -3.4e38 - 2; the call's pairs of floats can)."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from tests import beam_ref
from tests.test_gpu_beam_select import BF16, F32, Case, gen

pytestmark = pytest.mark.gpu
PAST = Fraction(float(np.finfo(np.float32).max)) + Fraction(2)**103  # rounds to infinity


@pytest.fixture(scope="module")
def pa(cuda_device):
    from paged_kv_cache_218_gb300 import binding
    return binding


def expect(c):
    """[(value, beam, token)] of each request, best first.  A row's best are its largest logits,
    so K of each row are enough; those whose values round to -infinity are none."""
    x, s = c.logits.double().cpu().numpy(), c.scores.double().cpu().numpy()
    fin = None if c.finished is None else c.finished.cpu().numpy().astype(bool)
    K, out = c.parents.shape[1], []
    for r in range(x.shape[0]):
        some = []
        for w in range(x.shape[1]):
            if not math.isfinite(s[r, w]):
                continue
            if fin is not None and fin[r, w]:
                some.append((Fraction(s[r, w]), w, c.end))
                continue
            row = np.where(np.isfinite(x[r, w]), x[r, w], -np.inf)
            top = row.max()
            if top == -np.inf:
                continue
            with np.errstate(over="ignore"):
                e = np.exp(row - top)
            lse = Fraction(top) + Fraction(math.log(math.fsum(e[e > 0])))
            for t in np.argsort(-row, kind="stable")[:K]:
                if row[t] > -np.inf:
                    some.append((Fraction(s[r, w]) + Fraction(row[t]) - lse, w, int(t)))
        some = [y for y in some if abs(y[0]) < PAST]
        out.append(sorted(some, key=lambda y: (-y[0], y[1], y[2]))[:K])
    return out


def check(c):
    par, tok, val, mark = (t.cpu().tolist() for t in (c.parents, c.tokens, c.out_scores, c.marks))
    fin = None if c.finished is None else c.finished.cpu().tolist()
    V, K = c.logits.shape[2], len(par[0])
    for r, best in enumerate(expect(c)):
        n = len(best)
        assert list(zip(par[r], tok[r])) == [(w, t) for _, w, t in best] + [(-1, -1)] * (K - n), r
        assert val[r][n:] == [-math.inf] * (K - n)
        for i, (v, w, t) in enumerate(best):
            tol = beam_ref.score_tolerance(float(v), V, c.logits.dtype == F32)
            assert abs(val[r][i] - float(v)) <= tol, (r, i, val[r][i], float(v))
            assert mark[r][i] == bool((fin and fin[r][w]) or t == c.end)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [40, 2000, 32000, 70000])
@pytest.mark.parametrize("low", ["lowest", -1e9, -math.inf])
@pytest.mark.parametrize("allowed", [1, 10])
def test_few_allowed_tokens_beside_ended_beams(pa, dtype, V, low, allowed):
    """Fewer allowed tokens than choices, in few blocks of the rows or in more than 256; beams
    that have ended, are absent, or both; the end token among the allowed ones or not."""
    low = torch.finfo(dtype).min if low == "lowest" else low
    g = gen(V + allowed)
    x = torch.full((5, 4, V), low, device="cuda")
    x[..., 10:10 + allowed] = 2 * torch.randn((5, 4, allowed), generator=g, device="cuda")
    x = x.to(dtype)
    scores = -5 * torch.rand((5, 4), generator=g, device="cuda")
    fin = torch.zeros((5, 4), dtype=torch.bool, device="cuda")
    fin[0, 1] = fin[1, 0] = fin[1, 2] = fin[2, 3] = fin[4, :] = True
    scores[2, 1] = scores[3, 0] = scores[4, 2] = -math.inf
    scores[1, 0] = math.nan
    for end in (0, 12, V - 1):
        for k in (1, 4, 9, 40):
            c = Case(x, scores, k, finished=fin, end=end)
            c.run(pa)
            check(c)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("low", [-math.inf, -1e9, float(np.finfo(np.float32).min)])
@pytest.mark.parametrize("R,W,V,K", [(3, 4, 32000, 4), (2, 6, 5, 20), (2, 4, 70001, 33)])
def test_beams_held_back_by_finite_scores(pa, dtype, low, R, W, V, K):
    """The first step of a search: one beam begun, the others held at a finite lowest score;
    beside them a request whose beams are all held so, and one with an ended beam."""
    g = gen(V)
    x = torch.randint(-40, 40, (R, W, V), generator=g, device="cuda").div(8.0).to(dtype)
    s = torch.full((R, W), low, device="cuda")
    s[0, 1] = -1.5
    fin = torch.zeros((R, W), dtype=torch.bool, device="cuda")
    fin[R - 1, 2] = True
    s[R - 1, 2] = -2.5
    c = Case(x, s, K, finished=fin, end=V // 2)
    c.run(pa)
    check(c)


@pytest.mark.parametrize("V", [40, 3000, 70000])
@pytest.mark.parametrize("K", [3, 8, 40])
def test_far_scores_and_far_logits_together(pa, V, K):
    """A score and a row's largest logit whose difference leaves fp32 where their candidates'
    values do not, on either side; beside them an ended and an ordinary beam."""
    x = torch.full((4, 4, V), -3e38, device="cuda")
    g = gen(V + K)
    x[0, 0, 3:9] = torch.tensor([3e38, 2e38, 1e38, 3e38, -1e38, 2.5e38], device="cuda")
    x[0, 1] = 1e38 * torch.rand(V, generator=g, device="cuda")
    x[1] = 3.4e38
    x[1, :, ::2] = 1.7e38
    x[2] = -3.4e38
    x[3] = 3e38 * (2 * torch.rand((4, V), generator=g, device="cuda") - 1)
    s = torch.tensor([[-1e38, -2e38, -5.0, -3e38], [-3.4e38, -3.3e38, -3.4e38, -1.0],
                      [3e38, 3.4e38, 1e38, -3e38], [-3e38, 3e38, 0.0, -1e38]], device="cuda")
    fin = torch.zeros((4, 4), dtype=torch.bool, device="cuda")
    fin[:, 2] = True
    c = Case(x, s, K, finished=fin, end=1)
    c.run(pa)
    check(c)


@pytest.mark.parametrize("low", [-1e9, float(np.finfo(np.float32).min)])
def test_held_back_beams_cost_no_more_than_others(pa, low):
    """Beams 1 .. 3 at a finite lowest score: the call reads their logits, as it does those of
    ordinary beams, and takes no longer (2 for noise; it took 4.5 times as long)."""
    R, W, V, K = 64, 4, 131072, 8
    x = (3 * torch.randn((R, W, V), generator=gen(1), device="cuda")).to(BF16)
    plain = -5.0 - 3.0 * torch.rand((R, W), generator=gen(2), device="cuda").cumsum(1)
    held = plain.clone()
    held[:, 1:] = low
    best = []
    for s in (plain, held):
        c, times = Case(x, s, K), []
        for _ in range(12):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            c.run(pa)
            a.record()
            for _ in range(5):
                c.run(pa)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        best.append(min(times))
    assert best[1] < 2 * best[0], best


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scores_within_the_stated_bound(pa, dtype):
    """One CTA for all 32 rows of a request, so that a lane sums as much as it ever does."""
    R, W, V, K = 160, 32, 40000, 4
    x = (3 * torch.randn((R, W, V), generator=gen(3), device="cuda")).to(dtype)
    s = -5.0 * torch.rand((R, W), generator=gen(4), device="cuda")
    c = Case(x, s, K)
    c.run(pa)
    lse = torch.stack([torch.logsumexp(y.double(), -1) for y in x])
    at = torch.arange(R, device="cuda")[:, None], c.parents.long(), c.tokens.long()
    value = s.double()[at[:2]] + x[at].double() - lse[at[:2]]
    bound = 2.0**-24 * value.abs() + 1.3e-5 + 2.5e-10 * V
    assert ((c.out_scores.double() - value).abs() <= bound).all()
