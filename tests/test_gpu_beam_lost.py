"""The loop of test_gpu_beam_loop where one request loses all its candidates: its beams are
empty from then on, its prompt still named by the call, and nothing is flagged; the other
requests go on as if it were not there."""
import numpy as np
import pytest
import torch

from tests import beam_ref, window_ref
from tests.test_gpu_beam_loop import D, END, HKV, HQ, LAYERS, V, W, Search

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa(cuda_device):
    from paged_kv_cache_218_gb300 import binding
    binding.pa_device_error_flags()
    return binding


class Losing(Search):
    """A beam without a parent gets no token."""

    def step(self):
        pa = self.pa
        pa.pa_beam_select(self.parents, self.tokens, self.scores, self.logits, self.scores,
                          finished=self.finished, out_finished=self.finished, end_token=END)
        pa.pa_beam_reorder(self.new_tables, self.new_lens, self.tables, self.lens, self.parents,
                           self.k, self.v)
        self.tables.copy_(self.new_tables)
        alive = self.parents.flatten() >= 0
        at = self.new_lens.long()
        block = torch.gather(self.tables, 1, (at // 16)[:, None])[:, 0].long()
        slots = torch.where(alive, block * 16 + at % 16, -1)
        self.lens.copy_(self.new_lens + alive)
        token = self.tokens.flatten().clamp(min=0).long()
        for layer in range(LAYERS):
            x = self.embed[layer][token]
            pa.pa_reshape_and_cache(x[:, HQ:HQ + HKV], x[:, HQ + HKV:], self.k[layer],
                                    self.v[layer], slots)
            self.q[layer].copy_(x[:, :HQ])
            pa.pa_decode_shared(self.out[layer], self.q[layer], self.k[layer], self.v[layer],
                                self.tables, self.lens, self.offsets, W, self.shared, D**-0.5,
                                self.workspace)
        self.logits.copy_((self.out.float().sum(0).flatten(1) @ self.head.float()).view(
            self.logits.shape))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("lost", [0, 1])
def test_a_request_without_candidates(pa, wide, lost):
    rng = np.random.default_rng(5)
    prompts = [rng.integers(8, V, n).tolist() for n in (700, 1500, 300)]
    s = Losing(pa, prompts, 12, wide)
    R = len(prompts)
    history = [[list(p)] + [[] for _ in range(W - 1)] for p in prompts]
    for n in range(12):
        if n == 3:
            s.logits[lost] = -float("inf")
        logits = window_ref.to64(s.logits)
        scores, finished = window_ref.to64(s.scores), s.finished.cpu().numpy()
        s.step()
        torch.cuda.synchronize()
        assert pa.pa_device_error_flags() == 0, n
        par, tok, _, _ = beam_ref.select(logits, scores, finished, END, W)
        assert np.array_equal(s.parents.cpu().numpy(), par)
        history = [[history[r][par[r, i]] + [int(tok[r, i])] if par[r, i] >= 0 else []
                    for i in range(W)] for r in range(R)]
        tables, lens = s.tables.cpu().numpy(), s.lens.cpu().numpy()
        for r in range(R):
            for i in range(W):
                line, row = history[r][i], r * W + i
                assert lens[row] == len(line)
                if n >= 3 and r == lost and not finished[r].any():
                    assert not line and (s.out[:, row] == 0).all()
                ids = torch.from_numpy(tables[row, :(len(line) + 15) // 16].astype(np.int64)).cuda()
                k = s.k[:, ids].flatten(1, 2)[:, :len(line)]
                v = s.v[:, ids].flatten(1, 2)[:, :len(line)]
                assert torch.equal(k, s.embed[:, line, HQ:HQ + HKV])
                if n in (2, 3, 11) and line:
                    q = window_ref.to64(s.q[0, row])
                    out, _, tol, _ = window_ref.attend(q[1], window_ref.to64(k[0])[:, 0],
                                                       window_ref.to64(v[0])[:, 0], D**-0.5,
                                                       2.0**-16)
                    window_ref.assert_within(s.out[0, row, 1], out, tol, (n, r, i))
