"""A beam search over a two-layer cache, the calls together as a serving loop makes them:
selection, reordering, scatter of the chosen tokens, attention behind the shared prompts,
eagerly and as one captured step.  After every step each beam's cache holds its own
history token for token, the attention is that of 64 bits over it, and the choice that of
the logits it was made from."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests import beam_ref, window_ref

pytestmark = pytest.mark.gpu
LAYERS, HQ, HKV, D, V, W = 2, 8, 2, 128, 501, 4
END = 7


@pytest.fixture(scope="module")
def pa(cuda_device):
    from paged_kv_cache_218_gb300 import binding
    binding.pa_device_error_flags()
    return binding


class Search:
    """The device's side of the loop: buffers that stay where they are."""

    def __init__(self, pa, prompts, steps, wide):
        self.pa, self.prompts = pa, prompts
        R = len(prompts)
        g = torch.Generator(device="cuda")
        g.manual_seed(3)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        # a token's query, key and value in each layer
        self.embed = rnd(LAYERS, V, HQ + 2 * HKV, D).bfloat16()
        self.head = (0.3 * rnd(HQ * D, V)).bfloat16()
        own = steps // 16 + 2
        need = sum(len(p) // 16 for p in prompts) + R * W * own
        place = torch.randperm(need + 5, generator=g, device="cuda").cpu().tolist()
        self.k = torch.full((LAYERS, need + 5, 16, HKV, D), float("nan"), dtype=torch.bfloat16,
                            device="cuda")
        self.v = torch.full_like(self.k, float("nan"))
        width = max(len(p) for p in prompts) // 16 + own
        if wide:  # (so that the decode takes the prompts apart)
            width = max(width, (96 << 20) // (R * W * HKV * 8192) + 1)
        tables = np.full((R * W, width), -1, np.int32)
        lens = np.zeros(R * W, np.int32)
        for r, p in enumerate(prompts):
            shared = [place.pop() for _ in range(len(p) // 16)]
            for w in range(W):
                mine = [place.pop() for _ in range(own)]
                row = (shared + mine) if w == 0 else mine  # only beam 0 has the prompt
                tables[r * W + w, :len(row)] = row
            lens[r * W] = len(p)
            for t, token in enumerate(p):
                b = int(tables[r * W, t // 16])
                self.k[:, b, t % 16] = self.embed[:, token, HQ:HQ + HKV]
                self.v[:, b, t % 16] = self.embed[:, token, HQ + HKV:]
        dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        self.tables, self.lens = dev(tables), dev(lens)
        self.new_tables, self.new_lens = torch.empty_like(self.tables), torch.empty_like(self.lens)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.offsets = torch.arange(0, R * W + 1, W, **i32)
        self.shared = torch.tensor([len(p) // 16 for p in prompts], **i32)
        self.scores = torch.full((R, W), -float("inf"), device="cuda")
        self.scores[:, 0] = 0.0
        self.finished = torch.zeros((R, W), dtype=torch.bool, device="cuda")
        self.parents, self.tokens = torch.zeros((R, W), **i32), torch.zeros((R, W), **i32)
        self.logits = rnd(R, W, V).bfloat16()
        self.q = torch.zeros((LAYERS, R * W, HQ, D), dtype=torch.bfloat16, device="cuda")
        self.out = torch.zeros_like(self.q)
        self.workspace = torch.empty(pa.pa_decode_shared_workspace_size(R * W, R, W, HQ, HKV, D),
                                     dtype=torch.uint8, device="cuda")

    def step(self):
        pa = self.pa
        pa.pa_beam_select(self.parents, self.tokens, self.scores, self.logits, self.scores,
                          finished=self.finished, out_finished=self.finished, end_token=END)
        pa.pa_beam_reorder(self.new_tables, self.new_lens, self.tables, self.lens, self.parents,
                           self.k, self.v)
        self.tables.copy_(self.new_tables)
        at = self.new_lens.long()
        block = torch.gather(self.tables, 1, (at // 16)[:, None])[:, 0].long()
        slots = block * 16 + at % 16
        self.lens.copy_(self.new_lens + 1)
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


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("wide", [False, True])
def test_beams_keep_their_histories(pa, captured, wide):
    rng = np.random.default_rng(4)
    prompts = [rng.integers(8, V, n).tolist() for n in (70, 33, 128, 5)]
    steps = 21
    s = Search(pa, prompts, steps, wide)
    R = len(prompts)
    history = [[list(p)] + [[] for _ in range(W - 1)] for p in prompts]
    graph = None
    for n in range(steps):
        logits = window_ref.to64(s.logits)
        scores, finished = window_ref.to64(s.scores), s.finished.cpu().numpy()
        if captured and n == 1:
            # (captured once the loop has run; the buffers it reads and writes stay)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                s.step()
        if graph:
            graph.replay()
        else:
            s.step()
        torch.cuda.synchronize()
        assert pa.pa_device_error_flags() == 0
        par, tok, val, mark = beam_ref.select(logits, scores, finished, END, W)
        assert np.array_equal(s.parents.cpu().numpy(), par)
        assert np.array_equal(s.tokens.cpu().numpy(), tok)
        assert np.array_equal(s.finished.cpu().numpy(), mark)
        history = [[history[r][par[r, i]] + [int(tok[r, i])] for i in range(W)] for r in range(R)]
        tables, lens = s.tables.cpu().numpy(), s.lens.cpu().numpy()
        for r in range(R):
            tails = set()
            for i in range(W):
                line, row = history[r][i], tables[r * W + i]
                assert lens[r * W + i] == len(line)
                ids = torch.from_numpy(row[:(len(line) + 15) // 16].astype(np.int64)).cuda()
                tails.add(int(ids[-1]))
                want = s.embed[:, line]
                k = s.k[:, ids].flatten(1, 2)[:, :len(line)]
                v = s.v[:, ids].flatten(1, 2)[:, :len(line)]
                assert torch.equal(k, want[:, :, HQ:HQ + HKV])
                assert torch.equal(v, want[:, :, HQ + HKV:])
                if n % 5 == 0:
                    for layer in range(LAYERS):
                        kk, vv = window_ref.to64(k[layer]), window_ref.to64(v[layer])
                        q = window_ref.to64(s.q[layer, r * W + i])
                        for h in range(HQ):
                            g = h // (HQ // HKV)
                            out, _, tol, _ = window_ref.attend(q[h], kk[:, g], vv[:, g], D**-0.5,
                                                               2.0**-8)
                            window_ref.assert_within(s.out[layer, r * W + i, h], out, tol,
                                                     (n, r, i, layer, h))
            assert len(tails) == W  # the next tokens go to blocks of the beams' own


FIRST = """
import torch
from paged_kv_cache_218_gb300 import binding as pa
dev = dict(device="cuda")
R, W, V, Hq, Hkv, D = 16, 4, 5000, 8, 2, 128
x = torch.randn((R, W, V), **dev)
scores = torch.zeros((R, W), **dev)
kc, vc = (torch.randn((2 * R * W + R, 16, Hkv, D), **dev).bfloat16() for _ in range(2))
tables = torch.full((R * W, (96 << 20) // (R * W * Hkv * 8192) + 1), -1, dtype=torch.int32, **dev)
tables[:, 0] = torch.arange(R, **dev).repeat_interleave(W)
tables[:, 1:3] = R + torch.arange(2 * R * W, **dev).view(-1, 2)
lens = torch.full((R * W,), 27, dtype=torch.int32, **dev)
q = torch.randn((R * W, Hq, D), **dev).bfloat16()
offsets = torch.arange(R + 1, dtype=torch.int32, **dev) * W
shared = torch.ones(R, dtype=torch.int32, **dev)
made = []
for members in (W, 20, R * W):  # the kernels of 16 query rows, of 128, of pairs
    out = torch.zeros_like(q)
    ws = torch.empty(pa.pa_decode_shared_workspace_size(R * W, R, members, Hq, Hkv, D),
                     dtype=torch.uint8, **dev)
    made.append((pa.pa_decode_shared, (out, q, kc, vc, tables, lens, offsets, members, shared,
                                       D ** -0.5, ws), (out,)))
for dtype in (torch.bfloat16, torch.float32):
    for choices in (4, 40):
        out = (torch.zeros((R, choices), dtype=torch.int32, **dev),
               torch.zeros((R, choices), dtype=torch.int32, **dev), torch.zeros((R, choices), **dev))
        made.append((pa.pa_beam_select, (*out, x.to(dtype), scores), out))
parents = torch.randint(0, W, (R, W), dtype=torch.int32, **dev)
out = (torch.zeros_like(tables), torch.zeros_like(lens))
made.append((pa.pa_beam_reorder, (*out, tables, lens, parents, None, None), out))
torch.cuda.synchronize()
for call, args, out in made:
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(*args)
    graph.replay()
    torch.cuda.synchronize()
    captured = [t.clone() for t in out]
    for t in out:
        t.zero_()
    call(*args)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(captured, out)), call.__name__
    assert any(t.ne(0).any() for t in out), call.__name__
assert pa.pa_device_error_flags() == 0
"""


def test_first_calls_captured(pa):
    """In a process of its own: a kernel's first launch sets its attributes, and asks how many
    of its clusters run at once."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True,
                          timeout=120)
    assert done.returncode == 0, done.stdout + done.stderr
