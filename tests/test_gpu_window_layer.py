"""A sliding-window attention layer served end to end: prompts in chunks, then
decode steps, each step pa_qk_norm_rope_cache followed by pa_prefill_window or
pa_decode_window, with blocks that left the window given back and reused.
Every output row is compared with dense fp64 attention over the whole
sequence's rotated keys, kept aside from k_out."""
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


class Manager:
    """Blocks of each sequence under a window: those without a key that a later
    query can see are freed, and the next block taken is the last one freed."""

    def __init__(self, blocks, width, seqs, window, sinks):
        self.free = list(range(blocks))
        self.tables = np.full((seqs, width), -1, dtype=np.int32)
        self.window, self.sinks = window, sinks

    def slots(self, s, start, count):
        out = []
        for p in range(start, start + count):
            if self.tables[s, p // 16] < 0:
                self.tables[s, p // 16] = self.free.pop()
            out.append(int(self.tables[s, p // 16]) * 16 + p % 16)
        return out

    def trim(self, s, length):
        """The next query stands at `length`."""
        for b in range(self.tables.shape[1]):
            last = b * 16 + 15
            if self.tables[s, b] >= 0 and b * 16 >= self.sinks and last <= length - self.window:
                self.free.append(int(self.tables[s, b]))
                self.tables[s, b] = -1


@pytest.mark.parametrize("Hq,Hkv,window,sinks,interleaved", [
    (8, 2, 100, 4, False), (4, 4, 33, 0, True), (8, 1, 64, 20, False), (2, 1, 1, 1, False)])
def test_chunks_then_decode_steps(pa, cuda_device, Hq, Hkv, window, sinks, interleaved):
    dev = cuda_device
    rng = np.random.default_rng(Hq + window)
    g = torch.Generator(device=dev)
    g.manual_seed(window)
    prompts = [333, 1, 150]
    steps, chunk = 20, 128
    S, scale = len(prompts), 1.0 / math.sqrt(D)
    inc, factor = pa.pa_rope_increments(64, base=10000.0, scaling="yarn", factor=4.0,
                                        original_context=256)
    inc = inc.to(dev)
    qw, kw = (1 + 0.1 * torch.randn(D, generator=g, device=dev) for _ in range(2))
    per_seq = (window + chunk + 31) // 16 + (sinks + 15) // 16 + 2
    man = Manager(S * per_seq, 32, S, window, sinks)
    kc, vc = (torch.full((S * per_seq, 16, Hkv, D), float("nan"), dtype=torch.bfloat16, device=dev)
              for _ in range(2))
    keys = [[] for _ in range(S)]
    values = [[] for _ in range(S)]
    done = [0] * S
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731

    def project(parts):
        """(sequence, first position, count) of the step's rows: norms, rotation, scatter."""
        T = sum(n for _, _, n in parts)
        qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=dev).bfloat16()
        slots = [x for s, p, n in parts for x in man.slots(s, p, n)]
        pos = [x for _, p, n in parts for x in range(p, p + n)]
        q = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
        k = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=dev)
        pa.pa_qk_norm_rope_cache(q, qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:],
                                 torch.tensor(pos, device=dev), inc, kc, vc,
                                 torch.tensor(slots, device=dev), q_weight=qw, k_weight=kw,
                                 interleaved=interleaved, rope_factor=factor, k_out=k)
        return q, k, qkv[:, Hq + Hkv:]

    def keep(parts, k, v):
        row = 0
        for s, _, n in parts:
            keys[s] += list(R.to64(k[row:row + n]))
            values[s] += list(R.to64(v[row:row + n]))
            row += n

    def check(parts, q, out, p_step):
        q, row = R.to64(q), 0
        got = R.to64(out)
        for s, p, n in parts:
            k, v = np.array(keys[s]), np.array(values[s])
            for i in range(n):
                j = R.visible(p + i, window, sinks)
                for h in range(Hq):
                    o, _, tol, _ = R.attend(q[row, h], k[j, h * Hkv // Hq], v[j, h * Hkv // Hq],
                                            scale, p_step)
                    R.assert_within(got[row, h], o, tol, (s, p + i, h))
                row += 1

    while any(d < n for d, n in zip(done, prompts)):
        parts = [(s, done[s], min(int(rng.integers(1, chunk + 1)), n - done[s]))
                 for s, n in enumerate(prompts) if done[s] < n]
        q, k, v = project(parts)
        out = torch.full_like(q, float("nan"))
        pa.pa_prefill_window(
            out, q, kc, vc, torch.from_numpy(man.tables[[s for s, _, _ in parts]]).to(dev),
            i32(np.cumsum([0] + [n for _, _, n in parts]).tolist()), i32([p for _, p, _ in parts]),
            i32([p + n for _, p, n in parts]), max(n for _, _, n in parts), window, sinks, scale)
        torch.cuda.synchronize()
        keep(parts, k, v)
        check(parts, q, out, 2.0**-8)
        for s, p, n in parts:
            done[s] += n
            man.trim(s, done[s])
    for _ in range(steps):
        parts = [(s, done[s], 1) for s in range(S)]
        q, k, v = project(parts)
        out = torch.full_like(q, float("nan"))
        pa.pa_decode_window(out, q, kc, vc, torch.from_numpy(man.tables).to(dev),
                            i32([d + 1 for d in done]), window, sinks, scale)
        torch.cuda.synchronize()
        keep(parts, k, v)
        check(parts, q, out, 2.0**-16)
        for s in range(S):
            done[s] += 1
            man.trim(s, done[s])
    assert pa.pa_device_error_flags() == 0
    # the prompts' middles were given back on the way
    assert (man.tables[0, :(done[0] - window) // 16] < 0).sum() > 0


def test_offsets_past_32_bits(pa, cuda_device):
    """Pools of more than 2^32 elements, of which the layer uses the last
    blocks, and a query tensor whose used rows lie past 2^31 elements: the
    bits of the same calls on a few blocks and rows."""
    Hq, Hkv, D, T, window, sinks = 16, 8, 128, 90, 40, 3
    g = torch.Generator(device=cuda_device)
    g.manual_seed(12)
    rnd = lambda *s: torch.randn(*s, generator=g, device=cuda_device).bfloat16()  # noqa: E731
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=cuda_device)  # noqa: E731
    q, k, v, w = rnd(T, Hq, D), rnd(T, Hkv, D), rnd(T, Hkv, D), torch.ones(D, device=cuda_device)
    pos = torch.arange(T, device=cuda_device)
    inc = pa.pa_rope_increments(D)[0].to(cuda_device)

    def run(blocks, first, stride):
        kc = torch.empty(blocks, 16, Hkv, D, dtype=torch.bfloat16, device=cuda_device)
        vc = torch.empty_like(kc)
        tail = blocks - 6
        kc[tail:], vc[tail:] = 0, 0
        table = torch.arange(blocks - 1, tail - 1, -1, dtype=torch.int32, device=cuda_device)[None]
        slots = table[0, pos // 16].long() * 16 + pos % 16
        wide = torch.empty(T, stride, dtype=torch.bfloat16, device=cuda_device)
        qs = wide[:, first:first + Hq * D].unflatten(1, (Hq, D))
        qs.copy_(q)
        rot, out, last = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q[:1])
        pa.pa_qk_norm_rope_cache(rot, qs, k, v, pos, inc, kc, vc, slots, w, w)
        pa.pa_prefill_window(out, rot, kc, vc, table, i32(0, T), i32(0), i32(T), T, window, sinks,
                             0.09)
        pa.pa_decode_window(last, rot[-1:].contiguous(), kc, vc, table, i32(T), window, sinks, 0.09)
        torch.cuda.synchronize()
        return rot, kc[tail:].clone(), vc[tail:].clone(), out, last

    small = run(6, 0, Hq * D)
    far = run(2**18 + 100, 2**24, 2**25)
    assert pa.pa_device_error_flags() == 0
    for a, b in zip(small, far):
        assert torch.equal(a, b)


def test_first_calls_of_a_process_may_be_captured(cuda_device):
    """Nothing that a first call sets up is forbidden while a graph is captured."""
    import os
    import subprocess
    import sys
    code = """
import torch
from paged_kv_cache_218_gb300 import binding as pa
T, Hq, Hkv, D = 64, 8, 2, 128
r = lambda *s: torch.randn(*s, device="cuda").bfloat16()
i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
q, k, kc, vc = r(T, Hq, D), r(T, Hkv, D), r(8, 16, Hkv, D), r(8, 16, Hkv, D)
bt, pos = torch.arange(4, dtype=torch.int32, device="cuda")[None], torch.arange(T, device="cuda")
inc = pa.pa_rope_increments(D)[0].cuda()
lens, cu, start = i(T), i(0, T), i(0)
outs = [torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q[:1])]
last = q[-1:].contiguous()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    pa.pa_decode_window(outs[2], last, kc, vc, bt, lens, 33, 2, 0.1)
    pa.pa_prefill_window(outs[1], q, kc, vc, bt, cu, start, lens, T, 33, 2, 0.1)
    pa.pa_qk_norm_rope_cache(outs[0], q, k, k, pos, inc, kc, vc, pos)
g.replay()
torch.cuda.synchronize()
assert all(o.abs().sum() > 0 for o in outs) and pa.pa_device_error_flags() == 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("Hq,Hkv,window,sinks,interleaved", [
    (16, 16, 100, 4, False), (16, 8, 33, 0, True), (64, 8, 64, 20, False)])
def test_a_layer_of_many_kv_heads(pa, cuda_device, Hq, Hkv, window, sinks, interleaved):
    """The same, with enough (token, kv head) pairs for tiles in most chunk steps."""
    test_chunks_then_decode_steps(pa, cuda_device, Hq, Hkv, window, sinks, interleaved)


@pytest.mark.parametrize("Hkv", [1, 8])
def test_first_prefill_of_a_process_may_be_captured(cuda_device, Hkv):
    """On both sides of the choice between queries one by one and in tiles (64
    and 512 (token, kv head) pairs)."""
    import os
    import subprocess
    import sys
    code = f"""
import torch
from paged_kv_cache_218_gb300 import binding as pa
T, Hkv, D = 64, {Hkv}, 128
r = lambda *s: torch.randn(*s, device="cuda").bfloat16()
i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
q, kc, vc = r(T, 2 * Hkv, D), r(8, 16, Hkv, D), r(8, 16, Hkv, D)
bt, lens, cu, start = torch.arange(4, dtype=torch.int32, device="cuda")[None], i(T), i(0, T), i(0)
out, again = torch.zeros_like(q), torch.zeros_like(q)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    pa.pa_prefill_window(out, q, kc, vc, bt, cu, start, lens, T, 33, 2, 0.1)
g.replay()
pa.pa_prefill_window(again, q, kc, vc, bt, cu, start, lens, T, 33, 2, 0.1)
torch.cuda.synchronize()
assert out.abs().sum() > 0 and torch.equal(out, again) and pa.pa_device_error_flags() == 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
