"""pa_qk_norm_rope_cache and its E4M3 form against the fp64 definition.

Tolerance of a bf16 output y' = f (a cos u -+ b sin u) of normed values a, b:
half a step of bf16 (2^-8 relative), plus fp32 arithmetic on |a| + |b|: the
sum of D squares is off by at most D 2^-24, rsqrt and the products by a few
2^-23, sincospif's argument by 2^-25 half turns (2^-23 rad) and its result by
two steps: (D 2^-24 + 2^-19) f (|a| + |b|) covers them.  An E4M3 code: half a
step, 2^-4 relative or 2^-10 among the subnormals, and the same fp32 part over
the scale."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa(cuda_device):
    from paged_kv_cache_218_gb300 import binding
    return binding


def to64(t):
    return t.detach().double().cpu().numpy()


def phases(positions, increments):
    """Exact angles in radians: whole turns dropped in integer arithmetic."""
    p = [[(int(x) * int(i)) % (1 << 64) for i in increments] for x in positions]
    return 2 * math.pi * (np.array(p, dtype=object) / 2**64).astype(np.float64)


def reference(x, w, eps, angle, rot, interleaved, factor):
    """(y, fp32 error bound of y) of rows x [T, H, D]."""
    x = to64(x)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * to64(w)
    D = x.shape[-1]
    y, size = x.copy(), np.abs(x)
    if rot:
        c, s = np.cos(angle)[:, None] * factor, np.sin(angle)[:, None] * factor
        i = np.arange(rot // 2)
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        size[..., ia] = size[..., ib] = abs(factor) * (np.abs(a) + np.abs(b))
    return y, (D * 2.0**-24 + 2.0**-19) * size


class Case:
    def __init__(self, T, Hq, Hkv, D, rot, device, seed=0, norm=True, fused=True, interleaved=False,
                 factor=1.0, positions=None, f8=False, pad=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
        self.T, self.Hq, self.Hkv, self.D, self.rot = T, Hq, Hkv, D, rot
        if fused:
            qkv = rnd(T, Hq + 2 * Hkv + pad, D).bfloat16()
            self.q, self.k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
            self.v = qkv[:, Hq + Hkv:Hq + 2 * Hkv]
        else:
            self.q, self.k, self.v = (rnd(T, h, D).bfloat16() for h in (Hq, Hkv, Hkv))
        self.qw = 1 + 0.2 * rnd(D) if norm else None
        self.kw = 1 + 0.2 * rnd(D) if norm else None
        self.eps, self.interleaved, self.factor, self.f8 = 1e-5, interleaved, factor, f8
        self.increments = self.positions = None
        if rot:
            f = 10000.0 ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
            self.increments = (f / (2 * math.pi) * 2.0**64).to(torch.int64).to(device)
            self.positions = torch.randint(0, 131072, (T,), generator=g, device=device)
            if positions is not None:
                self.positions = torch.tensor(positions, dtype=torch.int64, device=device)
        blocks = (T + 15) // 16 + 2
        self.slots = torch.randperm(blocks * 16, generator=g, device=device)[:T]
        shape = (blocks, 16, Hkv, D)
        self.scales = ()
        if f8:
            self.kc, self.vc = (torch.randint(0, 100, shape, generator=g, device=device,
                                              dtype=torch.uint8) for _ in range(2))
            self.scales = tuple(0.004 + 0.02 * torch.rand(Hkv, generator=g, device=device)
                                for _ in range(2))
        else:
            self.kc, self.vc = rnd(*shape).bfloat16(), rnd(*shape).bfloat16()
        self.q_out = torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16, device=device)
        self.k_out = None

    def call(self, pa, **change):
        a = dict(q_out=self.q_out, q=self.q, k=self.k, v=self.v, positions=self.positions,
                 increments=self.increments, k_cache=self.kc, v_cache=self.vc,
                 slot_mapping=self.slots, q_weight=self.qw, k_weight=self.kw, eps=self.eps,
                 interleaved=self.interleaved, rope_factor=self.factor, k_out=self.k_out)
        if self.f8:
            a.update(k_scales=self.scales[0], v_scales=self.scales[1])
        (pa.pa_qk_norm_rope_cache_fp8 if self.f8 else pa.pa_qk_norm_rope_cache)(**{**a, **change})

    def expect(self):
        angle = phases(self.positions, self.increments) if self.rot else None
        args = (self.eps, angle, self.rot, self.interleaved, self.factor)
        return reference(self.q, self.qw, *args), reference(self.k, self.kw, *args)

    def check(self, pa):
        (rq, bq), (rk, bk) = self.expect()
        v = self.v.clone()
        kc0, vc0 = self.kc.clone(), self.vc.clone()
        self.call(pa)
        torch.cuda.synchronize()
        assert pa.pa_device_error_flags() == 0
        close(self.q_out, rq, 2.0**-8 * np.abs(rq) + bq, "q")
        if self.k_out is not None:
            close(self.k_out, rk, 2.0**-8 * np.abs(rk) + bk, "k_out")
        kept = (self.slots >= 0).cpu().numpy()
        at = self.slots[self.slots >= 0]
        rows = lambda t: t.view(-1, self.Hkv, self.D)  # noqa: E731
        if self.f8:
            for pool, ref, b, s in ((self.kc, rk, bk, self.scales[0]),
                                    (self.vc, to64(v), 0 * bk, self.scales[1])):
                got = rows(pool.view(torch.float8_e4m3fn).float())[at]
                s = to64(s)[None, :, None]
                want = np.clip(ref / s, -448, 448)[kept]
                close(got, want, 2.0**-4 * np.abs(want) + 2.0**-10 + (b / s)[kept], "codes")
        else:
            close(rows(self.kc)[at], rk[kept], (2.0**-8 * np.abs(rk) + bk)[kept], "k")
            assert torch.equal(rows(self.vc)[at], v[self.slots >= 0])
        rest = torch.ones(self.kc.shape[0] * 16, dtype=torch.bool, device=self.kc.device)
        rest[at] = False
        assert torch.equal(rows(self.kc)[rest], rows(kc0)[rest])
        assert torch.equal(rows(self.vc)[rest], rows(vc0)[rest])


def close(got, ref, tol, what):
    got = to64(got)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.size,
                           [(i.tolist(), got[tuple(i)], ref[tuple(i)]) for i in np.argwhere(bad)[:4]])


@pytest.mark.parametrize("D,rot", [(16, 16), (64, 64), (64, 16), (80, 32), (96, 96), (96, 48),
                                   (128, 128), (128, 32), (128, 112), (192, 64), (256, 256),
                                   (256, 0), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_head_dims_and_layouts(pa, cuda_device, D, rot, interleaved, norm):
    Case(13, 6, 2, D, rot, cuda_device, seed=D + rot, norm=norm, interleaved=interleaved,
         factor=1.25).check(pa)


@pytest.mark.parametrize("T", [1, 2, 31, 500, 3001])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (7, 1), (32, 8), (9, 3)])
def test_token_and_head_counts(pa, cuda_device, T, Hq, Hkv):
    Case(T, Hq, Hkv, 128, 128, cuda_device, seed=T, fused=T % 2 == 0, pad=3).check(pa)


@pytest.mark.parametrize("D,rot", [(64, 64), (96, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_e4m3(pa, cuda_device, D, rot, interleaved):
    c = Case(77, 8, 2, D, rot, cuda_device, seed=1, interleaved=interleaved, f8=True)
    c.k[3] *= 100  # codes that saturate
    c.v[3] *= 100
    c.check(pa)


def test_far_and_negative_positions(pa, cuda_device):
    pos = [0, 1, 2**20 + 1, 2**31 - 1, 2**40 + 12345, -1, -131071, -2**63, 2**63 - 1]
    Case(len(pos), 4, 2, 128, 128, cuda_device, positions=pos, norm=False).check(pa)


def test_one_norm_only_padding_and_k_out(pa, cuda_device):
    c = Case(40, 4, 2, 64, 32, cuda_device, seed=2)
    c.qw = None
    c.slots[::3] = -1
    c.slots[1] = -2**63
    c.k_out = torch.empty(40, 2, 64, dtype=torch.bfloat16, device=cuda_device)
    c.check(pa)
    # the pool's keys are k_out's bits
    kept = c.slots >= 0
    assert torch.equal(c.kc.view(-1, 2, 64)[c.slots[kept]], c.k_out[kept])
    c.qw, c.kw = c.kw, None
    c.check(pa)


def test_no_scatter(pa, cuda_device):
    c = Case(20, 4, 2, 64, 64, cuda_device, seed=3)
    (_, _), (rk, bk) = c.expect()
    k_out = torch.empty(20, 2, 64, dtype=torch.bfloat16, device=cuda_device)
    c.call(pa, k_cache=None, v_cache=None, slot_mapping=None, v=None, k_out=k_out)
    close(k_out, rk, 2.0**-8 * np.abs(rk) + bk, "k_out")


def test_in_place(pa, cuda_device):
    c = Case(50, 4, 2, 128, 128, cuda_device, seed=4, fused=False)
    (rq, bq), (rk, bk) = c.expect()
    c.call(pa, q_out=c.q, k_out=c.k)
    close(c.q, rq, 2.0**-8 * np.abs(rq) + bq, "q")
    close(c.k, rk, 2.0**-8 * np.abs(rk) + bk, "k")


def test_nothing_to_do_is_a_copy_with_the_plain_scatters_bits(pa, cuda_device):
    for f8 in (False, True):
        c = Case(60, 4, 2, 64, 0, cuda_device, seed=5, norm=False, f8=f8)
        kc, vc = c.kc.clone(), c.vc.clone()
        c.call(pa)
        assert torch.equal(c.q_out, c.q)
        # (the plain scatters want 8-element strides and rows that are whole)
        scatter = pa.pa_reshape_and_cache_fp8 if f8 else pa.pa_reshape_and_cache
        scatter(c.k.contiguous(), c.v.contiguous(), kc, vc, c.slots, *c.scales)
        torch.cuda.synchronize()
        assert torch.equal(c.kc, kc) and torch.equal(c.vc, vc)


def test_zero_rows_and_extreme_values(pa, cuda_device):
    c = Case(4, 2, 1, 64, 64, cuda_device, seed=6, fused=False)
    c.q[0] = 0
    c.k[0] = 0
    c.q[1] *= 1e-20
    c.q[2] *= 1e15  # the sum of squares stays finite in fp32
    c.check(pa)
    assert (c.q_out[0] == 0).all()
    c.q[3, 0, 5] = float("nan")
    c.q[3, 1, 5] = float("inf")
    c.call(pa)
    assert c.q_out[3].isnan().any(-1).all() and not c.q_out[:3].isnan().any()


def test_slots_out_of_range_are_skipped_and_flagged(pa, cuda_device):
    c = Case(9, 2, 1, 64, 64, cuda_device, seed=7)
    cap = c.kc.shape[0] * 16
    c.slots[4] = cap
    c.slots[5] = 2**62
    kc = c.kc.clone()
    c.call(pa)
    assert pa.pa_device_error_flags() == pa.PA_DEVERR_SLOT
    good = [0, 1, 2, 3, 6, 7, 8]
    changed = (c.kc.view(cap, -1) != kc.view(cap, -1)).any(-1)
    assert set(torch.nonzero(changed)[:, 0].tolist()) <= set(c.slots[good].tolist())
    assert not c.q_out.isnan().any()


def test_graph_replay_reads_new_positions(pa, cuda_device):
    c = Case(33, 8, 2, 128, 128, cuda_device, seed=8)
    c.call(pa)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(pa)
    c.positions.add_(17)
    c.q.mul_(2)
    g.replay()
    torch.cuda.synchronize()
    (rq, bq), _ = c.expect()
    close(c.q_out, rq, 2.0**-8 * np.abs(rq) + bq, "q")


def test_scatter_then_read_on_one_stream(pa, cuda_device):
    """The windowed decode right behind it reads what it wrote."""
    from tests import window_ref as R
    S, Hq, Hkv, D = 16, 8, 2, 128
    lens = list(range(1, 17 * S, 17))
    kc, vc, bt = R.paged_cache(lens, 64, 4, Hkv, D, 3, cuda_device)
    sl = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    c = Case(S, Hq, Hkv, D, 128, cuda_device, seed=9)
    last = sl.long() - 1
    c.kc, c.vc, c.positions = kc, vc, last.clone()
    c.slots = torch.gather(bt.long(), 1, (last // 16)[:, None])[:, 0] * 16 + last % 16
    out = torch.empty_like(c.q_out)
    for _ in range(3):
        c.kc.view(-1, Hkv, D)[c.slots] = float("nan")
        c.call(pa)
        pa.pa_decode_window(out, c.q_out, kc, vc, bt, sl, 64, 4, 0.09)
        torch.cuda.synchronize()
        ro, _, to, _ = R.decode(c.q_out, kc, vc, bt, sl, 64, 4, 0.09)
        R.assert_within(out, ro, to, "decode behind the scatter")


def test_refusals(pa, cuda_device):
    c = Case(8, 4, 2, 64, 64, cuda_device, seed=10)
    q_out, kc = c.q_out.clone(), c.kc.clone()
    e = lambda *s, **k: torch.empty(*s, **{"device": cuda_device, **k})  # noqa: E731
    for bad in (dict(q_out=e(8, 4, 32, dtype=torch.bfloat16)), dict(slot_mapping=c.slots[:7]),
                dict(positions=c.positions[:7]), dict(v=c.v[:7]), dict(k=c.k[:, :, :32]),
                dict(q_weight=e(32)), dict(k_cache=c.kc[:, :, :1].contiguous()),
                dict(v_cache=c.vc[:-1]), dict(q=c.q.cpu()), dict(positions=c.positions.cpu()),
                dict(q=c.q.transpose(0, 1)), dict(k_out=e(8, 2, 32, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            c.call(pa, **bad)
    for bad in (dict(q=c.q.float()), dict(positions=c.positions.int()), dict(k_cache=None),
                dict(slot_mapping=None), dict(increments=c.increments.double()),
                dict(q_weight=e(64, dtype=torch.bfloat16)), dict(v=None)):
        with pytest.raises(TypeError):
            c.call(pa, **bad)
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(rope_factor=float("inf")),
                dict(k_cache=None, v_cache=None, slot_mapping=None),  # nothing receives k
                dict(q_out=c.kc.view(-1)[:8 * 4 * 64].view(8, 4, 64)),  # inside the pool
                dict(k_cache=c.vc)):
        with pytest.raises(pa.PAError) as err:
            c.call(pa, **bad)
        assert err.value.status == pa.PA_ERR_INVALID
    with pytest.raises(pa.PAError) as err:
        c.call(pa, increments=c.increments[:12])  # 24 rotary columns
    assert err.value.status == pa.PA_ERR_UNSUPPORTED
    torch.cuda.synchronize()
    assert q_out.isnan().all() and c.q_out.isnan().all() and torch.equal(c.kc, kc)
