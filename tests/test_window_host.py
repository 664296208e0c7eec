"""Refusals of the windowed-attention and norm-rotation entry points on a
machine without a GPU: every call here returns from its argument checks."""
import ctypes

import pytest

from paged_kv_cache_218_gb300 import build

OK, INVALID, UNSUPPORTED = 0, -1, -2
P = 0x10000  # a non-null, aligned stand-in that no refused call reads


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ctypes.CDLL(build.LIB)


def call(fn, defaults, types, **change):
    args = {**defaults, **change}
    fn.argtypes = [types[k] for k in defaults]
    fn.restype = ctypes.c_int
    return fn(*[args[k] for k in defaults])


V, I, L, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
DECODE = dict(out=P, q=P, k=P, v=P, bt=P, mb=4, sl=P, S=2, Hq=8, Hkv=2, D=128, bs=16, nb=64,
              window=100, sinks=4, scale=0.1, lse=None, stream=None)
DECODE_T = dict(zip(DECODE, [V, V, V, V, V, I, V, I, I, I, I, I, L, I, I, F, V, V]))


@pytest.mark.parametrize("change,want", [
    (dict(window=0), INVALID), (dict(window=-3), INVALID), (dict(sinks=-1), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(S=-1), INVALID), (dict(mb=0), INVALID),
    (dict(nb=0), INVALID), (dict(Hq=9), INVALID), (dict(Hkv=0), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(bs=32), UNSUPPORTED), (dict(Hq=18), UNSUPPORTED),
    (dict(nb=1 << 28), UNSUPPORTED), (dict(mb=1 << 28), UNSUPPORTED),
    (dict(S=1 << 28), UNSUPPORTED), (dict(S=0), OK), (dict(S=0, out=None, q=None), OK),
    (dict(out=None), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(bt=None), INVALID), (dict(sl=None), INVALID),
    (dict(out=P + 8), INVALID), (dict(q=P + 2), INVALID), (dict(k=P + 8), INVALID),
    (dict(v=P + 4), INVALID), (dict(bt=P + 2), INVALID), (dict(sl=P + 1), INVALID),
    (dict(lse=P + 2), INVALID)])
def test_decode_window_refuses(lib, change, want):
    assert call(lib.pa_decode_window, DECODE, DECODE_T, **change) == want


B = 1 << 20  # stand-ins far enough apart
ROPE = dict(q_out=B, k_out=None, q=2 * B, k=3 * B, v=4 * B, qs=1024, ks=256, vs=256, qw=None,
            kw=None, eps=1e-6, pos=5 * B, inc=6 * B, rot=128, il=0, factor=1.0, kc=7 * B,
            vc=20 * B, slots=40 * B, T=4, Hq=8, Hkv=2, D=128, bs=16, nb=64, stream=None)
ROPE_T = dict(zip(ROPE, [V, V, V, V, V, L, L, L, V, V, F, V, V, I, I, F, V, V, V, I, I, I, I, I, L,
                         V]))


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=-1), INVALID), (dict(D=0), INVALID),
    (dict(rot=-16), INVALID), (dict(rot=144), INVALID), (dict(D=72, rot=16), UNSUPPORTED),
    (dict(D=272), UNSUPPORTED), (dict(rot=24), UNSUPPORTED), (dict(bs=8), UNSUPPORTED),
    (dict(nb=0), INVALID), (dict(nb=1 << 62), INVALID), (dict(qw=B, eps=-1.0), INVALID),
    (dict(kw=B, eps=float("inf")), INVALID), (dict(factor=float("nan")), INVALID),
    (dict(T=0), OK), (dict(T=0, q=None, q_out=None), OK),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(q_out=None), INVALID),
    (dict(v=None), INVALID), (dict(slots=None), INVALID), (dict(kc=None), INVALID),
    (dict(vc=None), INVALID), (dict(pos=None), INVALID), (dict(inc=None), INVALID),
    (dict(kc=None, vc=None), INVALID),
    (dict(qs=1016), INVALID), (dict(qs=1028), INVALID), (dict(ks=128), INVALID),
    (dict(vs=12), INVALID), (dict(qs=1 << 40), INVALID),
    (dict(q=2 * B + 8), INVALID), (dict(q_out=B + 2), INVALID), (dict(kc=7 * B + 8), INVALID),
    (dict(qw=B + 4), INVALID), (dict(pos=5 * B + 4), INVALID), (dict(slots=40 * B + 4), INVALID),
    # overlaps: q_out inside q, over k, half in place, with the pools; the pools with each other
    (dict(q_out=2 * B + 2048), INVALID), (dict(q_out=3 * B), INVALID),
    (dict(q_out=2 * B, qs=2048), INVALID), (dict(q_out=7 * B + 4096), INVALID),
    (dict(k_out=B), INVALID), (dict(vc=7 * B + 16), INVALID), (dict(v=20 * B), INVALID)])
def test_norm_rope_refuses(lib, change, want):
    assert call(lib.pa_qk_norm_rope_cache, ROPE, ROPE_T, **change) == want


def test_norm_rope_fp8_refuses_missing_scales_and_pools(lib):
    names = list(ROPE)
    at = names.index("slots") + 1
    args = dict(ROPE)
    full = {k: args[k] for k in names[:at]} | {"kscale": B, "vscale": B} | {
        k: args[k] for k in names[at:]}
    types = {**ROPE_T, "kscale": V, "vscale": V}
    for change in (dict(kscale=None), dict(vscale=None), dict(kscale=B + 2), dict(kc=None),
                   dict(kc=None, vc=None, k_out=60 * B), dict(kc=7 * B + 4)):
        assert call(lib.pa_qk_norm_rope_cache_fp8, full, types, **change) == INVALID


def _increments(lib, rot, base=10000.0, scaling=0, factor=1.0, ctx=0.0, p0=0.0, p1=0.0):
    out = (ctypes.c_int64 * max(rot // 2, 1))()
    f = ctypes.c_float(0)
    fn = lib.pa_rope_increments
    fn.argtypes = [V, V, I] + [ctypes.c_double, I] + [ctypes.c_double] * 4
    fn.restype = ctypes.c_int
    rc = fn(out, ctypes.byref(f), rot, base, scaling, factor, ctx, p0, p1)
    return rc, [x / 2.0**64 * 2 * 3.141592653589793 for x in out], f.value


def test_rope_increments_follow_their_formulas(lib):
    import math
    rot, base = 64, 10000.0
    plain = [base ** (-2 * i / rot) for i in range(rot // 2)]

    def near(got, want):
        # doubles: pow and the quotient by 2 pi, a few steps of 2^-52; and the
        # rounding to whole units of 2^-64 turn: 2 pi 2^-65 = 1.7e-19 radians
        assert all(abs(a - b) <= 1e-14 * b + 2 * math.pi * 2.0**-65 for a, b in zip(got, want))

    rc, f, s = _increments(lib, rot)
    assert rc == OK and s == 1.0
    near(f, plain)
    near(_increments(lib, rot, scaling=1, factor=4.0)[1], [x / 4 for x in plain])
    ntk = base * 4.0 ** (rot / (rot - 2))
    near(_increments(lib, rot, scaling=2, factor=4.0)[1],
         [ntk ** (-2 * i / rot) for i in range(rot // 2)])
    rc, f, s = _increments(lib, rot, scaling=3, factor=16.0, ctx=4096.0, p0=32.0, p1=1.0)
    assert abs(s - (0.1 * math.log(16) + 1)) < 1e-7
    for i, (x, p) in enumerate(zip(f, plain)):
        turns = 4096 * p / (2 * math.pi)
        step = 1e-14 * p + 2 * math.pi * 2.0**-65
        assert p / 16 - step <= x <= p + step
        if turns > 32 * 2:  # well inside either part: kept, or interpolated whole
            near([x], [p])
        if turns < 0.5:
            near([x], [p / 16])
    assert f == sorted(f, reverse=True)
    rc, f, s = _increments(lib, rot, scaling=4, factor=8.0, ctx=8192.0, p0=1.0, p1=4.0)
    assert s == 1.0
    for x, p in zip(f, plain):
        wave = 2 * math.pi / p
        if wave < 8192 / 4:
            want = p
        elif wave > 8192:
            want = p / 8
        else:
            smooth = (8192 / wave - 1.0) / 3.0
            want = (1 - smooth) * p / 8 + smooth * p
        near([x], [want])


@pytest.mark.parametrize("kw,want", [
    (dict(rot=0), UNSUPPORTED), (dict(rot=24), UNSUPPORTED), (dict(rot=512), UNSUPPORTED),
    (dict(rot=64, base=1.0), INVALID), (dict(rot=64, base=float("nan")), INVALID),
    (dict(rot=64, scaling=5), INVALID), (dict(rot=64, scaling=-1), INVALID),
    (dict(rot=64, scaling=1, factor=0.5), INVALID),
    (dict(rot=64, scaling=3, factor=2.0), INVALID),
    (dict(rot=64, scaling=3, factor=2.0, ctx=4096.0, p0=1.0, p1=32.0), INVALID),
    (dict(rot=64, scaling=4, factor=2.0, ctx=4096.0, p0=4.0, p1=1.0), INVALID)])
def test_rope_increments_refuse(lib, kw, want):
    assert _increments(lib, **kw)[0] == want


PREFILL = dict(out=P, q=P, k=P, v=P, bt=P, mb=4, cu=P, start=P, sl=P, C=2, T=64, max_q=40, Hq=8,
               Hkv=2, D=128, bs=16, nb=64, window=100, sinks=4, scale=0.1, lse=None, stream=None)
PREFILL_T = dict(zip(PREFILL, [V, V, V, V, V, I, V, V, V, I, I, I, I, I, I, I, L, I, I, F, V, V]))


@pytest.mark.parametrize("change,want", [
    (dict(window=0), INVALID), (dict(sinks=-1), INVALID), (dict(scale=-1.0), INVALID),
    (dict(C=-1), INVALID), (dict(T=-1), INVALID), (dict(max_q=-1), INVALID), (dict(mb=0), INVALID),
    (dict(nb=0), INVALID), (dict(Hq=9), INVALID), (dict(D=64), UNSUPPORTED),
    (dict(bs=8), UNSUPPORTED), (dict(Hq=6), UNSUPPORTED), (dict(nb=1 << 28), UNSUPPORTED),
    (dict(mb=1 << 28), UNSUPPORTED), (dict(C=0), OK), (dict(T=0), OK), (dict(max_q=0), OK),
    (dict(out=None), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(bt=None), INVALID), (dict(cu=None), INVALID),
    (dict(start=None), INVALID), (dict(sl=None), INVALID), (dict(out=P + 8), INVALID),
    (dict(q=P + 8), INVALID), (dict(k=P + 8), INVALID), (dict(v=P + 8), INVALID),
    (dict(bt=P + 1), INVALID), (dict(cu=P + 2), INVALID), (dict(start=P + 2), INVALID),
    (dict(sl=P + 2), INVALID), (dict(lse=P + 1), INVALID)])
def test_prefill_window_refuses(lib, change, want):
    assert call(lib.pa_prefill_window, PREFILL, PREFILL_T, **change) == want


@pytest.mark.parametrize("limit", [0, 2000001])
def test_stalled_prefill_refuses_its_limit(lib, limit):
    names = [n for n in PREFILL if n not in ("lse", "stream")]
    args = {n: PREFILL[n] for n in names} | {"limit": limit, "stream": None}
    types = {n: PREFILL_T[n] for n in names} | {"limit": ctypes.c_uint, "stream": V}
    assert call(lib.pa_test_prefill_window_stalled, args, types) == INVALID


@pytest.mark.parametrize("bad,error", [
    (lambda t: None, TypeError), (lambda t: 3, TypeError), (lambda t: t.half(), TypeError),
    (lambda t: t, ValueError), (lambda t: t.to("meta"), ValueError),
    (lambda t: t.to_sparse(), ValueError), (lambda t: t[0], ValueError)])
def test_python_calls_refuse_what_is_no_cuda_tensor(lib, bad, error):
    torch = pytest.importorskip("torch")
    from paged_kv_cache_218_gb300 import binding as pa
    x = bad(torch.zeros(2, 4, 64, dtype=torch.bfloat16))
    for call_it in (lambda: pa.pa_decode_window(x, x, x, x, x, x, 8, 0, 0.1),
                    lambda: pa.pa_prefill_window(x, x, x, x, x, x, x, x, 1, 8, 0, 0.1),
                    lambda: pa.pa_qk_norm_rope_cache(x, x, x, x, None, None, None, None, None,
                                                     k_out=x),
                    lambda: pa.pa_qk_norm_rope_cache_fp8(x, x, x, x, None, None, x, x, x, x, x)):
        with pytest.raises(error):
            call_it()


@pytest.mark.parametrize("out", ["q_out", "k_out", "kc", "vc"])
@pytest.mark.parametrize("name,size", [("qw", 512), ("kw", 512), ("pos", 32), ("inc", 512),
                                       ("slots", 32), ("kscale", 8), ("vscale", 8)])
def test_norm_rope_refuses_outputs_over_its_small_inputs(lib, out, name, size):
    """Weights, positions, increments, slots and scales are inputs too: an
    output that begins on their last element, or ends on their first one."""
    names = list(ROPE)
    at = names.index("slots") + 1
    full = {k: ROPE[k] for k in names[:at]} | {"kscale": 50 * B, "vscale": 51 * B} | {
        k: ROPE[k] for k in names[at:]}
    full |= dict(k_out=60 * B, qw=52 * B, kw=53 * B)
    types = {**ROPE_T, "kscale": V, "vscale": V}
    bytes_ = dict(q_out=4 * 1024 * 2, k_out=4 * 256 * 2, kc=64 * 16 * 256, vc=64 * 16 * 256)[out]
    for where in (full[out] - size + 16, full[out] + bytes_ - 16):
        where -= where % 16
        assert call(lib.pa_qk_norm_rope_cache_fp8, full, types, **{name: where}) == INVALID, where
        if name not in ("kscale", "vscale"):
            bf16 = {k: x for k, x in full.items() if k not in ("kscale", "vscale")}
            assert call(lib.pa_qk_norm_rope_cache, bf16, ROPE_T, **{name: where}) == INVALID


@pytest.mark.parametrize("base", [3.7, 1e4, 5e5, 1e7])
@pytest.mark.parametrize("scaling,factor", [(0, 1.0), (1, 3.3), (2, 7.7)])
@pytest.mark.parametrize("rot", [16, 48, 64, 112, 128, 256])
def test_rope_increments_are_as_near_as_stated(lib, base, scaling, factor, rot):
    """Against 60 digits: (3 + ln base) 2^-53 relative and half a unit (the
    exponent's rounding grows by ln base; pow, quotient and constant)."""
    from decimal import Decimal, localcontext
    out = (ctypes.c_int64 * (rot // 2))()
    f = ctypes.c_float(0)
    fn = lib.pa_rope_increments
    fn.argtypes = [V, V, I] + [ctypes.c_double, I] + [ctypes.c_double] * 4
    fn.restype = ctypes.c_int
    assert fn(out, ctypes.byref(f), rot, base, scaling, factor, 0.0, 0.0, 0.0) == OK
    with localcontext() as ctx:
        ctx.prec = 60
        two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494")
        b = Decimal(base)
        if scaling == 2:
            b *= Decimal(factor) ** (Decimal(rot) / Decimal(rot - 2))
        for i, got in enumerate(out):
            want = (b.ln() * Decimal(-2 * i) / Decimal(rot)).exp() * 2**64 / two_pi
            want /= Decimal(factor) if scaling == 1 else 1
            assert abs(got - want) <= Decimal("0.5") + want * (3 + b.ln()) / 2**53, (i, got, want)
