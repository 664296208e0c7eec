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
