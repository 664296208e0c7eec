"""Refusals of the shared-prefix decode on a machine without a GPU: every call here
returns from its argument checks."""
import ctypes

import pytest

from paged_kv_cache_218_gb300 import build

OK, INVALID, UNSUPPORTED = 0, -1, -2
P = 0x10000  # a non-null, aligned stand-in that no refused call reads


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ctypes.CDLL(build.LIB)


V, I, L, F, S = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t)
ARGS = dict(out=P, q=P, k=P, v=P, bt=P, mb=4, sl=P, S=2, go=P, G=1, mg=2, sb=P, Hq=8, Hkv=2, D=128,
            bs=16, nb=64, scale=0.1, lse=None, ws=P, wsb=0, stream=None)
TYPES = [V, V, V, V, V, I, V, I, V, I, I, V, I, I, I, I, L, F, V, V, S, V]


@pytest.mark.parametrize("change,want", [
    (dict(S=-1), INVALID), (dict(mb=0), INVALID), (dict(nb=0), INVALID), (dict(G=-1), INVALID),
    (dict(mg=0), INVALID), (dict(Hq=9), INVALID), (dict(Hkv=0), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(D=64), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(bs=32), UNSUPPORTED),
    (dict(Hq=18), UNSUPPORTED), (dict(nb=1 << 28), UNSUPPORTED), (dict(mb=1 << 28), UNSUPPORTED),
    (dict(S=1 << 28), UNSUPPORTED), (dict(S=0), OK), (dict(S=0, out=None, ws=None), OK),
    (dict(out=None), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(bt=None), INVALID), (dict(sl=None), INVALID),
    (dict(go=None), INVALID), (dict(sb=None), INVALID),
    (dict(out=P + 8), INVALID), (dict(q=P + 2), INVALID), (dict(k=P + 8), INVALID),
    (dict(v=P + 4), INVALID), (dict(bt=P + 2), INVALID), (dict(sl=P + 1), INVALID),
    (dict(go=P + 2), INVALID), (dict(sb=P + 1), INVALID), (dict(lse=P + 2), INVALID)])
def test_decode_shared_refuses(lib, change, want):
    lib.pa_decode_shared.argtypes, lib.pa_decode_shared.restype = TYPES, ctypes.c_int
    assert lib.pa_decode_shared(*{**ARGS, **change}.values()) == want


def test_stalled_launch_refuses_its_limit(lib):
    fn = lib.pa_test_decode_shared_stalled
    fn.argtypes = TYPES[:18] + [V, S, ctypes.c_uint, V]
    args = [v for k, v in ARGS.items() if k not in ("lse", "stream")]
    for limit in (0, 2000001):
        assert fn(*args, limit, None) == INVALID


@pytest.mark.parametrize("args", [(2, 1, 2, 8, 2, 64, 16), (2, 1, 0, 8, 2, 128, 16),
                                  (-1, 1, 2, 8, 2, 128, 16), (2, -1, 2, 8, 2, 128, 16),
                                  (2, 1, 2, 9, 2, 128, 16), (2, 1, 2, 8, 2, 128, 8)])
def test_no_workspace_for_shapes_that_are_refused(lib, args):
    lib.pa_decode_shared_workspace_size.restype = S
    assert lib.pa_decode_shared_workspace_size(*args) == 0


def test_binding_refuses():
    torch = pytest.importorskip("torch")
    build.build()
    from paged_kv_cache_218_gb300 import binding as pa
    t = torch.zeros((2, 8, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_decode_shared(t, t, t, t, t, t, t, 2, t, 0.1, t)
    with pytest.raises(TypeError):
        pa.pa_decode_shared(t, 1, t, t, t, t, t, 2, t, 0.1, t)
