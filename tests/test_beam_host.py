"""Refusals of the beam-search entry points on a machine without a GPU: every call
here returns from its argument checks."""
import ctypes

import numpy as np
import pytest

from paged_kv_cache_218_gb300 import build
from tests import beam_ref

OK, INVALID, UNSUPPORTED = 0, -1, -2
B = 1 << 24  # stand-ins far enough apart, which no refused call reads


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ctypes.CDLL(build.LIB)


def call(fn, defaults, types, **change):
    args = {**defaults, **change}
    fn.argtypes = [types[k] for k in defaults]
    fn.restype = ctypes.c_int
    return fn(*[args[k] for k in defaults])


V, I, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
SELECT = dict(par=B, tok=2 * B, out=3 * B, of=4 * B, x=5 * B, f32=0, rs=4 * 1000, bs=1000,
              s=6 * B, fin=7 * B, end=2, R=3, W=4, K=4, vocab=1000, stream=None)
SELECT_T = dict(zip(SELECT, [V, V, V, V, V, I, L, L, V, V, I, I, I, I, I, V]))


@pytest.mark.parametrize("change,want", [
    (dict(R=-1), INVALID), (dict(W=0), INVALID), (dict(K=0), INVALID), (dict(vocab=0), INVALID),
    (dict(W=33), UNSUPPORTED), (dict(K=65), UNSUPPORTED), (dict(vocab=1 << 29), UNSUPPORTED),
    (dict(R=1 << 25), UNSUPPORTED), (dict(end=-1), INVALID), (dict(end=1000), INVALID),
    (dict(fin=None, end=-2), INVALID), (dict(fin=None, end=1000), INVALID),
    (dict(rs=-1), INVALID), (dict(bs=-1), INVALID), (dict(bs=1 << 40), INVALID),
    (dict(R=0), OK), (dict(R=0, x=None, par=None), OK),
    (dict(par=None), INVALID), (dict(tok=None), INVALID), (dict(out=None), INVALID),
    (dict(x=None), INVALID), (dict(s=None), INVALID),
    (dict(par=B + 2), INVALID), (dict(tok=2 * B + 1), INVALID), (dict(out=3 * B + 2), INVALID),
    (dict(s=6 * B + 2), INVALID), (dict(x=5 * B + 1), INVALID),
    (dict(x=5 * B + 2, f32=1), INVALID),
    # outputs over inputs or one another
    (dict(par=2 * B + 16), INVALID), (dict(tok=5 * B + 4), INVALID), (dict(out=6 * B + 4), INVALID),
    (dict(K=3, out=6 * B), INVALID), (dict(K=3, of=7 * B), INVALID), (dict(of=6 * B), INVALID),
    (dict(par=5 * B + 23996), INVALID), (dict(out=7 * B), INVALID)])
def test_beam_select_refuses(lib, change, want):
    assert call(lib.pa_beam_select, SELECT, SELECT_T, **change) == want


REORDER = dict(ot=B, ol=2 * B, bt=3 * B, sl=4 * B, par=5 * B, R=3, W=4, mb=10, k=6 * B, v=12 * B,
               layers=2, stride=64 * 16 * 2 * 64, Hkv=2, D=64, bs=16, nb=64, stream=None)
REORDER_T = dict(zip(REORDER, [V, V, V, V, V, I, I, I, V, V, I, L, I, I, I, L, V]))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("change,want", [
    (dict(R=-1), INVALID), (dict(W=0), INVALID), (dict(mb=0), INVALID), (dict(layers=-1), INVALID),
    (dict(Hkv=0), INVALID), (dict(D=0), INVALID), (dict(nb=0), INVALID), (dict(bs=0), INVALID),
    (dict(stride=-8), INVALID), (dict(nb=1 << 60), INVALID), (dict(W=33), UNSUPPORTED),
    (dict(bs=32), UNSUPPORTED), (dict(D=4), UNSUPPORTED), (dict(mb=1 << 28), UNSUPPORTED),
    (dict(W=32, mb=(1 << 25) + 1), UNSUPPORTED),
    (dict(R=1 << 25), UNSUPPORTED), (dict(layers=1 << 20), UNSUPPORTED),
    (dict(stride=64 * 16 * 2 * 64 - 16), INVALID), (dict(stride=64 * 16 * 2 * 64 + 4), INVALID),
    (dict(R=0), OK), (dict(R=0, ot=None, k=None), OK),
    (dict(ot=None), INVALID), (dict(ol=None), INVALID), (dict(bt=None), INVALID),
    (dict(sl=None), INVALID), (dict(par=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID),
    (dict(ot=B + 2), INVALID), (dict(ol=2 * B + 1), INVALID), (dict(bt=3 * B + 2), INVALID),
    (dict(sl=4 * B + 2), INVALID), (dict(par=5 * B + 2), INVALID), (dict(k=6 * B + 8), INVALID),
    (dict(v=12 * B + 4), INVALID),
    # overlaps
    (dict(ot=3 * B), INVALID), (dict(ot=3 * B + 476), INVALID), (dict(ol=4 * B), INVALID),
    (dict(ol=5 * B + 44), INVALID), (dict(ot=6 * B + 1024), INVALID), (dict(v=6 * B), INVALID),
    (dict(par=6 * B + 64), INVALID), (dict(ol=B + 4), INVALID)])
def test_beam_reorder_refuses(lib, change, want, fp8):
    fn = lib.pa_beam_reorder_fp8 if fp8 else lib.pa_beam_reorder
    assert call(fn, REORDER, REORDER_T, **change) == want


def test_binding_refuses():
    torch = pytest.importorskip("torch")
    build.build()
    from paged_kv_cache_218_gb300 import binding as pa
    i32 = torch.zeros((2, 4), dtype=torch.int32)
    with pytest.raises(TypeError):
        pa.pa_beam_select(i32, i32, None, "logits", None)
    with pytest.raises(TypeError, match="logits"):
        pa.pa_beam_select(i32, i32, None, torch.zeros((2, 4, 8), dtype=torch.float16), None)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_beam_select(i32, i32, None, torch.zeros((2, 4, 8)), None)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_beam_reorder(i32, i32, i32, i32, i32, None, None)


def test_reference_select_by_hand():
    """Two beams, three tokens of equal logits: every candidate of beam 0 at s0 - ln 3."""
    x = np.zeros((1, 2, 3))
    x[0, 1, 2] = -np.inf
    par, tok, val, mark = beam_ref.select(x, np.array([[-1.0, -1.5]]), None, -1, 6)
    assert par.tolist() == [[0, 0, 0, 1, 1, -1]] and tok.tolist() == [[0, 1, 2, 0, 1, -1]]
    assert np.allclose(val[0, :5], [-1 - np.log(3)] * 3 + [-1.5 - np.log(2)] * 2)
    par, tok, val, mark = beam_ref.select(x, np.array([[-1.0, -1.5]]), np.array([[True, False]]),
                                          2, 4)
    assert par.tolist() == [[0, 1, 1, -1]] and tok.tolist() == [[2, 0, 1, -1]]
    assert mark.tolist() == [[True, False, False, False]]


def test_reference_reorder_by_hand():
    """Beams 0 and 1 both continue beam 1; beam 2 begins anew; beam 0's block takes the copy."""
    tables = np.array([[7, 1, 4], [7, 2, 5], [7, 3, 6]])
    out, lens, copies = beam_ref.reorder(tables, np.array([20, 21, 19]), np.array([[1, 1, -1]]))
    assert out.tolist() == [[7, 2, 5], [7, 1, 4], [3, 6, -1]] and lens.tolist() == [21, 21, 0]
    assert copies == [(2, 1, 5)]
