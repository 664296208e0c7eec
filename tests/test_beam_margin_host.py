"""The bound that decides which rows of a beam selection are summed again: the error of an
exponential's argument, in the fp32 arithmetic that the pass uses (no GPU)."""
import os
import re

import numpy as np

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "paged_kv_cache_218_gb300", "csrc", "pa_beam_select.cu")


def steps_off(x, m):
    """Steps of 2^-24, for each unit of |x - m|, that 2^fl(fl(x - m) fl(log2 e)) is off e^(x - m)
    for its argument's roundings: |argument - (x - m) log2 e| ln 2 to first order."""
    x, m = x.astype(np.float32), m.astype(np.float32)
    arg = ((x - m) * np.float32(1.4426950408889634)).astype(np.float64)
    d = x.astype(np.float64) - m.astype(np.float64)
    off = np.abs(arg * np.log(2.0) - d)
    some = d != 0
    return (off[some] / np.abs(d[some])).max() * 2.0**24


def test_argument_of_the_exponentials():
    with open(SOURCE) as f:
        bound = float(re.search(r"kArgSteps = ([0-9.]+);", f.read()).group(1))
    rng = np.random.default_rng(0)
    n = 1 << 20
    m = rng.uniform(0, 30, n)
    worst = steps_off(m - rng.exponential(8.0, n), m)
    assert 1.3 < worst <= bound  # (the rounded difference counts, not its product alone)
    # bf16 logits: exact differences mostly, but not of a far and a tiny one
    cut = lambda a: (a.astype(np.float32).view(np.uint32) & 0xffff0000).view(np.float32)  # noqa: E731
    tiny = cut(np.exp(-rng.uniform(8, 30, n)))
    assert steps_off(tiny, cut(m)) <= bound
    assert steps_off(tiny, cut(m)) > 1.3
