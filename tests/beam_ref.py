"""64-bit references of the beam-search calls, written from their definitions with
numpy and plain loops, and the tolerance their tests use for scores.

A score is s + x - lse with lse = ln sum exp x from one fp32 pass.  Relative error of the
pass's sum, every rounding adding up: an exponential 2^-22 (the unit's bound), four of
them in a row (a term and three rescalings); their arguments, x - m rounded, times log2(e)
rounded, 1.3 * 2^-24 |x - m| with a weighted mean of |x - m| of at most ln V (a token at
depth d weighs e^-d of the largest, and there are V), and some units more for maxima
that moved; additions 2^-24 each: 9 in a lane's step, 3 more for each further step of it
(2048 loads of 16 or 8 elements at a time in a cluster of eight CTAs), 16 behind.  Then
the score's own rounding, 2^-24 of it.
"""
import math

import numpy as np


def score_tolerance(value, vocab, fp32):
    steps = math.ceil(vocab / (8 * 8 * 4 * 32 * (8 if fp32 else 16))) + 1
    err = 2.0**-20 + 2.0**-23 * math.log(vocab) + 1.3 * 2.0**-24 * (4 + math.log(vocab))
    err += (25 + 3 * steps) * 2.0**-24
    return err + 2.0**-24 * np.abs(value)


def select(logits, scores, finished, end_token, num_choices):
    """logits [R, W, V] float64 -> parents, tokens (int), scores (float64), marks (bool)."""
    R, W, V = logits.shape
    par = np.full((R, num_choices), -1)
    tok = np.full((R, num_choices), -1)
    val = np.full((R, num_choices), -np.inf)
    mark = np.zeros((R, num_choices), bool)
    x = np.where(np.isnan(logits) | (logits == np.inf), -np.inf, logits)
    for r in range(R):
        value = np.full((W, V), -np.inf)
        for w in range(W):
            s = float(scores[r, w])
            if not math.isfinite(s):
                continue
            if finished is not None and finished[r, w]:
                value[w, end_token] = s
                continue
            top = x[r, w].max()
            if top == -np.inf:
                continue
            # (in this order: s and the logarithm vanish next to a far logit)
            value[w] = (x[r, w] - top) + (s - math.log(math.fsum(np.exp(x[r, w] - top))))
        flat = value.ravel()
        best = np.argsort(-flat, kind="stable")[:num_choices]
        best = best[flat[best] > -np.inf]
        n = len(best)
        par[r, :n], tok[r, :n], val[r, :n] = best // V, best % V, flat[best]
        for i in range(n):
            w = best[i] // V
            mark[r, i] = (finished is not None and finished[r, w]) or tok[r, i] == end_token
    return par, tok, val, mark


def reorder(tables, lens, parents):
    """tables [R * W, M], lens [R * W], parents [R, W] (all in range) -> new tables, new lens,
    copies [(source block, destination block, tokens)]."""
    R, W = parents.shape
    M = tables.shape[1]
    out, new_lens, copies = np.full_like(tables, -1), np.zeros_like(lens), []
    for r in range(R):
        row = [int(p) for p in parents[r]]
        idle = [b for b in range(W) if b not in row]
        takes = {}
        for i, p in enumerate(row):
            if p >= 0 and p not in row[:i]:
                takes[i] = p
        for i in [i for i in range(W) if i not in takes and row[i] >= 0]:
            takes[i] = idle.pop(0)
        for i in [i for i in range(W) if i not in takes]:
            takes[i] = idle.pop(0)
        assert not idle
        for i, p in enumerate(row):
            n = int(lens[r * W + p]) if p >= 0 else 0
            o = takes[i]
            own = [int(b) for b in tables[r * W + o][int(lens[r * W + o]) // 16:]]
            line = ([int(b) for b in tables[r * W + p][:n // 16]] if p >= 0 else []) + own
            line = (line + [-1] * M)[:M]
            out[r * W + i], new_lens[r * W + i] = line, n
            if p >= 0 and o != p and n % 16:
                copies.append((int(tables[r * W + p][n // 16]), own[0] if own else -1, n % 16))
    return out, new_lens, copies
