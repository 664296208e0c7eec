"""fp64 reference of attention under a sliding window with sinks, written from
the definition with numpy, and the tolerance its tests use.

Rounding of a kernel that accumulates in fp32 and rounds once to bf16, per
output element, in terms of the data:

* a score x = scale * sum_d q_d k_d has exact products (bf16 * bf16 fits fp32)
  and D additions, each off by at most 2^-23 of the partial sum (truncation),
  so |dx| <= D * 2^-23 * scale * sum_d |q_d k_d|, plus 2^-22 |x| for the
  conversion to base 2;
* a weight is off by |dx| + 2^-21 (the exponential unit), plus `p_step` where
  weights are rounded before the product with V; so is its normalizer;
* the sums over L keys add L * 2^-23 of the largest |v|;
* the output's rounding to bf16: half a step, 2^-8 relative.
"""
import numpy as np
import torch


def to64(t):
    return t.detach().double().cpu().numpy()


def visible(p, window, sinks):
    """Key positions that a query at position p sees, ascending."""
    near = np.arange(max(0, p - window + 1), p + 1)
    far = np.arange(0, min(sinks, near[0]))
    return np.concatenate([far, near])


def attend(q, k, v, scale, p_step):
    """One query row q [D] over k, v [L, D]: (out, lse, tolerance of out, of lse)."""
    if k.shape[0] == 0:
        return np.zeros(v.shape[1]), -np.inf, np.zeros(v.shape[1]), 0.0
    x = scale * (k @ q)
    m = x.max()
    w = np.exp(x - m)
    out = (w[:, None] * v).sum(0) / w.sum()
    dx = len(q) * 2.0**-23 * scale * (np.abs(k) @ np.abs(q)).max() + 2.0**-22 * np.abs(x).max()
    dp = dx + 2.0**-21
    sums = k.shape[0] * 2.0**-23
    tol = 2.0**-8 * np.abs(out) + (2 * dp + p_step + sums) * np.abs(v).max()
    lse = m + np.log(w.sum())
    return out, lse, tol, dp + sums + 2.0**-22 * abs(lse)


def decode(q, kc, vc, tables, lens, window, sinks, scale):
    """Tensors in; (out, lse, tol_out, tol_lse) as numpy."""
    q, kc, vc = to64(q), to64(kc), to64(vc)
    tables, lens = tables.cpu().numpy(), lens.cpu().numpy()
    S, Hq, D = q.shape
    G = Hq // kc.shape[2]
    out, tol = np.zeros((S, Hq, D)), np.zeros((S, Hq, D))
    lse, tol_l = np.zeros((S, Hq)), np.zeros((S, Hq))
    for s in range(S):
        j = visible(lens[s] - 1, window, sinks) if lens[s] > 0 else np.arange(0)
        rows = tables[s, j // 16], j % 16
        for h in range(Hq):
            out[s, h], lse[s, h], tol[s, h], tol_l[s, h] = attend(
                q[s, h], kc[rows[0], rows[1], h // G], vc[rows[0], rows[1], h // G], scale,
                2.0**-16)
    return out, lse, tol, tol_l


def prefill(q, kc, vc, tables, cu, start, window, sinks, scale):
    """As decode, for chunks.  Weights are rounded to bf16 before the product with V: each is off
    by at most 2^-8 of itself, so an output by at most 2^-8 sum w |v| / sum w more."""
    q, kc, vc = to64(q), to64(kc), to64(vc)
    tables, cu, start = tables.cpu().numpy(), cu.cpu().numpy(), start.cpu().numpy()
    T, Hq, D = q.shape
    G = Hq // kc.shape[2]
    out, tol = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, tol_l = np.zeros((T, Hq)), np.zeros((T, Hq))
    for c in range(len(start)):
        rows = np.arange(cu[c], cu[c + 1])
        if len(rows) == 0:
            continue
        pos = start[c] + np.arange(len(rows))
        keys = np.union1d(np.arange(max(0, pos[0] - window + 1), pos[-1] + 1),
                          np.arange(min(sinks, pos[-1] + 1)))
        gap = pos[:, None] - keys
        seen = (gap >= 0) & ((keys < sinks) | (gap < window))
        at = tables[c, keys // 16], keys % 16
        for h in range(Hq):
            k, v = kc[at[0], at[1], h // G], vc[at[0], at[1], h // G]
            qh = q[rows, h]
            x = np.where(seen, scale * (qh @ k.T), -np.inf)
            m = x.max(1, keepdims=True)
            w = np.exp(x - m)
            l = w.sum(1, keepdims=True)
            out[rows, h] = w @ v / l
            lse[rows, h] = (m + np.log(l))[:, 0]
            size = np.where(seen, np.abs(qh) @ np.abs(k).T, 0).max(1, keepdims=True)
            dp = (D * 2.0**-23 * scale * size + 2.0**-21 +
                  2.0**-22 * np.where(seen, np.abs(x), 0).max(1, keepdims=True))
            sums = seen.sum(1, keepdims=True) * 2.0**-23
            tol[rows, h] = (2.0**-8 * np.abs(out[rows, h]) + (2 * dp + sums) * np.abs(v).max() +
                            2.0**-8 * (w @ np.abs(v)) / l)
            tol_l[rows, h] = (dp + sums)[:, 0] + 2.0**-22 * np.abs(lse[rows, h])
    return out, lse, tol, tol_l


def assert_within(got, ref, tol, what):
    got = to64(got) if isinstance(got, torch.Tensor) else got
    same = (got == ref) | (np.abs(got - ref) <= tol)
    assert same.all(), (what, int((~same).sum()), same.size,
                        [(i.tolist(), float(got[tuple(i)]), float(ref[tuple(i)]))
                         for i in np.argwhere(~same)[:4]])


def paged_cache(lens, window, sinks, Hkv, D, seed, device, first_query=None, poison=True,
                spare=3):
    """Pools and tables of sequences with `lens` keys whose queries stand at
    first_query[s] (default: the last key) and later.  Every slot that no such
    query sees is NaN, and the table entry of every block without a visible key
    is an id outside the pool."""
    rng = np.random.default_rng(seed)
    width = max(1, max((n + 15) // 16 for n in lens)) + 1
    first_query = [n - 1 for n in lens] if first_query is None else first_query
    tables = np.full((len(lens), width), -7, dtype=np.int32)
    tables[:, 1::2] = 2**31 - 1  # ids far outside, of both signs
    seen = []
    for n, p in zip(lens, first_query):
        keys = np.zeros(width * 16, dtype=bool)
        if n > 0:
            keys[max(0, p - window + 1):n] = True
            keys[:min(sinks, n)] = True
        seen.append(keys.reshape(width, 16))
    used = sum(int(k.any(1).sum()) for k in seen)
    order = rng.permutation(used + spare)[:used]
    kc = rng.standard_normal((used + spare, 16, Hkv, D)).astype(np.float32)
    vc = rng.standard_normal((used + spare, 16, Hkv, D)).astype(np.float32)
    hidden = np.ones((used + spare, 16), dtype=bool)
    at = 0
    for s, keys in enumerate(seen):
        for b in np.flatnonzero(keys.any(1)):
            tables[s, b] = order[at]
            hidden[order[at]] = ~keys[b]
            at += 1
    if poison:
        kc[hidden] = np.nan
        vc[hidden] = np.nan
    dev = lambda a: torch.from_numpy(a).to(device)  # noqa: E731
    return dev(kc).bfloat16(), dev(vc).bfloat16(), dev(tables)
