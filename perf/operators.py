"""The operators of a sliding-window attention layer, case by case.

Three operators, in the order a layer of a serving step runs them:

* ``norm_rope``: root-mean-square norms of queries and keys for each head, the
  position rotation, and the scatter of keys and values into the paged cache;
* ``decode``: one query per sequence over its last ``window`` keys and its first
  ``sinks`` keys, read from the paged cache;
* ``prefill``: the same mask for the queries of prefill chunks.

``own`` false: their plain form in torch.  ``own`` true: this package's calls.
"""
import math
import random

import torch

own = False

BLOCK = 16


def listed():
    return [
        # one decode step of a batch of 64: latency
        {"name": "rope step 64", "op": "norm_rope", "tokens": 64, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "interleaved": False, "norm": True, "scaling": "none", "fused": True,
         "kv": "bf16", "max_pos": 32768, "shape_seed": 1},
        # a large prefill batch: bandwidth
        {"name": "rope prefill 8192", "op": "norm_rope", "tokens": 8192, "hq": 32, "hkv": 8,
         "d": 128, "rot": 128, "interleaved": False, "norm": True, "scaling": "yarn",
         "fused": True, "kv": "bf16", "max_pos": 131072, "shape_seed": 2},
        # adjacent pairs, a quarter of a 64-wide head, no norm, an odd number of tokens
        {"name": "rope partial 4099", "op": "norm_rope", "tokens": 4099, "hq": 16, "hkv": 4,
         "d": 64, "rot": 16, "interleaved": True, "norm": False, "scaling": "none",
         "fused": False, "kv": "bf16", "max_pos": 1000000, "shape_seed": 3},
        # a prefill chunk written into an E4M3 cache
        {"name": "rope e4m3 2048", "op": "norm_rope", "tokens": 2048, "hq": 32, "hkv": 8,
         "d": 128, "rot": 64, "interleaved": False, "norm": True, "scaling": "linear",
         "fused": True, "kv": "e4m3", "max_pos": 65536, "shape_seed": 4},
        # one user, a short window: latency
        {"name": "decode one 128", "op": "decode", "seqs": 1, "hq": 32, "hkv": 8, "d": 128,
         "window": 128, "sinks": 4, "min_len": 5000, "max_len": 5000, "shape_seed": 5},
        # a batch under a common window, lengths on both sides of it
        {"name": "decode 128 x 1024", "op": "decode", "seqs": 128, "hq": 32, "hkv": 8, "d": 128,
         "window": 1024, "sinks": 4, "min_len": 300, "max_len": 8192, "shape_seed": 6},
        # the largest batch, every sequence past its window
        {"name": "decode 256 x 4096", "op": "decode", "seqs": 256, "hq": 32, "hkv": 8, "d": 128,
         "window": 4096, "sinks": 64, "min_len": 5000, "max_len": 32768, "shape_seed": 7},
        # odd everything: three query heads a kv head, 64-wide heads, no sinks, empty sequences
        {"name": "decode ragged 37", "op": "decode", "seqs": 37, "hq": 12, "hkv": 4, "d": 64,
         "window": 1001, "sinks": 0, "min_len": 0, "max_len": 3000, "shape_seed": 8},
        # few sequences, a long window: the key axis has to be split
        {"name": "decode 4 x 32768", "op": "decode", "seqs": 4, "hq": 32, "hkv": 8, "d": 128,
         "window": 32768, "sinks": 16, "min_len": 30000, "max_len": 131072, "shape_seed": 9},
        # the chunk of a hybrid batch
        {"name": "prefill 512 x 1024", "op": "prefill", "chunks": 1, "hq": 32, "hkv": 8,
         "window": 1024, "sinks": 4, "min_q": 512, "max_q": 512, "max_start": 1536,
         "shape_seed": 10},
        # a long prompt's chunk far into the sequence: the largest
        {"name": "prefill 8192 x 4096", "op": "prefill", "chunks": 1, "hq": 32, "hkv": 8,
         "window": 4096, "sinks": 128, "min_q": 8192, "max_q": 8192, "max_start": 24576,
         "shape_seed": 11},
        # several ragged chunks, eight query heads a kv head
        {"name": "prefill ragged 7", "op": "prefill", "chunks": 7, "hq": 16, "hkv": 2,
         "window": 333, "sinks": 5, "min_q": 1, "max_q": 900, "max_start": 3000,
         "shape_seed": 12},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "decode", "prefill"])
    shape_seed = rng.randrange(1 << 20)
    if op == "norm_rope":
        d = rng.choice([64, 96, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        return {"op": op, "tokens": _log_int(rng, 1, 8192), "hq": hkv * rng.randint(1, 4),
                "hkv": hkv, "d": d, "rot": 16 * rng.randint(1, d // 16),
                "interleaved": rng.random() < 0.4, "norm": rng.random() < 0.7,
                "scaling": rng.choice(["none", "linear", "yarn"]), "fused": rng.random() < 0.5,
                "kv": rng.choice(["bf16", "bf16", "e4m3"]),
                "max_pos": _log_int(rng, 100, 1000000), "shape_seed": shape_seed}
    if op == "decode":
        seqs = _log_int(rng, 1, 256)
        # seqs * window stays under the largest listed case's
        window = _log_int(rng, 1, min(32768, (256 * 4096) // seqs))
        hkv = rng.choice([1, 2, 4, 8])
        max_len = _log_int(rng, 16, 4 * window + 64)
        return {"op": op, "seqs": seqs, "hq": hkv * rng.randint(1, 4 if hkv == 8 else 8),
                "hkv": hkv, "d": rng.choice([64, 128, 128]), "window": window,
                "sinks": rng.choice([0, 1, 4, 16, rng.randint(0, 128)]),
                "min_len": rng.choice([0, 1, max_len // 2]), "max_len": max_len,
                "shape_seed": shape_seed}
    chunks = rng.randint(1, 8)
    max_q = _log_int(rng, 1, 8192 // chunks)
    hkv = rng.choice([1, 2, 4, 8])
    return {"op": op, "chunks": chunks, "hq": hkv * rng.choice([1, 2, 4] + [8] * (hkv < 8)),
            "hkv": hkv, "window": _log_int(rng, 1, 4096),
            "sinks": rng.choice([0, 1, 4, 16, rng.randint(0, 256)]),
            "min_q": rng.choice([1, max(1, max_q // 2), max_q]), "max_q": max_q,
            "max_start": _log_int(rng, 1, 24576), "shape_seed": shape_seed}


# ------------------------------------------------------------------ shapes of a case

def _lengths(case):
    """Sequence lengths of a decode case: spread evenly over their logarithm."""
    r = random.Random(case["shape_seed"])
    lo, hi = case["min_len"], case["max_len"]
    lens = [lo if r.random() < 0.05 else _log_int(r, max(lo, 1), max(hi, 1))
            for _ in range(case["seqs"])]
    lens[0] = max(hi, 1)
    return lens


def _chunk_shapes(case):
    """(query counts, start positions) of a prefill case."""
    r = random.Random(case["shape_seed"])
    q = [r.randint(case["min_q"], case["max_q"]) for _ in range(case["chunks"])]
    start = [r.randint(0, case["max_start"]) for _ in range(case["chunks"])]
    q[0], start[0] = case["max_q"], case["max_start"]
    return q, start


def _visible(p, window, sinks):
    """Number of keys that the query at position p sees."""
    first = max(0, p - window + 1)
    return p - first + 1 + min(sinks, first)


def _visible_sum(p0, n, window, sinks):
    return sum(_visible(p, window, sinks) for p in range(p0, p0 + n))


# ------------------------------------------------------------------ inputs

def _bf16(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)


def _frequencies(case):
    """Rotary frequencies in radians per position (Python floats) and the factor of the
    rotated values: base 10000 (500000 far out), position interpolation by 4, or the
    by-parts interpolation by 16 of a 4096-token context."""
    rot = case["rot"]
    base = 500000.0 if case["max_pos"] > 40000 else 10000.0
    freq = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == "linear":
        return [f / 4.0 for f in freq], 1.0
    if case["scaling"] == "yarn":
        factor, original = 16.0, 4096.0

        def turns_at(turns):  # the pair that makes `turns` turns over the original context
            return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))

        low = max(math.floor(turns_at(32.0)), 0)
        high = min(math.ceil(turns_at(1.0)), rot - 1)
        out = []
        for i, f in enumerate(freq):
            ramp = min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
            out.append(f / factor * ramp + f * (1.0 - ramp))
        return out, 0.1 * math.log(factor) + 1.0
    return freq, 1.0


def _increments(freq):
    """Frequencies as fixed-point turns: units of 2^-64 turn per position, as int64."""
    wrapped = [int(round(f / (2 * math.pi) * 2.0 ** 64)) % (1 << 64) for f in freq]
    return [w - (1 << 64) if w >= 1 << 63 else w for w in wrapped]


def _paged(gen, lens, first_kept, hkv, d, sinks):
    """Pools and tables that hold, of each sequence, the blocks of its first `sinks` keys
    and those from position first_kept[s] on; the other table entries are -1, as a cache
    manager leaves them that frees what left the window."""
    width = max(1, max((n + BLOCK - 1) // BLOCK for n in lens))
    keep = torch.zeros((len(lens), width), dtype=torch.bool)
    for s, n in enumerate(lens):
        keep[s, : min((sinks + BLOCK - 1) // BLOCK, (n + BLOCK - 1) // BLOCK)] = True
        keep[s, first_kept[s] // BLOCK:(n + BLOCK - 1) // BLOCK] = True
    keep = keep.cuda()
    used = int(keep.sum())
    blocks = used + max(8, used // 8)
    place = torch.randperm(blocks, generator=gen, device="cuda")[:used].to(torch.int32)
    tables = torch.full(keep.shape, -1, dtype=torch.int32, device="cuda")
    tables[keep] = place
    return (_bf16(gen, blocks, BLOCK, hkv, d), _bf16(gen, blocks, BLOCK, hkv, d), tables)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "norm_rope":
        t, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
        if case["fused"]:  # one projection's output, split by columns
            qkv = _bf16(gen, t, hq + 2 * hkv, d)
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            s["q"], s["k"], s["v"] = (_bf16(gen, t, h, d) for h in (hq, hkv, hkv))
        freq, s["factor"] = _frequencies(case)
        s["freq"] = torch.tensor(freq, dtype=torch.float64, device="cuda")
        s["increments"] = torch.tensor(_increments(freq), dtype=torch.int64, device="cuda")
        s["positions"] = torch.randint(0, case["max_pos"], (t,), generator=gen, device="cuda")
        s["qw"] = s["kw"] = None
        if case["norm"]:
            s["qw"], s["kw"] = (1 + 0.1 * torch.randn(d, generator=gen, device="cuda")
                                for _ in range(2))
        blocks = (t + BLOCK - 1) // BLOCK + 4
        s["slots"] = torch.randperm(blocks * BLOCK, generator=gen, device="cuda")[:t]
        s["slots"][torch.rand(t, generator=gen, device="cuda") < 0.02] = -1  # padding
        shape = (blocks, BLOCK, hkv, d)
        if case["kv"] == "e4m3":
            s["kc"], s["vc"] = (torch.randint(0, 120, shape, generator=gen, device="cuda",
                                              dtype=torch.uint8) for _ in range(2))
            s["ks"], s["vs"] = (0.01 + 0.02 * torch.rand(hkv, generator=gen, device="cuda")
                                for _ in range(2))
        else:
            s["kc"], s["vc"] = _bf16(gen, *shape), _bf16(gen, *shape)
        s["q_out"] = torch.empty((t, hq, d), dtype=torch.bfloat16, device="cuda")
        return s
    if case["op"] == "decode":
        lens, d = _lengths(case), case["d"]
        first = [max(0, n - case["window"]) for n in lens]
        s["q"] = _bf16(gen, len(lens), case["hq"], d)
        s["kc"], s["vc"], s["tables"] = _paged(gen, lens, first, case["hkv"], d, case["sinks"])
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    else:
        d = 128
        counts, start = _chunk_shapes(case)
        lens = [n + p for n, p in zip(counts, start)]
        first = [max(0, p - case["window"] + 1) for p in start]
        cu = [0]
        for n in counts:
            cu.append(cu[-1] + n)
        s["q"] = _bf16(gen, cu[-1], case["hq"], d)
        s["kc"], s["vc"], s["tables"] = _paged(gen, lens, first, case["hkv"], d, case["sinks"])
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
        s["max_q"] = max(counts)
    s["scale"] = 1.0 / math.sqrt(d)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms

def _plain_norm_rope(s):
    case = s["case"]
    angle = s["positions"].double()[:, None, None] * s["freq"]
    cos, sin = (f(angle).float() * s["factor"] for f in (torch.cos, torch.sin))
    rot = case["rot"]

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        y = x.clone()
        if case["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
        return y

    q, k, v = one(s["q"], s["qw"]), one(s["k"], s["kw"]), s["v"]
    kept = s["slots"] >= 0
    slots = s["slots"][kept]
    if case["kv"] == "e4m3":
        k = (k / s["ks"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        v = (v.float() / s["vs"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        k, v = k.view(torch.uint8), v.view(torch.uint8)
    else:
        k = k.to(torch.bfloat16)
    s["kc"].view(-1, case["hkv"], case["d"])[slots] = k[kept]
    s["vc"].view(-1, case["hkv"], case["d"])[slots] = v[kept]
    return q.to(torch.bfloat16)


def _plain_attention(s, q, start, counts):
    """q [C, M, Hq, D] float: row i of sequence c stands at start[c] + i (valid while
    i < counts[c]).  Keys: the first `sinks`, and `window` - 1 + M from the first row's
    window on."""
    case = s["case"]
    c, m, hq, d = q.shape
    hkv, window, sinks = case["hkv"], case["window"], case["sinks"]
    dev = q.device
    start, counts = start.long(), counts.long()
    # no key lies past the longest sequence, nor (under a long window) before position 0
    span = min(window - 1 + m, s["tables"].shape[1] * BLOCK)
    first = (start - (window - 1)).clamp(min=0)
    near = first[:, None] + torch.arange(span, device=dev)
    far = torch.arange(sinks, device=dev).expand(c, sinks)
    pos = torch.cat([far, near], 1)  # [C, L]
    held = pos < (start + counts)[:, None]
    held[:, sinks:] &= near >= sinks  # counted once
    block = (pos // BLOCK).clamp(max=s["tables"].shape[1] - 1)
    ids = torch.gather(s["tables"], 1, block).long().clamp(min=0)
    rows = ids * BLOCK + pos % BLOCK
    at = start[:, None] + torch.arange(m, device=dev)
    gap = at[:, :, None] - pos[:, None, :]
    seen = (gap >= 0) & ((pos[:, None, :] < sinks) | (gap < window)) & held[:, None, :]
    seen &= (torch.arange(m, device=dev) < counts[:, None])[:, :, None]
    some = seen.any(1)[:, :, None, None]
    k = torch.where(some, s["kc"].view(-1, hkv, d)[rows].float(), 0.0)  # [C, L, Hkv, D]
    v = torch.where(some, s["vc"].view(-1, hkv, d)[rows].float(), 0.0)
    qg = q.view(c, m, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(c, hkv, -1, d)
    score = torch.matmul(qg, k.permute(0, 2, 3, 1)) * s["scale"]  # [C, Hkv, G * M, L]
    score = score.view(c, hkv, hq // hkv, m, -1).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(score.sub_(top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(c, hkv, -1, p.shape[-1]), v.permute(0, 2, 1, 3))
    out = out.view(c, hkv, hq // hkv, m, d) / total.clamp(min=1e-30)
    lse = (top + torch.log(total)).squeeze(-1)
    return (out.permute(0, 3, 1, 2, 4).reshape(c, m, hq, d),
            lse.permute(0, 3, 1, 2).reshape(c, m, hq))


def _plain_decode(s):
    lens = s["lens"].long()
    out, lse = _plain_attention(s, s["q"].float()[:, None], (lens - 1).clamp(min=0),
                                (lens > 0).long())
    return out[:, 0].to(torch.bfloat16), lse[:, 0]


def _plain_prefill(s):
    counts = s["cu"].long().diff()
    steps = torch.arange(s["max_q"], device="cuda")
    rows = s["cu"].long()[:-1, None] + steps
    valid = steps < counts[:, None]
    q = s["q"].float()[rows.clamp(max=s["q"].shape[0] - 1)]
    out, lse = _plain_attention(s, q, s["start"], counts)
    return out[valid].to(torch.bfloat16), lse[valid]


def run(state):
    s = state
    case = s["case"]
    if case["op"] == "norm_rope":
        if own:
            from paged_kv_cache_218_gb300 import binding as pa
            if case["kv"] == "e4m3":
                pa.pa_qk_norm_rope_cache_fp8(
                    s["q_out"], s["q"], s["k"], s["v"], s["positions"], s["increments"],
                    s["kc"], s["vc"], s["slots"], s["ks"], s["vs"], q_weight=s["qw"],
                    k_weight=s["kw"], eps=1e-6, interleaved=case["interleaved"],
                    rope_factor=s["factor"])
            else:
                pa.pa_qk_norm_rope_cache(
                    s["q_out"], s["q"], s["k"], s["v"], s["positions"], s["increments"],
                    s["kc"], s["vc"], s["slots"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6,
                    interleaved=case["interleaved"], rope_factor=s["factor"])
            q = s["q_out"]
        else:
            q = _plain_norm_rope(s)
        if case["kv"] == "e4m3":
            return {"q": q, "k_cache": s["kc"].view(torch.float8_e4m3fn),
                    "v_cache": s["vc"].view(torch.float8_e4m3fn)}
        return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}
    if own:
        from paged_kv_cache_218_gb300 import binding as pa
        if case["op"] == "decode":
            pa.pa_decode_window(s["out"], s["q"], s["kc"], s["vc"], s["tables"], s["lens"],
                                case["window"], case["sinks"], s["scale"], out_lse=s["lse"])
        else:
            pa.pa_prefill_window(s["out"], s["q"], s["kc"], s["vc"], s["tables"], s["cu"],
                                 s["start"], s["lens"], s["max_q"], case["window"],
                                 case["sinks"], s["scale"], out_lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    out, lse = _plain_decode(s) if case["op"] == "decode" else _plain_prefill(s)
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        t, d, rot = case["tokens"], case["d"], case["rot"]
        freq = torch.tensor(_frequencies(case)[0], dtype=torch.float64)
        phase = torch.outer(s["positions"].cpu().double(), freq)
        turn = torch.polar(torch.full_like(phase, _frequencies(case)[1]), phase).cuda()[:, None]

        def one(x, w):
            x = x.double()
            if w is not None:
                x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / d + 1e-6) * w.double()
            head, rest = x[..., :rot], x[..., rot:]
            if case["interleaved"]:
                z = torch.view_as_complex(head.reshape(t, -1, rot // 2, 2).contiguous())
                head = torch.view_as_real(z * turn).reshape(t, -1, rot)
            else:
                z = torch.complex(head[..., :rot // 2], head[..., rot // 2:]) * turn
                head = torch.cat([z.real, z.imag], -1)
            return torch.cat([head, rest], -1)

        q, k, v = one(s["q"], s["qw"]), one(s["k"], s["kw"]), s["v"].double()
        if case["kv"] == "e4m3":
            kc, vc = (s[n].view(torch.float8_e4m3fn).double() for n in ("kc", "vc"))
            k = (k / s["ks"].double()[None, :, None]).clamp(-448, 448)
            v = (v / s["vs"].double()[None, :, None]).clamp(-448, 448)
        else:
            kc, vc = s["kc"].double(), s["vc"].double()
        kept = torch.nonzero(s["slots"] >= 0).squeeze(1)
        kc.flatten(0, 1).index_copy_(0, s["slots"][kept], k[kept])
        vc.flatten(0, 1).index_copy_(0, s["slots"][kept], v[kept])
        return {"q": q, "k_cache": kc, "v_cache": vc}

    # attention: one sequence at a time, its keys in order, rows in slices
    window, sinks, hkv = case["window"], case["sinks"], case["hkv"]
    g = case["hq"] // hkv
    if case["op"] == "decode":
        lens = _lengths(case)
        spans = [(i, i + 1, n - 1) for i, n in enumerate(lens)]
    else:
        counts, start = _chunk_shapes(case)
        spans, row = [], 0
        for n, p in zip(counts, start):
            spans.append((row, row + n, p))
            row += n
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for c, (row0, row1, p0) in enumerate(spans):
        for r0 in range(row0, row1, 512):
            r1 = min(row1, r0 + 512)
            p = p0 + r0 - row0
            last = p + r1 - r0 - 1
            if last < 0:
                continue
            near = max(0, p - window + 1)
            keys = list(range(min(sinks, near))) + list(range(near, last + 1))
            j = torch.tensor(keys, device="cuda")
            slot = s["tables"][c].long()[j // BLOCK] * BLOCK + j % BLOCK
            i = torch.arange(p, last + 1, device="cuda")[:, None]
            hide = (j > i) | ((j >= sinks) & (j <= i - window))
            for h in range(hkv):
                kk = s["kc"].flatten(0, 1)[slot, h].double()
                vv = s["vc"].flatten(0, 1)[slot, h].double()
                for e in range(h * g, h * g + g):
                    a = s["q"][r0:r1, e].double() @ kk.T * s["scale"]
                    a[hide] = -math.inf
                    z = torch.logsumexp(a, 1)
                    out[r0:r1, e] = torch.exp(a - z[:, None]) @ vv
                    lse[r0:r1, e] = z
    return {"out": out, "lse": lse}


def work(case):
    if case["op"] == "norm_rope":
        t, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
        to = 1 if case["kv"] == "e4m3" else 2
        per_token = (hq * 4 + 2 * hkv * (2 + to)) * d + 16
        flops = t * (hq + hkv) * (4 * d * case["norm"] + 3 * case["rot"])
        return {"bytes": t * per_token + 8 * d + 4 * case["rot"], "flops": flops}
    window, sinks, hq, hkv = case["window"], case["sinks"], case["hq"], case["hkv"]
    if case["op"] == "decode":
        d = case["d"]
        pairs = sum(_visible(n - 1, window, sinks) for n in _lengths(case) if n > 0)
        rows, keys = case["seqs"], pairs
    else:
        d = 128
        counts, start = _chunk_shapes(case)
        pairs = sum(_visible_sum(p, n, window, sinks) for n, p in zip(counts, start))
        keys = sum(_visible(p, window, sinks) + n - 1 for n, p in zip(counts, start))
        rows = sum(counts)
    return {"bytes": keys * hkv * d * 4 + rows * hq * (4 * d + 4) + keys // BLOCK * 4,
            "flops": 4 * d * hq * pairs}
