"""The operators of a beam-search step over the paged cache, case by case.

Three operators, in the order such a step runs them:

* ``shared``: decode attention of a batch whose sequences share long prefixes (the
  beams of a prompt, or every request behind one system prompt), the prefix attended
  once for all sequences of a group;
* ``select``: the best continuations of each request, over its beams and the
  vocabulary, from the logits and the beams' scores;
* ``reorder``: block tables, lengths and the partly filled blocks of the paged cache
  rearranged after the selection.

``own`` false: their plain form in torch.  ``own`` true: this package's calls.
"""
import math
import random

import torch

own = False

BLOCK = 16


def listed():
    return [
        # one request's four beams behind a prompt of a thousand tokens: latency
        {"name": "shared one 4 x 992", "op": "shared", "groups": 1, "min_members": 4,
         "max_members": 4, "hq": 32, "hkv": 8, "min_prefix": 62, "max_prefix": 62,
         "min_suffix": 1, "max_suffix": 40, "short": False, "shape_seed": 1},
        # a batch of 64 requests of four beams each, prompts of 256 to 2048 tokens: bandwidth
        {"name": "shared 64 x 4", "op": "shared", "groups": 64, "min_members": 4,
         "max_members": 4, "hq": 32, "hkv": 8, "min_prefix": 16, "max_prefix": 128,
         "min_suffix": 1, "max_suffix": 128, "short": False, "shape_seed": 2},
        # 256 requests behind one system prompt: the prefix is a dense product
        {"name": "shared 256 of 8192", "op": "shared", "groups": 1, "min_members": 256,
         "max_members": 256, "hq": 32, "hkv": 8, "min_prefix": 512, "max_prefix": 512,
         "min_suffix": 16, "max_suffix": 512, "short": False, "shape_seed": 3},
        # 32 questions about one long document: the key axis has to be split
        {"name": "shared 32 of 65536", "op": "shared", "groups": 1, "min_members": 32,
         "max_members": 32, "hq": 32, "hkv": 8, "min_prefix": 4096, "max_prefix": 4096,
         "min_suffix": 1, "max_suffix": 64, "short": False, "shape_seed": 4},
        # odd everything: three query heads a kv head, groups from nothing to 41 members,
        # groups without a prefix, members that end inside it or are empty
        {"name": "shared ragged 9", "op": "shared", "groups": 9, "min_members": 0,
         "max_members": 41, "hq": 15, "hkv": 5, "min_prefix": 0, "max_prefix": 37,
         "min_suffix": 0, "max_suffix": 333, "short": True, "shape_seed": 5},
        # one request, four beams, a small vocabulary: latency
        {"name": "select one 4 x 32000", "op": "select", "requests": 1, "beams": 4,
         "choices": 4, "vocab": 32000, "pad": 0, "logits": "bf16", "masked": False,
         "finished": True, "shape_seed": 6},
        # a batch of four beams over a large vocabulary, twice as many choices as beams so
        # that ended ones can be set aside: bandwidth
        {"name": "select 64 x 4 x 131072", "op": "select", "requests": 64, "beams": 4,
         "choices": 8, "vocab": 131072, "pad": 0, "logits": "bf16", "masked": False,
         "finished": False, "shape_seed": 7},
        # wide beams, fp32 logits
        {"name": "select 16 x 16 x 131072", "op": "select", "requests": 16, "beams": 16,
         "choices": 32, "vocab": 131072, "pad": 0, "logits": "fp32", "masked": False,
         "finished": False, "shape_seed": 8},
        # odd sizes, rows of a padded matrix, tokens that a grammar forbids, ended beams
        {"name": "select ragged 37 x 3 x 50001", "op": "select", "requests": 37, "beams": 3,
         "choices": 5, "vocab": 50001, "pad": 6, "logits": "bf16", "masked": True,
         "finished": True, "shape_seed": 9},
        # one request's four beams in a cache of 32 layers: latency
        {"name": "reorder one 4", "op": "reorder", "requests": 1, "beams": 4, "layers": 32,
         "hkv": 8, "d": 128, "kv": "bf16", "max_len": 2048, "shape_seed": 10},
        # a batch in a cache of 32 layers: bandwidth
        {"name": "reorder 64 x 4", "op": "reorder", "requests": 64, "beams": 4, "layers": 32,
         "hkv": 8, "d": 128, "kv": "bf16", "max_len": 2048, "shape_seed": 11},
        # an odd number of requests and beams in an E4M3 cache with few small heads
        {"name": "reorder ragged e4m3 37 x 5", "op": "reorder", "requests": 37, "beams": 5,
         "layers": 7, "hkv": 3, "d": 64, "kv": "e4m3", "max_len": 333, "shape_seed": 12},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared", "select", "reorder"])
    shape_seed = rng.randrange(1 << 20)
    if op == "shared":
        groups = _log_int(rng, 1, 64)
        members = _log_int(rng, 1, 256 // groups)
        hkv = rng.choice([1, 2, 4, 8])
        g = rng.randint(1, 4 if hkv == 8 else 8)
        # query-key pairs of the prefix, and its tokens, stay below the largest case's
        prefix = _log_int(rng, 1, min(4096, (256 * 512) // (groups * members),
                                      4096 // groups))
        suffix = _log_int(rng, 1, min(512, (256 * 512) // (groups * members)))
        return {"op": op, "groups": groups, "min_members": rng.choice([0, 1, members]),
                "max_members": members, "hq": hkv * g, "hkv": hkv,
                "min_prefix": rng.choice([0, prefix // 2, prefix]), "max_prefix": prefix,
                "min_suffix": rng.choice([0, 1, suffix // 2]), "max_suffix": suffix,
                "short": rng.random() < 0.3, "shape_seed": shape_seed}
    if op == "select":
        beams = _log_int(rng, 1, 32)
        vocab = _log_int(rng, 64, 131072)
        requests = _log_int(rng, 1, max(1, min(256, (256 * 131072) // (beams * vocab))))
        return {"op": op, "requests": requests, "beams": beams,
                "choices": min(vocab, rng.choice([beams, 2 * beams, rng.randint(1, 64)])),
                "vocab": vocab, "pad": rng.choice([0, 0, rng.randint(1, 64)]),
                "logits": rng.choice(["bf16", "fp32"]), "masked": rng.random() < 0.3,
                "finished": rng.random() < 0.5, "shape_seed": shape_seed}
    beams = _log_int(rng, 1, 32)
    requests = _log_int(rng, 1, max(1, 256 // beams))
    hkv = rng.choice([1, 2, 3, 8])
    return {"op": op, "requests": requests, "beams": beams, "layers": _log_int(rng, 1, 32),
            "hkv": hkv, "d": rng.choice([64, 128]), "kv": rng.choice(["bf16", "bf16", "e4m3"]),
            "max_len": _log_int(rng, 16, 4096), "shape_seed": shape_seed}


# ------------------------------------------------------------------ shapes of a case

def _group_shapes(case):
    """(members, shared blocks) of each group, and the sequences' lengths in order."""
    r = random.Random(case["shape_seed"])
    members, shared, lens = [], [], []
    for g in range(case["groups"]):
        first = g == 0
        m = case["max_members"] if first else r.randint(case["min_members"], case["max_members"])
        p = case["max_prefix"] if first else r.randint(case["min_prefix"], case["max_prefix"])
        members.append(m)
        shared.append(p)
        for _ in range(m):
            n = p * BLOCK + r.randint(case["min_suffix"], case["max_suffix"])
            if case["short"] and r.random() < 0.1:
                n = r.randint(0, p * BLOCK)  # ends inside the prefix
            lens.append(n)
    return members, shared, lens


def _parents(case):
    """Parents of a reorder case: beams with better scores have more children."""
    r = random.Random(case["shape_seed"])
    w = case["beams"]
    out = []
    for _ in range(case["requests"]):
        row = [min(w - 1, int(r.expovariate(2.5 / w))) for _ in range(w)]
        if r.random() < 0.1:
            row[w - 1] = -1  # fewer candidates than beams
        out.append(row)
    return out


def _beam_lens(case):
    """A request's beams are as long as one another."""
    r = random.Random(case["shape_seed"] + 1)
    return [r.randint(0, case["max_len"]) for _ in range(case["requests"])]


# ------------------------------------------------------------------ inputs

def _bf16(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)


def _prepare_shared(case, gen):
    s = {"case": case}
    hq, hkv, d = case["hq"], case["hkv"], 128
    members, shared, lens = _group_shapes(case)
    # the group's prefix blocks, then each sequence's own
    own_blocks = []
    i = 0
    for m, p in zip(members, shared):
        for _ in range(m):
            own_blocks.append(max(0, (lens[i] + BLOCK - 1) // BLOCK - p))
            i += 1
    used = sum(shared) + sum(own_blocks)
    blocks = used + max(8, used // 8)
    place = torch.randperm(blocks, generator=gen, device="cuda")[:used].to(torch.int32).cpu()
    width = max([1] + shared + [(n + BLOCK - 1) // BLOCK for n in lens])
    tables = torch.full((len(lens), width), -1, dtype=torch.int32)
    at, i = 0, 0
    for m, p in zip(members, shared):
        prefix = place[at:at + p]
        at += p
        for _ in range(m):
            tables[i, :p] = prefix
            tables[i, p:p + own_blocks[i]] = place[at:at + own_blocks[i]]
            at += own_blocks[i]
            i += 1
    offsets = [0]
    for m in members:
        offsets.append(offsets[-1] + m)
    s["q"] = _bf16(gen, len(lens), hq, d)
    s["kc"], s["vc"] = _bf16(gen, blocks, BLOCK, hkv, d), _bf16(gen, blocks, BLOCK, hkv, d)
    s["tables"] = tables.cuda()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    s["shared"] = torch.tensor(shared, dtype=torch.int32, device="cuda")
    s["max_members"], s["max_prefix"] = max(members), max(shared)
    s["max_suffix"] = max([0] + own_blocks) * BLOCK
    s["scale"] = 1.0 / math.sqrt(d)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    if own:
        from paged_kv_cache_218_gb300 import binding as pa
        s["workspace"] = torch.empty(pa.pa_decode_shared_workspace_size(
            len(lens), case["groups"], s["max_members"], hq, hkv, d), dtype=torch.uint8,
            device="cuda")
    return s


def _prepare_select(case, gen):
    r, w, v = case["requests"], case["beams"], case["vocab"]
    s = {"case": case}
    x = 2.5 * torch.randn((r, w, v + case["pad"]), generator=gen, device="cuda")
    # a few likely tokens stand out
    likely = torch.randint(0, v, (r, w, 8), generator=gen, device="cuda")
    x.scatter_add_(2, likely, 6.0 + 4.0 * torch.rand(likely.shape, generator=gen, device="cuda"))
    if case["masked"]:  # each row allows some share of the tokens
        share = torch.rand((r, w, 1), generator=gen, device="cuda") ** 4
        x.masked_fill_(torch.rand(x.shape, generator=gen, device="cuda") > share, -math.inf)
    s["logits"] = x.to(torch.bfloat16 if case["logits"] == "bf16" else torch.float32)[..., :v]
    scores = -5.0 - 3.0 * torch.rand((r, w), generator=gen, device="cuda").cumsum(1)
    shape = random.Random(case["shape_seed"])
    for i in range(r):  # some requests have just begun, with one beam
        if shape.random() < 0.1:
            scores[i, 0] = 0.0
            scores[i, 1:] = -math.inf
    s["scores"] = scores
    s["finished"] = None
    s["end"] = -1
    if case["finished"]:
        s["finished"] = torch.rand((r, w), generator=gen, device="cuda") < 0.2
        s["end"] = v // 2
    k = case["choices"]
    s["parents"], s["tokens"] = (torch.empty((r, k), dtype=torch.int32, device="cuda")
                                 for _ in range(2))
    s["out_scores"] = torch.empty((r, k), dtype=torch.float32, device="cuda")
    s["out_finished"] = torch.empty((r, k), dtype=torch.bool, device="cuda")
    return s


def _prepare_reorder(case, gen):
    r, w = case["requests"], case["beams"]
    s = {"case": case}
    lens = _beam_lens(case)
    s["parents"] = torch.tensor(_parents(case), dtype=torch.int32, device="cuda")
    s["lens"] = torch.tensor([n for n in lens for _ in range(w)], dtype=torch.int32,
                             device="cuda")
    width = (case["max_len"] + BLOCK) // BLOCK + 1
    blocks = 2 * r * w + 7
    place = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    # the block of the next token, and one behind it, are a beam's own; those before
    # are shared
    tables = place[2 * r * w:][torch.randint(0, 7, (r, 1, width), generator=gen, device="cuda")]
    tables = tables.expand(r, w, width).reshape(r * w, width).clone()
    col = torch.arange(width, device="cuda")
    tail = (s["lens"].long() // BLOCK)[:, None]
    tables = torch.where(col == tail, place[:r * w, None], tables)
    tables = torch.where(col == tail + 1, place[r * w:2 * r * w, None], tables)
    s["tables"] = torch.where(col > tail + 1, -1, tables)
    shape = (case["layers"], blocks, BLOCK, case["hkv"], case["d"])
    if case["kv"] == "e4m3":
        s["kc"], s["vc"] = (torch.randint(0, 120, shape, generator=gen, device="cuda",
                                          dtype=torch.uint8) for _ in range(2))
    else:
        s["kc"], s["vc"] = _bf16(gen, *shape), _bf16(gen, *shape)
    s["out_tables"], s["out_lens"] = torch.empty_like(s["tables"]), torch.empty_like(s["lens"])
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    return {"shared": _prepare_shared, "select": _prepare_select,
            "reorder": _prepare_reorder}[case["op"]](case, gen)


# ------------------------------------------------------------------ plain forms

def _softmax_part(q, k, v, seen, scale):
    """q [B, R, H, D], k and v [B, L, H, D], seen [B, R, L]: the attention over these keys
    alone as (reference maximum, sum of weights, weighted sum of v)."""
    x = torch.matmul(q.permute(0, 2, 1, 3), k.permute(0, 2, 3, 1)) * scale  # [B, H, R, L]
    x = x.masked_fill_(~seen[:, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38) if x.shape[-1] else \
        x.new_full(x.shape[:-1] + (1,), -3e38)
    p = torch.exp(x.sub_(top))
    return top, p.sum(-1, keepdim=True), torch.matmul(p, v.permute(0, 2, 1, 3))


def _plain_shared(s):
    case = s["case"]
    hq, hkv, d = case["hq"], case["hkv"], 128
    g = hq // hkv
    dev = s["q"].device
    tables, lens = s["tables"].long(), s["lens"].long()
    members = s["offsets"].long().diff()
    group = torch.repeat_interleave(torch.arange(case["groups"], device=dev), members,
                                    output_size=lens.shape[0])
    shared = s["shared"].long() * BLOCK  # tokens
    # ---- prefixes: a group's queries against its first member's leading blocks
    m = s["max_members"]
    row = s["offsets"].long()[:-1, None] + torch.arange(m, device=dev)
    present = torch.arange(m, device=dev) < members[:, None]
    row = row.clamp(max=lens.shape[0] - 1)
    pos = torch.arange(s["max_prefix"] * BLOCK, device=dev)
    limit = torch.minimum(lens[row], shared[:, None]) * present  # [groups, m]
    seen = pos < limit[:, :, None]
    slots = (tables[row[:, 0]][:, :s["max_prefix"]].clamp(min=0)[:, :, None] * BLOCK +
             torch.arange(BLOCK, device=dev)).flatten(1)
    any_row = seen.any(1)[:, :, None, None]
    kp = torch.where(any_row, s["kc"].view(-1, hkv, d)[slots].float(), 0.0)
    vp = torch.where(any_row, s["vc"].view(-1, hkv, d)[slots].float(), 0.0)
    q = s["q"].float().view(-1, hkv, g, d)
    qp = q[row].permute(0, 1, 3, 2, 4).reshape(case["groups"], m * g, hkv, d)
    tp, lp, op = _softmax_part(qp, kp, vp, seen.repeat_interleave(g, 1), s["scale"])

    def by_sequence(x):  # [groups, H, m * g, c] -> [S, H, g, c]
        return x.view(case["groups"], hkv, m, g, -1).permute(0, 2, 1, 3, 4)[present]

    tp, lp, op = by_sequence(tp), by_sequence(lp), by_sequence(op)
    # ---- suffixes: each sequence's own keys
    pos = shared[group][:, None] + torch.arange(s["max_suffix"], device=dev)
    seen = pos < lens[:, None]
    block = (pos // BLOCK).clamp(max=tables.shape[1] - 1)
    slots = torch.gather(tables, 1, block).clamp(min=0) * BLOCK + pos % BLOCK
    ks = torch.where(seen[:, :, None, None], s["kc"].view(-1, hkv, d)[slots].float(), 0.0)
    vs = torch.where(seen[:, :, None, None], s["vc"].view(-1, hkv, d)[slots].float(), 0.0)
    qs = q.permute(0, 2, 1, 3)
    ts, ls, os = _softmax_part(qs, ks, vs, seen[:, None].expand(-1, g, -1), s["scale"])
    # ---- joined
    top = torch.maximum(tp, ts)
    wp, ws = torch.exp(tp - top), torch.exp(ts - top)
    total = wp * lp + ws * ls
    out = (wp * op + ws * os) / total.clamp(min=1e-30)
    lse = (top + torch.log(total)).view(-1, hq)
    return {"out": out.reshape(-1, hq, d).to(torch.bfloat16), "lse": lse}


def _plain_select(s):
    case = s["case"]
    r, w, v, k = case["requests"], case["beams"], case["vocab"], case["choices"]
    dev = s["scores"].device
    x = s["logits"].float()
    # The k largest logits of a beam, equal ones in the order of their tokens: whole
    # numbers in the same order, the token below them.
    bits = x.view(torch.int32) if x.is_contiguous() else x.contiguous().view(torch.int32)
    order = torch.where(bits >= 0, bits, bits ^ 0x7fffffff).long()  # (-0 stands below +0)
    order = torch.where(x == 0, 0, order)
    key = order * (1 << 32) + ((1 << 31) - torch.arange(v, device=dev))
    best = torch.topk(key, k, 2).values
    token = (1 << 31) - best % (1 << 32)
    # Log-probabilities in 64 bits: two beams' sums often lie within 32 bits' rounding
    lse = torch.logsumexp(x.double(), 2, keepdim=True)
    alive = s["scores"] > -math.inf
    value = s["scores"].double()[..., None] + torch.gather(x, 2, token).double() - lse
    value = torch.where(alive[..., None] & (lse > -math.inf), value, -math.inf)
    if s["finished"] is not None:
        ended = s["finished"][..., None]
        only = torch.arange(k, device=dev) == 0
        value = torch.where(ended, torch.where(only, s["scores"].double()[..., None], -math.inf),
                            value)
        token = torch.where(ended, s["end"], token)
    # beams in order, each with its candidates in order: a stable sort keeps the
    # lowest beam and token of equal values first
    value, at = torch.sort(value.view(r, w * k), dim=1, descending=True, stable=True)
    value, at = value[:, :k], at[:, :k]
    if value.shape[1] < k:
        raise ValueError("more choices than candidates")
    some = value > -math.inf
    parent = torch.where(some, at // k, -1)
    token = torch.where(some, torch.gather(token.view(r, w * k), 1, at), -1)
    out = {"parents": parent.int(), "tokens": token.int(), "scores": value.float()}
    if s["finished"] is not None:
        was = torch.gather(s["finished"], 1, parent.clamp(min=0))
        out["finished"] = some & (was | (token == s["end"]))
    return out


def _plain_reorder(s):
    case = s["case"]
    r, w = case["requests"], case["beams"]
    dev = s["lens"].device
    par = s["parents"].long()
    beam = torch.arange(w, device=dev)
    lens = s["lens"].long().view(r, w)
    # whose own blocks each new beam takes: its parent's where it is the first child,
    # else those of beams without children, in order, beams without a parent last
    same = par[:, :, None] == par[:, None, :]
    first = ~(same & (beam[None, :] < beam[:, None])).any(2) & (par >= 0)
    childless = ~(par[:, None, :] == beam[:, None]).any(2)
    donors = torch.sort((~childless).long(), dim=1, stable=True).indices
    need = torch.where(first, 2, torch.where(par >= 0, 0, 1))
    takers = torch.sort(need, dim=1, stable=True).indices
    owner = torch.empty_like(par).scatter_(1, takers, donors)
    owner = torch.where(first, par, owner)
    base = torch.arange(r, device=dev)[:, None] * w
    new_len = torch.where(par >= 0, torch.gather(lens, 1, par.clamp(min=0)), 0)
    own_len = torch.gather(lens, 1, owner)
    src, own_row = (base + par.clamp(min=0)).flatten(), (base + owner).flatten()
    keep, tail = (new_len // BLOCK).flatten()[:, None], (own_len // BLOCK).flatten()[:, None]
    width = s["tables"].shape[1]
    col = torch.arange(width, device=dev)
    at = tail + col - keep
    own_part = torch.gather(s["tables"][own_row], 1, at.clamp(0, width - 1))
    own_part = torch.where(at < width, own_part, -1)
    tables = torch.where(col < keep, s["tables"][src], own_part)
    # the filled slots of the partly filled block, where it is not the parent's own
    filled = (new_len % BLOCK).flatten()[:, None]
    step = torch.arange(BLOCK, device=dev)
    copied = (step < filled) & ~first.flatten()[:, None]
    from_block = torch.gather(s["tables"][src], 1, keep.clamp(max=width - 1)).long()
    to_block = torch.gather(tables, 1, keep.clamp(max=width - 1)).long()
    source = (from_block * BLOCK + step)[copied]
    target = (to_block * BLOCK + step)[copied]
    for pool in (s["kc"], s["vc"]):
        flat = pool.flatten(1, 2)
        flat[:, target] = flat[:, source]
    return {"tables": tables, "lens": new_len.flatten().int(), "k": s["kc"], "v": s["vc"]}


def _values(case, pool):
    return pool.view(torch.float8_e4m3fn) if case["kv"] == "e4m3" else pool


def run(state):
    s = state
    case = s["case"]
    if not own:
        out = {"shared": _plain_shared, "select": _plain_select,
               "reorder": _plain_reorder}[case["op"]](s)
    else:
        from paged_kv_cache_218_gb300 import binding as pa
        if case["op"] == "shared":
            pa.pa_decode_shared(s["out"], s["q"], s["kc"], s["vc"], s["tables"], s["lens"],
                                s["offsets"], s["max_members"], s["shared"], s["scale"],
                                s["workspace"], out_lse=s["lse"])
            out = {"out": s["out"], "lse": s["lse"]}
        elif case["op"] == "select":
            ends = s["finished"] is not None
            pa.pa_beam_select(s["parents"], s["tokens"], s["out_scores"], s["logits"],
                              s["scores"], finished=s["finished"],
                              out_finished=s["out_finished"] if ends else None,
                              end_token=s["end"])
            out = {"parents": s["parents"], "tokens": s["tokens"], "scores": s["out_scores"]}
            if ends:
                out["finished"] = s["out_finished"]
        else:
            call = pa.pa_beam_reorder_fp8 if case["kv"] == "e4m3" else pa.pa_beam_reorder
            call(s["out_tables"], s["out_lens"], s["tables"], s["lens"], s["parents"], s["kc"],
                 s["vc"])
            out = {"tables": s["out_tables"], "lens": s["out_lens"], "k": s["kc"], "v": s["vc"]}
    if case["op"] == "reorder":
        out["k"], out["v"] = _values(case, out["k"]), _values(case, out["v"])
    return out


# ------------------------------------------------------------------ 64 bits

def _exact_shared(case, s):
    """One sequence at a time, over all its keys in order."""
    hkv, g = case["hkv"], case["hq"] // case["hkv"]
    _, _, lens = _group_shapes(case)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(lens):
        if n == 0:
            continue
        blocks = s["tables"][i, :(n + BLOCK - 1) // BLOCK].long()
        k = s["kc"][blocks].flatten(0, 1)[:n].double().transpose(0, 1)  # [H, n, D]
        v = s["vc"][blocks].flatten(0, 1)[:n].double().transpose(0, 1)
        a = torch.bmm(s["q"][i].double().view(hkv, g, -1), k.transpose(1, 2)) * s["scale"]
        z = torch.logsumexp(a, 2)
        out[i] = torch.bmm(torch.exp(a - z[..., None]), v).reshape(case["hq"], -1)
        lse[i] = z.flatten()
    return {"out": out, "lse": lse}


def _exact_select(case, s):
    """All candidates of a request in one sorted list."""
    k, v = case["choices"], case["vocab"]
    shape = (case["requests"], k)
    out = {"parents": torch.full(shape, -1, dtype=torch.int32, device="cuda"),
           "tokens": torch.full(shape, -1, dtype=torch.int32, device="cuda"),
           "scores": torch.full(shape, -math.inf, dtype=torch.float64, device="cuda")}
    if s["finished"] is not None:
        out["finished"] = torch.zeros(shape, dtype=torch.bool, device="cuda")
    for i in range(case["requests"]):
        x = s["logits"][i].double()
        total = torch.exp(x - x.amax(1, keepdim=True).clamp(min=-1e30)).sum(1)
        value = s["scores"][i].double()[:, None] + (
            x - x.amax(1, keepdim=True).clamp(min=-1e30) - torch.log(total)[:, None])
        value[torch.isnan(value)] = -math.inf
        if s["finished"] is not None:
            for w in torch.nonzero(s["finished"][i]).flatten().tolist():
                value[w] = -math.inf
                value[w, s["end"]] = s["scores"][i, w].double()
        best, at = torch.sort(value.flatten(), descending=True, stable=True)
        n = min(k, int((best > -math.inf).sum()))
        best, at = best[:n], at[:n]
        out["parents"][i, :n], out["tokens"][i, :n] = (at // v).int(), (at % v).int()
        out["scores"][i, :n] = best
        if s["finished"] is not None:
            out["finished"][i, :n] = s["finished"][i][at // v] | (at % v == s["end"])
    return out


def _exact_reorder(case, s):
    """Request by request, beam by beam; copies of whole slots."""
    w = case["beams"]
    lens = _beam_lens(case)
    old = s["tables"].cpu().tolist()
    width = len(old[0])
    tables, new_lens, copies = [], [], []
    for i, row in enumerate(_parents(case)):
        mine = old[i * w:(i + 1) * w]
        full, part = divmod(lens[i], BLOCK)
        idle = [b for b in range(w) if b not in row]
        taken = {}
        for c, p in enumerate(row):
            if p >= 0 and p not in row[:c]:
                taken[c] = p
        for c in [c for c in range(w) if c not in taken and row[c] >= 0]:
            taken[c] = idle.pop(0)
        for c in [c for c in range(w) if c not in taken]:
            taken[c] = idle.pop(0)
        for c, p in enumerate(row):
            tail = mine[taken[c]][full:]
            line = (mine[p][:full] if p >= 0 else []) + tail
            tables.append((line + [-1] * width)[:width])
            new_lens.append(lens[i] if p >= 0 else 0)
            if p >= 0 and taken[c] != p and part:
                copies.append((mine[p][full], tail[0], part))
    k, v = s["kc"].clone(), s["vc"].clone()
    for source, target, n in copies:
        for pool in (k, v):
            pool[:, target, :n] = pool[:, source, :n]
    return {"tables": torch.tensor(tables, dtype=torch.int32, device="cuda"),
            "lens": torch.tensor(new_lens, dtype=torch.int32, device="cuda"),
            "k": _values(case, k), "v": _values(case, v)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"shared": _exact_shared, "select": _exact_select,
            "reorder": _exact_reorder}[case["op"]](case, s)


def work(case):
    if case["op"] == "shared":
        members, shared, lens = _group_shapes(case)
        hq, hkv, d = case["hq"], case["hkv"], 128
        keys = pairs = i = 0
        for m, p in zip(members, shared):
            mine = lens[i:i + m]
            i += m
            keys += min(p * BLOCK, max(mine, default=0))
            keys += sum(max(0, n - p * BLOCK) for n in mine)
            pairs += sum(mine)
        rows = len(lens) * hq
        return {"bytes": keys * hkv * d * 4 + keys // BLOCK * 4 + rows * (4 * d + 4),
                "flops": 4 * d * hq * pairs}
    if case["op"] == "select":
        rows = case["requests"] * case["beams"]
        size = 2 if case["logits"] == "bf16" else 4
        return {"bytes": rows * (case["vocab"] * size + 4) + case["requests"] * case["choices"] * 12,
                "flops": rows * case["vocab"] * 4}
    w = case["beams"]
    size = 1 if case["kv"] == "e4m3" else 2
    slots = 0
    for row, n in zip(_parents(case), _beam_lens(case)):
        live = [p for p in row if p >= 0]
        slots += (len(live) - len(set(live))) * (n % BLOCK)
    width = (case["max_len"] + BLOCK) // BLOCK + 1
    moved = slots * 2 * case["layers"] * case["hkv"] * case["d"] * size
    return {"bytes": 2 * moved + case["requests"] * w * (8 * width + 12), "flops": 0}
