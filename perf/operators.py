"""What a ragged chunk of new tokens costs in one layer over the paged cache.

Three operators, used one after the other for every chunk (a prompt's piece, a
mixed batch of prompts and single tokens, drafts of different lengths):

* ``plan``: row offsets, positions, page tables and slot maps of the chunk,
  built on the GPU from the requests' lengths and a list of free pages;
* ``rope``: the chunk's q, k and v rows as the projection leaves them: per-head
  RMSNorm where the model has one, rotary positions (both layouts, part of the
  head, scaled for long contexts), keys and values stored into their slots;
* ``attn``: attention of the chunk's rows over the paged cache, causal, with an
  optional sliding window and per-head sinks.

``run`` is their plain form; with ``own`` true it makes the library's calls.
Geometries are those of this repository's workloads (32 query heads over 8 or 2
KV heads of 128, a tiny 4-over-2 of 64, pages of 64 or 16) and generic ones.
"""
import math
import random

import torch

own = False

GOLD = 0.6180339887498949


def listed():
    q8 = {"hq": 32, "nkv": 8, "hd": 128, "page": 64}
    head = {"gamma": True, "rot": 128, "layout": "half", "scaling": "plain", "factor": 1.0}
    return [
        # one new token in each of 64 running requests, some idle or finished
        {"name": "plan_decode_64", "op": "plan", "B": 64, "rows": 64, "singles": 64, "ctx": 8192, "page": 64},
        # a server's whole batch: 1000 single tokens and 24 pieces of prompts
        {"name": "plan_mixed_1024", "op": "plan", "B": 1024, "rows": 8192, "singles": 1000, "ctx": 8192, "page": 16},
        # four prompts of a long piece
        {"name": "plan_prompts_16k", "op": "plan", "B": 4, "rows": 16384, "singles": 0, "ctx": 32768, "page": 64},
        # a block's worth of rows, one layer of the decode step: latency
        dict(q8, name="rope_rows_16", op="rope", rows=16, ctx=32768, **head),
        # a prompt's piece with normed heads, whole-head rotation
        dict(q8, name="rope_rows_8192", op="rope", rows=8192, ctx=8192, **head),
        # odd rows, half of a 64-wide head rotated in neighbouring pairs, scaled eightfold past its trained context
        {"name": "rope_part_yarn_5003", "op": "rope", "rows": 5003, "hq": 24, "nkv": 4, "hd": 64, "page": 16, "ctx": 131072,
         "gamma": False, "rot": 32, "layout": "pairs", "scaling": "yarn", "factor": 8.0},
        # the smallest call: three short requests of a few tokens on the tiny geometry
        {"name": "attn_tiny", "op": "attn", "B": 3, "rows": 7, "singles": 1, "ctx": 100, "hq": 4, "nkv": 2, "hd": 64, "page": 16,
         "window": 0, "sinks": True},
        # a single new token of one request at a long context
        dict(q8, name="attn_single_32k", op="attn", B=1, rows=1, singles=1, ctx=32768, window=0, sinks=False),
        # 64 running requests with one to a few thousand keys each
        dict(q8, name="attn_decode_64", op="attn", B=64, rows=64, singles=64, ctx=8192, window=0, sinks=False),
        # a mixed batch: twelve single tokens beside odd pieces of prompts, sliding window and sinks
        {"name": "attn_mixed_window", "op": "attn", "B": 16, "rows": 2311, "singles": 12, "ctx": 8192, "hq": 32, "nkv": 2,
         "hd": 128, "page": 64, "window": 1024, "sinks": True},
        # a fresh prompt
        dict(q8, name="attn_prompt_4096", op="attn", B=1, rows=4096, singles=0, ctx=0, window=0, sinks=False),
        # a prompt's piece far into a long context
        dict(q8, name="attn_piece_1024_at_32k", op="attn", B=1, rows=1024, singles=0, ctx=32768, window=0, sinks=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "attn", "attn"])
    if op == "plan":
        B = _log(rng, 1, 1024)
        singles = rng.choice([0, B, rng.randint(0, B)])
        rows = singles + (0 if singles == B else _log(rng, B - singles, 16384 - singles))
        return {"op": op, "B": B, "rows": rows, "singles": singles, "ctx": _log(rng, 64, 32768), "page": rng.choice([16, 32, 64, 128])}
    if op == "rope":
        hd = rng.choice([64, 128])
        nkv = rng.choice([1, 2, 4, 8])
        return {"op": op, "rows": _log(rng, 1, 8192), "hq": nkv * rng.choice([1, 2, 3, 4]), "nkv": nkv, "hd": hd,
                "page": rng.choice([16, 32, 64]), "ctx": _log(rng, 16, 131072), "gamma": rng.random() < 0.5,
                "rot": rng.choice([hd, hd // 2, hd // 4, 24]), "layout": rng.choice(["half", "pairs"]),
                "scaling": rng.choice(["plain", "linear", "yarn"]), "factor": rng.choice([2.0, 4.0, 8.0])}
    nkv = rng.choice([1, 2, 4, 8])
    c = {"op": op, "hq": nkv * rng.choice([1, 2, 4, 5, 8][: 5 if nkv < 8 else 3]), "nkv": nkv, "hd": rng.choice([64, 128]),
         "page": rng.choice([16, 32, 64, 128]), "window": rng.choice([0, 0, _log(rng, 32, 4096)]), "sinks": rng.random() < 0.5}
    kind = rng.choice(["decode", "mixed", "prompt"])
    if kind == "decode":
        c["B"] = c["rows"] = c["singles"] = _log(rng, 1, 64)
        c["ctx"] = _log(rng, 16, 32768 if c["B"] <= 16 else 8192)
    elif kind == "mixed":
        c["B"] = rng.randint(2, 16)
        c["singles"] = rng.randint(0, c["B"] - 1)
        c["rows"] = c["singles"] + _log(rng, c["B"] - c["singles"], 2048)
        c["ctx"] = _log(rng, 16, 4096)
    else:
        c["B"], c["singles"], c["rows"] = 1, 0, _log(rng, 16, 4096)
        c["ctx"] = rng.choice([0, _log(rng, 16, 32768 if c["rows"] <= 1024 else 1024)])
    return c


# ------------------------------------------------------------------ lengths


def _lengths(case):
    """(new tokens, keys before) of each request, from the case alone."""
    B, singles = case["B"], case["singles"]
    n = [1] * singles
    many = B - singles
    if many:
        w = [0.25 + 1.5 * ((i + 1) * GOLD % 1.0) for i in range(many)]
        left = case["rows"] - singles - many  # each has one row at least
        part = [int(left * x / sum(w)) for x in w]
        part[0] += left - sum(part)
        n += [1 + x for x in part]
    ctx = [int(case["ctx"] * (1.0 if i == 0 else 0.125 + 0.875 * (i * GOLD % 1.0))) for i in range(B)]
    return n, ctx


def _pages(tokens, page):
    return -(-tokens // page)


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    return {"plan": _prepare_plan, "rope": _prepare_rope, "attn": _prepare_attn}[case["op"]](case, seed)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype=torch.bfloat16, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std + mean).to(dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _empty(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def _library(case, max_pages, pool_pages, layers=1):
    """The library and its geometry, where the library's calls are made."""
    if not own:
        return None, None
    import context_kv_update_gb300 as dl
    dl.load()
    hd = case.get("hd", 128)
    return dl, dl.make_geom(dict(kind="gqa", L=layers, D_in=case.get("hq", 1) * hd, D=case.get("hq", 1) * hd, hq=case.get("hq", 1),
                                 nkv=case.get("nkv", 1), hd=hd, P=case["page"], T=1, max_pages=max_pages, num_pool_pages=pool_pages,
                                 rope_theta=1e6, eps_h=1e-6, eps_k=1e-6))


def _prepare_plan(case, seed):
    n, ctx = _lengths(case)
    P, B = case["page"], case["B"]
    order = list(range(B))
    rnd = random.Random(seed)
    rnd.shuffle(order)
    n, ctx = [n[i] for i in order], [ctx[i] for i in order]
    # one request in sixteen has ended, one in sixteen brings nothing to this chunk
    valid = [0 if rnd.random() < 1 / 16 and B > 4 else 1 for _ in range(B)]
    n = [0 if rnd.random() < 1 / 16 and B > 4 else x for x in n]
    have = [_pages(c, P) for c in ctx]
    width = max(_pages(c + x, P) for c, x in zip(ctx, n)) + 2
    used = sum(have)
    pool_pages = used + sum(_pages(x, P) + 1 for x in n) + 8
    perm = torch.randperm(pool_pages, generator=_gen(seed), device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")[None, :]
    have_t = _ints(have)
    start = (have_t.cumsum(0) - have_t)[:, None]
    table = torch.where(col < have_t[:, None], perm[(start + col).clamp(max=pool_pages - 1)], -1).to(torch.int32).contiguous()
    head = 3  # some of the list is spent already
    s = {"op": "plan", "n_new": _ints(n), "ctx": _ints(ctx), "have": have_t, "table": table, "valid": torch.tensor(valid, dtype=torch.uint8, device="cuda"),
         "free": torch.cat([perm[:head], perm[used:]]).contiguous(), "range": _ints([head, head + pool_pages - used]), "P": P, "rows": case["rows"],
         "pool_pages": pool_pages}
    s["dl"], s["geom"] = _library(case, width, pool_pages)
    if own:
        R = case["rows"]
        s["out"] = {"cu_rows": _empty(B + 1), "n_pages": _empty(B), "alloc_limit": _empty(B), "seq_lens": _empty(B), "free_head": _empty(1),
                    "row_req": _empty(R), "row_pos": _empty(R), "row_page": _empty(R), "row_slot": _empty(R)}
    return s


def _spec(case):
    return {"rot": case["rot"], "layout": case["layout"], "scaling": case["scaling"], "factor": case["factor"], "trained": 8192,
            "beta_fast": 32.0, "beta_slow": 1.0, "theta": 1e6, "eps": 1e-6}


def _prepare_rope(case, seed):
    g = _gen(seed)
    rows, hq, nkv, hd, P = case["rows"], case["hq"], case["nkv"], case["hd"], case["page"]
    pages = _pages(rows, P) + 1
    pos = case["ctx"] + torch.arange(rows, device="cuda")
    perm = torch.randperm(pages + 2, generator=g, device="cuda")
    s = {"op": "rope", "qkv": _normal(g, (rows, (hq + 2 * nkv) * hd)), "pos": pos.to(torch.int32), "spec": _spec(case),
         "page": perm[pos // P - case["ctx"] // P].to(torch.int32), "slot": (pos % P).to(torch.int32),
         "pool": _normal(g, (1, pages + 2, 2, nkv, P, hd)), "gq": None, "gk": None, "hq": hq, "nkv": nkv, "hd": hd,
         "q_out": torch.zeros((rows, hq, hd), dtype=torch.bfloat16, device="cuda")}
    if case["gamma"]:
        s["gq"], s["gk"] = _normal(g, (hd,), std=0.02, mean=1.0), _normal(g, (hd,), std=0.02, mean=1.0)
    s["dl"], s["geom"] = _library(case, _pages(case["ctx"] + rows, P) + 1, pages + 2)
    if own:
        dl, sp = s["dl"], s["spec"]
        s["rope"] = dl.RopeSpec(layout=dl.ROPE_HALF if sp["layout"] == "half" else dl.ROPE_PAIRS, rot_dim=sp["rot"],
                                scaling={"plain": dl.ROPE_PLAIN, "linear": dl.ROPE_LINEAR, "yarn": dl.ROPE_YARN}[sp["scaling"]],
                                trained_ctx=sp["trained"], factor=sp["factor"], beta_fast=sp["beta_fast"], beta_slow=sp["beta_slow"], magnitude=0.0)
    return s


def _prepare_attn(case, seed):
    g = _gen(seed)
    n, ctx = _lengths(case)
    order = list(range(case["B"]))
    random.Random(seed).shuffle(order)
    n, ctx = [n[i] for i in order], [ctx[i] for i in order]
    hq, nkv, hd, P = case["hq"], case["nkv"], case["hd"], case["page"]
    kv = [c + x for c, x in zip(ctx, n)]
    have = [_pages(k, P) for k in kv]
    width, pool_pages = max(have) + 1, sum(have) + 4
    perm = torch.randperm(pool_pages, generator=g, device="cuda").to(torch.int32)
    col, have_t = torch.arange(width, device="cuda")[None, :], _ints(have)
    start = (have_t.cumsum(0) - have_t)[:, None]
    table = torch.where(col < have_t[:, None], perm[(start + col).clamp(max=pool_pages - 1)], -1).to(torch.int32).contiguous()
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    s = {"op": "attn", "q": _normal(g, (cu[-1], hq, hd)), "pool": _normal(g, (1, pool_pages, 2, nkv, P, hd)), "table": table, "cu": _ints(cu),
         "ctx": _ints(ctx), "kv": _ints(kv), "sinks": _normal(g, (hq,), torch.float32) if case["sinks"] else None, "window": case["window"],
         "most_rows": max(n), "most_keys": max(kv), "B": case["B"], "nkv": nkv, "P": P, "out": torch.zeros((cu[-1], hq, hd), dtype=torch.bfloat16, device="cuda")}
    s["dl"], s["geom"] = _library(case, width, pool_pages)
    if own:
        need = s["dl"].dflash_chunk_attention_workspace_bytes(s["geom"], case["B"], cu[-1])
        s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    if own:
        return _OWN[s["op"]](s)
    return _PLAIN[s["op"]](s)


def _own_plan(s):
    s["dl"].dflash_chunk_plan(s["geom"], s["n_new"], s["ctx"], s["have"], s["table"], s["free"], s["range"], s["valid"], 1 << 30, s["out"])
    return dict(s["out"], table=s["table"])


def _own_rope(s):
    hq, nkv, hd = s["hq"], s["nkv"], s["hd"]
    q, k, v = s["qkv"].split((hq * hd, nkv * hd, nkv * hd), dim=1)
    s["dl"].dflash_chunk_rope_store(s["geom"], 0, s["rope"], q, k, v, s["pos"], s["page"], s["slot"], s["q_out"], s["pool"], gamma_q=s["gq"], gamma_k=s["gk"])
    return s["q_out"], s["pool"]


def _own_attn(s):
    s["dl"].dflash_chunk_attention(s["geom"], 0, s["q"], s["pool"], s["table"], s["cu"], s["ctx"], s["kv"], s["out"], s["ws"], window=s["window"], sinks=s["sinks"])
    return s["out"]


_OWN = {"plan": _own_plan, "rope": _own_rope, "attn": _own_attn}


def _plain_plan(s):
    P, R, B = s["P"], s["rows"], s["n_new"].shape[0]
    M, dev = s["table"].shape[1], s["n_new"].device
    live = s["valid"] != 0
    n = torch.where(live, s["n_new"].long(), 0)
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), n.cumsum(0)])
    c, have = s["ctx"].long(), s["have"].long()
    want = torch.where(n > 0, ((c + n + P - 1) // P).clamp(max=M), have)
    need = (want - have).clamp(min=0)
    base = need.cumsum(0) - need
    head, tail = s["range"][0].long(), s["range"][1].long()
    got = torch.minimum(need, (tail - head - base).clamp(min=0))
    now = torch.where(live, have + got, 0)
    col = torch.arange(M, device=dev)[None, :]
    new = (col >= have[:, None]) & (col < (have + got)[:, None])
    table = torch.where(new, s["free"][(head + base[:, None] + col - have[:, None]).clamp(0, s["free"].shape[0] - 1)], s["table"])
    limit = (now * P).clamp(max=1 << 30)
    t = torch.arange(R, device=dev)
    req = (t[:, None] >= cu[None, 1:]).sum(1)
    inside = req < B
    r = req.clamp(max=B - 1)
    pos = c[r] + t - cu[r]
    placed = inside & (pos < limit[r])
    page = torch.where(placed, table[r, (pos // P).clamp(max=M - 1)].long(), -1)
    slot = torch.where(placed & (page >= 0), pos % P, -1)
    out = {"cu_rows": cu, "n_pages": now, "alloc_limit": limit, "seq_lens": torch.where(live, torch.minimum(c + n, limit), 0),
           "free_head": (head + got.sum()).reshape(1), "row_req": torch.where(inside, req, -1), "row_pos": torch.where(inside, pos, -1),
           "row_page": page, "row_slot": slot, "table": table}
    return {k: v.to(torch.int32) for k, v in out.items()}


def _frequencies(spec, device):
    """Angle a position turns each pair by, in 64 bits, and the factor on cos and sin."""
    d = spec["rot"]
    j = torch.arange(d // 2, device=device, dtype=torch.float64)
    f = spec["theta"] ** (-2.0 * j / d)
    if spec["scaling"] == "plain":
        return f, 1.0
    if spec["scaling"] == "linear":
        return f / spec["factor"], 1.0
    # the pair that turns b times over the trained context has this index
    low, high = [d * math.log(spec["trained"] / (2 * math.pi * b)) / (2 * math.log(spec["theta"])) for b in (spec["beta_fast"], spec["beta_slow"])]
    low, high = max(math.floor(low), 0), min(math.ceil(high), d - 1)
    ramp = ((j - low) / max(high - low, 1e-3)).clamp(0, 1)
    return f / spec["factor"] * ramp + f * (1 - ramp), 0.1 * math.log(spec["factor"]) + 1.0


def _plain_turn(x, gamma, pos, spec):
    """RMSNorm where gamma is given, then the rotation; x [rows, heads, hd]."""
    x = x.float()
    if gamma is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + spec["eps"]) * gamma.float()
    f, mag = _frequencies(spec, x.device)
    angle = pos.double()[:, None] * f
    cos, sin = (angle.cos() * mag).float()[:, None, :], (angle.sin() * mag).float()[:, None, :]
    d = spec["rot"]
    a, b = (x[..., : d // 2], x[..., d // 2:d]) if spec["layout"] == "half" else (x[..., 0:d:2], x[..., 1:d:2])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat([u, w], -1) if spec["layout"] == "half" else torch.stack([u, w], -1).flatten(-2)
    return torch.cat([turned, x[..., d:]], -1).to(torch.bfloat16)


def _plain_rope(s):
    hq, nkv, hd = s["hq"], s["nkv"], s["hd"]
    q, k, v = (x.unflatten(1, (-1, hd)) for x in s["qkv"].split((hq * hd, nkv * hd, nkv * hd), dim=1))
    page, slot = s["page"].long(), s["slot"].long()
    pool = s["pool"][0]
    pool[page, 0, :, slot] = _plain_turn(k, s["gk"], s["pos"], s["spec"])
    pool[page, 1, :, slot] = v
    return _plain_turn(q, s["gq"], s["pos"], s["spec"]), s["pool"]


def _plain_attn(s):
    B, nkv, P, q = s["B"], s["nkv"], s["P"], s["q"]
    N, hq, hd = q.shape
    G, dev = hq // nkv, q.device
    cu = s["cu"].long()
    i, j = torch.arange(s["most_rows"], device=dev), torch.arange(s["most_keys"], device=dev)
    row = cu[:-1, None] + i
    real = row < cu[1:, None]
    page = s["table"].long().gather(1, (j // P)[None, :].expand(B, -1))
    held = (j[None, :] < s["kv"][:, None]) & (page >= 0)
    pool, slot = s["pool"][0], (j % P)[None, :].expand(B, -1)
    K = pool[page.clamp(min=0), 0, :, slot].float().permute(0, 2, 3, 1)
    V = torch.where(held[:, :, None, None], pool[page.clamp(min=0), 1, :, slot].float(), 0.0).transpose(1, 2)
    x = q[row.clamp(max=N - 1)].float().unflatten(2, (nkv, G)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    score = (x @ K).unflatten(2, (G, -1)) * (1.0 / math.sqrt(hd))
    p = s["ctx"].long()[:, None] + i
    seen = held[:, None, :] & (j <= p[:, :, None])
    if s["window"] > 0:
        seen = seen & (j > p[:, :, None] - s["window"])
    score = score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].view(1, nkv, G, 1, 1)
        top = torch.maximum(top, sink)
    top = top.clamp(min=-1e30)
    w = score.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        total = total + (sink - top).exp()
    o = (w.flatten(2, 3) @ V).unflatten(2, (G, -1)) / total.clamp(min=1e-30)
    return o.permute(0, 3, 1, 2, 4).flatten(2, 3)[real].to(torch.bfloat16)


_PLAIN = {"plan": _plain_plan, "rope": _plain_rope, "attn": _plain_attn}


# ------------------------------------------------------------------ work and the definition in 64 bits


def work(case):
    if case["op"] == "plan":
        n, ctx = _lengths(case)
        touched = sum(_pages(c + x, case["page"]) - c // case["page"] for x, c in zip(n, ctx))
        new = sum(_pages(c + x, case["page"]) - _pages(c, case["page"]) for x, c in zip(n, ctx))
        return {"bytes": 13 * case["B"] + 4 * touched + 4 * new + 16 * case["B"] + 16 * case["rows"] + 16, "flops": 0}
    if case["op"] == "rope":
        vals = case["rows"] * (case["hq"] + 2 * case["nkv"]) * case["hd"]
        return {"bytes": 4 * vals + 12 * case["rows"], "flops": 6 * vals}
    n, ctx = _lengths(case)
    pairs = keys = 0
    for x, c in zip(n, ctx):
        W = case["window"]
        first = max(0, c - W + 1) if W else 0
        keys += c + x - first
        pairs += sum(min(c + i + 1, W) if W else c + i + 1 for i in range(x))
    return {"bytes": 4 * sum(n) * case["hq"] * case["hd"] + 4 * keys * case["nkv"] * case["hd"], "flops": 4 * pairs * case["hq"] * case["hd"]}


def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "rope": _exact_rope, "attn": _exact_attn}[case["op"]](s)


def _exact_plan(s):
    """Request by request and page by page, as the definition reads."""
    n_new, ctx, have, valid = (s[k].tolist() for k in ("n_new", "ctx", "have", "valid"))
    table, free, (head, tail), P = s["table"].tolist(), s["free"].tolist(), s["range"].tolist(), s["P"]
    out = {k: [] for k in ("n_pages", "alloc_limit", "seq_lens", "row_req", "row_pos", "row_page", "row_slot")}
    out["cu_rows"] = [0]
    for r in range(len(n_new)):
        n = n_new[r] if valid[r] else 0
        owned = have[r]
        while n and owned * P < ctx[r] + n and owned < len(table[r]) and head < tail:
            table[r][owned] = free[head]
            owned, head = owned + 1, head + 1
        limit = min(owned * P, 1 << 30) if valid[r] else 0
        out["n_pages"].append(owned if valid[r] else 0)
        out["alloc_limit"].append(limit)
        out["seq_lens"].append(min(ctx[r] + n, limit) if valid[r] else 0)
        out["cu_rows"].append(out["cu_rows"][-1] + n)
        for p in range(ctx[r], ctx[r] + n):
            ok = p < limit and table[r][p // P] >= 0
            out["row_req"].append(r)
            out["row_pos"].append(p)
            out["row_page"].append(table[r][p // P] if ok else -1)
            out["row_slot"].append(p % P if ok else -1)
    for k in ("row_req", "row_pos", "row_page", "row_slot"):
        out[k] += [-1] * (s["rows"] - len(out[k]))
    out["free_head"], out["table"] = [head], table
    return {k: _ints(v) for k, v in out.items()}


def _exact_rope(s):
    spec, hq, nkv, hd = s["spec"], s["hq"], s["nkv"], s["hd"]
    rows = s["qkv"].double().unflatten(1, (hq + 2 * nkv, hd))
    d = spec["rot"]
    turns = []
    mag = 0.1 * math.log(spec["factor"]) + 1.0 if spec["scaling"] == "yarn" else 1.0
    for j in range(d // 2):
        f = math.pow(spec["theta"], -2.0 * j / d)
        if spec["scaling"] == "linear":
            f /= spec["factor"]
        elif spec["scaling"] == "yarn":
            edge = [d / 2 * math.log(spec["trained"] / (b * 2 * math.pi)) / math.log(spec["theta"]) for b in (spec["beta_fast"], spec["beta_slow"])]
            a, b = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), d - 1)
            share = min(1.0, max(0.0, (j - a) / max(b - a, 1e-3)))
            f = share * f / spec["factor"] + (1.0 - share) * f
        turns.append(f)
    z = torch.polar(torch.full((rows.shape[0], d // 2), mag, dtype=torch.float64, device=rows.device),
                    s["pos"].double()[:, None] * torch.tensor(turns, dtype=torch.float64, device=rows.device))[:, None, :]

    def turned(x, gamma):
        if gamma is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / hd + spec["eps"]) * gamma.double()
        x = x.clone()
        even, odd = (slice(0, d // 2), slice(d // 2, d)) if spec["layout"] == "half" else (slice(0, d, 2), slice(1, d, 2))
        y = torch.complex(x[..., even].contiguous(), x[..., odd].contiguous()) * z
        x[..., even], x[..., odd] = y.real, y.imag
        return x

    pool = s["pool"].double()
    k = turned(rows[:, hq:hq + nkv], s["gk"])
    for h in range(nkv):
        pool[0, s["page"].long(), 0, h, s["slot"].long()] = k[:, h]
        pool[0, s["page"].long(), 1, h, s["slot"].long()] = rows[:, hq + nkv + h]
    return turned(rows[:, :hq], s["gq"]), pool


def _exact_attn(s):
    """Request by request, KV head by KV head, over the gathered keys."""
    q, pool, P = s["q"], s["pool"][0], s["P"]
    N, hq, hd = q.shape
    G = hq // s["nkv"]
    out = torch.zeros((N, hq, hd), dtype=torch.float64, device=q.device)
    cu, ctx, kv = s["cu"].tolist(), s["ctx"].tolist(), s["kv"].tolist()
    for r in range(s["B"]):
        a, b = cu[r], cu[r + 1]
        pages = s["table"][r, : _pages(kv[r], P)].long()
        keys = torch.arange(kv[r], device=q.device)
        at = ctx[r] + torch.arange(b - a, device=q.device)[:, None]
        seen = (keys <= at) if not s["window"] else (keys <= at) & (at - keys < s["window"])
        for h in range(s["nkv"]):
            K = pool[pages, 0, h].reshape(-1, hd)[: kv[r]].double()
            V = pool[pages, 1, h].reshape(-1, hd)[: kv[r]].double()
            for e in range(h * G, h * G + G):
                x = torch.where(seen, q[a:b, e].double() @ K.T / math.sqrt(hd), -math.inf)
                if s["sinks"] is not None:
                    x = torch.cat([x, s["sinks"][e].double().expand(b - a, 1)], 1)
                out[a:b, e] = torch.softmax(x, 1)[:, : kv[r]] @ V
    return out
