"""What a paged cache held in 8 bits costs in one layer: written, read back, attended to.

A cell of the cache is an e4m3 code; ``block`` tokens of a page share, head by head, K and
V apart, one power of two as their scale (an e8m0 byte: 2^(byte - 127)).  Three operators:

* ``store``: a chunk's q, k and v rows as the projection leaves them: per-head RMSNorm
  where the model has one, rotary positions, keys and values quantised into their slots.
  A block that a row begins is scaled by its rows; one that held tokens before keeps its
  scale or, where a row needs a larger one, has what it holds shifted to that.  What the
  blocks that were written then hold is read back, and that is what a pass returns;
* ``read``: rows of the cache as bf16, by page and slot (a prefix handed to another
  worker, or to a layer that keeps its cache in 16 bits);
* ``attn``: attention of a chunk's rows over the cache, causal or not, with an optional
  sliding window and per-head sinks.

``run`` is their plain form; with ``own`` true it makes the library's calls.  Geometries are
those of this repository's workloads (32 query heads over 8 or 2 KV heads of 128, a tiny
4-over-2 of 64, pages of 64 or 16) and generic ones.
"""
import math
import random

import torch

own = False

GOLD = 0.6180339887498949
TOP = 448.0  # the largest e4m3 value
LEAST, MOST = -124, 120  # exponents of the scales that are written


def listed():
    q8 = {"hq": 32, "nkv": 8, "hd": 128, "page": 64}
    head = {"gamma": True, "rot": 128, "layout": "half", "scaling": "plain", "factor": 1.0}
    return [
        # one new token in each of 64 running requests, in blocks that hold tokens already
        dict(q8, name="store_single_64", op="store", B=64, rows=64, singles=64, ctx=8192, block=16, **head),
        # a draft's 16 rows of one request at a long context: latency
        dict(q8, name="store_draft_16", op="store", B=1, rows=16, singles=0, ctx=32768, block=64, **head),
        # a fresh prompt's piece
        dict(q8, name="store_prompt_8192", op="store", B=1, rows=8192, singles=0, ctx=0, block=64, **head),
        # odd pieces of three prompts, half of a 64-wide head rotated in neighbouring pairs, scaled eightfold past its trained context
        {"name": "store_yarn_5003", "op": "store", "B": 3, "rows": 5003, "singles": 0, "ctx": 65536, "hq": 24, "nkv": 4, "hd": 64, "page": 16,
         "block": 16, "gamma": False, "rot": 32, "layout": "pairs", "scaling": "yarn", "factor": 8.0},
        # a short prefix read back
        {"name": "read_301", "op": "read", "rows": 301, "nkv": 2, "hd": 64, "page": 16, "block": 16},
        # a long one
        {"name": "read_32768", "op": "read", "rows": 32768, "nkv": 8, "hd": 128, "page": 64, "block": 32},
        # the smallest call: three short requests of a few tokens on the tiny geometry
        {"name": "attn_tiny", "op": "attn", "B": 3, "rows": 7, "singles": 1, "ctx": 100, "hq": 4, "nkv": 2, "hd": 64, "page": 16, "block": 16,
         "window": 0, "sinks": True, "causal": True},
        # a single new token of one request at a long context
        dict(q8, name="attn_single_32k", op="attn", B=1, rows=1, singles=1, ctx=32768, block=64, window=0, sinks=False, causal=True),
        # 64 running requests with one to a few thousand keys each
        dict(q8, name="attn_decode_64", op="attn", B=64, rows=64, singles=64, ctx=8192, block=16, window=0, sinks=False, causal=True),
        # drafts of 16 rows of eight requests, whose rows see one another
        dict(q8, name="attn_drafts_8x16", op="attn", B=8, rows=128, singles=0, ctx=16384, block=32, window=0, sinks=False, causal=False),
        # a mixed batch: twelve single tokens beside odd pieces of prompts, sliding window and sinks
        {"name": "attn_mixed_window", "op": "attn", "B": 16, "rows": 2311, "singles": 12, "ctx": 8192, "hq": 32, "nkv": 2, "hd": 128, "page": 64,
         "block": 64, "window": 1024, "sinks": True, "causal": True},
        # a prompt's piece far into a long context
        dict(q8, name="attn_piece_1024_at_32k", op="attn", B=1, rows=1024, singles=0, ctx=32768, block=64, window=0, sinks=False, causal=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "read", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    c = {"op": op, "nkv": rng.choice([1, 2, 4, 8]), "hd": rng.choice([64, 128]), "page": page,
         "block": rng.choice([b for b in (16, 32, 64) if b <= page])}
    if op == "read":
        return dict(c, rows=_log(rng, 1, 32768))
    c["hq"] = c["nkv"] * rng.choice([1, 2, 4, 5, 8][: 5 if c["nkv"] < 8 else 3])
    if op == "store":
        c["B"] = _log(rng, 1, 64)
        c["singles"] = rng.choice([0, c["B"], rng.randint(0, c["B"])])
        c["rows"] = c["singles"] + (0 if c["singles"] == c["B"] else _log(rng, c["B"] - c["singles"], 8192 - c["singles"]))
        return dict(c, ctx=_log(rng, 1, 65536), gamma=rng.random() < 0.5, rot=rng.choice([c["hd"], c["hd"] // 2, c["hd"] // 4, 24]),
                    layout=rng.choice(["half", "pairs"]), scaling=rng.choice(["plain", "linear", "yarn"]), factor=rng.choice([2.0, 4.0, 8.0]))
    c.update(window=rng.choice([0, 0, _log(rng, 32, 4096)]), sinks=rng.random() < 0.5, causal=rng.random() < 0.75)
    kind = rng.choice(["decode", "drafts", "mixed", "prompt"])
    if kind == "decode":
        c["B"] = c["rows"] = c["singles"] = _log(rng, 1, 64)
        c["ctx"] = _log(rng, 16, 32768 if c["B"] <= 16 else 8192)
    elif kind == "drafts":
        c["B"], c["singles"] = _log(rng, 1, 16), 0
        c["rows"], c["ctx"] = c["B"] * rng.randint(2, 16), _log(rng, 16, 16384)
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
    """(new tokens, tokens before) of each request, from the case alone."""
    B, singles = case["B"], case["singles"]
    n = [1] * singles
    many = B - singles
    if many and case["rows"] - singles == many * ((case["rows"] - singles) // many) and (case["rows"] - singles) // many <= 16:
        n += [(case["rows"] - singles) // many] * many  # drafts, all as long
    elif many:
        w = [0.25 + 1.5 * ((i + 1) * GOLD % 1.0) for i in range(many)]
        left = case["rows"] - singles - many  # each has one row at least
        part = [int(left * x / sum(w)) for x in w]
        part[0] += left - sum(part)
        n += [1 + x for x in part]
    ctx = [int(case["ctx"] * (1.0 if i == 0 else 0.125 + 0.875 * (i * GOLD % 1.0))) for i in range(B)]
    return n, ctx


def _pages(tokens, page):
    return -(-tokens // page)


def _held(n, ctx, block):
    """The positions that the blocks hold which a chunk writes, request by request."""
    return [range(c // block * block, c + x) for x, c in zip(n, ctx)]


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    return {"store": _prepare_store, "read": _prepare_read, "attn": _prepare_attn}[case["op"]](case, seed)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype=torch.bfloat16, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std + mean).to(dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cache(g, case, pages):
    """Codes and scales as the cache of a running server holds them: blocks of different size,
    the largest value of each between half of what its scale can hold and all of it."""
    nkv, P, hd, block = case["nkv"], case["page"], case["hd"], case["block"]
    size = torch.randint(-2, 3, (1, pages, 2, nkv, P // block), generator=g, device="cuda").float().exp2()
    x = torch.randn((1, pages, 2, nkv, P // block, block, hd), generator=g, device="cuda") * size[..., None, None]
    e = _exponent(x.abs().amax((-1, -2)))
    codes = (x * (-e.float()).exp2()[..., None, None]).to(torch.float8_e4m3fn).flatten(4, 5)
    return codes.contiguous(), (e + 127).to(torch.uint8).contiguous()


def _library(case, max_pages, pool_pages):
    """The library and its geometry, where the library's calls are made."""
    if not own:
        return None, None
    import context_kv_update_gb300 as dl
    dl.load()
    hq, hd = case.get("hq", case["nkv"]), case["hd"]
    return dl, dl.make_geom(dict(kind="gqa", L=1, D_in=hq * hd, D=hq * hd, hq=hq, nkv=case["nkv"], hd=hd, P=case["page"], T=1, max_pages=max_pages,
                                 num_pool_pages=pool_pages, rope_theta=1e6, eps_h=1e-6, eps_k=1e-6))


def _requests(case, seed, g):
    """New tokens, tokens before, the page table and the pages of the pool."""
    n, ctx = _lengths(case)
    order = list(range(case["B"]))
    random.Random(seed).shuffle(order)
    n, ctx = [n[i] for i in order], [ctx[i] for i in order]
    have = [_pages(c + x, case["page"]) for c, x in zip(ctx, n)]
    width, pool_pages = max(have) + 1, sum(have) + 4
    perm = torch.randperm(pool_pages, generator=g, device="cuda").to(torch.int32)
    col, have_t = torch.arange(width, device="cuda")[None, :], _ints(have)
    start = (have_t.cumsum(0) - have_t)[:, None]
    table = torch.where(col < have_t[:, None], perm[(start + col).clamp(max=pool_pages - 1)], -1).to(torch.int32).contiguous()
    return n, ctx, table, pool_pages


def _spec(case):
    return {"rot": case["rot"], "layout": case["layout"], "scaling": case["scaling"], "factor": case["factor"], "trained": 8192,
            "beta_fast": 32.0, "beta_slow": 1.0, "theta": 1e6, "eps": 1e-6}


def _prepare_store(case, seed):
    g = _gen(seed)
    n, ctx, table, pool_pages = _requests(case, seed, g)
    rows, hq, nkv, hd, P = case["rows"], case["hq"], case["nkv"], case["hd"], case["page"]

    def places(spans):  # position, page and slot of each row
        req = torch.tensor([r for r, s in enumerate(spans) for _ in s], device="cuda")
        pos = torch.tensor([p for s in spans for p in s], device="cuda")
        return pos.to(torch.int32), table[req, pos // P].contiguous(), (pos % P).to(torch.int32)

    held = _held(n, ctx, case["block"])
    s = {"op": "store", "spec": _spec(case), "gq": None, "gk": None, "hq": hq, "nkv": nkv, "hd": hd, "P": P, "block": case["block"],
         "q_out": torch.zeros((rows, hq, hd), dtype=torch.bfloat16, device="cuda")}
    s["pos"], s["page"], s["slot"] = places([range(c, c + x) for x, c in zip(n, ctx)])
    _, s["held_page"], s["held_slot"] = places(held)
    s["k_held"], s["v_held"] = (torch.zeros((sum(map(len, held)), nkv, hd), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    # rows of different size: some raise the scale of the block that they join
    size = torch.randint(-2, 3, (rows, 1), generator=g, device="cuda").float().exp2()
    s["qkv"] = (torch.randn((rows, (hq + 2 * nkv) * hd), generator=g, device="cuda") * size).to(torch.bfloat16)
    s["codes"], s["scales"] = _cache(g, case, pool_pages)
    if case["gamma"]:
        s["gq"], s["gk"] = _normal(g, (hd,), std=0.02, mean=1.0), _normal(g, (hd,), std=0.02, mean=1.0)
    s["dl"], s["geom"] = _library(case, table.shape[1], pool_pages)
    if own:
        dl, sp = s["dl"], s["spec"]
        s["rope"] = dl.RopeSpec(layout=dl.ROPE_HALF if sp["layout"] == "half" else dl.ROPE_PAIRS, rot_dim=sp["rot"],
                                scaling={"plain": dl.ROPE_PLAIN, "linear": dl.ROPE_LINEAR, "yarn": dl.ROPE_YARN}[sp["scaling"]],
                                trained_ctx=sp["trained"], factor=sp["factor"], beta_fast=sp["beta_fast"], beta_slow=sp["beta_slow"], magnitude=0.0)
    return s


def _prepare_read(case, seed):
    g = _gen(seed)
    rows, nkv, hd, P = case["rows"], case["nkv"], case["hd"], case["page"]
    pages = _pages(rows, P) + 2
    pos = torch.arange(rows, device="cuda") + 1
    perm = torch.randperm(pages, generator=g, device="cuda")
    s = {"op": "read", "page": perm[pos // P].to(torch.int32), "slot": (pos % P).to(torch.int32), "block": case["block"]}
    s["codes"], s["scales"] = _cache(g, case, pages)
    s["k"], s["v"] = (torch.zeros((rows, nkv, hd), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    s["dl"], s["geom"] = _library(case, pages, pages)
    return s


def _prepare_attn(case, seed):
    g = _gen(seed)
    n, ctx, table, pool_pages = _requests(case, seed, g)
    hq, nkv, hd = case["hq"], case["nkv"], case["hd"]
    kv = [c + x for c, x in zip(ctx, n)]
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    s = {"op": "attn", "q": _normal(g, (cu[-1], hq, hd)), "table": table, "cu": _ints(cu), "ctx": _ints(ctx), "kv": _ints(kv),
         "sinks": _normal(g, (hq,), torch.float32) if case["sinks"] else None, "window": case["window"], "causal": case["causal"],
         "most_rows": max(n), "most_keys": max(kv), "B": case["B"], "nkv": nkv, "P": case["page"], "block": case["block"],
         "out": torch.zeros((cu[-1], hq, hd), dtype=torch.bfloat16, device="cuda")}
    s["codes"], s["scales"] = _cache(g, case, pool_pages)
    s["dl"], s["geom"] = _library(case, table.shape[1], pool_pages)
    if own:
        need = s["dl"].dflash_chunk_attention8_workspace_bytes(s["geom"], case["B"], cu[-1])
        s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    if own:
        return _OWN[s["op"]](s)
    return _PLAIN[s["op"]](s)


def _own_store(s):
    hq, nkv, hd, dl = s["hq"], s["nkv"], s["hd"], s["dl"]
    q, k, v = s["qkv"].split((hq * hd, nkv * hd, nkv * hd), dim=1)
    dl.dflash_chunk_rope_store8(s["geom"], 0, s["rope"], q, k, v, s["pos"], s["page"], s["slot"], s["q_out"], s["codes"], s["scales"], s["block"],
                                gamma_q=s["gq"], gamma_k=s["gk"])
    dl.dflash_chunk_read8(s["geom"], 0, s["codes"], s["scales"], s["block"], s["held_page"], s["held_slot"], s["k_held"], s["v_held"])
    return s["q_out"], s["k_held"], s["v_held"]


def _own_read(s):
    s["dl"].dflash_chunk_read8(s["geom"], 0, s["codes"], s["scales"], s["block"], s["page"], s["slot"], s["k"], s["v"])
    return s["k"], s["v"]


def _own_attn(s):
    dl = s["dl"]
    dl.dflash_chunk_attention8(s["geom"], 0, s["q"], s["codes"], s["scales"], s["block"], s["table"], s["cu"], s["ctx"], s["kv"], s["out"], s["ws"],
                               window=s["window"], sinks=s["sinks"], mask_mode=dl.MASK_CAUSAL_TAIL if s["causal"] else dl.MASK_BLOCK_BIDIR)
    return s["out"]


_OWN = {"store": _own_store, "read": _own_read, "attn": _own_attn}


def _exponent(amax):
    """The smallest power of two that brings amax to 448 or below, of those that are written."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m from 0.5
    return torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), LEAST).clamp(LEAST, MOST)


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


def _turn(x, gamma, pos, spec):
    """RMSNorm where gamma is given, then the rotation, in 32 bits; x [rows, heads, hd]."""
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
    return torch.cat([turned, x[..., d:]], -1)


def _values(codes, scales, block, page, slot, kv):
    """Rows [n, nkv, hd] of the cache in 32 bits."""
    return codes[0, page, kv, :, slot].float() * (scales[0, page, kv, :, slot // block].float() - 127.0).exp2()[..., None]


def _plain_store(s):
    hq, nkv, hd, P, block = s["hq"], s["nkv"], s["hd"], s["P"], s["block"]
    q, k, v = (x.unflatten(1, (-1, hd)) for x in s["qkv"].split((hq * hd, nkv * hd, nkv * hd), dim=1))
    x = torch.stack([_turn(k, s["gk"], s["pos"], s["spec"]), v.float()], 1)  # [rows, 2, nkv, hd]
    page, slot = s["page"].long(), s["slot"].long()
    # the blocks that get rows, each once, and what they need
    at, row_at = torch.unique(page * (P // block) + slot // block, return_inverse=True)
    most = torch.zeros((at.shape[0], 2, nkv), device=x.device).index_reduce_(0, row_at, x.abs().amax(-1), "amax")
    begun = torch.zeros(at.shape[0], device=x.device).index_reduce_(0, row_at, (slot % block == 0).float(), "amax") > 0
    in_page, b = at // (P // block), at % (P // block)
    before = s["scales"][0, in_page, :, :, b].int() - 127
    e = _exponent(most)
    e = torch.where(begun[:, None, None], e, torch.maximum(before, e))
    # what they held, shifted to the scale that they have now; a block begun anew is left as it is
    cells = s["codes"][0].unflatten(3, (P // block, block))
    old = cells[in_page, :, :, b]
    shift = torch.where(begun[:, None, None], 0, before - e).float().exp2()[..., None, None]
    cells[in_page, :, :, b] = (old.float() * shift).to(torch.float8_e4m3fn)
    s["scales"][0, in_page, :, :, b] = (e + 127).to(torch.uint8)
    s["codes"][0, page, :, :, slot] = (x * (-e[row_at].float()).exp2()[..., None]).to(torch.float8_e4m3fn)
    held = [_values(s["codes"], s["scales"], block, s["held_page"].long(), s["held_slot"].long(), i).to(torch.bfloat16) for i in (0, 1)]
    return _turn(q, s["gq"], s["pos"], s["spec"]).to(torch.bfloat16), held[0], held[1]


def _plain_read(s):
    k, v = (_values(s["codes"], s["scales"], s["block"], s["page"].long(), s["slot"].long(), i).to(torch.bfloat16) for i in (0, 1))
    return k, v


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
    flat, slot = page.clamp(min=0).flatten(), (j % P)[None, :].expand(B, -1).flatten()
    K, V = (_values(s["codes"], s["scales"], s["block"], flat, slot, e).unflatten(0, (B, -1)) for e in (0, 1))
    K, V = K.permute(0, 2, 3, 1), torch.where(held[:, :, None, None], V, 0.0).transpose(1, 2)
    x = q[row.clamp(max=N - 1)].float().unflatten(2, (nkv, G)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    score = (x @ K).unflatten(2, (G, -1)) * (1.0 / math.sqrt(hd))
    p = s["ctx"].long()[:, None] + i
    seen = held[:, None, :].expand(-1, i.shape[0], -1)
    if s["causal"]:
        seen = seen & (j <= p[:, :, None])
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


_PLAIN = {"store": _plain_store, "read": _plain_read, "attn": _plain_attn}


# ------------------------------------------------------------------ work and the definition in 64 bits


def work(case):
    cell = 2 * case["nkv"] * case["hd"]  # bytes that a token's codes take
    if case["op"] == "read":
        return {"bytes": case["rows"] * (3 * cell + 8) + 2 * case["nkv"] * _pages(case["rows"], case["block"]), "flops": case["rows"] * cell}
    n, ctx = _lengths(case)
    if case["op"] == "store":
        held = sum(map(len, _held(n, ctx, case["block"])))
        vals = case["rows"] * (case["hq"] + 2 * case["nkv"]) * case["hd"]
        back = held * (3 * cell + 8)  # the codes read, their values and the places of the rows
        return {"bytes": 2 * vals + 2 * case["rows"] * case["hq"] * case["hd"] + case["rows"] * (cell + 12) + back, "flops": 6 * vals + held * cell}
    pairs = keys = 0
    for x, c in zip(n, ctx):
        W = case["window"]
        first = max(0, c - W + 1) if W else 0
        keys += c + x - first
        for i in range(x):
            pairs += (c + i + 1 if case["causal"] else c + x) - (max(0, c + i - W + 1) if W else 0)
    return {"bytes": 4 * sum(n) * case["hq"] * case["hd"] + keys * (cell + 2 * case["nkv"] / case["block"]), "flops": 4 * pairs * case["hq"] * case["hd"]}


def exact(case, seed):
    s = prepare(case, seed)
    return {"store": _exact_store, "read": _exact_read, "attn": _exact_attn}[case["op"]](s)


def _exact_code(x):
    """x rounded to the nearest e4m3 value (three bits after the first one, steps of 2^-9 at the least)."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step  # to even where two are as near


def _exact_turn(x, gamma, pos, spec):
    hd, d = x.shape[-1], spec["rot"]
    x = x.double()
    if gamma is not None:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / hd + spec["eps"]) * gamma.double()
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
    z = torch.polar(torch.full((x.shape[0], d // 2), mag, dtype=torch.float64, device=x.device),
                    pos.double()[:, None] * torch.tensor(turns, dtype=torch.float64, device=x.device))[:, None, :]
    x = x.clone()
    even, odd = (slice(0, d // 2), slice(d // 2, d)) if spec["layout"] == "half" else (slice(0, d, 2), slice(1, d, 2))
    y = torch.complex(x[..., even].contiguous(), x[..., odd].contiguous()) * z
    x[..., even], x[..., odd] = y.real, y.imag
    return x


def _exact_store(s):
    """Block by block, in the order of the rows, the values themselves held in place of codes."""
    hq, nkv, hd, P, block = s["hq"], s["nkv"], s["hd"], s["P"], s["block"]
    rows = s["qkv"].unflatten(1, (hq + 2 * nkv, hd))
    new = torch.stack([_exact_turn(rows[:, hq:hq + nkv], s["gk"], s["pos"], s["spec"]), rows[:, hq + nkv:].double()])
    e_all = s["scales"][0].double() - 127
    cells = s["codes"][0].double() * torch.exp2(e_all).repeat_interleave(block, -1)[..., None]
    page, slot = s["page"].tolist(), s["slot"].tolist()
    t = 0
    while t < len(page):
        end = t + 1
        while end < len(page) and page[end] == page[t] and slot[end] // block == slot[t] // block:
            end += 1
        p, b, a = page[t], slot[t] // block, slot[t]
        most = new[:, t:end].abs().amax((1, 3))
        need = torch.ceil(torch.log2(most / TOP)).clamp(LEAST, MOST)
        if a % block:
            need = torch.maximum(need, e_all[p, :, :, b])
            step = torch.exp2(need)[..., None, None]
            cells[p, :, :, b * block:a] = _exact_code(cells[p, :, :, b * block:a] / step) * step
        step = torch.exp2(need)[..., None, None]
        cells[p, :, :, a:a + end - t] = _exact_code(new[:, t:end].transpose(1, 2) / step) * step
        t = end
    at, of = s["held_page"].long(), s["held_slot"].long()
    return _exact_turn(rows[:, :hq], s["gq"], s["pos"], s["spec"]), cells[at, 0, :, of], cells[at, 1, :, of]


def _exact_read(s):
    cells = s["codes"][0].double()
    for i in range(cells.shape[3]):
        cells[:, :, :, i] *= torch.exp2(s["scales"][0, :, :, :, i // s["block"]].double() - 127)[..., None]
    at, of = s["page"].long(), s["slot"].long()
    return cells[at, 0, :, of], cells[at, 1, :, of]


def _exact_attn(s):
    """Request by request, KV head by KV head, over the gathered keys."""
    q, P = s["q"], s["P"]
    N, hq, hd = q.shape
    G = hq // s["nkv"]
    out = torch.zeros((N, hq, hd), dtype=torch.float64, device=q.device)
    cu, ctx, kv = s["cu"].tolist(), s["ctx"].tolist(), s["kv"].tolist()
    for r in range(s["B"]):
        a, b = cu[r], cu[r + 1]
        pages = s["table"][r, : _pages(kv[r], P)].long()
        keys = torch.arange(kv[r], device=q.device)
        at = ctx[r] + torch.arange(b - a, device=q.device)[:, None]
        seen = keys <= (at if s["causal"] else torch.full_like(at, kv[r]))
        if s["window"]:
            seen = seen & (at - keys < s["window"])
        for h in range(s["nkv"]):
            K, V = (torch.ldexp(s["codes"][0, pages, e, h].double(), (s["scales"][0, pages, e, h].int() - 127).repeat_interleave(s["block"], -1)[..., None])
                    .reshape(-1, hd)[: kv[r]] for e in (0, 1))
            for e in range(h * G, h * G + G):
                x = torch.where(seen, q[a:b, e].double() @ K.T / math.sqrt(hd), -math.inf)
                if s["sinks"] is not None:
                    x = torch.cat([x, s["sinks"][e].double().expand(b - a, 1)], 1)
                out[a:b, e] = torch.softmax(x, 1)[:, : kv[r]] @ V
    return out
