"""CPU definitions of the ragged-chunk calls (plan, RoPE + paged store,
attention), in Python integers and numpy float64, request by request.  Test
infrastructure like the rest of this package: no code is shared with the CUDA
path."""
import math

import numpy as np


def chunk_plan(n_new, ctx_len, n_pages, table, free_pages, free_range, valid, max_ctx, *, n_rows,
               P, NP):
    """Outputs of dflash_chunk_plan as a dict of int32 arrays, the table after
    the call under "block_table", the status bits under "flags"."""
    BAD_CTX, BAD_PAGE, BAD_ROWS, NO_PAGES = 2, 8, 128, 256
    table = np.array(table, np.int64)
    B, M = table.shape
    nf = len(free_pages)
    head = min(max(int(free_range[0]), 0), nf)
    tail = min(max(int(free_range[1]), head), nf)
    flags, used = 0, 0
    out = {k: np.zeros(B, np.int64) for k in ("n_pages", "alloc_limit", "seq_lens")}
    rows = {k: np.full(n_rows, -1, np.int64) for k in ("row_req", "row_pos", "row_page",
                                                       "row_slot")}
    cu = [0]
    for r in range(B):
        n, c, have = int(n_new[r]), int(ctx_len[r]), int(n_pages[r])
        live = valid is None or valid[r] != 0
        if live:
            flags |= BAD_ROWS if n < 0 else 0
            flags |= BAD_PAGE if not 0 <= have <= M else 0
            if c < 0 or c > 2 ** 31 - 1 - n_rows - 1:
                flags |= BAD_CTX
                live = False
        have = min(max(have, 0), M)
        ask = max(n, 0) if live else 0
        if cu[r] + ask > n_rows:
            flags |= BAD_ROWS
        n = min(ask, n_rows - cu[r])
        cu.append(cu[r] + n)
        now = have
        if n > 0:
            want = -(-(c + n) // P)
            if want > M:
                flags |= NO_PAGES
            while now < min(want, M):
                if head + used >= tail:
                    flags |= NO_PAGES
                    break
                pg = int(free_pages[head + used])
                used += 1
                if not 0 <= pg < NP:
                    flags |= BAD_PAGE
                    pg = -1
                table[r, now] = pg
                now += 1
        if live:
            out["n_pages"][r] = now
            out["alloc_limit"][r] = min(now * P, max_ctx)
            out["seq_lens"][r] = min(c + n, out["alloc_limit"][r])
        for i in range(n):
            t, p = cu[r] + i, c + i
            rows["row_req"][t], rows["row_pos"][t] = r, p
            if p < out["alloc_limit"][r]:
                pg = table[r, p // P]
                if 0 <= pg < NP:
                    rows["row_page"][t], rows["row_slot"][t] = pg, p % P
                else:
                    flags |= BAD_PAGE
    out.update(rows)
    out["cu_rows"] = np.array(cu)
    out["free_head"] = np.array([head + used])
    out["block_table"] = table
    out = {k: v.astype(np.int32) for k, v in out.items()}
    out["flags"] = flags
    return out


def rope_angles(rot, theta, scaling="plain", factor=1.0, trained_ctx=1, beta_fast=32.0,
                beta_slow=1.0, magnitude=0.0):
    """(radians per position of each pair, factor on cos and sin)."""
    f = np.array([theta ** (-2.0 * j / rot) for j in range(rot // 2)])
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        def index(beta):  # of the pair that turns beta times over trained_ctx
            return rot * math.log(trained_ctx / (2 * math.pi * beta)) / (2 * math.log(theta))
        j0 = max(0.0, math.floor(index(beta_fast)))
        j1 = min(rot - 1.0, math.ceil(index(beta_slow)))
        u = np.clip((np.arange(rot // 2) - j0) / max(j1 - j0, 1e-3), 0.0, 1.0)
        return f * (1 - u + u / factor), (magnitude if magnitude > 0
                                          else 0.1 * math.log(factor) + 1.0)
    return f, 1.0


def turn(x, gamma, pos, eps, *, layout, rot, angles, mag):
    """x float64 [rows, heads, hd] -> normed (gamma given) and rotated; second
    result: sum of the magnitudes each output is formed from."""
    x = np.array(x, np.float64)
    if gamma is not None:
        x = x * gamma / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    a = np.asarray(pos, np.float64)[:, None] * angles[None, :]
    cos, sin = (mag * np.cos(a))[:, None, :], (mag * np.sin(a))[:, None, :]
    i, j = ((np.arange(rot // 2), np.arange(rot // 2) + rot // 2) if layout == "half"
            else (np.arange(0, rot, 2), np.arange(1, rot, 2)))
    y, size = x.copy(), np.abs(x)
    y[..., i] = x[..., i] * cos - x[..., j] * sin
    y[..., j] = x[..., j] * cos + x[..., i] * sin
    size[..., i] = size[..., j] = mag * (np.abs(x[..., i]) + np.abs(x[..., j]))
    return y, size


def chunk_attention(q, pool, table, cu, ctx, kv_len, *, scale, window=0, sinks=None, causal=True):
    """q float64 [n_rows, hq, hd]; pool float64 [NP, 2, nkv, P, hd] (one layer).
    Returns (out, weight): weight[t, h, d] = sum_j p_j |v_jd| / sum, the size of
    what each output is formed from; rows of no request are NaN."""
    N, hq, hd = q.shape
    NP, _, nkv, P, _ = pool.shape
    G = hq // nkv
    out = np.full(q.shape, np.nan)
    size = np.full(q.shape, np.nan)
    M = table.shape[1]
    for r in range(len(ctx)):
        kv = min(max(int(kv_len[r]), 0), M * P)
        pages = [int(table[r, j // P]) for j in range(kv)]
        ok = np.array([0 <= pg < NP for pg in pages], bool)
        at = [(pg if o else 0, j % P) for j, (pg, o) in enumerate(zip(pages, ok))]
        pg = np.array([x[0] for x in at], np.int64)
        sl = np.array([x[1] for x in at], np.int64)
        j = np.arange(kv)
        for i in range(int(cu[r + 1]) - int(cu[r])):
            t, p = int(cu[r]) + i, int(ctx[r]) + i
            seen = ok & (j <= p if causal else True)
            if window > 0:
                seen &= j > p - window
            w = np.nonzero(seen)[0]
            for h in range(hq):
                s = scale * (pool[pg[w], 0, h // G, sl[w]] @ q[t, h])
                m = max(s.max() if len(w) else -np.inf,
                        sinks[h] if sinks is not None else -np.inf)
                if len(w) == 0:
                    out[t, h] = size[t, h] = 0.0
                    continue
                e = np.exp(s - m)
                den = e.sum() + (np.exp(sinks[h] - m) if sinks is not None else 0.0)
                v = pool[pg[w], 1, h // G, sl[w]]
                out[t, h] = e @ v / den
                size[t, h] = e @ np.abs(v) / den
    return out, size
