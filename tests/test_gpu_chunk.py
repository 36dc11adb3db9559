"""GPU parity of the ragged-chunk calls (dflash_chunk_plan,
dflash_chunk_rope_store, dflash_chunk_attention) against the float64
definitions in oracle/chunk.py, at the sizes and masks where they can go wrong,
and of a run of the three together.

Tolerances.  Rounding to bf16 is off by at most 2^-8 of the value.  RoPE: one
rounding of each output, plus fp32 arithmetic: the angle (2^-24 of half a turn,
4e-7 with the magnitude), the norm's sum over at most 256 values and the
products, together below 1e-5 of the magnitudes the output is formed from.
Attention: the weights and the output are rounded to bf16 once each, and fp32
scores of size |s| are off by at most (hd + 2) 2^-24 |s|_1 and the exponential by 2^-22, so
with |s|_1 <= 100 below 128 * 2^-24 * 100 < 8e-4 relative of a weight and as
much again of the sum: in all 2^-8 |out| + (2^-8 + 2e-3) sum p|v|, which is at
most (2^-7 + 2e-3) sum p|v|."""
import numpy as np
import pytest

from oracle import chunk
from tests.gpu_helpers import bf16_f64, bits

pytestmark = pytest.mark.gpu

ATTN_TOL = 2.0 ** -7 + 2e-3


@pytest.fixture(scope="module")
def dl():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from context_kv_update_gb300 import build
    build.build()
    import context_kv_update_gb300 as dl
    dl.load()
    return dl


def geom(dl, *, hq=4, nkv=2, hd=64, P=16, M=8, NP=32, L=1, theta=1e6):
    return dl.make_geom(dict(kind="gqa", L=L, D_in=64, D=64, hq=hq, nkv=nkv, hd=hd, P=P, T=1,
                             max_pages=M, num_pool_pages=NP, rope_theta=theta, eps_h=1e-6,
                             eps_k=1e-6))


def dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def bf16(a):
    """float64 array -> (bf16 CUDA tensor, its values in float64)."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


# ------------------------------------------------------------------ plan

ROW_KEYS = ("row_req", "row_pos", "row_page", "row_slot")


def plan_outputs(dl, B, n_rows, fill=-77):
    import torch
    size = {"cu_rows": B + 1, "free_head": 1, **{k: n_rows for k in ROW_KEYS}}
    return {k: torch.full((size.get(k, B),), fill, dtype=torch.int32, device="cuda")
            for k in dl.CHUNK_OUTPUT_FIELDS}


def run_plan(dl, case, n_rows, P, NP, max_ctx=1 << 30):
    import torch
    B, M = case["table"].shape
    g = geom(dl, P=P, M=M, NP=NP)
    tbl = dev(case["table"])
    out = plan_outputs(dl, B, n_rows)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dl.dflash_chunk_plan(g, dev(case["n_new"]), dev(case["ctx"]), dev(case["have"]), tbl,
                         dev(case["free"]), dev(case["range"]),
                         None if case["valid"] is None else dev(case["valid"]), max_ctx, out, st)
    torch.cuda.synchronize()
    got = {k: v.cpu().numpy() for k, v in out.items()}
    got["block_table"] = tbl.cpu().numpy()
    got["flags"] = int(st.item())
    want = chunk.chunk_plan(case["n_new"], case["ctx"], case["have"], case["table"], case["free"],
                            case["range"], case["valid"], max_ctx, n_rows=n_rows, P=P, NP=NP)
    for k in want:
        np.testing.assert_array_equal(got[k], want[k], err_msg=k)
    return got


def plan_case(rng, B, P, most_new, most_ctx, *, dead=0.1, idle=0.2):
    n = rng.integers(1, most_new + 1, B) * (rng.random(B) >= idle)
    ctx = rng.integers(0, most_ctx + 1, B)
    have = -(-ctx // P)
    want = -(-(ctx + n) // P)
    M = int(max(want.max(), 1)) + 1
    new = int((want - have).sum())
    NP = int(have.sum()) + new + 5
    perm = rng.permutation(NP).astype(np.int32)
    table = np.full((B, M), -1, np.int32)
    at = 0
    for r in range(B):
        table[r, :have[r]] = perm[at:at + have[r]]
        at += have[r]
    i32 = lambda a: np.asarray(a, np.int32)  # noqa: E731
    return dict(n_new=i32(n), ctx=i32(ctx), have=i32(have), table=table,
                free=np.concatenate([perm[:2], perm[at:]]), range=i32([2, 2 + NP - at]),
                valid=(rng.random(B) >= dead).astype(np.uint8)), NP


@pytest.mark.parametrize("B,P,most_new,most_ctx,extra", [
    (1, 16, 1, 0, 0), (1, 64, 700, 33, 3), (3, 8, 5, 40, 0), (31, 16, 1, 500, 1),
    (33, 128, 90, 1000, 2), (257, 64, 40, 300, 0), (1025, 16, 3, 100, 64), (3000, 16, 2, 60, 0),
    (8192, 16, 1, 40, 5)])
def test_plan(dl, B, P, most_new, most_ctx, extra):
    rng = np.random.default_rng(B + P)
    case, NP = plan_case(rng, B, P, most_new, most_ctx)
    rows = int((case["n_new"] * (case["valid"] != 0)).sum()) + extra
    run_plan(dl, case, rows, P, NP)


def test_plan_without_requests_or_rows(dl):
    rng = np.random.default_rng(1)
    case, NP = plan_case(rng, 5, 16, 4, 50, idle=1.0)
    got = run_plan(dl, case, 0, 16, NP)
    assert got["free_head"][0] == 2
    case = dict(n_new=np.zeros(0, np.int32), ctx=np.zeros(0, np.int32), have=np.zeros(0, np.int32),
                table=np.zeros((0, 4), np.int32), free=np.zeros(0, np.int32),
                range=np.array([0, 0], np.int32), valid=None)
    run_plan(dl, case, 7, 16, 4)
    got = run_plan(dl, case, 0, 16, 4)   # neither
    assert got["cu_rows"][0] == 0 and got["free_head"][0] == 0


def test_plan_lengths_out_of_range(dl):
    """Bad lengths, an exhausted free list, a full table, bad pages: flagged,
    and everything else as defined."""
    rng = np.random.default_rng(2)
    case, NP = plan_case(rng, 40, 16, 30, 200, dead=0.0, idle=0.0)
    case["valid"] = None
    rows = int(case["n_new"].sum())
    bad = {k: v.copy() for k, v in case.items() if v is not None}
    bad["valid"] = None
    bad["n_new"][3] = -5
    bad["n_new"][7] = 2 ** 31 - 1      # more rows than there are: the rest gets none
    assert run_plan(dl, bad, rows, 16, NP)["flags"] & 128
    bad["n_new"] = case["n_new"].copy()
    bad["ctx"][5], bad["ctx"][6] = -1, 2 ** 31 - 1
    assert run_plan(dl, bad, rows, 16, NP)["flags"] & 2
    bad["ctx"] = case["ctx"].copy()
    bad["range"] = np.array([2, 9], np.int32)
    assert run_plan(dl, bad, rows, 16, NP)["flags"] & 256
    bad["range"] = np.array([-4, 2 ** 31 - 1], np.int32)
    run_plan(dl, bad, rows, 16, NP)
    bad["range"] = case["range"]
    bad["table"] = case["table"][:, :4].copy()
    bad["have"] = np.minimum(case["have"], 4)
    assert run_plan(dl, bad, rows, 16, NP)["flags"] & 256
    bad["have"] = case["have"].copy()
    bad["have"][9], bad["have"][10] = -3, 1000
    bad["table"] = case["table"].copy()
    bad["table"][11, :] = NP
    bad["free"] = case["free"].copy()
    bad["free"][4] = NP + 7
    assert run_plan(dl, bad, rows, 16, NP)["flags"] & 8
    run_plan(dl, case, rows, 16, NP, max_ctx=100)


# ------------------------------------------------------------------ RoPE + store


def rope_spec(dl, layout, rot, scaling="plain", factor=1.0, trained=64):
    return dl.RopeSpec(layout=dl.ROPE_HALF if layout == "half" else dl.ROPE_PAIRS, rot_dim=rot,
                       scaling={"plain": dl.ROPE_PLAIN, "linear": dl.ROPE_LINEAR,
                                "yarn": dl.ROPE_YARN}[scaling],
                       trained_ctx=trained, factor=factor, beta_fast=32.0, beta_slow=1.0,
                       magnitude=0.0)


def check_rope(dl, *, rows, hq, nkv, hd, rot, layout, scaling="plain", factor=1.0, gamma=True,
               P=16, L=2, layer=1, top=4000, pad=0, in_place=False, packed=True, seed=0):
    """One call with unplaced, absent and out-of-pool rows among the others."""
    import torch
    rng = np.random.default_rng(seed)
    NP = -(-rows // P) + 3
    g = geom(dl, hq=hq, nkv=nkv, hd=hd, P=P, NP=NP, L=L, theta=1e4)
    W = (hq + 2 * nkv) * hd
    qkv, x = bf16(rng.standard_normal((rows, W + pad)))
    x = x[:, :W].reshape(rows, hq + 2 * nkv, hd)
    pos = rng.integers(0, top + 1, rows).astype(np.int32)
    place = rng.permutation(NP * P)[:rows]
    page, slot = (place // P).astype(np.int32), (place % P).astype(np.int32)
    bad = 0
    if rows > 4:
        pos[1] = -1                     # past the last request
        page[2], slot[2] = -1, -1       # not placed
        page[3] = NP                    # outside the pool
        bad = 8
    gq, gqv = bf16(1 + 0.1 * rng.standard_normal(hd))
    gk, gkv = bf16(1 + 0.1 * rng.standard_normal(hd))
    pool, poolv = bf16(rng.standard_normal((L, NP, 2, nkv, P, hd)))
    q, k, v = qkv[:, :hq * hd], qkv[:, hq * hd:(hq + nkv) * hd], qkv[:, (hq + nkv) * hd:W]
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    q_out = q if in_place else torch.full((rows, hq, hd), 7.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dl.dflash_chunk_rope_store(g, layer, rope_spec(dl, layout, rot, scaling, factor), q, k, v,
                               dev(pos), dev(page), dev(slot), q_out, pool,
                               gamma_q=gq if gamma else None, gamma_k=gk if gamma else None,
                               dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == bad
    ang, mag = chunk.rope_angles(rot, 1e4, scaling, factor, 64)
    kw = dict(layout=layout, rot=rot, angles=ang, mag=mag)
    yq, sq = chunk.turn(x[:, :hq], gqv if gamma else None, pos, 1e-6, **kw)
    yk, sk = chunk.turn(x[:, hq:hq + nkv], gkv if gamma else None, pos, 1e-6, **kw)
    got = bf16_f64(bits(q_out)).reshape(rows, hq, hd)
    here = pos >= 0
    tol = 2.0 ** -8 * np.abs(yq) + 1e-5 * sq
    assert np.all(np.abs(got - yq)[here] <= tol[here])
    left = x[:, :hq] if in_place else np.full_like(yq, 7.0)
    np.testing.assert_array_equal(got[~here], left[~here])
    want, slack = poolv.copy(), np.zeros_like(poolv)
    for t in range(rows):
        if here[t] and 0 <= page[t] < NP:
            want[layer, page[t], 0, :, slot[t]] = yk[t]
            slack[layer, page[t], 0, :, slot[t]] = (2.0 ** -8 * np.abs(yk) + 1e-5 * sk)[t]
            want[layer, page[t], 1, :, slot[t]] = x[t, hq + nkv:]
    got = bf16_f64(bits(pool)).reshape(want.shape)
    assert np.all(np.abs(got - want) <= slack)


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("hd,rot", [(128, 128), (64, 64), (64, 32), (128, 24), (64, 24), (96, 80),
                                    (64, 2), (128, 12), (64, 6), (256, 256), (8, 8), (256, 2),
                                    (24, 16)])
def test_rope_widths(dl, layout, hd, rot):
    check_rope(dl, rows=37, hq=3, nkv=1, hd=hd, rot=rot, layout=layout, pad=8)


@pytest.mark.parametrize("scaling,factor", [("plain", 1.0), ("linear", 4.0), ("yarn", 8.0),
                                            ("yarn", 1.0)])
@pytest.mark.parametrize("gamma", [True, False])
def test_rope_scaling(dl, scaling, factor, gamma):
    check_rope(dl, rows=50, hq=8, nkv=2, hd=128, rot=128, layout="half", scaling=scaling,
               factor=factor, gamma=gamma, top=1 << 20)


@pytest.mark.parametrize("rows,hq,nkv,in_place,packed", [
    (1, 1, 1, False, True), (1, 32, 8, True, False), (2, 7, 7, True, True), (300, 40, 8, True, True),
    (65, 32, 4, False, False), (1000, 6, 2, False, True)])
def test_rope_rows_and_heads(dl, rows, hq, nkv, in_place, packed):
    check_rope(dl, rows=rows, hq=hq, nkv=nkv, hd=64, rot=64, layout="half", in_place=in_place,
               packed=packed, P=64, L=1, layer=0)
    check_rope(dl, rows=rows, hq=hq, nkv=nkv, hd=128, rot=64, layout="pairs", in_place=in_place,
               packed=packed, P=8)


def test_rope_far_positions(dl):
    """The angle of a position near 2^31 keeps its low bits."""
    check_rope(dl, rows=40, hq=2, nkv=1, hd=128, rot=128, layout="half", top=2 ** 31 - 2, seed=5)


def test_rope_queries_or_keys_alone(dl):
    import torch
    rng = np.random.default_rng(8)
    g = geom(dl, hq=4, nkv=2, hd=64, P=16, NP=4)
    sp = rope_spec(dl, "half", 64)
    q, _ = bf16(rng.standard_normal((9, 256)))
    k, _ = bf16(rng.standard_normal((9, 128)))
    v, _ = bf16(rng.standard_normal((9, 128)))
    pos, page, slot = (dev(a.astype(np.int32)) for a in (np.arange(9) + 5, np.arange(9) % 2,
                                                         np.arange(9)))
    pool, _ = bf16(rng.standard_normal((1, 4, 2, 2, 16, 64)))
    both, out = pool.clone(), torch.zeros_like(q)
    dl.dflash_chunk_rope_store(g, 0, sp, q, k, v, pos, page, slot, out, both)
    alone, keys = torch.zeros_like(q), pool.clone()
    dl.dflash_chunk_rope_store(g, 0, sp, q, None, None, pos, None, None, alone, None)
    dl.dflash_chunk_rope_store(g, 0, sp, None, k, v, pos, page, slot, None, keys)
    torch.cuda.synchronize()
    assert torch.equal(out, alone) and torch.equal(both, keys) and not torch.equal(keys, pool)


# ------------------------------------------------------------------ attention


def attn_problem(rng, n, ctx, *, hq, nkv, hd, P, extra_pages=2, L=1, layer=0, stale=np.nan):
    """A paged cache whose unused slots hold `stale`."""
    kv = [c + x for c, x in zip(ctx, n)]
    have = [-(-k // P) for k in kv]
    NP, M = sum(have) + extra_pages, max(have + [1]) + 1
    perm = rng.permutation(NP).astype(np.int32)
    table = np.full((len(n), M), -1, np.int32)
    pool = np.full((L, NP, 2, nkv, P, hd), stale)
    at = 0
    for r, h in enumerate(have):
        table[r, :h] = perm[at:at + h]
        at += h
        for j in range(kv[r]):
            pool[layer, table[r, j // P], :, :, j % P] = rng.standard_normal((2, nkv, hd))
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    q = rng.standard_normal((int(cu[-1]), hq, hd))
    return dict(cu=cu, ctx=np.array(ctx, np.int32), kv=np.array(kv, np.int32), table=table,
                pool=pool, q=q, NP=NP, M=M)


def run_attn(dl, pb, *, hq, nkv, hd, P, window=0, sinks=None, causal=True, S=0, L=1, layer=0,
             scale=None, pad_rows=0, stride_pad=0, flags=0, check=True, stream=None):
    import torch
    g = geom(dl, hq=hq, nkv=nkv, hd=hd, P=P, M=pb["M"], NP=pb["NP"], L=L)
    B, N = len(pb["ctx"]), pb["q"].shape[0]
    qt, qv = bf16(np.concatenate([pb["q"], np.ones((pad_rows, hq, hd))]))
    pool, poolv = bf16(pb["pool"])
    if stride_pad:  # rows of a wider tensor
        wide = torch.zeros((N + pad_rows, hq * hd + stride_pad), dtype=torch.bfloat16, device="cuda")
        wide[:, :hq * hd] = qt.flatten(1)
        qt = wide[:, :hq * hd].unflatten(1, (hq, hd))
    full = torch.full((N + pad_rows, hq * hd + stride_pad), 7.0, dtype=torch.bfloat16, device="cuda")
    out = full[:, :hq * hd].unflatten(1, (hq, hd))
    need = dl.dflash_chunk_attention_workspace_bytes(g, B, N + pad_rows, S)
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")  # NaN everywhere
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dl.dflash_chunk_attention(
        g, layer, qt, pool, dev(pb["table"]), dev(pb["cu"]), dev(pb["ctx"]), dev(pb["kv"]), out,
        ws, window=window, sinks=None if sinks is None else dev(sinks.astype(np.float32)),
        scale=scale, mask_mode=dl.MASK_CAUSAL_TAIL if causal else dl.MASK_BLOCK_BIDIR,
        num_segments=S, dev_status=st, stream=stream)
    torch.cuda.synchronize()
    assert int(st.item()) == flags
    got = bf16_f64(bits(out)).reshape(N + pad_rows, hq, hd)
    if check:
        want, size = chunk.chunk_attention(
            qv, poolv[layer], pb["table"], pb["cu"], pb["ctx"], pb["kv"], window=window,
            scale=hd ** -0.5 if scale is None else scale,
            sinks=None if sinks is None else sinks.astype(np.float32).astype(np.float64),
            causal=causal)
        rows = ~np.isnan(want).any((1, 2))
        err = np.abs(got - want)[rows] - ATTN_TOL * size[rows]
        assert np.all(err <= 1e-30), f"worst excess {np.nanmax(err)}"
        np.testing.assert_array_equal(got[~rows], 7.0)  # rows of no request
        if stride_pad:
            assert torch.all(full[:, hq * hd:] == 7.0)
    return got


SHAPES = {
    "one": ([1], [0]), "one_of_many": ([1], [700]), "tile_edge": ([1, 1, 1], [126, 127, 128]),
    "short": ([1, 4, 2], [100, 0, 31]), "chunk": ([130], [0]), "chunk_on_ctx": ([67], [300]),
    "mixed": ([1, 150, 1, 33, 0, 1], [400, 0, 5, 129, 50, 255]), "empty": ([0, 3, 0], [7, 0, 0]),
}


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("hq,nkv,hd,P", [(4, 2, 64, 16), (8, 2, 128, 64)])
def test_attention_lengths(dl, shape, hq, nkv, hd, P):
    rng = np.random.default_rng(11)
    n, ctx = SHAPES[shape]
    pb = attn_problem(rng, n, ctx, hq=hq, nkv=nkv, hd=hd, P=P)
    run_attn(dl, pb, hq=hq, nkv=nkv, hd=hd, P=P)


@pytest.mark.parametrize("window", [1, 5, 128, 1000])
@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_masks(dl, window, sinks, causal):
    rng = np.random.default_rng(12)
    hq, nkv, hd, P = 6, 2, 64, 8
    pb = attn_problem(rng, [1, 90, 3], [300, 45, 0], hq=hq, nkv=nkv, hd=hd, P=P)
    run_attn(dl, pb, hq=hq, nkv=nkv, hd=hd, P=P, window=window, causal=causal,
             sinks=rng.standard_normal(hq) if sinks else None)


@pytest.mark.parametrize("hq,nkv,hd,P", [(1, 1, 64, 128), (5, 1, 128, 256), (7, 7, 64, 32),
                                         (48, 1, 128, 16), (40, 8, 64, 64), (160, 1, 64, 16)])
def test_attention_heads_and_pages(dl, hq, nkv, hd, P):
    rng = np.random.default_rng(13)
    pb = attn_problem(rng, [3, 40], [200, 17], hq=hq, nkv=nkv, hd=hd, P=P, L=2, layer=1)
    run_attn(dl, pb, hq=hq, nkv=nkv, hd=hd, P=P, L=2, layer=1, sinks=rng.standard_normal(hq))


@pytest.mark.parametrize("S", [1, 2, 3, 9, 40])
def test_attention_segments(dl, S):
    """Any number of segments, more than there are key tiles among them."""
    rng = np.random.default_rng(14)
    hq, nkv, hd, P = 4, 1, 128, 64
    pb = attn_problem(rng, [1, 2, 0, 50], [1200, 63, 3, 700], hq=hq, nkv=nkv, hd=hd, P=P)
    for sinks in (None, rng.standard_normal(hq)):
        run_attn(dl, pb, hq=hq, nkv=nkv, hd=hd, P=P, S=S, sinks=sinks, pad_rows=2)
        run_attn(dl, pb, hq=hq, nkv=nkv, hd=hd, P=P, S=S, sinks=sinks, window=200)


@pytest.mark.parametrize("S", [0, 1, 4])
def test_attention_rows_without_keys(dl, S):
    """A cache cut off before the chunk (no free pages): the window leaves the
    last rows nothing, and they are 0; a request without any key too."""
    rng = np.random.default_rng(15)
    hq, nkv, hd, P = 4, 2, 64, 16
    pb = attn_problem(rng, [20, 30, 4], [40, 100, 0], hq=hq, nkv=nkv, hd=hd, P=P)
    pb["kv"] = np.array([60, 104, 0], np.int32)
    for sinks in (None, rng.standard_normal(hq)):
        got = run_attn(dl, pb, hq=hq, nkv=nkv, hd=hd, P=P, window=8, S=S, sinks=sinks, pad_rows=3)
        assert np.all(got[20 + 11:54] == 0)  # rows at 111.. see keys 104.. only


def test_attention_extreme_scores(dl):
    """Scores far apart, a sink far above and far below them, and masked keys
    that would win."""
    rng = np.random.default_rng(16)
    hq, nkv, hd, P = 4, 2, 64, 16
    pb = attn_problem(rng, [70], [500], hq=hq, nkv=nkv, hd=hd, P=P, stale=np.inf)
    pb["q"] *= 6.0
    pb["pool"][:, :, 0] = np.where(np.isfinite(pb["pool"][:, :, 0]), pb["pool"][:, :, 0] * 2, np.inf)
    # |s|_1 here is up to 64 * 6 * 3 * 2 * 3 / 8, 900: 64 * 2^-24 * 900 = 3.5e-3 of a weight
    for sink in (-1e30, 0.0, 90.0):
        sinks = np.full(hq, sink)
        got = run_attn(dl, pb, hq=hq, nkv=nkv, hd=hd, P=P, sinks=sinks, check=False)
        qv, poolv = bf16(pb["q"])[1], bf16(pb["pool"])[1]
        want, size = chunk.chunk_attention(qv, poolv[0], pb["table"], pb["cu"], pb["ctx"], pb["kv"],
                                           scale=hd ** -0.5, sinks=sinks)
        assert np.all(np.abs(got - want) <= (ATTN_TOL + 7e-3) * size + 1e-30)


def test_attention_bad_pages_and_lengths(dl):
    """Pages outside the pool are masked and flagged; where no row sees them
    they are neither; lengths out of range are clamped or give no rows."""
    rng = np.random.default_rng(17)
    hq, nkv, hd, P = 4, 2, 64, 16
    kw = dict(hq=hq, nkv=nkv, hd=hd, P=P)
    pb = attn_problem(rng, [5, 140], [200, 150], **kw)
    pb["table"][0, 3], pb["table"][1, 2] = -1, pb["NP"]
    run_attn(dl, pb, **kw, flags=8)
    run_attn(dl, pb, **kw, flags=8, S=3)
    pb = attn_problem(rng, [5, 9], [200, 150], **kw)
    pb["table"][0, :10], pb["table"][1, :3] = -1, 10 ** 9   # before every window
    run_attn(dl, pb, **kw, window=30)
    pb = attn_problem(rng, [5, 9], [200, 150], **kw)
    pb["kv"][0] = -3
    run_attn(dl, pb, **kw, flags=16)
    pb["kv"][0] = pb["M"] * P + 1   # clamped; the causal rows see no further than before
    run_attn(dl, pb, **kw, flags=16)
    pb = attn_problem(rng, [5, 9], [200, 150], **kw)
    pb["ctx"][0] = -1
    got = run_attn(dl, pb, **kw, flags=128, check=False)
    assert np.all(got[:5] == 7.0) and not np.any(got[5:] == 7.0)
    pb["ctx"][0], pb["cu"] = 200, np.array([0, 5, 15], np.int32)   # past the last row
    got = run_attn(dl, pb, **kw, flags=128, check=False)
    assert np.all(got[5:] == 7.0) and not np.any(got[:5] == 7.0)


def test_attention_padded_and_strided_rows(dl):
    rng = np.random.default_rng(18)
    kw = dict(hq=8, nkv=2, hd=128, P=64)
    pb = attn_problem(rng, [1, 35], [90, 64], **kw)
    a = run_attn(dl, pb, **kw, pad_rows=5, stride_pad=64)
    b = run_attn(dl, pb, **kw)
    np.testing.assert_array_equal(a[:36], b)


def test_attention_is_repeatable_and_on_another_stream(dl):
    import torch
    rng = np.random.default_rng(19)
    kw = dict(hq=32, nkv=8, hd=128, P=64)
    pb = attn_problem(rng, [1, 1, 80], [900, 30, 64], **kw)
    a = run_attn(dl, pb, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = run_attn(dl, pb, **kw, check=False, stream=s)
    np.testing.assert_array_equal(a, b)


def test_attention_long_cache(dl):
    """Pool offsets past 2^31 elements: the requests' pages sit at both ends of
    a large pool.  The definition is evaluated on the pages in use."""
    import torch
    rng = np.random.default_rng(20)
    hq, nkv, hd, P = 4, 2, 128, 64
    NP = (1 << 31) // (2 * nkv * P * hd) + 40      # > 2^31 values
    pb = attn_problem(rng, [3, 20], [170, 500], hq=hq, nkv=nkv, hd=hd, P=P, extra_pages=0)
    small = pb["pool"].shape[1]
    far = np.where(np.arange(small) % 2 == 0, np.arange(small), NP - 1 - np.arange(small))
    g = geom(dl, hq=hq, nkv=nkv, hd=hd, P=P, M=pb["M"], NP=NP)
    pool = torch.empty((1, NP, 2, nkv, P, hd), dtype=torch.bfloat16, device="cuda")
    pool[0, dev(far)] = bf16(pb["pool"][0])[0]
    table = np.where(pb["table"] >= 0, far[pb["table"]], -1).astype(np.int32)
    qt, _ = bf16(pb["q"])
    out = torch.empty_like(qt)
    ws = torch.empty(max(16, dl.dflash_chunk_attention_workspace_bytes(g, 2, 23)),
                     dtype=torch.uint8, device="cuda")
    dl.dflash_chunk_attention(g, 0, qt, pool, dev(table), dev(pb["cu"]), dev(pb["ctx"]),
                              dev(pb["kv"]), out, ws)
    near = run_attn(dl, pb, hq=hq, nkv=nkv, hd=hd, P=P)
    np.testing.assert_array_equal(bf16_f64(bits(out)).reshape(near.shape), near)


# Work tiles of 256 rows (the mean request fills more than one tile of 128), with a
# remainder of each kind, and requests of a few rows among them.
WIDE = {"full_and_rest": ([130, 3], [0, 700]), "one_over": ([65], [500]),
        "half": ([96, 64], [40, 0]), "long": ([200, 1, 0, 70], [129, 1000, 9, 3])}


@pytest.mark.parametrize("shape", WIDE)
@pytest.mark.parametrize("window,sinks,causal", [(0, False, True), (150, True, True),
                                                 (1, False, True), (40, True, False)])
def test_attention_wide_tiles(dl, shape, window, sinks, causal):
    rng = np.random.default_rng(23)
    n, ctx = WIDE[shape]
    kw = dict(hq=4, nkv=1, hd=128, P=16)
    pb = attn_problem(rng, n, ctx, **kw)
    run_attn(dl, pb, **kw, window=window, causal=causal, pad_rows=1,
             sinks=rng.standard_normal(4) if sinks else None)


@pytest.mark.parametrize("hq,nkv,rows", [(4, 1, 20), (16, 2, 9), (16, 1, 5), (128, 1, 1),
                                         (3, 3, 70), (64, 1, 3), (256, 1, 1)])
def test_attention_fewer_rows_than_a_box(dl, hq, nkv, rows):
    """More than 64 rows of a KV head's group, of fewer tokens than 128 rows hold."""
    rng = np.random.default_rng(34)
    kw = dict(hq=hq, nkv=nkv, hd=128, P=32)
    pb = attn_problem(rng, [rows], [150], **kw)
    run_attn(dl, pb, **kw, S=1)
    run_attn(dl, pb, **kw, S=2, stride_pad=64, window=70)


@pytest.mark.parametrize("S", [2, 5])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_wide_tiles_in_segments(dl, S, hd):
    rng = np.random.default_rng(24)
    kw = dict(hq=8, nkv=1, hd=hd, P=64)
    pb = attn_problem(rng, [70, 1, 5], [600, 300, 0], **kw)
    for sinks in (None, rng.standard_normal(8)):
        run_attn(dl, pb, **kw, S=S, sinks=sinks, pad_rows=2)
        run_attn(dl, pb, **kw, S=S, sinks=sinks, window=130)


def test_attention_wide_tiles_bad_pages_and_cut_cache(dl):
    rng = np.random.default_rng(25)
    kw = dict(hq=8, nkv=2, hd=64, P=16)
    pb = attn_problem(rng, [90, 40], [200, 150], **kw)
    pb["table"][0, 3], pb["table"][0, 15], pb["table"][1, 9] = -1, pb["NP"] + 5, -7
    run_attn(dl, pb, **kw, flags=8)
    run_attn(dl, pb, **kw, flags=8, S=3)
    pb = attn_problem(rng, [90, 40], [200, 150], **kw)
    pb["kv"] = np.array([250, 0], np.int32)
    for S in (1, 3):
        got = run_attn(dl, pb, **kw, window=20, S=S)
        assert np.all(got[69:] == 0)   # rows at 269 on see keys 250 on; the second request none


def test_attention_many_requests(dl):
    """More requests than a warp searches at once, some empty, tiles of each."""
    rng = np.random.default_rng(26)
    kw = dict(hq=2, nkv=1, hd=64, P=16)
    n = [int(x) for x in rng.integers(0, 4, 1100)]
    n[500] = 150
    pb = attn_problem(rng, n, [int(x) for x in rng.integers(0, 30, 1100)], **kw)
    run_attn(dl, pb, **kw)
    run_attn(dl, pb, **kw, S=2)


@pytest.mark.parametrize("hq,nkv,hd,P,window,S", [
    (16, 8, 128, 64, 0, 1), (15, 5, 64, 16, 37, 1), (8, 8, 128, 32, 200, 1), (24, 8, 64, 16, 0, 3),
    (64, 8, 128, 64, 0, 2)])
def test_attention_blocks_with_many_works(dl, hq, nkv, hd, P, window, S):
    """More work tiles than the GPU runs at once, so a block goes from one to the
    next: one and two row tiles, rows without keys, pages outside the pool and
    empty requests after one another, key spans from none to several rounds of the ring."""
    rng = np.random.default_rng(29)
    kw = dict(hq=hq, nkv=nkv, hd=hd, P=P)
    n = [int(x) for x in rng.choice([0, 1, 2, 5, 33, 65, 129, 140, 200], 34)]
    ctx = [int(x) for x in rng.integers(0, 900, 34)]
    pb = attn_problem(rng, n, ctx, **kw)
    pb["kv"][[5, 11]] = 0
    pb["kv"][17] //= 2
    live = [r for r in range(34) if n[r] > 0 and pb["kv"][r] == n[r] + ctx[r]]
    # the last key's page: causal rows before it and windows that end there see it
    bad = [r for r in live if n[r] > 1][3:6]
    for r in bad:
        pb["table"][r, (pb["kv"][r] - 1) // P] = pb["NP"] + 9
    sinks = rng.standard_normal(hq)
    got = [run_attn(dl, pb, **kw, window=window, S=S, sinks=sinks, pad_rows=1, flags=8,
                    check=check) for check in (True, False)]
    np.testing.assert_array_equal(got[0], got[1])


@pytest.mark.parametrize("nkv,rows,ctx", [(40, 600, 900), (20, 1300, 3000), (9, 4000, 300),
                                          (30, 1500, 500)])
@pytest.mark.parametrize("window,causal", [(0, True), (90, True), (0, False)])
def test_attention_uneven_segments(dl, nkv, rows, ctx, window, causal):
    """Two segments of one request whose work tiles leave SMs over: most keys in the
    first, the rest (or none of a short span) in the second.  Three of the heads are
    compared."""
    rng = np.random.default_rng(31)
    kw = dict(hq=nkv, nkv=nkv, hd=64, P=64)
    pb = attn_problem(rng, [rows], [ctx], **kw)
    got = run_attn(dl, pb, **kw, window=window, causal=causal, S=2, check=False)
    heads = [0, nkv // 2, nkv - 1]
    pool, q = bf16(pb["pool"][0][:, :, heads])[1], bf16(pb["q"][:, heads])[1]
    want, size = chunk.chunk_attention(q, pool, pb["table"], pb["cu"], pb["ctx"], pb["kv"],
                                       window=window, scale=0.125, sinks=None, causal=causal)
    assert np.all(np.abs(got[:, heads] - want) <= ATTN_TOL * size)
    np.testing.assert_array_equal(
        got, run_attn(dl, pb, **kw, window=window, causal=causal, S=2, check=False))


@pytest.mark.parametrize("B", [2, 33, 65, 256, 257])
def test_attention_bad_lengths_among_many_works(dl, B):
    """Lengths and offsets out of range where blocks take the requests' work tiles in
    the order of their cost (up to 256) and in their own: flagged, the other requests as ever."""
    rng = np.random.default_rng(32)
    kw = dict(hq=48, nkv=24, hd=64, P=16)
    n = [int(x) for x in rng.integers(1, 4, B)]
    n[0] = 400 if B == 2 else 70
    ctx = [int(x) for x in rng.integers(0, 300, B)]
    ctx[0] = 20
    pb = attn_problem(rng, n, ctx, **kw)
    right = run_attn(dl, pb, **kw, S=1, check=B < 256)
    last = int(pb["cu"][B - 1])
    bad = dict(pb, ctx=pb["ctx"].copy(), kv=pb["kv"].copy(), cu=pb["cu"].copy())
    bad["ctx"][B - 1] = -1
    got = run_attn(dl, bad, **kw, S=1, flags=128, check=False)
    np.testing.assert_array_equal(got[:last], right[:last])
    assert np.all(got[last:] == 7.0)
    bad["ctx"][B - 1], bad["cu"][B] = ctx[B - 1], bad["cu"][B] + 5   # past the last row
    got = run_attn(dl, bad, **kw, S=1, flags=128, check=False)
    np.testing.assert_array_equal(got[:last], right[:last])
    assert np.all(got[last:] == 7.0)
    bad["cu"][B] -= 5
    bad["kv"][0] = -7
    got = run_attn(dl, bad, **kw, S=1, flags=16, check=False)
    np.testing.assert_array_equal(got[n[0]:], right[n[0]:])
    assert np.all(got[:n[0]] == 0.0)
    # offsets that go back: flagged, nothing outside the rows is written
    bad = dict(pb, cu=pb["cu"].copy())
    bad["cu"][1:B] = bad["cu"][1:B][::-1] if B > 2 else pb["cu"][B] + 3
    run_attn(dl, bad, **kw, S=1, flags=128, check=False)


def test_attention_calls_at_once(dl):
    """Two calls on two streams with a workspace each, many times over, give what
    each gives alone."""
    import torch
    rng = np.random.default_rng(27)
    kw = dict(hq=8, nkv=2, hd=128, P=64)
    pbs = [attn_problem(rng, [1, 2], [900, 1500], **kw), attn_problem(rng, [40, 3], [300, 64], **kw)]
    want = [run_attn(dl, pb, **kw, S=4) for pb in pbs]
    streams, outs, keep = [torch.cuda.Stream() for _ in pbs], [], []
    for s, pb in zip(streams, pbs):
        g = geom(dl, P=64, hq=8, nkv=2, hd=128, M=pb["M"], NP=pb["NP"])
        n = pb["q"].shape[0]
        a = [bf16(pb["q"])[0], bf16(pb["pool"])[0], *(dev(pb[k]) for k in ("table", "cu", "ctx", "kv"))]
        ws = torch.empty(dl.dflash_chunk_attention_workspace_bytes(g, 2, n, 4), dtype=torch.uint8,
                         device="cuda")
        outs.append([torch.empty_like(a[0]) for _ in range(20)])
        keep.append((g, a, ws))
    torch.cuda.synchronize()
    for i in range(20):
        for s, o, (g, a, ws) in zip(streams, outs, keep):
            dl.dflash_chunk_attention(g, 0, *a, o[i], ws, num_segments=4, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for x in o:
            np.testing.assert_array_equal(bf16_f64(bits(x)).reshape(w.shape), w)


@pytest.mark.parametrize("B,S", [(40, 1), (40, 2), (100, 1), (300, 1)])
def test_attention_many_works_captured_and_at_once(dl, B, S):
    """Calls with more work tiles than the GPU runs at once, in two graphs replayed on
    two streams at the same time, give what each gives alone."""
    import torch
    rng = np.random.default_rng(33)
    kw = dict(hq=16, nkv=8, hd=128, P=32)
    pbs = [attn_problem(rng, [int(x) for x in rng.choice([1, 2, 90, 150], B)],
                        [int(x) for x in rng.integers(0, 500, B)], **kw) for _ in range(2)]
    want = [run_attn(dl, pb, **kw, S=S, check=False) for pb in pbs]
    graphs, outs, streams, keep = [], [], [torch.cuda.Stream() for _ in pbs], []
    for pb, s in zip(pbs, streams):
        g = geom(dl, M=pb["M"], NP=pb["NP"], **kw)
        a = [bf16(pb["q"])[0], bf16(pb["pool"])[0],
             *(dev(pb[k]) for k in ("table", "cu", "ctx", "kv"))]
        need = dl.dflash_chunk_attention_workspace_bytes(g, B, pb["q"].shape[0], S)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        o = torch.empty_like(a[0])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for _ in range(3):
                dl.dflash_chunk_attention(g, 0, *a, o, ws, num_segments=S, stream=s)
        graphs.append(graph)
        outs.append(o)
        keep.append((a, ws))
    for _ in range(5):
        for o in outs:
            o.fill_(7.0)
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            np.testing.assert_array_equal(bf16_f64(bits(o)).reshape(w.shape), w)


def test_a_workspace_serves_captured_graphs_in_turn(dl):
    """Two graphs captured on one workspace and replayed one after the other: each
    leaves nothing there that the other needs."""
    import torch
    rng = np.random.default_rng(28)
    kw = dict(hq=8, nkv=2, hd=64, P=16)
    pbs = [attn_problem(rng, [1, 1], [500, 800], **kw), attn_problem(rng, [2], [300], **kw)]
    want = [run_attn(dl, pb, **kw, S=3) for pb in pbs]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    graphs, outs, keep = [], [], []
    for pb in pbs:
        g = geom(dl, P=16, hq=8, nkv=2, hd=64, M=pb["M"], NP=pb["NP"])
        a = [bf16(pb["q"])[0], bf16(pb["pool"])[0], *(dev(pb[k]) for k in ("table", "cu", "ctx", "kv"))]
        o = torch.empty_like(a[0])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            dl.dflash_chunk_attention(g, 0, *a, o, ws, num_segments=3)
        graphs.append(graph)
        outs.append(o)
        keep.append((g, a))
    for _ in range(3):
        for graph, o, w in zip(graphs, outs, want):
            o.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            np.testing.assert_array_equal(bf16_f64(bits(o)).reshape(w.shape), w)


@pytest.mark.parametrize("rows", [1, 90])
def test_attention_unloaded_tile_times_out_cleanly(dl, rows):
    """The bounded waits: the producer leaves one key tile unloaded, the kernel
    winds down and sets its status, and the next call is right."""
    rng = np.random.default_rng(22)
    kw = dict(hq=4, nkv=2, hd=64, P=16)
    pb = attn_problem(rng, [rows], [1000], **kw)
    dl.dflash_test_attention_skip_tile(2)
    try:
        run_attn(dl, pb, **kw, S=1, check=False, flags=dl._lib.DEV_WAIT_TIMEOUT)
    finally:
        dl.dflash_test_attention_skip_tile(-1)
    run_attn(dl, pb, **kw, S=1)


def test_attention_unloaded_tile_among_many_works(dl):
    """A wait that runs out in blocks that hold, or have claimed, other works: the
    call ends, sets its status, and the next one is right."""
    rng = np.random.default_rng(30)
    kw = dict(hq=8, nkv=8, hd=64, P=16)
    n = [1] * 30
    pb = attn_problem(rng, n, [100] * 29 + [900], **kw)
    dl.dflash_test_attention_skip_tile(5)
    try:
        run_attn(dl, pb, **kw, S=1, check=False, flags=dl._lib.DEV_WAIT_TIMEOUT)
    finally:
        dl.dflash_test_attention_skip_tile(-1)
    run_attn(dl, pb, **kw, S=1)


# ------------------------------------------------------------------ together


def test_chunks_of_a_prompt_in_a_captured_graph(dl):
    """Plan, RoPE + store and attention of one layer, captured once and replayed
    for the pieces of two prompts and single tokens between them, against the
    definition over all tokens at once."""
    import torch
    rng = np.random.default_rng(21)
    hq, nkv, hd, P, M, R = 4, 2, 64, 16, 12, 96
    W = (hq + 2 * nkv) * hd
    pieces = [[70, 1], [3, 80], [1, 1], [25, 0], [1, 40]]
    total = np.sum(pieces, 0)
    NP = 2 * M + 3
    g = geom(dl, hq=hq, nkv=nkv, hd=hd, P=P, M=M, NP=NP, theta=1e4)
    sp = rope_spec(dl, "half", hd, "yarn", 4.0)
    gq, gqv = bf16(1 + 0.1 * rng.standard_normal(hd))
    gk, gkv = bf16(1 + 0.1 * rng.standard_normal(hd))
    tokens = [bf16(rng.standard_normal((t, W)))[0] for t in total]
    pool, _ = bf16(np.full((1, NP, 2, nkv, P, hd), np.nan))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    tbl = torch.full((2, M), -1, dtype=torch.int32, device="cuda")
    n_new, ctx, have, rng_t = i32([0, 0]), i32([0, 0]), i32([0, 0]), i32([0, NP])
    free = dev(rng.permutation(NP).astype(np.int32))
    out = plan_outputs(dl, 2, R)
    qkv = torch.zeros((R, W), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((R, hq, hd), dtype=torch.bfloat16, device="cuda")
    o = torch.zeros_like(q)
    ws = torch.empty(max(16, dl.dflash_chunk_attention_workspace_bytes(g, 2, R)),
                     dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def layer():
        dl.dflash_chunk_plan(g, n_new, ctx, have, tbl, free, rng_t, None, M * P, out, st)
        x, k, v = qkv.split((hq * hd, nkv * hd, nkv * hd), 1)
        dl.dflash_chunk_rope_store(g, 0, sp, x, k, v, out["row_pos"], out["row_page"],
                                   out["row_slot"], q, pool, gamma_q=gq, gamma_k=gk, dev_status=st)
        dl.dflash_chunk_attention(g, 0, q, pool, tbl, out["cu_rows"], ctx, out["seq_lens"], o, ws,
                                  dev_status=st)

    layer()  # no rows: one-time set-up
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        layer()
    got, turned = [[], []], [[], []]
    at = [0, 0]
    for piece in pieces:
        n_new.copy_(i32(piece))
        x = torch.cat([tokens[r][at[r]:at[r] + piece[r]] for r in range(2)])
        qkv[:x.shape[0]] = x
        o.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        cu = out["cu_rows"].tolist()
        for r in range(2):
            got[r].append(bf16_f64(bits(o[cu[r]:cu[r + 1]])).reshape(-1, hq, hd))
            turned[r].append(bf16_f64(bits(q[cu[r]:cu[r + 1]])).reshape(-1, hq, hd))
            at[r] += piece[r]
        assert torch.all(o[cu[2]:] == 7.0)
        ctx.copy_(out["seq_lens"])
        have.copy_(out["n_pages"])
        rng_t[0:1].copy_(out["free_head"])
    assert int(st.item()) == 0 and at == total.tolist()
    # the rotated rows against the definition, the attention against the
    # definition over the rows as the device stored them
    ang, mag = chunk.rope_angles(hd, 1e4, "yarn", 4.0, 64)
    kw = dict(layout="half", rot=hd, angles=ang, mag=mag)
    table, rows = tbl.cpu().numpy(), bf16_f64(bits(pool)).reshape(NP, 2, nkv, P, hd)
    for r in range(2):
        x = tokens[r].double().cpu().numpy().reshape(-1, hq + 2 * nkv, hd)
        n = len(x)
        pos = np.arange(n)
        qr = np.concatenate(turned[r])
        kr = rows[table[r, pos // P], 0, :, pos % P]
        for have_rows, raw, g64 in ((qr, x[:, :hq], gqv), (kr, x[:, hq:hq + nkv], gkv)):
            y, size = chunk.turn(raw, g64, pos, 1e-6, **kw)
            assert np.all(np.abs(have_rows - y) <= 2.0 ** -8 * np.abs(y) + 1e-5 * size)
        np.testing.assert_array_equal(rows[table[r, pos // P], 1, :, pos % P], x[:, hq + nkv:])
        want, size = chunk.chunk_attention(qr, rows, table[r:r + 1], [0, n], [0], [n],
                                           scale=hd ** -0.5)
        assert np.all(np.abs(np.concatenate(got[r]) - want) <= ATTN_TOL * size)
