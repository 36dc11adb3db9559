"""GPU parity of the chunk calls over a cache held in 8 bits (dflash_chunk_rope_store8,
dflash_chunk_read8, dflash_chunk_attention8) against the definitions in oracle/chunk8.py and
oracle/chunk.py, at the sizes and masks where they can go wrong, and of a run of them together.

Tolerances.  What is stored without norm and rotation (v always) is exact: codes and scales are
compared bit by bit.  Normed and turned keys carry fp32 arithmetic, below 1e-5 of the
magnitudes that each is formed from (tests/test_gpu_chunk.py), so a block's largest value may
fall on the other side of a power of two: its exponent is that of the largest value less or
more 1e-5 of them, and a code is off by half a step of e4m3 at most, 2^-4 |x| or 2^(e - 10), with
1e-5 of the magnitudes beside it.  Reading back is exact.  Attention: the values are
bf16 numbers exactly, so the 16-bit call's bound holds, (2^-7 + 2e-3) sum p|v|."""
import numpy as np
import pytest

from oracle import chunk, chunk8
from tests.gpu_helpers import bf16_f64, bits
from tests.test_gpu_chunk import (ATTN_TOL, SHAPES, WIDE, attn_problem, bf16, dev, dl,  # noqa: F401
                                  geom, plan_outputs, rope_spec)

pytestmark = pytest.mark.gpu


def code_bits(t):
    import torch
    return t.view(torch.uint8).cpu().numpy()


# ------------------------------------------------------------------ store


def spans(rng, n, ctx, P, extra=3):
    """Places of n[r] rows from ctx[r] on of each request, on pages of their own."""
    pos = np.concatenate([np.arange(c, c + x) for x, c in zip(n, ctx)]).astype(np.int32)
    need = [-(-(c + x) // P) for x, c in zip(n, ctx)]
    NP = sum(need) + extra
    perm = rng.permutation(NP)
    first = np.concatenate([[0], np.cumsum(need)])
    req = np.repeat(np.arange(len(n)), n)
    page = perm[first[req] + pos // P].astype(np.int32)
    return pos, page, (pos % P).astype(np.int32), NP


def check_store(dl, *, n, ctx, hq, nkv, hd, P, block, rot, layout="half", scaling="plain",  # noqa: F811
                factor=1.0, gamma=True, L=2, layer=1, pad=0, in_place=False, seed=0, size=None,
                edit=None, flags=0, q=True, f8=False):
    """One call into a cache that is in use.  edit(pos, page, slot, x) changes the places or the
    rows; size: the exponents rows are drawn from."""
    import torch
    rng = np.random.default_rng(seed)
    pos, page, slot, NP = spans(rng, n, ctx, P)
    rows, W = len(pos), (hq + 2 * nkv) * hd
    x = rng.standard_normal((rows, W + pad))
    lo, hi = size or (-3, 4)
    x *= 2.0 ** rng.integers(lo, hi, (rows, 1))
    if edit:
        edit(pos, page, slot, x[:, :W].reshape(rows, hq + 2 * nkv, hd))
    qkv, x = bf16(x)
    x = x[:, :W].reshape(rows, hq + 2 * nkv, hd)
    g = geom(dl, hq=hq, nkv=nkv, hd=hd, P=P, NP=NP, L=L, theta=1e4)
    shape = (L, NP, 2, nkv, P, hd)
    codes0 = rng.integers(0, 256, shape).astype(np.uint8)      # NaN among them
    scales0 = rng.integers(100, 140, shape[:4] + (P // block,)).astype(np.uint8)
    codes, scales = dev(codes0), dev(scales0)
    if f8:
        codes, scales = codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)
    assert codes.numel() == dl.dflash_cache8_code_bytes(g)
    assert scales.numel() == dl.dflash_cache8_scale_bytes(g, block)
    gq, gqv = bf16(1 + 0.1 * rng.standard_normal(hd))
    gk, gkv = bf16(1 + 0.1 * rng.standard_normal(hd))
    xq, k, v = qkv[:, :hq * hd], qkv[:, hq * hd:(hq + nkv) * hd], qkv[:, (hq + nkv) * hd:W]
    q_out = xq if in_place else torch.full((rows, hq, hd), 7.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dl.dflash_chunk_rope_store8(
        g, layer, None if rot == 0 else rope_spec(dl, layout, rot, scaling, factor),
        xq if q else None, k, v, dev(pos), dev(page), dev(slot), q_out if q else None, codes, scales,
        block, gamma_q=gq if gamma else None, gamma_k=gk if gamma else None, dev_status=st)
    torch.cuda.synchronize()
    ang, mag = chunk.rope_angles(rot, 1e4, scaling, factor, 64)
    kw = dict(layout=layout, rot=rot, angles=ang, mag=mag)
    with np.errstate(invalid="ignore"):
        yq, sq = chunk.turn(x[:, :hq], gqv if gamma else None, pos, 1e-6, **kw)
        yk, sk = chunk.turn(x[:, hq:hq + nkv], gkv if gamma else None, pos, 1e-6, **kw)
    if not rot:  # what is not turned is as large as it is itself
        sq, sk = np.abs(yq), np.abs(yk)
    if q:
        got = bf16_f64(bits(q_out)).reshape(rows, hq, hd)
        here = pos >= 0
        fine = np.isfinite(yq) & here[:, None, None]
        assert np.all(np.abs(got - yq)[fine] <= (2.0 ** -8 * np.abs(yq) + 1e-5 * sq)[fine])
        left = x[:, :hq] if in_place else np.full_like(yq, 7.0)
        np.testing.assert_array_equal(got[~here], left[~here])
    exact_k = not gamma and rot == 0
    new = [yk, x[:, hq + nkv:]]
    slack = [1e-5 * sk, 0 * sk]
    got_c, got_s = code_bits(codes), code_bits(scales)
    want_c, want_s = codes0.copy(), scales0.copy()
    loose = []
    found, bad = chunk8.runs(pos, page, slot, block, P, NP)
    assert int(st.item()) == flags == bad
    for a, b, pg, i in found:
        at, begun = slot[a:b], np.any(slot[a:b] % block == 0)
        others = np.setdiff1d(np.arange(i * block, (i + 1) * block), at)
        for kv in (0, 1):
            for h in range(nkv):
                y, d = new[kv][a:b, h], slack[kv][a:b, h]
                ok = np.isfinite(y)
                amax = lambda s: np.abs(np.where(ok, np.abs(y) + s * d, 0)).max()  # noqa: E731, B023
                may = {chunk8.exponent(amax(s)) for s in ((-1, 0, 1) if not exact_k and kv == 0
                                                          else (0,))}
                before = int(scales0[layer, pg, kv, h, i]) - 127
                if not begun:
                    may = {max(e, before) for e in may}
                e = int(got_s[layer, pg, kv, h, i]) - 127
                assert e in may, (e, may)
                want_s[layer, pg, kv, h, i] = e + 127
                cell = (layer, pg, kv, h)
                if not begun and e != before:
                    old = chunk8.VALUES[codes0[cell][others]]
                    want_c[cell][others] = np.where(
                        np.isnan(old), got_c[cell][others], chunk8.encode(old * 2.0 ** (before - e)))
                    assert np.all(got_c[cell][others][np.isnan(old)] & 0x7f == 0x7f)
                if kv == 1 or exact_k:
                    with np.errstate(invalid="ignore"):
                        want_c[cell][at] = chunk8.encode(y * 2.0 ** -e)
                else:
                    val = chunk8.VALUES[got_c[cell][at]] * 2.0 ** e
                    assert np.all(np.isnan(val[~ok]))
                    tol = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** (e - 10)) + 1.1 * d
                    assert np.all(np.abs(val - y)[ok] <= tol[ok])
                    loose.append((*cell, at))
    for c in loose:
        want_c[c] = got_c[c]
    np.testing.assert_array_equal(got_s, want_s)
    np.testing.assert_array_equal(got_c, want_c)


@pytest.mark.parametrize("block,P", [(16, 16), (16, 64), (32, 32), (32, 96), (64, 64), (64, 256)])
@pytest.mark.parametrize("gamma", [True, False])
def test_store_blocks(dl, block, P, gamma):  # noqa: F811
    """Blocks begun, gone on with, filled, and left in the middle."""
    check_store(dl, n=[1, 1, 37, 150, 2], ctx=[0, 5, 60, 11, 31], hq=4, nkv=2, hd=128, P=P,
                block=block, rot=128, gamma=gamma, pad=8)


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("hd,rot", [(128, 128), (64, 64), (64, 32), (128, 24), (96, 80), (64, 2),
                                    (128, 12), (64, 6), (256, 256), (16, 16), (256, 2), (48, 40),
                                    (128, 0), (80, 0)])
def test_store_widths(dl, layout, hd, rot):  # noqa: F811
    check_store(dl, n=[21, 1, 16], ctx=[7, 40, 0], hq=3, nkv=1, hd=hd, P=32, block=16, rot=rot,
                layout=layout)
    check_store(dl, n=[1], ctx=[70], hq=2, nkv=2, hd=hd, P=32, block=32, rot=rot, layout=layout,
                gamma=False, L=1, layer=0)


@pytest.mark.parametrize("scaling,factor", [("linear", 4.0), ("yarn", 8.0)])
def test_store_scaling(dl, scaling, factor):  # noqa: F811
    check_store(dl, n=[50], ctx=[1 << 16], hq=8, nkv=2, hd=128, P=1 << 15, block=64, rot=128,
                scaling=scaling, factor=factor)


@pytest.mark.parametrize("n,ctx,hq,nkv,in_place", [
    ([1], [0], 1, 1, False), ([1] * 70, list(range(3, 73)), 32, 8, True), ([3, 0, 2], [9, 1, 0], 7, 7, True),
    ([300], [33], 40, 8, True), ([700, 1, 900], [1, 500, 16], 6, 3, False), ([16], [100], 32, 8, False)])
def test_store_rows_and_heads(dl, n, ctx, hq, nkv, in_place):  # noqa: F811
    check_store(dl, n=n, ctx=ctx, hq=hq, nkv=nkv, hd=64, P=64, block=64, rot=64, in_place=in_place)
    check_store(dl, n=n, ctx=ctx, hq=hq, nkv=nkv, hd=128, P=16, block=16, rot=64, layout="pairs",
                in_place=in_place, L=1, layer=0, f8=True)


def test_store_keys_alone_and_many_heads(dl):  # noqa: F811
    check_store(dl, n=[20, 3], ctx=[5, 8], hq=2, nkv=2, hd=64, P=16, block=16, rot=64, q=False)
    check_store(dl, n=[20, 3], ctx=[5, 8], hq=40, nkv=40, hd=64, P=16, block=16, rot=64)


def test_store_queries_alone(dl):  # noqa: F811
    import torch
    rng = np.random.default_rng(3)
    g = geom(dl, hq=4, nkv=2, hd=64, P=16, NP=4)
    q, qv = bf16(rng.standard_normal((9, 256)))
    pos, out = dev(np.arange(9, dtype=np.int32) + 5), torch.zeros_like(q)
    dl.dflash_chunk_rope_store8(g, 0, rope_spec(dl, "half", 64), q, None, None, pos, None, None, out,
                                None, None, 16)
    want = torch.zeros_like(q)
    dl.dflash_chunk_rope_store(g, 0, rope_spec(dl, "half", 64), q, None, None, pos, None, None, want,
                               None)
    assert torch.equal(out, want)


def test_store_rows_without_a_place(dl):  # noqa: F811
    """Rows past the last request, not placed, and outside the pool, between blocks."""
    def edit(pos, page, slot, x):
        pos[8:10] = -1
        page[24:26], slot[24:26] = -1, -1
        page[40] = 10 ** 6
        slot[56] = 64
        slot[57] = -1
    kw = dict(n=[64, 20], ctx=[0, 3], hq=2, nkv=2, hd=64, P=64, block=16, rot=64, flags=8)

    def cut(pos, page, slot, x):
        """the same, with what follows in a block left out: the rows of a block follow one another"""
        edit(pos, page, slot, x)
        for a, b in ((10, 16), (26, 32), (41, 48), (58, 64)):
            pos[a:b] = -1
    check_store(dl, edit=cut, **kw)


def test_store_any_order_of_slots_and_a_slot_too_often(dl):  # noqa: F811
    def backwards(pos, page, slot, x):
        slot[:16] = slot[:16][::-1].copy()
        slot[20:26] = slot[20:26][::-1].copy()
    check_store(dl, n=[40], ctx=[0], hq=2, nkv=1, hd=64, P=16, block=16, rot=64, edit=backwards)
    import torch
    rng = np.random.default_rng(4)
    g = geom(dl, hq=1, nkv=1, hd=64, P=16, NP=3)
    k, _ = bf16(rng.standard_normal((40, 64)))
    codes = torch.full((1, 3, 2, 1, 16, 64), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((1, 3, 2, 1, 1), 127, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ones = torch.ones(40, dtype=torch.int32, device="cuda")
    dl.dflash_chunk_rope_store8(g, 0, None, None, k, k, ones, ones, ones * 3, None, codes, scales, 16,
                                dev_status=st)
    assert int(st.item()) == dl._lib.DEV_BAD_ROWS
    got = codes.cpu().numpy()
    assert np.all(got[0, [0, 2]] == 9) and np.all(scales.cpu().numpy()[0, [0, 2]] == 127)


def test_store_extreme_values(dl):  # noqa: F811
    """Zeros, the largest and smallest bf16 numbers, infinities and NaN: the others of a block are
    stored as without them."""
    def edit(pos, page, slot, x):
        x[0:16] = 0
        x[16:32] *= 2.0 ** -127
        x[32:48] = np.clip(x[32:48] * 2.0 ** 127, -3.38e38, 3.38e38)
        x[50, :, 3], x[51, :, 5], x[52, :, 9] = np.inf, -np.inf, np.nan
        x[64:80] = np.nan
        x[80] = -0.0
    for begun in (True, False):
        check_store(dl, n=[96 - (not begun)], ctx=[int(not begun)], hq=2, nkv=2, hd=64, P=32,
                    block=16, rot=0, gamma=False, edit=edit, size=(0, 1))
    check_store(dl, n=[64], ctx=[0], hq=2, nkv=2, hd=64, P=32, block=16, rot=0, gamma=False,
                size=(-140, 100))


def test_store_scale_only_rises_while_a_block_goes_on(dl):  # noqa: F811
    """Token by token, a block ends with the scale that its largest token asks for, and what it
    held is within a step of what it would be stored at once."""
    import torch
    rng = np.random.default_rng(6)
    x = rng.standard_normal((64, 2, 64)) * 2.0 ** np.arange(-8, 8).repeat(4)[:, None, None]
    k, kv = bf16(x.reshape(64, 128))
    g = geom(dl, hq=2, nkv=2, hd=64, P=64, NP=1)
    codes = torch.zeros((1, 1, 2, 2, 64, 64), dtype=torch.uint8, device="cuda")
    scales = torch.full((1, 1, 2, 2, 1), 255, dtype=torch.uint8, device="cuda")   # stale
    i32 = torch.arange(64, dtype=torch.int32, device="cuda")
    for t in range(64):
        dl.dflash_chunk_rope_store8(g, 0, None, None, k[t:t + 1], k[t:t + 1], i32[t:t + 1],
                                    i32[:1], i32[t:t + 1], None, codes, scales, 64)
    want, s = chunk8.quantise(kv.reshape(64, 2, 64).transpose(1, 0, 2), 64)
    np.testing.assert_array_equal(code_bits(scales)[0, 0], np.stack([s, s]))
    got = chunk8.VALUES[code_bits(codes)[0, 0, 0]]
    err = np.abs(got - kv.reshape(64, 2, 64).transpose(1, 0, 2) / chunk8.factor(s)[:, :, None])
    # raised at most once a doubling: a shift is exact but for values below 2^-6, where each of up
    # to 16 shifts rounds by half a step of 2^-9, halved by every later one
    assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(got) * (1 + 2.0 ** -3), 2.0 ** -9))


# ------------------------------------------------------------------ read


@pytest.mark.parametrize("rows,nkv,hd,P,block", [(1, 1, 16, 16, 16), (37, 2, 64, 32, 16), (300, 8, 128, 64, 64),
                                                 (1000, 3, 96, 96, 32), (5, 40, 256, 64, 32), (4000, 8, 128, 16, 16)])
def test_read(dl, rows, nkv, hd, P, block):  # noqa: F811
    """Every code and scale, rows in any order and more than once, with absent and bad ones."""
    import torch
    rng = np.random.default_rng(7)
    L, NP, layer = 2, max(2, rows // P // 2), 1
    g = geom(dl, hq=nkv, nkv=nkv, hd=hd, P=P, NP=NP, L=L)
    codes = rng.integers(0, 256, (L, NP, 2, nkv, P, hd)).astype(np.uint8)
    scales = rng.integers(0, 256, (L, NP, 2, nkv, P // block)).astype(np.uint8)
    page, slot = (rng.integers(0, m, rows).astype(np.int32) for m in (NP, P))
    flags = 0
    if rows > 4:
        page[1], page[2], slot[3], slot[4], flags = -1, NP, P, -1, 8
    with np.errstate(over="ignore", invalid="ignore"):
        val = chunk8.values(codes[layer], scales[layer], block)
    here = (page >= 0) & (page < NP) & (slot >= 0) & (slot < P)
    pads, st = (0, 64), torch.zeros(1, dtype=torch.int32, device="cuda")
    for which in ((1, 1), (1, 0), (0, 1)):
        full = [torch.full((rows, nkv * hd + p), 7.0, dtype=torch.bfloat16, device="cuda") for p in pads]
        out = [f[:, :nkv * hd].unflatten(1, (nkv, hd)) if w else None for f, w in zip(full, which)]
        dl.dflash_chunk_read8(g, layer, dev(codes), dev(scales), block, dev(page), dev(slot), *out,
                              dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == flags
        for kv in (0, 1):
            got = bits(full[kv])[:, :nkv * hd].reshape(rows, nkv, hd)
            if not which[kv]:
                assert torch.all(full[kv] == 7.0)
                continue
            assert torch.all(full[kv][:, nkv * hd:] == 7.0)
            want = val[np.where(here, page, 0), kv, :, np.where(here, slot, 0)]
            want = torch.from_numpy(want).to(torch.float32)     # exact, or beyond bf16 as well
            want = bits(want.to(torch.bfloat16))
            want[~here] = 0x40e0
            nan = (want & 0x7fff) > 0x7f80
            np.testing.assert_array_equal((got & 0x7fff) > 0x7f80, nan)
            np.testing.assert_array_equal(got[~nan], want[~nan])


# ------------------------------------------------------------------ attention


def run_attn8(dl, pb, *, hq, nkv, hd, P, block=16, window=0, sinks=None, causal=True, S=0,  # noqa: F811
              L=1, layer=0, scale=None, pad_rows=0, stride_pad=0, flags=0, check=True, stream=None,
              cache=None, tol=ATTN_TOL):
    import torch
    g = geom(dl, hq=hq, nkv=nkv, hd=hd, P=P, M=pb["M"], NP=pb["NP"], L=L)
    B, N = len(pb["ctx"]), pb["q"].shape[0]
    qt, qv = bf16(np.concatenate([pb["q"], np.ones((pad_rows, hq, hd))]))
    codes, scales = cache or chunk8.quantise(pb["pool"], block)
    if stride_pad:  # rows of a wider tensor
        wide = torch.zeros((N + pad_rows, hq * hd + stride_pad), dtype=torch.bfloat16, device="cuda")
        wide[:, :hq * hd] = qt.flatten(1)
        qt = wide[:, :hq * hd].unflatten(1, (hq, hd))
    full = torch.full((N + pad_rows, hq * hd + stride_pad), 7.0, dtype=torch.bfloat16, device="cuda")
    out = full[:, :hq * hd].unflatten(1, (hq, hd))
    need = dl.dflash_chunk_attention8_workspace_bytes(g, B, N + pad_rows, S)
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")  # NaN everywhere
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dl.dflash_chunk_attention8(
        g, layer, qt, dev(codes), dev(scales), block, dev(pb["table"]), dev(pb["cu"]),
        dev(pb["ctx"]), dev(pb["kv"]), out, ws, window=window,
        sinks=None if sinks is None else dev(sinks.astype(np.float32)), scale=scale,
        mask_mode=dl.MASK_CAUSAL_TAIL if causal else dl.MASK_BLOCK_BIDIR, num_segments=S,
        dev_status=st, stream=stream)
    torch.cuda.synchronize()
    assert int(st.item()) == flags
    got = bf16_f64(bits(out)).reshape(N + pad_rows, hq, hd)
    if check:
        val = chunk8.values(codes[layer], scales[layer], block)
        want, size = chunk.chunk_attention(
            qv, val, pb["table"], pb["cu"], pb["ctx"], pb["kv"], window=window,
            scale=hd ** -0.5 if scale is None else scale,
            sinks=None if sinks is None else sinks.astype(np.float32).astype(np.float64),
            causal=causal)
        rows = ~np.isnan(want).any((1, 2))
        err = np.abs(got - want)[rows] - tol * size[rows]
        assert np.all(err <= 1e-30), f"worst excess {np.nanmax(err)}"
        np.testing.assert_array_equal(got[~rows], 7.0)  # rows of no request
        if stride_pad:
            assert torch.all(full[:, hq * hd:] == 7.0)
    return got


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("hq,nkv,hd,P,block", [(4, 2, 64, 16, 16), (8, 2, 128, 64, 32),
                                               (4, 1, 128, 64, 64)])
def test_attention_lengths(dl, shape, hq, nkv, hd, P, block):  # noqa: F811
    rng = np.random.default_rng(11)
    n, ctx = SHAPES[shape]
    pb = attn_problem(rng, n, ctx, hq=hq, nkv=nkv, hd=hd, P=P)
    run_attn8(dl, pb, hq=hq, nkv=nkv, hd=hd, P=P, block=block)


@pytest.mark.parametrize("window", [1, 5, 128, 1000])
@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_masks(dl, window, sinks, causal):  # noqa: F811
    rng = np.random.default_rng(12)
    hq, nkv, hd, P = 6, 2, 64, 16
    pb = attn_problem(rng, [1, 90, 3], [300, 45, 0], hq=hq, nkv=nkv, hd=hd, P=P)
    run_attn8(dl, pb, hq=hq, nkv=nkv, hd=hd, P=P, window=window, causal=causal,
              sinks=rng.standard_normal(hq) if sinks else None)


@pytest.mark.parametrize("hq,nkv,hd,P,block", [(1, 1, 64, 128, 64), (5, 1, 128, 256, 32),
                                               (7, 7, 64, 32, 32), (48, 1, 128, 16, 16),
                                               (40, 8, 64, 64, 64), (160, 1, 64, 16, 16)])
def test_attention_heads_and_pages(dl, hq, nkv, hd, P, block):  # noqa: F811
    rng = np.random.default_rng(13)
    pb = attn_problem(rng, [3, 40], [200, 17], hq=hq, nkv=nkv, hd=hd, P=P, L=2, layer=1)
    run_attn8(dl, pb, hq=hq, nkv=nkv, hd=hd, P=P, block=block, L=2, layer=1,
              sinks=rng.standard_normal(hq))


@pytest.mark.parametrize("S", [1, 2, 3, 9, 40])
def test_attention_segments(dl, S):  # noqa: F811
    rng = np.random.default_rng(14)
    kw = dict(hq=4, nkv=1, hd=128, P=64, block=64)
    pb = attn_problem(rng, [1, 2, 0, 50], [1200, 63, 3, 700], **{k: kw[k] for k in ("hq", "nkv", "hd", "P")})
    for sinks in (None, rng.standard_normal(4)):
        run_attn8(dl, pb, **kw, S=S, sinks=sinks, pad_rows=2)
        run_attn8(dl, pb, **kw, S=S, sinks=sinks, window=200)


@pytest.mark.parametrize("block", [16, 32, 64])
@pytest.mark.parametrize("hd,hq,nkv,rows", [(64, 4, 2, 3), (128, 8, 2, 3), (128, 4, 2, 150), (64, 6, 1, 90)])
def test_attention_scales_far_apart(dl, block, hd, hq, nkv, rows):  # noqa: F811
    """Blocks whose scales differ by many powers of two, K and V apart; keys large enough that the
    scores follow, and scales at the ends of what the store writes."""
    rng = np.random.default_rng(40)
    P = 64
    pb = attn_problem(rng, [rows], [600], hq=hq, nkv=nkv, hd=hd, P=P)
    codes, scales = chunk8.quantise(pb["pool"], block)
    shape = scales.shape[:2] + scales.shape[3:]
    up = rng.integers(-30, 3, shape)
    scales[:, :, 0] = np.clip(scales[:, :, 0].astype(int) + up, 3, 247)
    scales[:, :, 1] = np.clip(scales[:, :, 1].astype(int) + rng.integers(-30, 25, shape), 3, 247)
    # |s|_1 up to 64 * 4 * 2^2 * 3 / 8, 400 and more: 4 times the 16-bit call's scores
    kw = dict(hq=hq, nkv=nkv, hd=hd, P=P, block=block, tol=ATTN_TOL + 6e-3)
    run_attn8(dl, pb, cache=(codes, scales), **kw)
    run_attn8(dl, pb, cache=(codes, scales), **kw, S=3, window=300, sinks=rng.standard_normal(hq))
    for v in (3, 120, 247):        # every value the store can write, in V
        scales[:, :, 1] = v
        run_attn8(dl, pb, cache=(codes, scales), **kw) if v < 247 else None
    scales[:, :, 1], codes[:, :, 1] = 240, np.minimum(codes[:, :, 1] & 0x7f, 0x20)
    run_attn8(dl, pb, cache=(codes, scales), **kw)


def test_attention_every_code(dl):  # noqa: F811
    """Single keys: the output is that key's value, whatever the code, bit by bit."""
    rng = np.random.default_rng(41)
    for hd in (64, 128):
        pb = attn_problem(rng, [1] * 8, [0] * 8, hq=1, nkv=1, hd=hd, P=16)
        all_codes = np.array([c for c in range(256) if c & 0x7f != 0x7f] + [0, 1], np.uint8)
        for part in range(4):
            for s in (3, 9, 100, 120, 127, 134, 135, 190, 247):
                codes = np.zeros((1, pb["NP"], 2, 1, 16, hd), np.uint8)
                scales = np.full((1, pb["NP"], 2, 1, 1), s, np.uint8)
                use = np.resize(np.roll(all_codes, 64 * part), 8 * hd).reshape(8, hd)
                codes[0, pb["table"][:, 0], 1, 0, 0] = use
                val = chunk8.VALUES[use] * 2.0 ** (s - 127)
                val = np.where(np.abs(val) < 2.0 ** 128, val, np.copysign(np.inf, val))  # past bf16
                got = run_attn8(dl, pb, hq=1, nkv=1, hd=hd, P=16, cache=(codes, scales), check=False)
                np.testing.assert_array_equal(got[:, 0], val)


@pytest.mark.parametrize("S", [0, 1, 4])
def test_attention_rows_without_keys(dl, S):  # noqa: F811
    rng = np.random.default_rng(15)
    kw = dict(hq=4, nkv=2, hd=64, P=16)
    pb = attn_problem(rng, [20, 30, 4], [40, 100, 0], **kw)
    pb["kv"] = np.array([60, 104, 0], np.int32)
    for sinks in (None, rng.standard_normal(4)):
        got = run_attn8(dl, pb, **kw, window=8, S=S, sinks=sinks, pad_rows=3)
        assert np.all(got[20 + 11:54] == 0)  # rows at 111.. see keys 104.. only


def test_attention_stale_scales_and_codes(dl):  # noqa: F811
    """What no row sees is never used: NaN codes in the slots of a block that is not full, NaN
    scales in blocks and pages that hold nothing."""
    rng = np.random.default_rng(42)
    for hd, block, S in ((64, 16, 1), (128, 64, 1), (128, 16, 3)):
        kw = dict(hq=4, nkv=2, hd=hd, P=64)
        pb = attn_problem(rng, [5, 150, 1], [33, 0, 700], **kw)
        codes, scales = chunk8.quantise(pb["pool"], block)
        empty = np.isnan(pb["pool"]).all(-1).reshape(*scales.shape, block).all(-1)
        scales[empty] = 255
        run_attn8(dl, pb, **kw, block=block, S=S, cache=(codes, scales))
        run_attn8(dl, pb, **kw, block=block, S=S, cache=(codes, scales), window=40, causal=False)


@pytest.mark.parametrize("kv", [0, 1])
@pytest.mark.parametrize("hd,rows", [(64, 40), (128, 4), (128, 7), (128, 40), (128, 90)])
def test_attention_scale_of_nan(dl, hd, rows, kv):  # noqa: F811
    """A scale of 255 among finite codes: NaN for the rows that see the block, and nothing for the
    requests (and, K's, for the rows) that do not."""
    rng = np.random.default_rng(35)
    kw = dict(hq=4, nkv=1, hd=hd, P=16)
    pb = attn_problem(rng, [rows, rows], [150, 150], **kw)
    codes, scales = chunk8.quantise(pb["pool"], 16)
    want = run_attn8(dl, pb, **kw, check=False, cache=(codes, scales))
    broken = scales.copy()
    at = 150 + rows // 2   # the block of the middle row's own key: seen from its first slot on
    broken[0, pb["table"][1, at // 16], kv] = 255
    got = run_attn8(dl, pb, **kw, check=False, cache=(codes, broken))
    np.testing.assert_array_equal(got[:rows], want[:rows])
    sees = np.maximum(at // 16 * 16 - 150, 0)
    assert np.all(np.isnan(got[rows + sees:]))
    if kv == 0:
        np.testing.assert_array_equal(got[rows:rows + sees], want[rows:rows + sees])


def test_attention_extreme_scores(dl):  # noqa: F811
    rng = np.random.default_rng(16)
    hq, nkv, hd, P = 4, 2, 64, 16
    pb = attn_problem(rng, [70], [500], hq=hq, nkv=nkv, hd=hd, P=P)
    pb["q"] *= 6.0
    pb["pool"][:, :, 0] *= 2
    for sink in (-1e30, 0.0, 90.0):
        run_attn8(dl, pb, hq=hq, nkv=nkv, hd=hd, P=P, sinks=np.full(hq, sink), tol=ATTN_TOL + 7e-3)


@pytest.mark.parametrize("exp", [-100, -30, 20, 90])
def test_attention_query_sizes(dl, exp):  # noqa: F811
    """Queries of any size of bf16, a row of zeros and rows with one large value among them."""
    rng = np.random.default_rng(43)
    kw = dict(hq=4, nkv=1, hd=128, P=32, block=32)
    pb = attn_problem(rng, [40, 1], [100, 300], **{k: kw[k] for k in ("hq", "nkv", "hd", "P")})
    pb["q"][3] = 0
    pb["q"][5, :, 7] *= 2.0 ** 8
    pb["q"][6, :, 9:] *= 2.0 ** -12
    pb["q"] *= 2.0 ** exp
    # |s|_1 with one value 2^8 times the others, below 300
    run_attn8(dl, pb, **kw, scale=2.0 ** -exp / 11.3, tol=ATTN_TOL + 5e-3)


def test_attention_bad_pages_and_lengths(dl):  # noqa: F811
    rng = np.random.default_rng(17)
    hq, nkv, hd, P = 4, 2, 64, 16
    kw = dict(hq=hq, nkv=nkv, hd=hd, P=P)
    pb = attn_problem(rng, [5, 140], [200, 150], **kw)
    pb["table"][0, 3], pb["table"][1, 2] = -1, pb["NP"]
    run_attn8(dl, pb, **kw, flags=8)
    run_attn8(dl, pb, **kw, flags=8, S=3)
    pb = attn_problem(rng, [5, 9], [200, 150], **kw)
    pb["table"][0, :10], pb["table"][1, :3] = -1, 10 ** 9   # before every window
    run_attn8(dl, pb, **kw, window=30)
    pb = attn_problem(rng, [5, 9], [200, 150], **kw)
    pb["kv"][0] = -3
    run_attn8(dl, pb, **kw, flags=16)
    pb["kv"][0] = pb["M"] * P + 1   # clamped; the causal rows see no further than before
    run_attn8(dl, pb, **kw, flags=16)
    pb = attn_problem(rng, [5, 9], [200, 150], **kw)
    pb["ctx"][0] = -1
    got = run_attn8(dl, pb, **kw, flags=128, check=False)
    assert np.all(got[:5] == 7.0) and not np.any(got[5:] == 7.0)
    pb["ctx"][0], pb["cu"] = 200, np.array([0, 5, 15], np.int32)   # past the last row
    got = run_attn8(dl, pb, **kw, flags=128, check=False)
    assert np.all(got[5:] == 7.0) and not np.any(got[:5] == 7.0)


def test_attention_padded_and_strided_rows(dl):  # noqa: F811
    rng = np.random.default_rng(18)
    kw = dict(hq=8, nkv=2, hd=128, P=64)
    pb = attn_problem(rng, [1, 35], [90, 64], **kw)
    a = run_attn8(dl, pb, **kw, pad_rows=5, stride_pad=64)
    b = run_attn8(dl, pb, **kw)
    np.testing.assert_array_equal(a[:36], b)


def test_attention_is_repeatable_and_on_another_stream(dl):  # noqa: F811
    import torch
    rng = np.random.default_rng(19)
    kw = dict(hq=32, nkv=8, hd=128, P=64, block=64)
    pb = attn_problem(rng, [1, 1, 80], [900, 30, 64], **{k: kw[k] for k in ("hq", "nkv", "hd", "P")})
    a = run_attn8(dl, pb, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = run_attn8(dl, pb, **kw, check=False, stream=s)
    np.testing.assert_array_equal(a, b)


def test_long_cache(dl):  # noqa: F811
    """Code offsets past 2^32 bytes: the requests' pages sit at both ends of a large pool, which
    the store, the reading and the attention all reach."""
    import torch
    rng = np.random.default_rng(20)
    hq, nkv, hd, P, block = 4, 2, 128, 64, 32
    NP = (1 << 32) // (2 * nkv * P * hd) + 40
    pb = attn_problem(rng, [3, 20], [170, 500], hq=hq, nkv=nkv, hd=hd, P=P, extra_pages=0)
    small = pb["pool"].shape[1]
    far = np.where(np.arange(small) % 2 == 0, np.arange(small), NP - 1 - np.arange(small))
    g = geom(dl, hq=hq, nkv=nkv, hd=hd, P=P, M=pb["M"], NP=NP)
    codes = torch.empty((1, NP, 2, nkv, P, hd), dtype=torch.uint8, device="cuda")
    scales = torch.empty((1, NP, 2, nkv, P // block), dtype=torch.uint8, device="cuda")
    c, s = chunk8.quantise(pb["pool"], block)
    codes[0, dev(far)], scales[0, dev(far)] = dev(c[0]), dev(s[0])
    table = np.where(pb["table"] >= 0, far[pb["table"]], -1).astype(np.int32)
    qt, _ = bf16(pb["q"])
    out = torch.empty_like(qt)
    ws = torch.empty(max(16, dl.dflash_chunk_attention8_workspace_bytes(g, 2, 23)),
                     dtype=torch.uint8, device="cuda")
    dl.dflash_chunk_attention8(g, 0, qt, codes, scales, block, dev(table), dev(pb["cu"]),
                               dev(pb["ctx"]), dev(pb["kv"]), out, ws)
    near = run_attn8(dl, pb, hq=hq, nkv=nkv, hd=hd, P=P, block=block)
    np.testing.assert_array_equal(bf16_f64(bits(out)).reshape(near.shape), near)
    k, _ = bf16(rng.standard_normal((64, nkv * hd)))
    page = dev(np.full(64, NP - 1, np.int32))
    slot = dev(np.arange(64, dtype=np.int32))
    dl.dflash_chunk_rope_store8(g, 0, None, None, k, k, slot, page, slot, None, codes, scales, block)
    back = [torch.zeros((64, nkv, hd), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    dl.dflash_chunk_read8(g, 0, codes, scales, block, page, slot, *back)
    torch.cuda.synchronize()
    x = k.float().cpu().numpy().reshape(64, nkv, hd).transpose(1, 0, 2)
    want = chunk8.values(*chunk8.quantise(x, block), block).transpose(1, 0, 2)
    for b in back:
        np.testing.assert_array_equal(bf16_f64(bits(b)).reshape(want.shape), want)


@pytest.mark.parametrize("shape", WIDE)
@pytest.mark.parametrize("window,sinks,causal", [(0, False, True), (150, True, True),
                                                 (1, False, True), (40, True, False)])
def test_attention_wide_tiles(dl, shape, window, sinks, causal):  # noqa: F811
    rng = np.random.default_rng(23)
    n, ctx = WIDE[shape]
    kw = dict(hq=4, nkv=1, hd=128, P=16)
    pb = attn_problem(rng, n, ctx, **kw)
    run_attn8(dl, pb, **kw, window=window, causal=causal, pad_rows=1,
              sinks=rng.standard_normal(4) if sinks else None)


@pytest.mark.parametrize("hq,nkv,rows", [(4, 1, 20), (16, 2, 9), (16, 1, 5), (128, 1, 1),
                                         (3, 3, 70), (64, 1, 3), (256, 1, 1)])
def test_attention_fewer_rows_than_a_box(dl, hq, nkv, rows):  # noqa: F811
    rng = np.random.default_rng(34)
    kw = dict(hq=hq, nkv=nkv, hd=128, P=32)
    pb = attn_problem(rng, [rows], [150], **kw)
    run_attn8(dl, pb, **kw, block=32, S=1)
    run_attn8(dl, pb, **kw, S=2, stride_pad=64, window=70)


@pytest.mark.parametrize("S", [2, 5])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_wide_tiles_in_segments(dl, S, hd):  # noqa: F811
    rng = np.random.default_rng(24)
    kw = dict(hq=8, nkv=1, hd=hd, P=64)
    pb = attn_problem(rng, [70, 1, 5], [600, 300, 0], **kw)
    for sinks in (None, rng.standard_normal(8)):
        run_attn8(dl, pb, **kw, block=64, S=S, sinks=sinks, pad_rows=2)
        run_attn8(dl, pb, **kw, S=S, sinks=sinks, window=130)


def test_attention_wide_tiles_bad_pages_and_cut_cache(dl):  # noqa: F811
    rng = np.random.default_rng(25)
    kw = dict(hq=8, nkv=2, hd=64, P=16)
    pb = attn_problem(rng, [90, 40], [200, 150], **kw)
    pb["table"][0, 3], pb["table"][0, 15], pb["table"][1, 9] = -1, pb["NP"] + 5, -7
    run_attn8(dl, pb, **kw, flags=8)
    run_attn8(dl, pb, **kw, flags=8, S=3)
    pb = attn_problem(rng, [90, 40], [200, 150], **kw)
    pb["kv"] = np.array([250, 0], np.int32)
    for S in (1, 3):
        got = run_attn8(dl, pb, **kw, window=20, S=S)
        assert np.all(got[69:] == 0)   # rows at 269 on see keys 250 on; the second request none


def test_attention_many_requests(dl):  # noqa: F811
    rng = np.random.default_rng(26)
    kw = dict(hq=2, nkv=1, hd=64, P=16)
    n = [int(x) for x in rng.integers(0, 4, 1100)]
    n[500] = 150
    pb = attn_problem(rng, n, [int(x) for x in rng.integers(0, 30, 1100)], **kw)
    run_attn8(dl, pb, **kw)
    run_attn8(dl, pb, **kw, S=2)


@pytest.mark.parametrize("hq,nkv,hd,P,window,S", [
    (16, 8, 128, 64, 0, 1), (15, 5, 64, 16, 37, 1), (8, 8, 128, 32, 200, 1), (24, 8, 64, 16, 0, 3),
    (64, 8, 128, 64, 0, 2)])
def test_attention_blocks_with_many_works(dl, hq, nkv, hd, P, window, S):  # noqa: F811
    rng = np.random.default_rng(29)
    kw = dict(hq=hq, nkv=nkv, hd=hd, P=P)
    n = [int(x) for x in rng.choice([0, 1, 2, 5, 33, 65, 129, 140, 200], 34)]
    ctx = [int(x) for x in rng.integers(0, 900, 34)]
    pb = attn_problem(rng, n, ctx, **kw)
    pb["kv"][[5, 11]] = 0
    pb["kv"][17] //= 2
    live = [r for r in range(34) if n[r] > 0 and pb["kv"][r] == n[r] + ctx[r]]
    bad = [r for r in live if n[r] > 1][3:6]
    for r in bad:
        pb["table"][r, (pb["kv"][r] - 1) // P] = pb["NP"] + 9
    sinks = rng.standard_normal(hq)
    got = [run_attn8(dl, pb, **kw, window=window, S=S, sinks=sinks, pad_rows=1, flags=8,
                     check=check) for check in (True, False)]
    np.testing.assert_array_equal(got[0], got[1])


@pytest.mark.parametrize("nkv,rows,ctx", [(20, 1300, 3000), (9, 4000, 300)])
def test_attention_uneven_segments(dl, nkv, rows, ctx):  # noqa: F811
    rng = np.random.default_rng(31)
    kw = dict(hq=nkv, nkv=nkv, hd=64, P=64, block=64)
    pb = attn_problem(rng, [rows], [ctx], hq=nkv, nkv=nkv, hd=64, P=64)
    cache = chunk8.quantise(pb["pool"], 64)
    got = run_attn8(dl, pb, **kw, S=2, check=False, cache=cache)
    heads = [0, nkv // 2, nkv - 1]
    pool, q = chunk8.values(cache[0][0], cache[1][0], 64)[:, :, heads], bf16(pb["q"][:, heads])[1]
    want, size = chunk.chunk_attention(q, pool, pb["table"], pb["cu"], pb["ctx"], pb["kv"],
                                       scale=0.125)
    assert np.all(np.abs(got[:, heads] - want) <= ATTN_TOL * size)
    np.testing.assert_array_equal(got, run_attn8(dl, pb, **kw, S=2, check=False, cache=cache))


@pytest.mark.parametrize("B,S", [(2, 4), (100, 1), (300, 1)])
def test_attention_captured_and_at_once(dl, B, S):  # noqa: F811
    """Calls in two graphs replayed on two streams at the same time, a workspace each, give what
    each gives alone."""
    import torch
    rng = np.random.default_rng(33)
    kw = dict(hq=16, nkv=8, hd=128, P=32)
    pbs = [attn_problem(rng, [int(x) for x in rng.choice([1, 2, 90, 150], B)],
                        [int(x) for x in rng.integers(0, 500, B)], **kw) for _ in range(2)]
    caches = [chunk8.quantise(pb["pool"], 32) for pb in pbs]
    want = [run_attn8(dl, pb, **kw, block=32, S=S, check=False, cache=c) for pb, c in zip(pbs, caches)]
    graphs, outs, streams, keep = [], [], [torch.cuda.Stream() for _ in pbs], []
    for pb, c, s in zip(pbs, caches, streams):
        g = geom(dl, M=pb["M"], NP=pb["NP"], **kw)
        a = [bf16(pb["q"])[0], dev(c[0]), dev(c[1]), 32,
             *(dev(pb[k]) for k in ("table", "cu", "ctx", "kv"))]
        need = dl.dflash_chunk_attention8_workspace_bytes(g, B, pb["q"].shape[0], S)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        o = torch.empty_like(a[0])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for _ in range(3):
                dl.dflash_chunk_attention8(g, 0, *a, o, ws, num_segments=S, stream=s)
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


# ------------------------------------------------------------------ together


def test_chunks_of_a_prompt_in_a_captured_graph(dl):  # noqa: F811
    """Plan, store, attention and reading of one layer, captured once and replayed for the pieces
    of two prompts and single tokens between them: the rows read back are the tokens' to
    within e4m3, and every piece's output is the definition's over the cache as it then was."""
    import torch
    rng = np.random.default_rng(21)
    hq, nkv, hd, P, M, R, block = 4, 2, 64, 32, 6, 96, 16
    W = (hq + 2 * nkv) * hd
    pieces = [[70, 1], [3, 80], [1, 1], [25, 0], [1, 40]]
    total = np.sum(pieces, 0)
    NP = 2 * M + 3
    g = geom(dl, hq=hq, nkv=nkv, hd=hd, P=P, M=M, NP=NP, theta=1e4)
    sp = rope_spec(dl, "half", hd, "yarn", 4.0)
    gq, _ = bf16(1 + 0.1 * rng.standard_normal(hd))
    gk, gkv = bf16(1 + 0.1 * rng.standard_normal(hd))
    tokens = [bf16(rng.standard_normal((t, W)) * 2.0 ** rng.integers(-2, 3, (t, 1)))[0] for t in total]
    codes = torch.full((1, NP, 2, nkv, P, hd), 255, dtype=torch.uint8, device="cuda")
    scales = torch.full((1, NP, 2, nkv, P // block), 255, dtype=torch.uint8, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    tbl = torch.full((2, M), -1, dtype=torch.int32, device="cuda")
    n_new, ctx, have, rng_t = i32([0, 0]), i32([0, 0]), i32([0, 0]), i32([0, NP])
    free = dev(rng.permutation(NP).astype(np.int32))
    out = plan_outputs(dl, 2, R)
    qkv = torch.zeros((R, W), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((R, hq, hd), dtype=torch.bfloat16, device="cuda")
    o = torch.zeros_like(q)
    back = [torch.zeros((R, nkv, hd), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    ws = torch.empty(max(16, dl.dflash_chunk_attention8_workspace_bytes(g, 2, R)),
                     dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def layer():
        dl.dflash_chunk_plan(g, n_new, ctx, have, tbl, free, rng_t, None, M * P, out, st)
        x, k, v = qkv.split((hq * hd, nkv * hd, nkv * hd), 1)
        dl.dflash_chunk_rope_store8(g, 0, sp, x, k, v, out["row_pos"], out["row_page"],
                                    out["row_slot"], q, codes, scales, block, gamma_q=gq,
                                    gamma_k=gk, dev_status=st)
        dl.dflash_chunk_attention8(g, 0, q, codes, scales, block, tbl, out["cu_rows"], ctx,
                                   out["seq_lens"], o, ws, dev_status=st)
        dl.dflash_chunk_read8(g, 0, codes, scales, block, out["row_page"], out["row_slot"], *back,
                              dev_status=st)

    layer()  # no rows: one-time set-up
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        layer()
    ang, mag = chunk.rope_angles(hd, 1e4, "yarn", 4.0, 64)
    kw = dict(layout="half", rot=hd, angles=ang, mag=mag)
    at = [0, 0]
    for piece in pieces:
        n_new.copy_(i32(piece))
        x = torch.cat([tokens[r][at[r]:at[r] + piece[r]] for r in range(2)])
        qkv[:x.shape[0]] = x
        o.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        cu, table = out["cu_rows"].cpu().numpy(), tbl.cpu().numpy()
        val = chunk8.values(code_bits(codes)[0], code_bits(scales)[0], block)
        want, size = chunk.chunk_attention(
            bf16_f64(bits(q)).reshape(R, hq, hd), val, table, cu, ctx.cpu().numpy(),
            out["seq_lens"].cpu().numpy(), scale=hd ** -0.5)
        n = int(cu[2])
        got = bf16_f64(bits(o)).reshape(R, hq, hd)
        assert np.all(np.abs(got - want)[:n] <= ATTN_TOL * size[:n])
        assert torch.all(o[n:] == 7.0)
        page, slot, pos = (out[k].cpu().numpy()[:n] for k in ("row_page", "row_slot", "row_pos"))
        raw = x.double().cpu().numpy().reshape(-1, hq + 2 * nkv, hd)
        yk, sk = chunk.turn(raw[:, hq:hq + nkv], gkv, pos, 1e-6, **kw)
        step = chunk8.factor(code_bits(scales)[0])
        for kv, y, d in ((0, yk, 1e-5 * sk), (1, raw[:, hq + nkv:], 0.0)):
            np.testing.assert_array_equal(bf16_f64(bits(back[kv])).reshape(R, nkv, hd)[:n],
                                          val[page, kv, :, slot])
            e = step[page, kv, :, slot // block][:, :, None]
            assert np.all(np.abs(val[page, kv, :, slot] - y) <=
                          np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * e) + 1.1 * d)
        for r in range(2):
            at[r] += piece[r]
        ctx.copy_(out["seq_lens"])
        have.copy_(out["n_pages"])
        rng_t[0:1].copy_(out["free_head"])
    assert int(st.item()) == 0 and at == total.tolist()
