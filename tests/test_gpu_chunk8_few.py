"""dflash_chunk_attention8 where the mean request has few rows of a KV head's group (its forms for
16, 32 and 64 of them): every mask, odd numbers of rows, requests of many rows among them,
segments, scales and scores that change from tile to tile, many works a block, waits that run out."""
import numpy as np
import pytest

from oracle import chunk8
from tests.test_gpu_chunk import ATTN_TOL, attn_problem, dl  # noqa: F401
from tests.test_gpu_chunk8 import run_attn8

pytestmark = pytest.mark.gpu

# rows of a request, query heads of a KV head: 1 to 64 flat rows
ROWS = [(1, 1), (1, 4), (3, 5), (1, 16), (5, 4), (1, 31), (2, 16), (7, 9), (16, 4), (64, 1), (4, 16)]


@pytest.mark.parametrize("rows,G", ROWS)
@pytest.mark.parametrize("ctx", [0, 100, 127, 128, 700])
def test_rows_and_heads(dl, rows, G, ctx):  # noqa: F811
    rng = np.random.default_rng(rows * G + ctx)
    kw = dict(hq=2 * G, nkv=2, hd=128, P=32)
    pb = attn_problem(rng, [rows], [ctx], **kw)
    run_attn8(dl, pb, **kw, block=32, S=1, sinks=rng.standard_normal(2 * G), pad_rows=2)
    run_attn8(dl, pb, **kw, block=16, S=2, stride_pad=64)


@pytest.mark.parametrize("window", [1, 9, 150])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("rows,G", [(2, 8), (5, 6), (15, 4)])
def test_masks(dl, rows, G, causal, window):  # noqa: F811
    rng = np.random.default_rng(5)
    kw = dict(hq=G, nkv=1, hd=128, P=16)
    pb = attn_problem(rng, [rows, 1, rows, 0], [300, 64, 0, 5], **kw)
    for S in (1, 3):
        run_attn8(dl, pb, **kw, window=window, causal=causal, S=S, sinks=rng.standard_normal(G))
        run_attn8(dl, pb, **kw, window=window, causal=causal, S=S)


@pytest.mark.parametrize("S", [1, 2, 7])
def test_many_rows_among_few(dl, S):  # noqa: F811
    """A request of hundreds of rows in tiles of 16 or 64, and requests without rows or keys."""
    rng = np.random.default_rng(6)
    kw = dict(hq=4, nkv=2, hd=128, P=64, block=64)
    for n in ([1] * 30 + [70], [8] * 12 + [200, 0], [1, 0, 1, 1, 1, 1, 33]):
        ctx = [int(x) for x in rng.integers(0, 500, len(n))]
        pb = attn_problem(rng, n, ctx, **{k: kw[k] for k in ("hq", "nkv", "hd", "P")})
        pb["kv"][2] = 0
        run_attn8(dl, pb, **kw, S=S, pad_rows=1)
        run_attn8(dl, pb, **kw, S=S, window=33, sinks=rng.standard_normal(4))


@pytest.mark.parametrize("rows,G", [(1, 4), (6, 4), (13, 4)])
def test_references_and_units_that_move(dl, rows, G):  # noqa: F811
    """Scores that grow from tile to tile, by a little and by much, and V's scales with them: the
    accumulators are scaled again and again, and past fp16's reach the values go over to bf16."""
    rng = np.random.default_rng(7)
    kw = dict(hq=G, nkv=1, hd=128, P=16)
    for up, v_up in ((0.2, 0), (1.5, 1), (0.0, 3), (-1.0, -2), (1.0, 6)):
        pb = attn_problem(rng, [rows], [900], **kw)
        pb["q"] = np.abs(pb["q"])
        tile = np.repeat(np.arange(8), 128)[:900 + rows]
        kv = 900 + rows
        pages = pb["table"][0, np.arange(kv) // 16]
        slot = np.arange(kv) % 16
        # |s|_1 up to 128 * 0.8 * 12 * 0.1 / 11.3 + noise: well below the bound's 100
        pb["pool"][0, pages, 0, :, slot] = (0.1 * pb["pool"][0, pages, 0, :, slot]
                                            + 0.1 * up * tile[:, None, None])
        pb["pool"][0, pages, 1, :, slot] *= 2.0 ** (v_up * tile[:, None, None])
        run_attn8(dl, pb, **kw, S=1)
        run_attn8(dl, pb, **kw, S=2, window=500)


def test_zero_values_and_zero_keys(dl):  # noqa: F811
    """Blocks of zeros have the smallest scale there is: they count in the weights all the same."""
    rng = np.random.default_rng(8)
    for rows, G, hd in ((1, 4, 128), (10, 4, 128), (90, 2, 128), (3, 4, 64), (150, 2, 64)):
        kw = dict(hq=G, nkv=1, hd=hd, P=32)
        pb = attn_problem(rng, [rows], [400], **kw)
        for kv, at in ((1, [0, 3, 4]), (0, [1, 5]), (1, [9])):
            pb["pool"][0, pb["table"][0, at], kv] = 0
        run_attn8(dl, pb, **kw, block=32, S=1)
        pb["pool"][0, pb["table"][0, :(400 + rows) // 32], 1] = 0
        got = run_attn8(dl, pb, **kw, block=32, S=1, check=False)
        assert np.all(np.isfinite(got))


@pytest.mark.parametrize("rows,G", [(1, 4), (5, 4), (16, 4)])
def test_bad_pages_and_stale_cells(dl, rows, G):  # noqa: F811
    rng = np.random.default_rng(9)
    kw = dict(hq=G, nkv=1, hd=128, P=16)
    pb = attn_problem(rng, [rows, rows], [333, 140], **kw)
    codes, scales = chunk8.quantise(pb["pool"], 16)
    scales[np.isnan(pb["pool"]).all((-1, -2))[..., None]] = 255
    pb["table"][0, 3], pb["table"][0, 20], pb["table"][1, 8] = -1, pb["NP"] + 3, 10 ** 9
    for S in (1, 3):
        run_attn8(dl, pb, **kw, S=S, flags=8, cache=(codes, scales))
    # a page that is bad all over: nothing to see but the last
    pb["table"][1, :8] = -1
    run_attn8(dl, pb, **kw, S=1, flags=8, cache=(codes, scales))


@pytest.mark.parametrize("rows,G,B,S", [(1, 4, 60, 1), (1, 4, 300, 1), (5, 4, 50, 2), (16, 4, 45, 1),
                                        (1, 8, 40, 3)])
def test_many_works(dl, rows, G, B, S):  # noqa: F811
    """More work tiles than the GPU runs at once, lengths from none to several tiles; twice the
    same bits."""
    rng = np.random.default_rng(10)
    kw = dict(hq=8 * G, nkv=8, hd=128, P=64)
    n = [int(x) for x in rng.choice([0, rows, rows], B)]
    ctx = [int(x) for x in rng.integers(0, 600, B)]
    n[1], ctx[1], n[2] = rows, 0, rows
    pb = attn_problem(rng, n, ctx, **kw)
    pb["kv"][2] = 0
    cache = chunk8.quantise(pb["pool"], 64)
    args = dict(kw, block=64, S=S, window=400, sinks=rng.standard_normal(8 * G), cache=cache)
    a = run_attn8(dl, pb, **args, check=B < 100)
    np.testing.assert_array_equal(a, run_attn8(dl, pb, **args, check=False))


@pytest.mark.parametrize("rows,hd", [(1, 128), (10, 128), (16, 128), (1, 64), (90, 128), (90, 64)])
def test_unloaded_tile_times_out_cleanly(dl, rows, hd):  # noqa: F811
    """The bounded waits: one key tile stays unloaded, the kernel winds down and sets its status, and
    the next call is right."""
    rng = np.random.default_rng(22)
    kw = dict(hq=4, nkv=1, hd=hd, P=16)
    pb = attn_problem(rng, [rows], [1000], **kw)
    dl.dflash_test_attention_skip_tile(2)
    try:
        run_attn8(dl, pb, **kw, S=1, check=False, flags=dl._lib.DEV_WAIT_TIMEOUT)
    finally:
        dl.dflash_test_attention_skip_tile(-1)
    run_attn8(dl, pb, **kw, S=1)


@pytest.mark.parametrize("hd", [64, 128])
def test_unloaded_tile_among_many_works(dl, hd):  # noqa: F811
    rng = np.random.default_rng(30)
    kw = dict(hq=8, nkv=8, hd=hd, P=16)
    pb = attn_problem(rng, [1] * 30, [100] * 29 + [900], **kw)
    dl.dflash_test_attention_skip_tile(5)
    try:
        run_attn8(dl, pb, **kw, S=1, check=False, flags=dl._lib.DEV_WAIT_TIMEOUT)
    finally:
        dl.dflash_test_attention_skip_tile(-1)
    run_attn8(dl, pb, **kw, S=1)
