"""Attention of a ragged chunk where scores are NaN, over the cache in 16 and in 8 bits: a row that
sees such a key is NaN, whatever else it sees and however its keys are cut; the others are as
without it."""
import numpy as np
import pytest

from oracle import chunk, chunk8
from tests.test_gpu_chunk import ATTN_TOL, attn_problem, bf16, dl, run_attn  # noqa: F401
from tests.test_gpu_chunk8 import run_attn8

pytestmark = pytest.mark.gpu

# heads and rows of a request that take each kernel and form of a call: few rows (16 and 32 of a
# token and head), one row tile, two
FORMS = [(128, 4, 3), (128, 4, 8), (128, 4, 20), (128, 4, 90), (64, 4, 2), (64, 2, 150)]


def compare(got, q, values, pb, **kw):
    """Rows that the definition makes NaN are NaN in every dim, the others within the tolerance."""
    with np.errstate(invalid="ignore"):
        want, size = chunk.chunk_attention(q, values, pb["table"], pb["cu"], pb["ctx"], pb["kv"], **kw)
    lost = np.isnan(want)
    assert np.array_equal(lost.any(-1), lost.all(-1))
    np.testing.assert_array_equal(np.isnan(got), lost)
    assert np.all((np.abs(got - want) <= ATTN_TOL * size + 1e-30)[~lost])
    return lost.all(-1)


def page_of(pb, r, key, P):
    return pb["table"][r, key // P], key % P


@pytest.mark.parametrize("S", [1, 2, 3, 9, 30])
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("hd,hq,rows", FORMS)
def test_a_key_of_nan_among_others(dl, hd, hq, rows, bits, S):  # noqa: F811
    """One key's K is NaN: the rows that see it, whichever segment it falls into."""
    rng = np.random.default_rng(50)
    P, ctx = 32, 700
    kw = dict(hq=hq, nkv=1, hd=hd, P=P)
    for key in (3, 450, ctx + rows // 2):
        pb = attn_problem(rng, [rows, rows], [ctx, 100], **kw)
        page, slot = page_of(pb, 0, key, P)
        if bits == 16:
            pb["pool"][0, page, 0, 0, slot, 5] = np.nan
            got, values = run_attn(dl, pb, **kw, S=S, check=False), bf16(pb["pool"])[1][0]
        else:
            codes, scales = chunk8.quantise(pb["pool"], 16)
            codes[0, page, 0, 0, slot, 5] = 0x7f
            values = chunk8.values(codes[0], scales[0], 16)
            got = run_attn8(dl, pb, **kw, S=S, check=False, cache=(codes, scales))
        lost = compare(got, bf16(pb["q"])[1], values, pb, scale=hd ** -0.5)
        assert lost.sum() == hq * (rows if key < ctx else rows - rows // 2)


@pytest.mark.parametrize("S", [1, 3])
@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("hd,hq,rows", FORMS)
def test_queries_that_are_not_finite_8(dl, hd, hq, rows, sinks, S):  # noqa: F811
    rng = np.random.default_rng(51)
    kw = dict(hq=hq, nkv=1, hd=hd, P=32)
    pb = attn_problem(rng, [rows, rows], [300, 0], **kw)
    q = pb["q"]
    q[0, 1, hd - 1], q[rows - 1, 0, 3], q[rows, 1, 0] = np.nan, np.nan, np.nan
    if not sinks:  # (a sink makes rows whose scores are all -inf 0)
        q[rows + 1, 0, 17], q[2 * rows - 1, 1, 40] = np.inf, -np.inf
    sk = rng.standard_normal(hq).astype(np.float32) if sinks else None
    codes, scales = chunk8.quantise(pb["pool"], 16)
    got = run_attn8(dl, pb, **kw, S=S, sinks=sk, check=False, cache=(codes, scales))
    lost = compare(got, bf16(q)[1], chunk8.values(codes[0], scales[0], 16), pb, scale=hd ** -0.5,
                   sinks=None if sk is None else sk.astype(np.float64))
    assert lost.sum() == (3 if sinks else 5)


@pytest.mark.parametrize("S", [1, 2, 3])
@pytest.mark.parametrize("window", [0, 1, 20])
@pytest.mark.parametrize("hd,hq,rows", FORMS)
def test_every_visible_block_of_nan_8(dl, hd, hq, rows, window, S):  # noqa: F811
    """K's scales are 255 in all that some rows see: the whole context, or the window's blocks; rows
    without keys are 0 beside them."""
    rng = np.random.default_rng(52)
    kw = dict(hq=hq, nkv=1, hd=hd, P=16)
    pb = attn_problem(rng, [rows, rows, 2, 1], [200, 40, 3, 0], **kw)
    pb["kv"][2] = 0
    codes, scales = chunk8.quantise(pb["pool"], 16)
    at = np.arange(0, 200 + rows) if window == 0 else np.arange(200, 200 + (rows + 1) // 2)
    scales[0, pb["table"][0, np.unique(at // 16)], 0] = 255
    scales[0, pb["table"][3, 0], 0] = 255  # a request's first token
    got = run_attn8(dl, pb, **kw, S=S, window=window, check=False, cache=(codes, scales))
    lost = compare(got, bf16(pb["q"])[1], chunk8.values(codes[0], scales[0], 16), pb,
                   scale=hd ** -0.5, window=window)
    assert lost[0].all() and lost[-1].all() and not lost[rows:-1].any()
    assert np.all(got[2 * rows:-1] == 0)


@pytest.mark.parametrize("S", [1, 3])
def test_first_tokens_that_were_not_finite_8(dl, S):  # noqa: F811
    """Stored as NaN, such a key is all that its own row sees."""
    rng = np.random.default_rng(53)
    for hd, rows in ((128, 4), (128, 60), (64, 4)):
        kw = dict(hq=4, nkv=2, hd=hd, P=16)
        pb = attn_problem(rng, [rows] * 3, [0] * 3, **kw)
        codes, scales = chunk8.quantise(pb["pool"], 16)
        codes[0, pb["table"][1, 0], 0, 0, 0] = 0x7f
        got = run_attn8(dl, pb, **kw, S=S, check=False, cache=(codes, scales))
        lost = compare(got, bf16(pb["q"])[1], chunk8.values(codes[0], scales[0], 16), pb,
                       scale=hd ** -0.5)
        assert lost[rows:2 * rows, :2].all() and lost.sum() == 2 * rows


@pytest.mark.parametrize("S", [1, 2, 3])
@pytest.mark.parametrize("hd,hq,rows", FORMS)
def test_every_score_of_nan_16(dl, hd, hq, rows, S):  # noqa: F811
    """Queries of NaN, a window whose keys are all NaN, and a first token's."""
    rng = np.random.default_rng(54)
    P = 16
    kw = dict(hq=hq, nkv=1, hd=hd, P=P)
    for window in (0, 1, 20):
        for sinks in (None, rng.standard_normal(hq).astype(np.float32)):
            pb = attn_problem(rng, [rows, rows, 2, 1], [300, 40, 3, 0], **kw)
            pb["kv"][2] = 0
            pb["q"][0, 1, hd - 1], pb["q"][2 * rows - 1, 0, 3] = np.nan, np.nan
            pages = pb["table"][0, np.arange(300 - 32, 300 + 16) // P]
            pb["pool"][0, pages, 0] = np.nan
            pb["pool"][0, pb["table"][3, 0], 0, 0, 0, 7] = np.nan
            got = run_attn(dl, pb, **kw, S=S, window=window, sinks=sinks, check=False)
            lost = compare(got, bf16(pb["q"])[1], bf16(pb["pool"])[1][0], pb, scale=hd ** -0.5,
                           window=window, sinks=None if sinks is None else sinks.astype(np.float64))
            assert lost[0].all() and lost[-1].all() and lost[2 * rows - 1, 0]
            assert np.all(got[2 * rows:-1] == 0)


@pytest.mark.parametrize("S", [1, 2, 5])
@pytest.mark.parametrize("run", [run_attn8, run_attn])
@pytest.mark.parametrize("rows,hd", [(1, 128), (10, 128), (40, 128), (20, 64)])
def test_sinks_at_the_ends(dl, rows, hd, run, S):  # noqa: F811
    """-inf is no sink, one of 1e30 takes all weight; NaN and infinity make their head's rows NaN,
    but those that see no key."""
    rng = np.random.default_rng(74)
    kw = dict(hq=4, nkv=1, hd=hd, P=32)
    pb = attn_problem(rng, [rows, 2], [200, 40], **kw)
    pb["kv"][1] = 0
    none = run(dl, pb, **kw, S=S)
    got = run(dl, pb, **kw, S=S, check=False, sinks=np.array([-np.inf, 1e30, np.nan, np.inf]))
    np.testing.assert_array_equal(got[:, 0], none[:, 0])
    assert np.all(got[:, 1] == 0) and np.all(got[rows:] == 0)
    assert np.all(np.isnan(got[:rows, 2:]))
