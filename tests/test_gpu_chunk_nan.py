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
