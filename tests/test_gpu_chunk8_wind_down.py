"""dflash_chunk_attention8 with few rows: waits that run out while a block has more works to take."""
import numpy as np
import pytest

from tests.test_gpu_chunk import attn_problem, dl  # noqa: F401
from tests.test_gpu_chunk8 import run_attn8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,tile", [(1, 0), (1, 5), (8, 1)])
def test_works_after_an_unloaded_tile(dl, rows, tile):  # noqa: F811
    """Each block goes through works of one to eight key tiles, the given one of which stays
    unloaded: it ends with its status set, and the next call is right."""
    rng = np.random.default_rng(60)
    kw = dict(hq=32, nkv=8, hd=128, P=64)
    ctx = [int(x) for x in rng.integers(0, 1000, 24)]
    ctx[0] = 1000
    pb = attn_problem(rng, [rows] * 24, ctx, **kw)
    dl.dflash_test_attention_skip_tile(tile)
    try:
        run_attn8(dl, pb, **kw, S=1, check=False, flags=dl._lib.DEV_WAIT_TIMEOUT)
    finally:
        dl.dflash_test_attention_skip_tile(-1)
    some = [0, 1, 17, 23]  # compared, in a call of their own, too
    few = dict(pb, ctx=pb["ctx"][some], kv=pb["kv"][some], table=pb["table"][some],
               cu=np.arange(len(some) + 1, dtype=np.int32) * rows,
               q=np.concatenate([pb["q"][rows * r:rows * r + rows] for r in some]))
    got = run_attn8(dl, pb, **kw, S=1, check=False)
    want = run_attn8(dl, few, **kw, S=1)
    np.testing.assert_array_equal(np.concatenate([got[rows * r:rows * r + rows] for r in some]), want)
