"""dflash_chunk_attention8 against its definition where the other tests compare calls with each other
or look at less: more requests than are sorted, in the kernel of few rows; values that are zero for
most keys; V's largest scale; pages of other sizes."""
import numpy as np
import pytest

from oracle import chunk, chunk8
from tests.test_gpu_chunk import ATTN_TOL, attn_problem, bf16, dl  # noqa: F401
from tests.test_gpu_chunk8 import run_attn8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,G,S", [(1, 4, 1), (1, 4, 3), (4, 8, 1)])
def test_more_requests_than_are_sorted(dl, rows, G, S):  # noqa: F811
    rng = np.random.default_rng(70)
    B, kw = 300, dict(hq=4 * G, nkv=4, hd=128, P=32)
    n = [int(x) for x in rng.choice([0, rows, rows], B)]
    n[1], n[2], n[7] = rows, rows, rows + 20
    pb = attn_problem(rng, n, [int(x) for x in rng.integers(0, 600, B)], **kw)
    pb["kv"][2] = 0
    cache, sinks = chunk8.quantise(pb["pool"], 32), rng.standard_normal(4 * G).astype(np.float32)
    got = run_attn8(dl, pb, **kw, block=32, S=S, window=300, sinks=sinks, check=False, cache=cache)
    values, q = chunk8.values(cache[0][0], cache[1][0], 32), bf16(pb["q"])[1]
    for h in (0, 2 * G + 1, 4 * G - 1):  # a head of each request
        want, size = chunk.chunk_attention(
            q[:, h:h + 1], values[:, :, h // G:h // G + 1], pb["table"], pb["cu"], pb["ctx"], pb["kv"],
            scale=128 ** -0.5, window=300, sinks=sinks[h:h + 1].astype(np.float64))
        assert np.all(np.abs(got[:, h:h + 1] - want) <= ATTN_TOL * size + 1e-30)


@pytest.mark.parametrize("S", [1, 2])
@pytest.mark.parametrize("rows,G,hd", [(1, 4, 128), (10, 4, 128), (90, 2, 128), (3, 4, 64), (150, 2, 64)])
def test_values_of_zero_but_for_a_few(dl, rows, G, hd, S):  # noqa: F811
    """V is zero, and its scales the smallest, in all blocks but one: the weights of the others count
    in the sum."""
    rng = np.random.default_rng(71)
    kw = dict(hq=G, nkv=1, hd=hd, P=32)
    pb = attn_problem(rng, [rows], [400], **kw)
    have = -(-(400 + rows) // 32)
    for left in (0, 5, 12):
        one = dict(pb, pool=pb["pool"].copy())
        one["pool"][0, pb["table"][0, [b for b in range(have - 1) if b != left]], 1] = 0
        run_attn8(dl, one, **kw, block=32, S=S)


@pytest.mark.parametrize("rows,G,hd", [(1, 4, 128), (10, 4, 128), (90, 4, 128), (90, 2, 64)])
def test_largest_scale_of_values(dl, rows, G, hd):  # noqa: F811
    """2^120, the largest that the store writes, with codes up to 2^-3: no sum passes fp32."""
    rng = np.random.default_rng(72)
    kw = dict(hq=G, nkv=1, hd=hd, P=32)
    pb = attn_problem(rng, [rows], [300], **kw)
    codes, scales = chunk8.quantise(pb["pool"], 32)
    codes[:, :, 1] = np.minimum(codes[:, :, 1] & 0x7f, 0x20) | (codes[:, :, 1] & 0x80)
    scales[:, :, 1] = 247
    for S in (1, 3):
        run_attn8(dl, pb, **kw, block=32, S=S, cache=(codes, scales))


@pytest.mark.parametrize("P,block", [(384, 64), (640, 16), (32, 16)])
@pytest.mark.parametrize("rows,G,hd", [(1, 4, 128), (40, 4, 128), (20, 2, 64)])
def test_pages_of_other_sizes(dl, rows, G, hd, P, block):  # noqa: F811
    rng = np.random.default_rng(73)
    kw = dict(hq=2 * G, nkv=2, hd=hd, P=P)
    pb = attn_problem(rng, [rows, rows, 0, 2], [700, 383, 5, 0], **kw)
    run_attn8(dl, pb, **kw, block=block)
    run_attn8(dl, pb, **kw, block=block, S=2, window=100, causal=False)
