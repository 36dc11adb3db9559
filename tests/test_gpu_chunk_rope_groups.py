"""dflash_chunk_rope_store where a CTA goes through several groups of rows: both
shared-memory stages filled, freed and filled again, the last group partial, groups of
8, 4, 2 and 1 rows, and rows that do not turn, are not stored or lie outside the
pool in groups that are not a CTA's first.

Tolerances as in test_gpu_chunk.py: one rounding to bf16 (2^-8 of the value) and
fp32 arithmetic below 1e-5 of the magnitudes an output is formed from."""
import numpy as np
import pytest

from oracle import chunk
from tests.gpu_helpers import bf16_f64, bits
from tests.test_gpu_chunk import bf16, dev, dl, geom, rope_spec  # noqa: F401

pytestmark = pytest.mark.gpu

SMEM = 208 * 1024   # of a CTA's two stages, half of it where two CTAs share an SM


def rows_of_a_group(rows, row_bytes, sms):
    """The launcher's choice, so that a case here can say what it covers."""
    n = 1
    while n < 8 and rows > 2 * sms * n and 4 * n * row_bytes <= SMEM // 2:
        n *= 2
    return n


def check(dl, *, rows, hq, nkv, hd, rot, layout, gamma, in_place, packed, scaling="plain",  # noqa: F811
          factor=1.0, P=16, seed=0):
    import torch
    rng = np.random.default_rng(seed)
    NP = -(-rows // P) + 3
    g = geom(dl, hq=hq, nkv=nkv, hd=hd, P=P, NP=NP, theta=1e4)
    W, pad = (hq + 2 * nkv) * hd, 8
    qkv, x = bf16(rng.standard_normal((rows, W + pad), np.float32))
    x = x[:, :W].reshape(rows, hq + 2 * nkv, hd)
    pos = rng.integers(0, 1 << 17, rows).astype(np.int32)
    place = rng.permutation(NP * P)[:rows]
    page, slot = (place // P).astype(np.int32), (place % P).astype(np.int32)
    pos[3::17] = -1                        # rows of no request, in every group of some CTA
    page[5::23], slot[5::23] = -1, -1      # not placed
    page[7::101] = NP                      # outside the pool
    slot[9::103] = P
    gq, gqv = bf16(1 + 0.1 * rng.standard_normal(hd))
    gk, gkv = bf16(1 + 0.1 * rng.standard_normal(hd))
    pool, poolv = bf16(rng.standard_normal((1, NP, 2, nkv, P, hd), np.float32))
    q, k, v = qkv[:, :hq * hd], qkv[:, hq * hd:(hq + nkv) * hd], qkv[:, (hq + nkv) * hd:W]
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    q_out = q if in_place else torch.full((rows, hq, hd), 7.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dl.dflash_chunk_rope_store(g, 0, rope_spec(dl, layout, rot, scaling, factor), q, k, v,
                               dev(pos), dev(page), dev(slot), q_out, pool,
                               gamma_q=gq if gamma else None, gamma_k=gk if gamma else None,
                               dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == dl._lib.DEV_BAD_PAGE
    if packed and not in_place:            # the inputs are as they were
        np.testing.assert_array_equal(bf16_f64(bits(qkv)).reshape(rows, -1)[:, :W],
                                      x.reshape(rows, W))
    ang, mag = chunk.rope_angles(rot, 1e4, scaling, factor, 64)
    kw = dict(layout=layout, rot=rot, angles=ang, mag=mag)
    here = pos >= 0
    y, size = chunk.turn(x[:, :hq], gqv if gamma else None, pos, 1e-6, **kw)
    got = bf16_f64(bits(q_out)).reshape(rows, hq, hd)
    assert np.all((np.abs(got - y) <= 2.0 ** -8 * np.abs(y) + 1e-5 * size)[here])
    left = x[:, :hq] if in_place else np.full_like(y, 7.0)
    np.testing.assert_array_equal(got[~here], left[~here])
    y, size = chunk.turn(x[:, hq:hq + nkv], gkv if gamma else None, pos, 1e-6, **kw)
    kept = here & (page >= 0) & (page < NP) & (slot >= 0) & (slot < P)
    want, slack = poolv[0], np.zeros(poolv.shape[1:])
    at, on = page[kept], slot[kept]
    want[at, 0, :, on] = y[kept]
    slack[at, 0, :, on] = (2.0 ** -8 * np.abs(y) + 1e-5 * size)[kept]
    want[at, 1, :, on] = x[kept, hq + nkv:]
    got = bf16_f64(bits(pool)).reshape(want.shape)
    assert np.all(np.abs(got - want) <= slack)


def sm_count():
    import torch
    return torch.cuda.get_device_properties(0).multi_processor_count


# rows of a group, heads: more groups than three for every CTA, the last one partial
CASES = [(8, 2, 1, 64), (4, 24, 4, 128), (2, 40, 8, 128), (1, 96, 8, 128)]


@pytest.mark.parametrize("group,hq,nkv,hd", CASES)
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("in_place,packed", [(False, True), (True, True), (False, False)])
def test_rope_groups(dl, group, hq, nkv, hd, layout, in_place, packed):  # noqa: F811
    sms = sm_count()
    rows = 3 * 2 * sms * group + group * 5 + group // 2 + 1
    rows -= rows % group == 0 and group > 1
    assert rows_of_a_group(rows, 2 * hd * (hq + 2 * nkv), sms) == group
    check(dl, rows=rows, hq=hq, nkv=nkv, hd=hd, rot=hd, layout=layout, gamma=True,
          in_place=in_place, packed=packed, seed=group)


@pytest.mark.parametrize("layout,hd,rot,gamma", [
    ("half", 64, 24, False), ("pairs", 64, 4, True), ("half", 128, 32, True),
    ("pairs", 128, 24, False), ("half", 96, 80, True)])
def test_rope_groups_widths(dl, layout, hd, rot, gamma):  # noqa: F811
    """Chunks of 8 and of 4 values, heads partly turned, with and without norms."""
    check(dl, rows=3 * 2 * 8 * sm_count() + 61, hq=3, nkv=1, hd=hd, rot=rot, layout=layout,
          gamma=gamma, in_place=False, packed=True, scaling="yarn", factor=4.0, seed=rot)


def test_rope_one_cta_an_sm(dl):  # noqa: F811
    """Rows so wide that two stages fill an SM's shared memory: the second half of
    the CTAs begins when the first has ended."""
    check(dl, rows=2 * sm_count() * 2 + 7, hq=220, nkv=4, hd=128, rot=64, layout="half",
          gamma=True, in_place=True, packed=True, seed=3)


def test_rope_rows_wider_than_shared_memory(dl):  # noqa: F811
    for layout in ("half", "pairs"):
        check(dl, rows=21, hq=420, nkv=2, hd=128, rot=128, layout=layout, gamma=True,
              in_place=True, packed=True, seed=4)


@pytest.mark.parametrize("group", [0, 1, 3])
def test_unloaded_group_times_out_cleanly(dl, group):  # noqa: F811
    """The bounded waits: one group of rows is not loaded, the CTAs wind down with
    their copies landed, the status is set, and the next call is right."""
    import torch
    rows = 8 * 2 * sm_count() * 5 + 3
    g = geom(dl, hq=2, nkv=1, hd=64, P=16, NP=4)
    q, _ = bf16(np.ones((rows, 128), np.float32))
    pos, out = dev(np.zeros(rows, np.int32)), torch.empty_like(q)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda: dl.dflash_chunk_rope_store(  # noqa: E731
        g, 0, rope_spec(dl, "half", 64), q, None, None, pos, None, None, out, None, dev_status=st)
    dl.dflash_test_attention_skip_tile(group)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        dl.dflash_test_attention_skip_tile(-1)
    assert int(st.item()) == dl._lib.DEV_WAIT_TIMEOUT
    st.zero_()
    out.zero_()
    call()
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and torch.equal(out, q)
