"""dflash_chunk_attention8 called with offsets that make no sense, as test_gpu_chunk_guards.py calls the
16-bit one: rows and columns that nobody owns stay as they were, the bytes behind the workspace too,
and a request whose own offsets are right has its result or nothing new."""
import numpy as np
import pytest

from oracle import chunk8
from tests.gpu_helpers import bf16_f64, bits
from tests.test_gpu_chunk import attn_problem, bf16, dev, dl, geom  # noqa: F401
from tests.test_gpu_chunk_guards import GUARD, PAD_COLS, PAD_ROWS, offsets

pytestmark = pytest.mark.gpu


def run(dl, pb, cache, cu, *, S, hq, nkv, hd, P):  # noqa: F811
    """(rows, flags) with every guard checked."""
    import torch
    N, B = pb["q"].shape[0], len(pb["ctx"])
    rows, W = N + PAD_ROWS, hq * hd
    g = geom(dl, hq=hq, nkv=nkv, hd=hd, P=P, M=pb["M"], NP=pb["NP"])
    q = torch.zeros((rows, W), dtype=torch.bfloat16, device="cuda")
    q[:N] = bf16(pb["q"])[0].flatten(1)
    full = torch.full((rows, W + PAD_COLS), 7.0, dtype=torch.bfloat16, device="cuda")
    need = dl.dflash_chunk_attention8_workspace_bytes(g, B, rows, S)
    ws = torch.full((need + GUARD,), 165, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dl.dflash_chunk_attention8(g, 0, q.view(rows, hq, hd), *map(dev, cache), 16, dev(pb["table"]),
                               dev(cu.astype(np.int32)), dev(pb["ctx"]), dev(pb["kv"]),
                               full[:, :W].unflatten(1, (hq, hd)), ws[:need] if need else None,
                               num_segments=S, dev_status=st)
    torch.cuda.synchronize()
    assert torch.all(full[:, W:] == 7.0)
    assert torch.all(ws[need:] == 165)
    return bf16_f64(bits(full[:, :W])).reshape(rows, W), int(st.item())


@pytest.mark.parametrize("S", [1, 3])
@pytest.mark.parametrize("B,hd,G", [(2, 128, 2), (31, 128, 1), (70, 128, 4), (300, 128, 8), (70, 64, 2)])
@pytest.mark.parametrize("kind", ["past_the_rows", "far_past", "negative", "back", "reversed", "last"])
def test_offsets_out_of_order(dl, kind, B, hd, G, S):  # noqa: F811
    rng = np.random.default_rng(B)
    kw = dict(hq=3 * G, nkv=3, hd=hd, P=16)
    n = [int(x) for x in rng.integers(1, 4, B)]
    n[B // 2] = 9 if hd == 128 else 90
    pb = attn_problem(rng, n, [int(x) for x in rng.integers(0, 200, B)], **kw)
    cache, cu, N = chunk8.quantise(pb["pool"], 16), pb["cu"], pb["q"].shape[0]
    right, flags = run(dl, pb, cache, cu, S=S, **kw)
    assert flags == 0 and np.all(right[N:] == 7.0) and not np.any(np.all(right[:N] == 7.0, 1))
    bad = offsets(kind, cu, rng)
    got, flags = run(dl, pb, cache, bad, S=S, **kw)
    assert flags == dl._lib.DEV_BAD_ROWS
    owners, known = np.zeros(N + PAD_ROWS, int), np.zeros(N + PAD_ROWS, bool)
    for r in range(B):
        a, b = int(bad[r]), int(bad[r + 1])
        if 0 <= a <= b <= N + PAD_ROWS:
            owners[a:b] += 1
            known[a:b] |= (a, b) == (cu[r], cu[r + 1])
    assert np.all(got[owners == 0] == 7.0)
    one = (owners == 1) & known
    as_ever = np.all(got == right, 1)
    assert np.all(as_ever[one] | np.all(got == 7.0, 1)[one])
    if kind == "last":     # the last request's alone: all others as ever
        assert np.all(as_ever[:cu[B - 1]])
