"""dflash_chunk_attention called with offsets that make no sense: what it may not touch.
Rows behind the last request and columns behind the heads stay as they were, the bytes
behind the workspace too, rows that only requests without a place claim as well; a row of a
request whose own offsets are right holds its result or, since offsets are what
places the work, nothing new."""
import numpy as np
import pytest

from tests.gpu_helpers import bf16_f64, bits
from tests.test_gpu_chunk import attn_problem, bf16, dev, dl, geom  # noqa: F401

pytestmark = pytest.mark.gpu

PAD_ROWS, PAD_COLS, GUARD = 4, 32, 4096


def run(dl, pb, cu, *, S, hq, nkv, hd, P):  # noqa: F811
    """(rows, flags) with every guard checked."""
    import torch
    N, B = pb["q"].shape[0], len(pb["ctx"])
    rows, W = N + PAD_ROWS, hq * hd
    g = geom(dl, hq=hq, nkv=nkv, hd=hd, P=P, M=pb["M"], NP=pb["NP"])
    q = torch.zeros((rows, W), dtype=torch.bfloat16, device="cuda")
    q[:N] = bf16(pb["q"])[0].flatten(1)
    full = torch.full((rows, W + PAD_COLS), 7.0, dtype=torch.bfloat16, device="cuda")
    need = dl.dflash_chunk_attention_workspace_bytes(g, B, rows, S)
    ws = torch.full((need + GUARD,), 165, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dl.dflash_chunk_attention(g, 0, q.view(rows, hq, hd), bf16(pb["pool"])[0], dev(pb["table"]),
                              dev(cu.astype(np.int32)), dev(pb["ctx"]), dev(pb["kv"]),
                              full[:, :W].unflatten(1, (hq, hd)), ws[:need] if need else None,
                              num_segments=S, dev_status=st)
    torch.cuda.synchronize()
    assert torch.all(full[:, W:] == 7.0)
    assert torch.all(ws[need:] == 165)
    return bf16_f64(bits(full[:, :W])).reshape(rows, W), int(st.item())


def offsets(kind, cu, rng):
    """The offsets of one request or of many in the wrong place."""
    bad, B = cu.astype(np.int64).copy(), len(cu) - 1
    i = int(rng.integers(1, B))
    if kind == "past_the_rows":
        bad[i] = cu[B] + PAD_ROWS + 1
    elif kind == "far_past":
        bad[i] = 2 ** 31 - 1
    elif kind == "negative":
        bad[i] = -1 - int(rng.integers(0, 2 ** 30))
    elif kind == "back":
        bad[i] = cu[i + 1] + 1
    elif kind == "reversed":
        bad = bad[::-1].copy()
    elif kind == "last":
        bad[B] = cu[B] + PAD_ROWS + 7
    return bad


@pytest.mark.parametrize("S", [1, 3])
@pytest.mark.parametrize("B", [2, 31, 70, 300])
@pytest.mark.parametrize("kind", ["past_the_rows", "far_past", "negative", "back", "reversed",
                                  "last"])
def test_offsets_out_of_order(dl, kind, B, S):  # noqa: F811
    rng = np.random.default_rng(B)
    kw = dict(hq=24, nkv=12, hd=64, P=16)
    n = [int(x) for x in rng.integers(1, 4, B)]
    n[B // 2] = 90
    pb = attn_problem(rng, n, [int(x) for x in rng.integers(0, 200, B)], **kw)
    cu, N = pb["cu"], pb["q"].shape[0]
    right, flags = run(dl, pb, cu, S=S, **kw)
    assert flags == 0 and np.all(right[N:] == 7.0) and not np.any(np.all(right[:N] == 7.0, 1))
    bad = offsets(kind, cu, rng)
    got, flags = run(dl, pb, bad, S=S, **kw)
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
