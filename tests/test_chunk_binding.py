"""What the Python binding of the ragged-chunk calls turns away (CPU only): tensors of
another type, with gaps between their values, shorter than the call reads or writes
them, or on more than one device.  A kernel would read or write past them, or take
their bytes for something else."""
import pytest


@pytest.fixture(scope="module")
def dl():
    from context_kv_update_gb300 import build
    build.build()
    import context_kv_update_gb300 as dl
    dl.load()
    return dl


B, R, M, HQ, NKV, HD, P, NP, L = 3, 5, 8, 4, 2, 64, 16, 32, 2


def geom(dl):
    return dl.make_geom(dict(kind="gqa", L=L, D_in=64, D=64, hq=HQ, nkv=NKV, hd=HD, P=P, T=1,
                             max_pages=M, num_pool_pages=NP, rope_theta=1e4, eps_h=1e-6,
                             eps_k=1e-6))


def ints(n):
    import torch
    return torch.zeros(n, dtype=torch.int32)


def half(*shape):
    import torch
    return torch.zeros(shape, dtype=torch.bfloat16)


def plan_args(dl):
    import torch
    a = dict(n_new=ints(B), ctx_len=ints(B), n_pages=ints(B), block_table=ints(B * M).view(B, M),
             free_pages=ints(6), free_range=ints(2), valid=torch.ones(B, dtype=torch.uint8),
             dev_status=ints(1))
    out = {k: ints({"cu_rows": B + 1, "free_head": 1}.get(k, R if k.startswith("row_") else B))
           for k in dl.CHUNK_OUTPUT_FIELDS}
    return {**a, **{"out." + k: v for k, v in out.items()}}


def plan(dl, a):
    out = {k[4:]: v for k, v in a.items() if k.startswith("out.")}
    dl.dflash_chunk_plan(geom(dl), a["n_new"], a["ctx_len"], a["n_pages"], a["block_table"],
                         a["free_pages"], a["free_range"], a["valid"], 100, out, a["dev_status"])


def rope_args(dl):
    return dict(q=half(R, HQ * HD), k=half(R, NKV * HD), v=half(R, NKV * HD), row_pos=ints(R),
                row_page=ints(R), row_slot=ints(R), q_out=half(R, HQ, HD),
                kv_pool=half(L, NP, 2, NKV, P, HD), gamma_q=half(HD), gamma_k=half(HD),
                dev_status=ints(1))


def rope(dl, a):
    dl.dflash_chunk_rope_store(geom(dl), 0, dl.RopeSpec(rot_dim=HD), a["q"], a["k"], a["v"],
                               a["row_pos"], a["row_page"], a["row_slot"], a["q_out"],
                               a["kv_pool"], gamma_q=a["gamma_q"], gamma_k=a["gamma_k"],
                               dev_status=a["dev_status"])


def attn_args(dl):
    import torch
    return dict(q=half(R, HQ, HD), kv_pool=half(L, NP, 2, NKV, P, HD),
                block_table=ints(B * M).view(B, M), cu_rows=ints(B + 1), ctx_len=ints(B),
                kv_len=ints(B), out=half(R, HQ, HD),
                workspace=torch.zeros(1 << 16, dtype=torch.uint8),
                sinks=torch.zeros(HQ), dev_status=ints(1))


def attn(dl, a):
    dl.dflash_chunk_attention(geom(dl), 0, a["q"], a["kv_pool"], a["block_table"], a["cu_rows"],
                              a["ctx_len"], a["kv_len"], a["out"], a["workspace"],
                              sinks=a["sinks"], dev_status=a["dev_status"])


CALLS = {"plan": (plan, plan_args), "rope": (rope, rope_args), "attn": (attn, attn_args)}
# what sets a count has no length of its own to be short of
COUNTS = {("plan", "n_new"), ("plan", "free_pages"), ("plan", "out.row_req"), ("rope", "row_pos"),
          ("attn", "q"), ("attn", "kv_len"), ("attn", "workspace")}


def arguments():
    import context_kv_update_gb300 as dl
    return [(c, k) for c, (_, args) in CALLS.items() for k in args(dl)]


def spread(t):
    """The same values with a gap behind each."""
    import torch
    wide = torch.zeros((*t.shape, 2), dtype=t.dtype)
    return wide[..., 0]


@pytest.mark.parametrize("call,name", arguments())
def test_gaps_between_values(dl, call, name):
    f, args = CALLS[call]
    a = args(dl)
    if a[name].numel() == 1:
        pytest.skip("one value has no gaps")
    a[name] = spread(a[name])
    assert not a[name].is_contiguous()
    with pytest.raises(AssertionError, match=name.replace("out.", "")):
        f(dl, a)


@pytest.mark.parametrize("call,name", arguments())
def test_types(dl, call, name):
    import torch
    f, args = CALLS[call]
    a = args(dl)
    if name == "workspace":
        pytest.skip("scratch of any type")
    for t in (torch.int64, torch.float16, torch.float64):
        a[name] = args(dl)[name].to(t)
        with pytest.raises(TypeError, match=name.replace("out.", "")):
            f(dl, a)
    a[name] = [0, 1, 2]
    with pytest.raises(TypeError, match=name.replace("out.", "")):
        f(dl, a)


@pytest.mark.parametrize("call,name", arguments())
def test_too_short(dl, call, name):
    f, args = CALLS[call]
    if (call, name) in COUNTS:
        pytest.skip("sets the count")
    a = args(dl)
    a[name] = a[name][:-1]
    with pytest.raises(ValueError, match=name.replace("out.", "")):
        f(dl, a)


@pytest.mark.parametrize("call,name,width", [
    ("rope", "q", HQ), ("rope", "k", NKV), ("rope", "v", NKV), ("rope", "q_out", HQ),
    ("attn", "q", HQ), ("attn", "out", HQ)])
def test_rows_too_narrow(dl, call, name, width):
    """Rows of fewer heads than the geometry has, with or without other columns behind
    them: a row stride that is wide enough says nothing about the last row."""
    f, args = CALLS[call]
    for t in (half(R, width - 1, HD), half(R, width, HD)[:, :-1],
              half(R, 4 * HQ * HD)[:, :width * HD - 8]):
        a = args(dl)
        a[name] = t
        with pytest.raises(ValueError, match=name):
            f(dl, a)


@pytest.mark.parametrize("call", CALLS)
def test_devices(dl, call):
    """All on one device, and that the current CUDA device."""
    f, args = CALLS[call]
    with pytest.raises(ValueError, match="device"):
        f(dl, args(dl))
    for name in args(dl):
        a = args(dl)
        a[name] = a[name].to("meta")
        with pytest.raises(ValueError, match="device"):
            f(dl, a)


@pytest.mark.parametrize("call", CALLS)
def test_structures(dl, call):
    """A structure of another size in the place of the geometry, or of the RoPE
    specification."""
    import context_kv_update_gb300 as pkg
    f, args = CALLS[call]
    real = geom
    try:
        globals()["geom"] = lambda dl: pkg.RopeSpec()
        with pytest.raises(TypeError):
            f(dl, args(dl))
    finally:
        globals()["geom"] = real
