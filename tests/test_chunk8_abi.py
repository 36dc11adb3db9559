"""What the chunk calls over a cache held in 8 bits refuse, before touching a GPU (CPU only):
by the C entry points, and by the Python binding, whose tensors must be of the right type, without
gaps, as long as the call reads or writes them, and on the current device."""
import ctypes

import pytest

P16 = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10002)
BIG = 1 << 40
B, R, M, HQ, NKV, HD, P, NP, L, BLOCK = 3, 5, 8, 4, 2, 64, 32, 32, 2, 16


@pytest.fixture(scope="module")
def lib():
    from context_kv_update_gb300 import build, _lib
    build.build()
    return _lib.load()


@pytest.fixture(scope="module")
def dl(lib):
    import context_kv_update_gb300 as dl
    return dl


def _geom(**over):
    from context_kv_update_gb300 import make_geom
    g = dict(kind="gqa", L=L, D_in=64, D=64, hq=HQ, nkv=NKV, hd=HD, P=P, T=1, max_pages=M,
             num_pool_pages=NP, rope_theta=1e4, eps_h=1e-6, eps_k=1e-6)
    g.update(over)
    return make_geom(g)


def _cache(codes=P16, scales=ODD, block=BLOCK):
    from context_kv_update_gb300 import Cache8
    return ctypes.byref(Cache8(codes=codes, scales=scales, block=block))


def _codes(lib):
    return lib.DFLASH_ERR_INVALID_ARG, lib.DFLASH_ERR_UNSUPPORTED_GEOM, lib.DFLASH_OK


def test_sizes(lib):
    from context_kv_update_gb300 import _lib
    assert ctypes.sizeof(_lib.Cache8) == 24
    g = _geom()
    assert lib.dflash_cache8_code_bytes(g) == 2 * L * NP * NKV * P * HD
    assert lib.dflash_cache8_scale_bytes(g, 16) == 2 * L * NP * NKV * (P // 16)
    for g, block in ((_geom(), 64), (_geom(), 8), (_geom(), 0), (_geom(), -16), (_geom(P=24), 16),
                     (_geom(kind="mla"), 16), (_geom(hd=72), 16), (_geom(hd=272), 16)):
        assert lib.dflash_cache8_scale_bytes(g, block) == 0
    assert lib.dflash_cache8_code_bytes(_geom(kind="mla")) == 0
    assert lib.dflash_cache8_code_bytes(None) == lib.dflash_cache8_scale_bytes(None, 16) == 0


def _store(lib, spec=None, n_rows=3, layer=0, g=None, q=P16, qs=256, k=P16, ks=128, v=P16, vs=128,
           gq=None, gk=None, pos=P16, page=P16, slot=P16, qo=P16, qos=256, rope=True, **cache):
    from context_kv_update_gb300 import _lib
    g = g or _geom()
    s = dict(layout=0, rot_dim=64, scaling=0, trained_ctx=0, factor=1.0, beta_fast=32.0,
             beta_slow=1.0, magnitude=0.0)
    s.update(spec or {})
    return lib.dflash_chunk_rope_store8(
        ctypes.byref(g), layer, n_rows, ctypes.byref(_lib.RopeSpec(**s)) if rope else None, q, qs, k,
        ks, v, vs, gq, gk, pos, page, slot, qo, qos, _cache(**cache), None, None)


def test_store_refusals(lib):
    from context_kv_update_gb300 import _lib
    bad, geo, ok = _codes(_lib)
    nothing = dict(n_rows=0, q=None, k=None, v=None, qo=None, codes=None, scales=None)
    assert _store(lib, **nothing) == _store(lib, rope=False, **nothing) == ok
    yarn = dict(scaling=2, trained_ctx=64, factor=2.0)
    for kw in (dict(n_rows=-1), dict(layer=2), dict(layer=-1), dict(spec=dict(layout=2)),
               dict(spec=dict(scaling=3)), dict(spec=dict(scaling=1, factor=0.5)),
               dict(spec=dict(yarn, trained_ctx=0)), dict(spec=dict(yarn, beta_slow=0.0)),
               dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(codes=None),
               dict(scales=None), dict(codes=ODD), dict(q=None, qo=None, k=None, v=None),
               dict(pos=None), dict(page=None), dict(slot=None), dict(q=ODD), dict(qo=ODD),
               dict(k=ODD), dict(v=ODD), dict(gq=ODD), dict(gk=ODD), dict(qs=255), dict(qs=260),
               dict(qos=248), dict(ks=120), dict(vs=132), dict(qs=512)):
        assert _store(lib, **kw) == bad, kw
        if "spec" not in kw:
            assert _store(lib, rope=False, **kw) == bad, kw
    for kw in (dict(spec=dict(rot_dim=0)), dict(spec=dict(rot_dim=66)), dict(g=_geom(hd=72)),
               dict(g=_geom(hd=272)), dict(g=_geom(kind="mla")), dict(n_rows=1 << 30),
               dict(block=8), dict(block=128), dict(block=0), dict(block=64), dict(block=-16),
               dict(g=_geom(P=24))):
        assert _store(lib, **kw) == geo, kw
    a = [None] * 4 + [0]
    assert lib.dflash_chunk_rope_store8(ctypes.byref(_geom()), 0, 0, None, None, 0, None, 0, None, 0,
                                        *a[:4], None, None, 0, None, None, None) == bad
    assert lib.dflash_chunk_rope_store8(None, 0, 0, None, None, 0, None, 0, None, 0, *a[:4], None,
                                        None, 0, _cache(), None, None) == bad


def _read(lib, n_rows=3, layer=0, g=None, page=P16, slot=P16, k=P16, ks=128, v=P16, vs=128, **cache):
    return lib.dflash_chunk_read8(ctypes.byref(g or _geom()), layer, n_rows, _cache(**cache), page,
                                  slot, k, ks, v, vs, None, None)


def test_read_refusals(lib):
    from context_kv_update_gb300 import _lib
    bad, geo, ok = _codes(_lib)
    assert _read(lib, n_rows=0, page=None, slot=None, k=None, v=None, codes=None) == ok
    for kw in (dict(n_rows=-1), dict(layer=-1), dict(layer=2), dict(page=None), dict(slot=None),
               dict(k=None, v=None), dict(k=ODD), dict(v=ODD), dict(ks=120), dict(vs=130),
               dict(codes=None), dict(codes=ODD), dict(scales=None)):
        assert _read(lib, **kw) == bad, kw
    for kw in (dict(block=48), dict(block=64), dict(g=_geom(hd=24)), dict(g=_geom(kind="mla")),
               dict(n_rows=1 << 30)):
        assert _read(lib, **kw) == geo, kw
    assert lib.dflash_chunk_read8(ctypes.byref(_geom()), 0, 1, None, P16, P16, P16, 128, P16, 128,
                                  None, None) == bad


def _attn(lib, B=2, layer=0, n_rows=6, g=None, q=P16, qs=256, tbl=P16, cu=P16, ctx=P16, kv=P16,
          window=0, scale=0.0, mask=0, S=0, ws=P16, nb=BIG, out=P16, os=256, **cache):
    return lib.dflash_chunk_attention8(ctypes.byref(g or _geom()), B, layer, n_rows, q, qs,
                                       _cache(**cache), tbl, cu, ctx, kv, window, None, scale,
                                       mask, S, ws, nb, out, os, None, None)


def test_attention_refusals(lib):
    from context_kv_update_gb300 import _lib
    bad, geo, ok = _codes(_lib)
    none = dict(q=None, codes=None, scales=None, tbl=None, cu=None, ctx=None, kv=None, ws=None,
                out=None)
    assert _attn(lib, B=0, **none) == _attn(lib, n_rows=0, **none) == ok
    for kw in (dict(B=-1), dict(n_rows=-1), dict(layer=2), dict(layer=-1), dict(window=-1),
               dict(mask=2), dict(S=-1), dict(scale=float("inf")), dict(scale=float("nan")),
               dict(q=None), dict(codes=None), dict(scales=None), dict(tbl=None), dict(cu=None),
               dict(ctx=None), dict(kv=None), dict(out=None), dict(q=ODD), dict(out=ODD),
               dict(codes=ODD), dict(qs=248), dict(qs=260), dict(os=0), dict(os=257),
               dict(S=65536)):
        assert _attn(lib, **kw) == bad, kw
    for kw in (dict(g=_geom(kind="mla")), dict(g=_geom(hd=96)), dict(g=_geom(P=48)),
               dict(g=_geom(P=192)), dict(g=_geom(P=8)), dict(g=_geom(num_pool_pages=1 << 24)),
               dict(g=_geom(max_pages=(1 << 26) - 7)), dict(n_rows=1 << 29), dict(B=1 << 29),
               dict(block=64), dict(block=24)):
        assert _attn(lib, **kw) == geo, kw
    assert lib.dflash_chunk_attention8(ctypes.byref(_geom()), 2, 0, 6, P16, 256, None, P16, P16, P16,
                                       P16, 0, None, 0.0, 0, 0, P16, BIG, P16, 256, None, None) == bad


def test_attention_workspace(lib):
    G = ctypes.byref(_geom())
    ws = lib.dflash_chunk_attention8_workspace_bytes
    assert ws(G, 2, 6, 1) == 0            # one segment writes out directly
    assert ws(G, 2, 6, -1) == ws(None, 2, 6, 3) == 0
    assert lib.dflash_chunk_attention8_num_segments(G, 2, 6) >= 1
    assert lib.dflash_chunk_attention8_num_segments(G, 0, 6) == 0
    assert lib.dflash_chunk_attention8_num_segments(None, 1, 6) == 0


# ------------------------------------------------------------------ the binding


def ints(n):
    import torch
    return torch.zeros(n, dtype=torch.int32)


def half(*shape):
    import torch
    return torch.zeros(shape, dtype=torch.bfloat16)


def cache_args():
    import torch
    return dict(codes=torch.zeros((L, NP, 2, NKV, P, HD), dtype=torch.uint8),
                scales=torch.zeros((L, NP, 2, NKV, P // BLOCK), dtype=torch.uint8))


def store_args():
    return dict(q=half(R, HQ * HD), k=half(R, NKV * HD), v=half(R, NKV * HD), row_pos=ints(R),
                row_page=ints(R), row_slot=ints(R), q_out=half(R, HQ, HD), **cache_args(),
                gamma_q=half(HD), gamma_k=half(HD), dev_status=ints(1))


def store(dl, a, block=BLOCK, rope=True):
    dl.dflash_chunk_rope_store8(_geom(), 0, dl.RopeSpec(rot_dim=HD) if rope else None, a["q"],
                                a["k"], a["v"], a["row_pos"], a["row_page"], a["row_slot"],
                                a["q_out"], a["codes"], a["scales"], block, gamma_q=a["gamma_q"],
                                gamma_k=a["gamma_k"], dev_status=a["dev_status"])


def read_args():
    return dict(**cache_args(), row_page=ints(R), row_slot=ints(R), k_out=half(R, NKV, HD),
                v_out=half(R, NKV, HD), dev_status=ints(1))


def read(dl, a, block=BLOCK):
    dl.dflash_chunk_read8(_geom(), 0, a["codes"], a["scales"], block, a["row_page"], a["row_slot"],
                          a["k_out"], a["v_out"], dev_status=a["dev_status"])


def attn_args():
    import torch
    return dict(q=half(R, HQ, HD), **cache_args(), block_table=ints(B * M).view(B, M),
                cu_rows=ints(B + 1), ctx_len=ints(B), kv_len=ints(B), out=half(R, HQ, HD),
                workspace=torch.zeros(1 << 16, dtype=torch.uint8), sinks=torch.zeros(HQ),
                dev_status=ints(1))


def attn(dl, a, block=BLOCK):
    dl.dflash_chunk_attention8(_geom(), 0, a["q"], a["codes"], a["scales"], block, a["block_table"],
                               a["cu_rows"], a["ctx_len"], a["kv_len"], a["out"], a["workspace"],
                               sinks=a["sinks"], dev_status=a["dev_status"])


CALLS = {"store": (store, store_args), "read": (read, read_args), "attn": (attn, attn_args)}
COUNTS = {("store", "row_pos"), ("read", "row_page"), ("attn", "q"), ("attn", "kv_len"),
          ("attn", "workspace")}
ARGUMENTS = [(c, k) for c, (_, args) in CALLS.items() for k in
             {"store": ("q", "k", "v", "row_pos", "row_page", "row_slot", "q_out", "codes", "scales",
                        "gamma_q", "gamma_k", "dev_status"),
              "read": ("codes", "scales", "row_page", "row_slot", "k_out", "v_out", "dev_status"),
              "attn": ("q", "codes", "scales", "block_table", "cu_rows", "ctx_len", "kv_len", "out",
                       "workspace", "sinks", "dev_status")}[c]]


@pytest.mark.parametrize("call,name", ARGUMENTS)
def test_binding_gaps_types_lengths(dl, call, name):
    import torch
    f, args = CALLS[call]
    a = args()
    if a[name].numel() > 1:
        a[name] = torch.zeros((*a[name].shape, 2), dtype=a[name].dtype)[..., 0]
        with pytest.raises(AssertionError, match=name):
            f(dl, a)
    if name != "workspace":
        for t in (torch.int64, torch.float16, torch.float64, torch.int8):
            a = args()
            a[name] = a[name].to(t)
            with pytest.raises(TypeError, match=name):
                f(dl, a)
        a[name] = [0, 1, 2]
        with pytest.raises(TypeError, match=name):
            f(dl, a)
    if (call, name) not in COUNTS:
        a = args()
        a[name] = a[name][:-1]
        with pytest.raises(ValueError, match=name):
            f(dl, a)


@pytest.mark.parametrize("call", CALLS)
def test_binding_devices_and_blocks(dl, call):
    """All on one device, and that the current CUDA device; a block that does not fit 32 bits."""
    import torch
    f, args = CALLS[call]
    with pytest.raises(ValueError, match="device"):
        f(dl, args())
    for name in args():
        a = args()
        a[name] = a[name].to("meta")
        with pytest.raises(ValueError, match="device"):
            f(dl, a)
    with pytest.raises(OverflowError):
        f(dl, args(), block=1 << 40)
    # the 8-bit types of torch are taken as what they are, each in its own place only
    a = args()
    a["codes"], a["scales"] = a["codes"].view(torch.float8_e4m3fn), a["scales"].view(torch.float8_e8m0fnu)
    with pytest.raises(ValueError, match="device"):
        f(dl, a)
    a["codes"] = a["codes"].view(torch.float8_e5m2)
    with pytest.raises(TypeError, match="codes"):
        f(dl, a)
    a["codes"], a["scales"] = a["scales"], a["codes"]
    with pytest.raises(TypeError, match="codes"):
        f(dl, a)
    if call == "store":
        with pytest.raises(ValueError, match="device"):
            store(dl, args(), rope=False)


def test_binding_smaller_blocks_need_more_scales(dl):
    a = cache_args()
    a = dict(read_args(), scales=a["scales"][..., :1].contiguous())
    with pytest.raises(ValueError, match="scales"):
        read(dl, a, block=16)
    with pytest.raises(ValueError, match="device"):
        read(dl, a, block=32)
