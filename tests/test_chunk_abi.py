"""What the ragged-chunk calls refuse, before touching a GPU (CPU only)."""
import ctypes

import pytest

P16 = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10002)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from context_kv_update_gb300 import build, _lib
    build.build()
    return _lib.load()


def _geom(**over):
    from context_kv_update_gb300 import make_geom
    g = dict(kind="gqa", L=2, D_in=64, D=64, hq=4, nkv=2, hd=64, P=16, T=1, max_pages=8,
             num_pool_pages=32, rope_theta=1e4, eps_h=1e-6, eps_k=1e-6)
    g.update(over)
    return make_geom(g)


def _plan(lib, B=2, n_rows=6, n_free=4, max_ctx=100, g=None, drop=None, alias=None, valid=None):
    """Every pointer distinct and far apart unless named; never reaches a launch
    in these tests."""
    from context_kv_update_gb300 import _lib
    o = {k: 0x1000000 * (i + 1) for i, k in enumerate(_lib.CHUNK_OUTPUT_FIELDS)}
    a = {k: 0x100000 * (i + 1) for i, k in enumerate(
        ("n_new", "ctx_len", "n_pages", "block_table", "free_pages", "free_range"))}
    for k in (drop or ()):
        (o if k.startswith("out_") else a)[k.replace("out_", "")] = None
    for k, v in (alias or {}).items():
        o[k] = a[v]
    out = _lib.ChunkOutputs(*[o[k] for k in _lib.CHUNK_OUTPUT_FIELDS])
    g = g or _geom()
    return lib.dflash_chunk_plan(ctypes.byref(g), B, n_rows, a["n_new"], a["ctx_len"],
                                 a["n_pages"], a["block_table"], a["free_pages"], n_free,
                                 a["free_range"], valid, max_ctx, ctypes.byref(out), None, None)


def test_struct_sizes(lib):
    from context_kv_update_gb300 import _lib
    assert ctypes.sizeof(_lib.ChunkOutputs) == 9 * 8
    assert ctypes.sizeof(_lib.RopeSpec) == 4 * 4 + 4 * 8


def test_plan_refusals(lib):
    from context_kv_update_gb300 import _lib
    bad, geo = _lib.DFLASH_ERR_INVALID_ARG, _lib.DFLASH_ERR_UNSUPPORTED_GEOM
    assert lib.dflash_chunk_plan(None, 1, 1, *[P16] * 5, 1, P16, None, 1, None, None, None) == bad
    for kw in (dict(B=-1), dict(n_rows=-1), dict(n_free=-1), dict(max_ctx=-1)):
        assert _plan(lib, **kw) == bad, kw
    for k in ("n_new", "ctx_len", "n_pages", "block_table", "free_pages", "free_range",
              "out_cu_rows", "out_n_pages", "out_alloc_limit", "out_seq_lens", "out_free_head",
              "out_row_req", "out_row_pos", "out_row_page", "out_row_slot"):
        assert _plan(lib, drop=[k]) == bad, k
    # an output in an input's memory: other threads still read it
    for o, i in (("n_pages", "n_pages"), ("free_head", "free_range"), ("seq_lens", "ctx_len"),
                 ("row_page", "free_pages")):
        assert _plan(lib, alias={o: i}) == bad, (o, i)
    assert _plan(lib, B=8193) == geo
    assert _plan(lib, n_rows=1 << 30) == geo
    assert _plan(lib, valid=0x1000000) == bad   # the memory of cu_rows
    assert _plan(lib, g=_geom(max_pages=1 << 27, P=16)) == geo


def _rope(lib, spec=None, n_rows=3, layer=0, g=None, q=P16, qs=256, k=P16, ks=128, v=P16, vs=128,
          gq=None, gk=None, pos=P16, page=P16, slot=P16, qo=P16, qos=256, pool=P16):
    from context_kv_update_gb300 import _lib
    g = g or _geom()
    s = dict(layout=0, rot_dim=64, scaling=0, trained_ctx=0, factor=1.0, beta_fast=32.0,
             beta_slow=1.0, magnitude=0.0)
    s.update(spec or {})
    return lib.dflash_chunk_rope_store(ctypes.byref(g), layer, n_rows,
                                       ctypes.byref(_lib.RopeSpec(**s)), q, qs, k, ks, v, vs, gq,
                                       gk, pos, page, slot, qo, qos, pool, None, None)


def test_rope_refusals(lib):
    from context_kv_update_gb300 import _lib
    bad, geo = _lib.DFLASH_ERR_INVALID_ARG, _lib.DFLASH_ERR_UNSUPPORTED_GEOM
    assert _rope(lib, n_rows=0, q=None, k=None, v=None, qo=None) == _lib.DFLASH_OK
    yarn = dict(scaling=2, trained_ctx=64, factor=2.0)
    for kw in (dict(n_rows=-1), dict(layer=2), dict(layer=-1), dict(spec=dict(layout=2)),
               dict(spec=dict(scaling=3)), dict(spec=dict(scaling=1, factor=0.5)),
               dict(spec=dict(scaling=1, factor=float("nan"))), dict(spec=dict(yarn, trained_ctx=0)),
               dict(spec=dict(yarn, beta_slow=0.0)), dict(spec=dict(yarn, beta_slow=64.0)),
               dict(spec=dict(yarn, beta_fast=float("inf"))),
               dict(spec=dict(yarn, magnitude=float("nan"))),
               dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(pool=None),
               dict(q=None, qo=None, k=None, v=None), dict(pos=None), dict(page=None),
               dict(slot=None), dict(q=ODD), dict(qo=ODD), dict(k=ODD), dict(v=ODD),
               dict(pool=ODD), dict(gq=ODD), dict(gk=ODD), dict(qs=255), dict(qs=260),
               dict(qos=248), dict(ks=120), dict(vs=132),
               dict(qs=512)):   # in place with another stride
        assert _rope(lib, **kw) == bad, kw
    for kw in (dict(spec=dict(rot_dim=0)), dict(spec=dict(rot_dim=7)), dict(spec=dict(rot_dim=66)),
               dict(g=_geom(hd=60)), dict(g=_geom(hd=264)), dict(g=_geom(kind="mla")),
               dict(spec=yarn, g=_geom(rope_theta=1.0)), dict(n_rows=1 << 30)):
        assert _rope(lib, **kw) == geo, kw


def _attn(lib, B=2, layer=0, n_rows=6, g=None, q=P16, qs=256, pool=P16, tbl=P16, cu=P16, ctx=P16,
          kv=P16, window=0, scale=0.0, mask=0, S=0, ws=P16, nb=BIG, out=P16, os=256):
    g = g or _geom()
    return lib.dflash_chunk_attention(ctypes.byref(g), B, layer, n_rows, q, qs, pool, tbl, cu, ctx,
                                      kv, window, None, scale, mask, S, ws, nb, out, os, None, None)


def test_attention_refusals(lib):
    from context_kv_update_gb300 import _lib
    bad, geo = _lib.DFLASH_ERR_INVALID_ARG, _lib.DFLASH_ERR_UNSUPPORTED_GEOM
    none = dict(q=None, pool=None, tbl=None, cu=None, ctx=None, kv=None, ws=None, out=None)
    assert _attn(lib, B=0, **none) == _lib.DFLASH_OK
    assert _attn(lib, n_rows=0, **none) == _lib.DFLASH_OK
    for kw in (dict(B=-1), dict(n_rows=-1), dict(layer=2), dict(layer=-1), dict(window=-1),
               dict(mask=2), dict(S=-1), dict(scale=float("inf")), dict(scale=float("nan")),
               dict(q=None), dict(pool=None), dict(tbl=None), dict(cu=None), dict(ctx=None),
               dict(kv=None), dict(out=None), dict(q=ODD), dict(out=ODD), dict(pool=ODD),
               dict(qs=248), dict(qs=260), dict(os=0), dict(os=257), dict(S=65536), dict(S=3, ws=None),
               dict(S=3, ws=ODD)):
        assert _attn(lib, **kw) == bad, kw
    assert _attn(lib, S=3, nb=64) == _lib.DFLASH_ERR_WORKSPACE_TOO_SMALL
    for kw in (dict(g=_geom(kind="mla")), dict(g=_geom(hd=96)), dict(g=_geom(P=12)),
               dict(g=_geom(P=48)), dict(g=_geom(P=192)), dict(g=_geom(num_pool_pages=1 << 25)),
               dict(g=_geom(max_pages=(1 << 27) - 15)), dict(n_rows=1 << 29), dict(B=1 << 29)):
        assert _attn(lib, **kw) == geo, kw


def test_attention_workspace(lib):
    g = _geom()
    G = ctypes.byref(g)
    ws = lib.dflash_chunk_attention_workspace_bytes
    assert ws(G, 2, 6, 1) == 0            # one segment writes out directly
    assert ws(G, 2, 6, 3) >= 3 * 6 * 4 * (64 + 2) * 4
    assert ws(G, 2, 6, -1) == ws(None, 2, 6, 3) == 0
    assert lib.dflash_chunk_attention_num_segments(G, 2, 6) >= 1
    assert lib.dflash_chunk_attention_num_segments(G, 0, 6) == 0
    assert lib.dflash_chunk_attention_num_segments(None, 1, 6) == 0


def test_binding_refuses_what_it_cannot_pass_on(lib):
    """Arguments the marshalling itself turns away: tensors that are not on the
    current device (a CPU pointer would reach a kernel), views whose rows are not
    contiguous, structures of another type, counts past 32 bits."""
    import torch

    import context_kv_update_gb300 as dl
    from context_kv_update_gb300 import _lib
    g = _geom()
    i32 = torch.zeros(4, dtype=torch.int32)
    q = torch.zeros((4, 4, 64), dtype=torch.bfloat16)
    pool = torch.zeros((2, 32, 2, 2, 16, 64), dtype=torch.bfloat16)
    out = {k: i32 for k in dl.CHUNK_OUTPUT_FIELDS}
    tbl = torch.zeros((4, 8), dtype=torch.int32)
    spec = dl.RopeSpec(rot_dim=64)
    plan = lambda **kw: dl.dflash_chunk_plan(*[kw.get(k, d) for k, d in (  # noqa: E731
        ("g", g), ("n", i32), ("ctx", i32), ("have", i32), ("tbl", tbl), ("free", i32),
        ("range", i32), ("valid", None), ("max_ctx", 100), ("out", out))])
    rope = lambda **kw: dl.dflash_chunk_rope_store(  # noqa: E731
        kw.get("g", g), 0, kw.get("spec", spec), kw.get("q", q), None, None, i32, None, None, q,
        kw.get("pool"))
    attn = lambda **kw: dl.dflash_chunk_attention(  # noqa: E731
        g, kw.get("layer", 0), kw.get("q", q), pool, tbl, i32, i32, i32, q)
    # no CUDA device here, or tensors that are not on it
    for f in (plan, rope, attn):
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            f()
    for f, kw in ((plan, dict(tbl=tbl[:, ::2])), (rope, dict(q=q.transpose(0, 1))),
                  (rope, dict(q=q[:, ::2])), (rope, dict(pool=pool[:, :, :1])),
                  (attn, dict(q=q[:, :, ::2]))):
        with pytest.raises(AssertionError):
            f(**kw)
    with pytest.raises(KeyError):
        plan(out={})
    with pytest.raises(OverflowError):
        attn(layer=1 << 40)
    with pytest.raises(TypeError):
        _lib._calls.chunk_plan(g)
