"""The chunk calls over a cache held in 8 bits, made by two threads at once, with a stream, a RoPE
specification, a cache and a workspace each: a thread gets what it gets alone, bit by bit."""
import threading

import numpy as np
import pytest

from oracle import chunk8
from tests.test_gpu_chunk import attn_problem, bf16, dev, dl, geom, rope_spec  # noqa: F401

pytestmark = pytest.mark.gpu


def test_calls_from_two_threads(dl):  # noqa: F811
    import torch

    def problem(seed, hd, layout, scaling, block, n, ctx):
        rng = np.random.default_rng(seed)
        kw = dict(hq=8, nkv=2, hd=hd, P=32)
        pb = attn_problem(rng, n, ctx, **kw)
        g = geom(dl, M=pb["M"], NP=pb["NP"], **kw)
        N, sp = pb["q"].shape[0], rope_spec(dl, layout, hd, scaling, 4.0)
        q = bf16(rng.standard_normal((N, 8 * hd)))[0]
        k, v = (bf16(rng.standard_normal((N, 2 * hd)))[0] for _ in "kv")
        at = np.concatenate([np.arange(c, c + x) for x, c in zip(n, ctx)])
        req = np.repeat(np.arange(len(n)), n)
        pos, page, slot = (dev(a.astype(np.int32)) for a in (at, pb["table"][req, at // 32], at % 32))
        cache = chunk8.quantise(pb["pool"], block)
        ints = [dev(pb[x]) for x in ("table", "cu", "ctx", "kv")]
        ws = torch.empty(dl.dflash_chunk_attention8_workspace_bytes(g, len(n), N, 3),
                         dtype=torch.uint8, device="cuda")

        def new():
            zeros = [torch.zeros((N, h, hd), dtype=torch.bfloat16, device="cuda") for h in (8, 8, 2, 2)]
            return zeros + [dev(cache[0]), dev(cache[1])]

        def layer(out, stream):
            turned, o, k_back, v_back, codes, scales = out
            dl.dflash_chunk_rope_store8(g, 0, sp, q, k, v, pos, page, slot, turned, codes, scales,
                                        block, stream=stream)
            dl.dflash_chunk_attention8(g, 0, turned, codes, scales, block, *ints, o, ws,
                                       num_segments=3, stream=stream)
            dl.dflash_chunk_read8(g, 0, codes, scales, block, page, slot, k_back, v_back,
                                  stream=stream)
        return new, layer

    work = [problem(1, 128, "half", "plain", 16, [1, 1, 3], [700, 30, 64]),
            problem(2, 64, "pairs", "yarn", 32, [3, 1, 90], [300, 900, 0])]
    streams, want, got = [torch.cuda.Stream() for _ in work], [], []
    for (new, layer), s in zip(work, streams):
        want.append(new())
        torch.cuda.synchronize()
        layer(want[-1], s)
        torch.cuda.synchronize()
    times = 100
    got = [[new() for _ in range(times)] for new, _ in work]
    torch.cuda.synchronize()
    ready, failed = threading.Barrier(2), []

    def caller(i):
        try:
            ready.wait()
            for out in got[i]:
                work[i][1](out, streams[i])
        except Exception as e:  # told below: the other thread is to end too
            failed.append(e)

    threads = [threading.Thread(target=caller, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for outs, w in zip(got, want):
        for out in outs:
            for a, b in zip(out, w):
                assert torch.equal(a, b)
