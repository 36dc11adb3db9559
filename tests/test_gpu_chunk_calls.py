"""The ragged-chunk calls as a program of several threads and streams makes them."""
import threading
import time

import numpy as np
import pytest

from tests.test_gpu_chunk import (attn_problem, bf16, dev, dl, geom, plan_case,  # noqa: F401
                                  plan_outputs, rope_spec)

pytestmark = pytest.mark.gpu


def test_other_threads_run_while_a_call_waits(dl):  # noqa: F811
    """A call that waits for room in the GPU's queue keeps no other Python thread
    from running: the work it waits for may need one."""
    import torch
    case, NP = plan_case(np.random.default_rng(0), 4, 16, 3, 40)
    g = geom(dl, P=16, M=case["table"].shape[1], NP=NP)
    a = [dev(case[k]) for k in ("n_new", "ctx", "have", "table", "free", "range")]
    out = plan_outputs(dl, 4, 12)
    dl.dflash_chunk_plan(g, *a, None, 1 << 20, out)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    start, took = threading.Event(), []

    def caller():
        start.wait()
        for _ in range(40):
            t0 = time.perf_counter()
            for _ in range(100):
                dl.dflash_chunk_plan(g, *a, None, 1 << 20, out, stream=s)
            took.append(time.perf_counter() - t0)

    t = threading.Thread(target=caller)
    t.start()
    with torch.cuda.stream(s):
        torch.cuda._sleep(int(1.6e9))    # 0.8 s and more
    start.set()
    gaps, last = [], time.perf_counter()
    while t.is_alive():
        time.sleep(1e-3)
        now = time.perf_counter()
        gaps.append(now - last)
        last = now
    t.join()
    torch.cuda.synchronize()
    assert max(took) > 0.3, "the queue took all calls at once"
    assert max(gaps) < 0.15, max(gaps)


def test_calls_from_two_threads(dl):  # noqa: F811
    """Two threads, each with a stream, a RoPE specification and a workspace of its own,
    call at the same time: each gets what it gets alone."""
    import torch

    def problem(seed, hd, layout, scaling, n, ctx):
        rng = np.random.default_rng(seed)
        kw = dict(hq=8, nkv=2, hd=hd, P=16)
        pb = attn_problem(rng, n, ctx, **kw)
        g = geom(dl, M=pb["M"], NP=pb["NP"], **kw)
        N = pb["q"].shape[0]
        x = bf16(rng.standard_normal((N, 8 * hd)))[0]
        sp = rope_spec(dl, layout, hd, scaling, 4.0)
        pos = dev(rng.integers(0, 5000, N).astype(np.int32))
        pool, ints = bf16(pb["pool"])[0], [dev(pb[k]) for k in ("table", "cu", "ctx", "kv")]
        ws = torch.empty(dl.dflash_chunk_attention_workspace_bytes(g, len(n), N, 3),
                         dtype=torch.uint8, device="cuda")

        def layer(q, out, stream):
            dl.dflash_chunk_rope_store(g, 0, sp, x, None, None, pos, None, None, q, None,
                                       stream=stream)
            dl.dflash_chunk_attention(g, 0, q, pool, *ints, out, ws, num_segments=3,
                                      stream=stream)
        return layer, (N, 8, hd)

    work = [problem(1, 128, "half", "plain", [1, 40], [700, 30]),
            problem(2, 64, "pairs", "yarn", [3, 1, 20], [300, 900, 0])]
    new = lambda shape: torch.zeros(shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    streams, want = [torch.cuda.Stream() for _ in work], []
    for layer, shape in work:
        q, out = new(shape), new(shape)
        layer(q, out, None)
        torch.cuda.synchronize()
        assert out.any()
        want.append((q, out))
    rounds = 100
    got = [[(new(shape), new(shape)) for _ in range(rounds)] for _, shape in work]
    torch.cuda.synchronize()
    failed = []

    def caller(i):
        try:
            for q, out in got[i]:
                work[i][0](q, out, streams[i])
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=caller, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for (q, out), all_of_them in zip(want, got):
        for a, b in all_of_them:
            assert torch.equal(a, q) and torch.equal(b, out)
