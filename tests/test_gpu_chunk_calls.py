"""The ragged-chunk calls as a program of several threads and streams makes them."""
import threading
import time

import numpy as np
import pytest

from tests.test_gpu_chunk import dev, dl, geom, plan_case, plan_outputs  # noqa: F401

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
