"""What loading the library needs (CPU only): the shared library alone.  The module
that marshals the ragged-chunk calls, and torch, are needed by the calls that use
them and not before."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.fixture(scope="module", autouse=True)
def built():
    from context_kv_update_gb300 import build
    build.build()


GEOM = """
g = dl.make_geom(dict(kind="gqa", L=2, D_in=64, D=64, hq=4, nkv=2, hd=64, P=16, T=1, max_pages=8,
                      num_pool_pages=32, rope_theta=1e4, eps_h=1e-6, eps_k=1e-6))
"""


def test_load_needs_the_shared_library_alone():
    run("""
import sys
sys.modules["context_kv_update_gb300._calls"] = None   # as if it were not there
import context_kv_update_gb300 as dl
assert dl.load() is dl.load()
assert "torch" not in sys.modules
""" + GEOM + """
assert dl.dflash_ctx_workspace_bytes(g, 2) > 0
assert dl.dflash_attention_workspace_bytes(g, 2, 4, 3) > 0
assert dl.dflash_chunk_attention_workspace_bytes(g, 2, 6, 3) > 0
assert dl.dflash_chunk_attention_num_segments(g, 2, 6) >= 1
assert "torch" not in sys.modules
""")


def test_a_missing_module_is_named_by_the_calls_that_need_it():
    run("""
import sys
sys.modules["context_kv_update_gb300._calls"] = None
import context_kv_update_gb300 as dl
""" + GEOM + """
import torch
i32, q = torch.zeros(4, dtype=torch.int32), torch.zeros((4, 4, 64), dtype=torch.bfloat16)
calls = [lambda: dl.dflash_chunk_plan(g, *[i32] * 6, None, 100, {}),
         lambda: dl.dflash_chunk_rope_store(g, 0, dl.RopeSpec(), q, None, None, i32, None, None, q, None),
         lambda: dl.dflash_chunk_attention(g, 0, q, q, i32, i32, i32, i32, q)]
for f in calls:
    try:
        f()
    except ImportError as e:
        assert "context_kv_update_gb300.build" in str(e), e
    else:
        raise SystemExit("no error")
""")
