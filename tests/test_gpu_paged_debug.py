"""The KVQ_DEBUG build's range checks in the paged cache's kernels: none fires on a
correct call (the paged suites' calls, each ending with a clear error word, in a child
process), and an access outside what they allow is reported and left out."""

import ctypes
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEBUG = os.environ.get("KVQ_DEBUG_LIB") == "1"

SUBSET = ("(test_attn_pairs and fp16 and 128) or test_attn_heads_and_pages or test_attn_window or test_attn_long or test_attn_many or "
          "test_append_one_row_each or test_append_prompts or test_append_rotations or test_append_heads or test_append_and_read or "
          "test_read or test_prefill or test_captured or test_pages_past or test_bad_pages or test_ends_that or test_the_checks")


def test_paged_subset_under_the_debug_build():
    if DEBUG:
        pytest.skip("runs the debug build itself")
    from mixed_precision_quantized_quant_gb300 import build
    assert build.build(debug=True).endswith("libkvq_debug.so")
    r = subprocess.run(
        [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "tests/test_gpu_paged.py",
         "tests/test_gpu_paged_edges.py", "tests/test_gpu_paged_debug.py", "-k", SUBSET],
        cwd=ROOT, env=dict(os.environ, KVQ_DEBUG_LIB="1"), capture_output=True, text=True, timeout=1200)
    tail = (r.stdout + r.stderr)[-4000:]
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and "deselected" in r.stdout and "skipped" not in r.stdout, tail


@pytest.mark.skipif(not DEBUG, reason="of the debug build (run by the test above)")
@pytest.mark.parametrize("width", [None, 200])
@pytest.mark.parametrize("kb,vb", [(16, 16), (4, 2)])
def test_the_checks_report_and_leave_out(kb, vb, width):
    # pages from the third on count as outside the pool (though they are there): sequence 1's are,
    # sequence 0's are not
    import torch

    from mixed_precision_quantized_quant_gb300 import kvq as K
    from test_gpu_paged import Case
    c = Case([32, 32], [32, 32], kb=kb, vb=vb, d=64, page=16, width=width)
    c.table[:, :2] = [[0, 1], [2, 3]]
    c.batch = K.PagedBatch(torch.from_numpy(c.table).cuda(), *c.batch._keep[1:])
    lib = K.load()
    lib.kvq_paged_debug_limit.argtypes = [ctypes.c_void_p, ctypes.c_int64]
    before = c.download().copy()
    k, q = c.rows(64, 2), c.rows(2, 8)
    assert lib.kvq_paged_debug_limit(c.cache.h, 2 * c.cache.view(0)["page_stride"]) == 0
    c.cache.append(0, c.batch, k, k)
    assert c.cache.device_error() == 3
    got = c.download()
    assert (got[2:] == before[2:]).all() and not (got[:2] == before[:2]).all()
    out = torch.full((64, 2, 64), 7.0, dtype=c.dtype, device="cuda")
    rk, _ = c.cache.read(0, c.batch, 64, K=out)
    assert c.cache.device_error() == 3 and bool((rk[32:] == 7).all()) and not bool((rk[:32] == 7).all(2).any())
    c.cache.decode_attn(0, c.batch, q)
    assert c.cache.device_error() == 3
    assert lib.kvq_paged_debug_limit(c.cache.h, before.size) == 0
    c.cache.append(0, c.batch, k, k)
    c.cache.read(0, c.batch, 64)
    c.cache.decode_attn(0, c.batch, q)
    assert c.cache.device_error() == 0
