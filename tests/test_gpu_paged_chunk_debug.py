"""The KVQ_DEBUG build's range checks in the kernels for runs of new tokens: none
fires on a correct call, and pages outside what they allow are reported and left out."""

import ctypes
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEBUG = os.environ.get("KVQ_DEBUG_LIB") == "1"

SUBSET = ("(test_chunk_pairs and fp16 and 128) or test_chunk_pages or test_chunk_window or test_chunk_long or test_chunk_many or "
          "test_chunk_keeps or test_prompt or test_norm_prompts or test_norm_one_row or test_keys_out or test_rows_that or "
          "(test_few_rows and 128) or test_the_checks")


def test_chunk_subset_under_the_debug_build():
    if DEBUG:
        pytest.skip("runs the debug build itself")
    from mixed_precision_quantized_quant_gb300 import build
    assert build.build(debug=True).endswith("libkvq_debug.so")
    r = subprocess.run(
        [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "tests/test_gpu_paged_chunk.py",
         "tests/test_gpu_paged_norm.py", "tests/test_gpu_paged_chunk_long.py", "tests/test_gpu_paged_chunk_debug.py", "-k", SUBSET],
        cwd=ROOT, env=dict(os.environ, KVQ_DEBUG_LIB="1"), capture_output=True, text=True, timeout=1200)
    tail = (r.stdout + r.stderr)[-4000:]
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and "deselected" in r.stdout, tail


@pytest.mark.skipif(not DEBUG, reason="of the debug build (run by the test above)")
@pytest.mark.parametrize("kb,vb", [(16, 16), (4, 2)])
def test_the_checks_report_and_leave_out(kb, vb):
    # pages from the third on count as outside the pool (though they are there)
    import torch

    from mixed_precision_quantized_quant_gb300 import kvq as K
    from test_gpu_paged import Case
    c = Case([32, 32], [32, 32], kb=kb, vb=vb, d=64, page=16)
    c.table[:, :2] = [[0, 1], [2, 3]]
    c.batch = K.PagedBatch(torch.from_numpy(c.table).cuda(), *c.batch._keep[1:])
    lib = K.load()
    lib.kvq_paged_debug_limit.argtypes = [ctypes.c_void_p, ctypes.c_int64]
    q = c.rows(64, 8)
    good = c.cache.chunk_attn(0, c.batch, q)
    assert c.cache.device_error() == 0
    assert lib.kvq_paged_debug_limit(c.cache.h, 2 * c.cache.view(0)["page_stride"]) == 0
    got = c.cache.chunk_attn(0, c.batch, q)
    assert c.cache.device_error() == 3 and torch.equal(got[:32], good[:32])
    assert lib.kvq_paged_debug_limit(c.cache.h, 1 << 40) == 0
    assert torch.equal(c.cache.chunk_attn(0, c.batch, q), good) or not bool(torch.isfinite(good.float()).all())
    assert c.cache.device_error() == 0
