"""The host side of the calls for runs of new tokens: null handles, sizes, the
binding's struct and its refusals, without a GPU."""

import ctypes
import math
import os
import shutil
import subprocess

import pytest

from mixed_precision_quantized_quant_gb300 import kvq as K

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(K.LIB_PATH):
        from mixed_precision_quantized_quant_gb300 import build
        build.build()
    return K.load()


def test_null_handles_are_refused(lib):
    assert lib.kvq_paged_append_norm(None, 0, None, None, None, None, None, None, None, None, 1, None) == 1
    assert lib.kvq_paged_chunk_attn(None, 0, None, None, None, None, 0.0, 0, 1, None, 0, None) == 1
    assert lib.kvq_paged_prompt_attn(None, None, None, None, None, None, None, 0.0, 0, 1, None, 0, None) == 1
    assert lib.kvq_paged_chunk_workspace_bytes(None, 1, 1) == 0


def test_norm_struct_matches_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = [f for f, _ in K.HeadNormArgs._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "kvq.h"\nint main(void) {\n'
                   '  printf("%zu", sizeof(kvq_head_norm));\n' +
                   "".join(f'  printf(" %zu", offsetof(kvq_head_norm, {f}));\n' for f in names) + "  return 0;\n}\n")
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(K.HeadNormArgs)] + [getattr(K.HeadNormArgs, f).offset for f in names]


def test_norm_refuses():
    torch = pytest.importorskip("torch")
    for eps in (-1e-9, math.nan, math.inf, 1e39):
        with pytest.raises(ValueError):
            K.HeadNorm(eps=eps)
    with pytest.raises(ValueError, match="CUDA"):
        K.HeadNorm(torch.ones(64))
    assert K.HeadNorm(eps=0.0).args.q_weight is None


def test_model_reads_what_it_wrote():
    # the vectorised reading of the pages against the plain model's
    import numpy as np
    import torch

    import chunk_testutil as C
    import paged_testutil as T
    for kb, vb in ((16, 16), (8, 8), (8, 4), (4, 2), (2, 8)):
        for d in (64, 128):
            p = T.Pages(kb, vb, 2, d, 32, 3, torch.float16)
            g = torch.Generator().manual_seed(kb + vb)
            for page in range(3):
                for slot in range(32):
                    for h in range(2):
                        for is_v in (False, True):
                            p.put(page, slot, h, is_v, torch.randn(d, generator=g).half().float())

            class Cache:
                Hkv, num_pages, dtype = 2, 3, torch.float16
                buf = torch.from_numpy(p.data.reshape(-1).copy())

                def view(self, layer):
                    return dict(k_bits=kb, v_bits=vb, page_size=32, head_dim=d, tile_bytes=p.tile, pages=self.buf.data_ptr(),
                                page_stride=2 * 2 * p.tile)

            for is_v in (False, True):
                got, size = C.dense(Cache(), 0, [2, 0], 50, is_v)
                for h in range(2):
                    want, code, _ = p.rows([2, 0], 0, 50, h, is_v)
                    assert np.array_equal(got[h].numpy(), want)
                    assert np.allclose(size[h].numpy(), np.abs(code) + (np.abs(want - code) if kb != 16 else 0))
