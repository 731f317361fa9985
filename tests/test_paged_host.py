"""The paged cache's host side: sizes, argument checks, the binding's structs."""

import ctypes
import os

import pytest

from mixed_precision_quantized_quant_gb300 import kvq as K

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(K.LIB_PATH):
        from mixed_precision_quantized_quant_gb300 import build
        build.build()
    return K.load()


def _cfg(**kw):
    base = dict(layers=[(16, 16), (4, 2)], num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=32, num_pages=5)
    base.update(kw)
    return K.make_paged_config(base.pop("layers"), **base)


def test_bytes_by_hand(lib):
    # 5 pages x 2 heads x 2 tiles; a 16-bit tile 16 x 2 x 256 B, a K4V2 one 16 x (64 + 32) + 128 B
    assert K.kvq_paged_bytes(_cfg()) == 20 * 8192 + (20 * 1664 + 255) // 256 * 256 + 256
    assert K.kvq_paged_bytes(_cfg(layers=[(8, 8)], head_dim=64, num_pages=1, page_size=16)) == \
        (2 * (16 * 128 + 128) + 255) // 256 * 256 + 256
    # far past 32 bits
    assert K.kvq_paged_bytes(_cfg(layers=[(16, 16)] * 80, num_pages=1 << 20)) == 80 * (4 << 20) * 8192 + 256


def test_bytes_refuses_bad_configs(lib):
    bad = [dict(head_dim=96), dict(page_size=8), dict(page_size=48), dict(page_size=256), dict(num_pages=0),
           dict(num_q_heads=6, num_kv_heads=4), dict(num_q_heads=18, num_kv_heads=2), dict(num_q_heads=0),
           dict(num_kv_heads=0), dict(num_q_heads=2 ** 17, num_kv_heads=2 ** 16), dict(layers=[(3, 4)]), dict(layers=[(4, 3)]), dict(layers=[(16, 8)]),
           dict(layers=[(8, 16)]), dict(layers=[(0, 0)]), dict(dtype=2), dict(dtype=-1), dict(layers=[]),
           dict(layers=[(16, 16)] * 60000, num_pages=2 ** 31 - 1, num_q_heads=2 ** 16, num_kv_heads=2 ** 16)]
    for b in bad:
        assert K.kvq_paged_bytes(_cfg(**b)) == 0, b
    assert lib.kvq_paged_bytes(None) == 0


def test_create_refuses(lib):
    h = ctypes.c_void_p()
    cfg = _cfg()
    buf = ctypes.c_void_p
    assert lib.kvq_paged_create(ctypes.byref(cfg), None, 0, ctypes.byref(h)) == 1 and not h.value
    assert lib.kvq_paged_create(ctypes.byref(cfg), buf(256), 16, ctypes.byref(h)) == 4 and not h.value
    assert lib.kvq_paged_create(ctypes.byref(cfg), buf(128), 1 << 40, ctypes.byref(h)) == 3 and not h.value
    assert lib.kvq_paged_create(ctypes.byref(cfg), buf(256), 1 << 40, None) == 1
    for layers, code in (([(5, 4)], 2), ([(16, 4)], 7), ([(4, 16)], 7)):
        bad = _cfg(layers=layers)
        assert lib.kvq_paged_create(ctypes.byref(bad), buf(256), 1 << 40, ctypes.byref(h)) == code and not h.value
    wide = _cfg(num_q_heads=32, num_kv_heads=2)
    assert lib.kvq_paged_create(ctypes.byref(wide), buf(256), 1 << 40, ctypes.byref(h)) == 7


def test_null_handles_are_refused(lib):
    assert lib.kvq_paged_append(None, 0, None, None, None, None, None, None, 1, None) == 1
    assert lib.kvq_paged_decode_attn(None, 0, None, None, None, None, 0.0, 0, None, 0, None) == 1
    assert lib.kvq_paged_read(None, 0, None, None, None, 1, None) == 1
    assert lib.kvq_paged_view_get(None, 0, None) == 1
    assert lib.kvq_paged_device_error(None, None, None) == 1
    assert lib.kvq_paged_destroy(None) == 1
    assert lib.kvq_paged_workspace_bytes(None, 4) == 0


def test_paged_structs_match_the_header(tmp_path):
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    fields = {"kvq_paged_layer_cfg": K.PagedLayerCfg, "kvq_paged_config": K.PagedConfig, "kvq_paged_view": K.PagedView,
              "kvq_paged_batch": K.PagedBatchArgs, "kvq_rotation": K.RotationArgs, "kvq_rows": K.Rows}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "kvq.h"', "int main(void) {"]
    for cname, py in fields.items():
        lines.append(f'  printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'  printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    lines.append("  return 0;\n}")
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines))
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = {tuple(l.split()[:2]): int(l.split()[2])
           for l in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n") if l}
    for cname, py in fields.items():
        assert got[(cname, "size")] == ctypes.sizeof(py), cname
        for f, _ in py._fields_:
            assert got[(cname, f)] == getattr(py, f).offset, (cname, f)


def test_batch_and_rotation_refuse_cpu_tensors():
    torch = pytest.importorskip("torch")
    t = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        K.PagedBatch(t, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        K.Rotation(torch.zeros(4, 64))


def test_model_rows_are_a_permutation():
    # the plain model's row order and offsets: no two bytes of a tile share a place
    import numpy as np
    import torch

    import paged_testutil as T
    for d in (64, 128):
        for kb, vb in ((16, 16), (8, 8), (8, 4), (4, 2), (2, 8)):
            p = T.Pages(kb, vb, 1, d, 16, 1, torch.float16)
            seen = np.zeros(p.tile, int)
            for i in range(16):
                for is_v in (False, True):
                    start, n, xor = p._row(is_v, i)
                    seen[start + (np.arange(n) ^ xor)] += 1
                    if kb != 16:
                        off = 16 * (p.rk + p.rv) + T.key_row(i) * 8 + (4 if is_v else 0)
                        seen[off:off + 4] += 1
            assert (seen == 1).all()
