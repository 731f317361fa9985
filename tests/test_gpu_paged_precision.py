"""How near the paged attention is to 64 bits: weights far below the largest,
weights in two parts, queries of a wide range."""

import math

import numpy as np
import pytest
import torch

import paged_testutil as T
from test_gpu_paged import PAIRS, Case

pytestmark = pytest.mark.gpu


def attend_closely(pages, table, lens, q, scale=0.0, window=0, dtype=torch.float16):
    """`attend` with tolerances for weights held in two 16-bit parts.

    Counted, element by element, w_j being what weight j multiplies (the value,
    or the scale, with the code c_j):
      * the output's rounding, u_out |o|, at least half a step of fp16's
        subnormals, 2^-25;
      * a weight in two parts of a type with half step u: u^2 of it.  In fp16 the
        second part is off by 2^-25 at least, of weights whose running maximum
        is kept at 2^7 or higher: 2^-32 max(p w) sum_j |c_j|;
      * the scores' sums, as in `attend`: a factor exp(2 e) of every weight;
      * the products with the values: 2 (n / 16 + 1) MMAs after one another at
        the most.  Each adds two groups of 8 products to its sum and drops what
        lies below 2^-24 of the largest exponent, so it is off by at most 9 * 2^-23 of
        that.  Codes are subnormals: their exponent stands for 2^(10 - field)
        codes, which is G = 4, 64 / 15 or 64 / 3 times the largest code;
      * the sums of zeros and of weights, a thread's n / 8 additions and the
        merges' of a few dozen: (n / 8 + 64) 2^-23 of sum_j p_j (|v_j| + |z_j|).
    """
    B, hq, d = q.shape
    g = hq // pages.hkv
    out, lse, _, ltol = T.attend(pages, table, lens, q, scale, window, dtype)
    tol = np.zeros((B, hq, d))
    sc = scale or 1 / math.sqrt(d)
    quant = pages.kb != 16
    u_out = torch.finfo(dtype).eps / 2
    half = quant or dtype == torch.float16
    u2 = 2.0 ** -22 if half else 2.0 ** -16
    G = {16: 1.0, 8: 4.0, 4: 64 / 15, 2: 64 / 3}[pages.vb]
    for b in range(B):
        n = int(lens[b])
        lo = max(0, n - window) if window else 0
        if n == 0:
            continue
        for h in range(pages.hkv):
            k, kc, _ = pages.rows(table[b], lo, n, h, False)
            v, vc, vs = pages.rows(table[b], lo, n, h, True)
            c = np.abs(vc) / np.where(vs > 0, vs, 1.0)[:, None]
            top = (vs * (2 ** pages.vb - 1))[:, None] * (c > 0) if quant else np.abs(v)
            for j in range(h * g, h * g + g):
                qq = q[b, j].double().numpy()
                t = k @ qq * sc
                p = np.exp(t - t.max())
                e = (d + 16) * 2.0 ** -23 * abs(sc) * ((np.abs(kc) + np.abs(k - kc)) @ np.abs(qq)).max() + 2.0 ** -20
                chain = 2 * ((n - lo) / 16 + 1) * 9 * 2.0 ** -23 * G * (p @ top)
                sums = ((n - lo) / 8 + 64) * 2.0 ** -23
                tol[b, j] = (u_out * np.abs(out[b, j]) + 2.0 ** -25
                             + (u2 * (p @ np.abs(vc)) + (2.0 ** -32 * (p * vs).max() * c.sum(0) if half else 0.0)
                                + chain + (2 * e + sums) * (p @ (np.abs(v) + np.abs(v - vc)))) / p.sum())
    return out, lse, tol, ltol


def _check(c, q, scale=0.0):
    out, lse = c.cache.decode_attn(c.layer, c.batch, q, scale=scale, return_lse=True)
    torch.cuda.synchronize()
    eo, el, tol, ltol = attend_closely(c.model, c.table, c.lens, q.cpu(), scale, 0, c.dtype)
    far = np.abs(out.double().cpu().numpy() - eo) / tol
    assert (far <= 1).all(), float(far.max())
    assert (np.abs(lse.double().cpu().numpy() - el) <= ltol).all()
    assert c.cache.device_error() == 0


@pytest.mark.parametrize("width", [None, 100])
@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 8), (8, 4)])
def test_weights_far_below_the_largest_count(kb, vb, width):
    # one token has nearly all the weight and value 0 in every channel but one; 400 others have 2^-26 of
    # it each and are the whole of the other channels' output
    c = Case([401], kb=kb, vb=vb, d=64, hq=2, hkv=1, fill=False, width=width)
    top = 2 ** min(vb, 8) - 1
    for p in range(401):
        at = (c.table[0, p // 16], p % 16, 0)
        k, v = torch.zeros(64), torch.zeros(64)
        if p == 0:
            k[0], v[63] = 18.0, float(top)
        else:
            v[:63] = 400 + 600 * torch.rand(63, generator=c.g)
        c.model.put(*at, False, k.half().float())
        c.model.put(*at, True, v.half().float())
    c.upload()
    q = torch.zeros(1, 2, 64, dtype=torch.float16, device="cuda")
    q[:, :, 0] = 1.0
    _check(c, q, scale=1.0)


@pytest.mark.parametrize("width", [None, 100])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kb,vb", PAIRS)
def test_weights_keep_more_than_16_bits(kb, vb, d, dtype, width):
    # few tokens, so that sums cancel in many channels, and small queries, so that scores are near exact: one
    # rounding of a weight to 16 bits is far outside the tolerance for 16-bit, 8-bit and 4-bit values
    c = Case([2, 3, 3, 4, 5, 7, 16, 17, 40], kb=kb, vb=vb, d=d, dtype=dtype, width=width)
    _check(c, c.rows(len(c.lens), c.hq) / 64)
