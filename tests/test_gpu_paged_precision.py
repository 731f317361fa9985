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


def _wide_queries(kb, below, d, width, small):
    """Keys that are 0 where the row's largest query, 1, is; the others, 2^-below times `small`, make the scores."""
    c = Case([60], kb=kb, vb=8, d=d, hq=4, hkv=1, dtype="bf16", fill=False, width=width)
    top = 2 ** kb - 1
    for p in range(60):
        at = (c.table[0, p // 16], p % 16, 0)
        k = torch.randint(0, top + 1, (d,), generator=c.g).float()
        k[0], k[1] = 0, top
        c.model.put(*at, False, k)
        c.model.put(*at, True, torch.randn(d, generator=c.g))
    c.upload()
    q = small(c.g, (1, 4, d)) * 2.0 ** -below
    q[:, :, 0] = 1.0
    q = q.bfloat16()
    scale = 2.0 ** below / (top * 8)
    out, lse = c.cache.decode_attn(0, c.batch, q.cuda(), scale=scale, return_lse=True)
    eo, el, tol, ltol = T.attend(c.model, c.table, c.lens, q, scale, 0, c.dtype)
    k, _, _ = c.model.rows(c.table[0], 0, 60, 0, False)
    v, _, _ = c.model.rows(c.table[0], 0, 60, 0, True)
    return (np.abs(out.double().cpu().numpy() - eo), tol, np.abs(lse.double().cpu().numpy() - el), ltol,
            scale * np.abs(k).sum(1).max(), np.abs(v).max())


@pytest.mark.parametrize("width", [None, 100])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kb,below", [(8, 31), (4, 31), (2, 27)])
def test_queries_keep_their_bits_far_below_the_largest(kb, below, d, width):
    # 8 significant bits whose first is `below` under the row's largest fit fp16 exactly: no term for their rounding
    def small(g, shape):
        return (1 + torch.randint(0, 128, shape, generator=g) / 128) * (1 - 2 * torch.randint(0, 2, shape, generator=g))

    o, tol, l, ltol, _, _ = _wide_queries(kb, below, d, width, small)
    assert (l <= ltol).all() and (o <= tol).all() and (ltol < 2e-3).all()


@pytest.mark.parametrize("width", [None, 100])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kb,below", [(8, 29), (4, 29), (2, 25)])
def test_queries_below_fp16_steps(kb, below, d, width):
    # smaller ones lose what lies below fp16's half step of 2^-25: 2^-40 (2-bit keys: 2^-36) of the row's
    # largest, 1, a channel, so that a score is off by r = that times scale * sum_c |k_c| at the most, every weight by
    # exp(2 r), the log-sum-exp by r and an output by under 3 r of the largest value
    o, tol, l, ltol, keys, value = _wide_queries(kb, below, d, width, lambda g, s: torch.randn(s, generator=g).clamp(-3, 3))
    r = 2.0 ** (-36 if kb == 2 else -40) * keys
    assert (l <= ltol + r).all() and (o <= tol + 3 * r * value).all() and r < 1e-2


@pytest.mark.parametrize("width", [None, 100])
@pytest.mark.parametrize("d", [64, 128])
def test_one_score_of_8_bit_keys(d, width):
    # One token a sequence, whose score is the log-sum-exp, with strong channels, so that the codes' part s q.c is
    # R times the score and the zeros' part takes most of it off.  An MMA cuts 2^-24 of its sum off each product, in
    # [0, 1) of that and of either sign: over d products in two chains of d / 2, whose sums are half of s q.c
    # at the end and a quarter on the way, sqrt(d / 3) 2^-24 R / 4 of the score in the 2-norm; the zeros' part, its
    # factor and the scale round by 2^-24 R / 3 each.  One chain has twice the first part.
    S, g = 24, torch.Generator().manual_seed(9)
    c = Case([1] * S, kb=8, vb=8, d=d, hq=32, hkv=8, fill=False, width=width)
    mu, sigma, strong = torch.randn(8, d, generator=g) * 0.5, torch.exp(torch.randn(8, d, generator=g) * 0.5), torch.ones(8, d)
    for h in range(8):
        strong[h, torch.randperm(d, generator=g)[:4]] = 10.0
    for b in range(S):
        for h in range(8):
            c.model.put(c.table[b, 0], 0, h, False, ((mu[h] + sigma[h] * torch.randn(d, generator=g)) * strong[h]).half().float())
            c.model.put(c.table[b, 0], 0, h, True, torch.randn(d, generator=g).half().float())
    c.upload()
    q = c.rows(S, 32)
    _, lse = c.cache.decode_attn(0, c.batch, q, return_lse=True)
    score, codes = np.zeros((S, 32)), np.zeros((S, 32))
    for b in range(S):
        for h in range(8):
            k, kc, _ = c.model.rows(c.table[b], 0, 1, h, False)
            x = q[b, 4 * h:4 * h + 4].double().cpu().numpy() / math.sqrt(d)
            score[b, 4 * h:4 * h + 4], codes[b, 4 * h:4 * h + 4] = x @ k[0], x @ kc[0]
    R = np.linalg.norm(codes) / np.linalg.norm(score)
    off = np.linalg.norm(lse.double().cpu().numpy() - score) / np.linalg.norm(score)
    assert off <= 2.0 ** -24 * R * math.sqrt(d / 48 + 1 / 3), (off, R)
