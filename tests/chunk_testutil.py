"""Attention of runs of new tokens in 64 bits, with what a kernel may be off by."""

from __future__ import annotations

import math

import torch


def attend(q, k, v, first, last, dtype, scale=0.0, quant=False, parts=None, v_scale=None):
    """q [m, hq, d]; k, v [hkv, t, d] (64 bits); the query row i sees first[i] .. last[i].
    Returns out [m, hq, d], lse [m, hq] and the tolerance of each.

    The tolerances count what a kernel may round, element by element, with u_out
    the half step of the output's type and u that of the type in which the
    weights meet the values (fp16 on quantized layers):
      * the output's own rounding, u_out |o|;
      * each weight's rounding, u p_j |v_j|, and in fp16, where a weight under
        2^-14 is off by up to 2^-25: they are held at least 2^7 above what
        weighs one, so by at most 2^-32 of the greatest weight, 2^-32 |v_j|;
      * the rounding of a dequantized value to fp16, 2^-11 |v_j| + 2^-25, and
        the sum's that it is part of;
      * the scores' fp32 sums over d channels, e = (d + 16) 2^-23 |scale| sum_c
        |q_c| |k_jc| (`parts`: |code * scale| + |zero| for dequantized keys), and
        the largest score's own rounding in base 2, which move every weight by
        at most a factor exp(2 e);
      * fp32 sums over n tokens in tiles of 128 and pieces of the sequence:
        (n / 16 + 64) 2^-23 of sum_j p_j |v_j|.
    """
    m, hq, d = q.shape
    hkv, n, _ = k.shape
    sc = scale or 1 / math.sqrt(d)
    u_out = torch.finfo(dtype).eps / 2
    u = torch.finfo(torch.float16).eps / 2 if quant else u_out
    kk, vv = (x.repeat_interleave(hq // hkv, 0) for x in (k, v))
    ka = kk.abs() if parts is None else parts.repeat_interleave(hq // hkv, 0)
    qq = q.double().transpose(0, 1)
    at = torch.arange(n)
    seen = (at >= first[:, None]) & (at <= last[:, None])
    t = (qq @ kk.transpose(1, 2) * sc).masked_fill(~seen, -math.inf)
    top = t.amax(-1, keepdim=True)
    safe = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p = (t - safe).exp()
    total = p.sum(-1, keepdim=True)
    some = total > 0
    div = torch.where(some, total, torch.ones_like(total))
    va = vv.abs()
    out = (p @ vv) / div
    lse = (safe + total.log()).squeeze(-1)
    size = (qq.abs() @ ka.transpose(1, 2) * abs(sc)).masked_fill(~seen, 0.0).nan_to_num(0.0, 0.0, 0.0)
    e = (d + 16) * 2.0 ** -23 * size.amax(-1, keepdim=True) + 2.0 ** -22 * (1 + safe.abs())
    f = (n / 16 + 64) * 2.0 ** -23
    pv = (p @ va) / div
    w = (seen.double() @ va)
    tol = u_out * out.abs() + (u + 2 * e + f) * pv + 2.0 ** -24
    if dtype == torch.float16 or quant:
        tol = tol + 2.0 ** -32 * w
    if quant:
        tol = tol + 2.0 ** -11 * pv + 2.0 ** -25
    ltol = (2 * e + f).squeeze(-1) + 2.0 ** -20 * (1 + torch.where(torch.isfinite(lse), lse, torch.zeros_like(lse)).abs())
    return out.transpose(0, 1), lse.transpose(0, 1), tol.transpose(0, 1), ltol.transpose(0, 1)


def close(got, lse, exp):
    """Every element within its tolerance; infinities and zeros of empty rows exactly."""
    out, l64, tol, ltol = exp
    got, lse = got.double().cpu(), lse.double().cpu()
    err = (got - out).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (int(bad.sum()), float((err / tol)[bad].max()), torch.nonzero(bad)[:4].tolist())
    empty = torch.isinf(l64)
    assert torch.equal(torch.isinf(lse), empty)
    if bool(empty.any()):
        assert bool((got[empty] == 0).all()) and bool((lse[empty] == -math.inf).all())
    lerr = (lse - l64).abs()
    bad = ~((lerr <= ltol) | empty)
    assert not bool(bad.any()), (float((lerr / ltol)[bad].max()), torch.nonzero(bad)[:4].tolist())
