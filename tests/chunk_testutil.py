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
    at = torch.arange(n, device=q.device)
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
    got, lse = got.double().to(out.device), lse.double().to(out.device)
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


def dense(cache, layer, table_row, n, is_value):
    """Rows [hkv, n, d] of a sequence's positions 0 .. n - 1 from the cache's bytes, in 64 bits, and the sizes
    |scale code| + |zero| that they are made of, all on the GPU."""
    v = cache.view(layer)
    kb, vb, P, d, tile = v["k_bits"], v["v_bits"], v["page_size"], v["head_dim"], v["tile_bytes"]
    off = v["pages"] - cache.buf.data_ptr()
    data = cache.buf[off:off + cache.num_pages * v["page_stride"]].view(cache.num_pages, cache.Hkv, P // 16, tile)
    pages = torch.as_tensor(table_row[:-(-n // P)], dtype=torch.int64, device=data.device)
    t = data[pages].transpose(0, 1).reshape(cache.Hkv, -1, tile)  # [hkv, tiles, bytes]
    dev = data.device
    i = torch.arange(16, device=dev)
    if kb == 16:
        rows = t.view(cache.dtype).view(cache.Hkv, -1, 2, 16, d)[:, :, int(is_value)]
        c = torch.arange(d, device=dev)
        at = (((c // 8)[None] ^ (i & 7)[:, None]) * 8 + c % 8).expand(rows.shape)
        x = torch.gather(rows, -1, at).reshape(cache.Hkv, -1, d)[:, :n].double()
        return x, x.abs()
    row = 2 * (i & 3) + (i >> 2 & 1) + (i & 8)
    rk, rv = d * kb // 8, d * vb // 8
    bits, rb, start, place = (vb, rv, 16 * rk, i) if is_value else (kb, rk, 0, row)
    raw = t[..., start:start + 16 * rb].reshape(cache.Hkv, -1, 16, rb)[:, :, place]
    b = torch.arange(rb, device=dev)
    if is_value:
        xor = (i & 3) * 32 if rb == 128 else (i >> 1 & 1) * 32 if rb == 64 else i * 0
    else:
        xor = (row & 1) * 64 if rb == 128 else row * 0
    raw = torch.gather(raw, -1, (b[None] ^ xor[:, None]).expand(raw.shape))
    sh = torch.arange(8 // bits, device=dev) * bits
    code = ((raw.int()[..., None] >> sh) & ((1 << bits) - 1)).reshape(cache.Hkv, -1, 16, d).double()
    sz = t[..., 16 * (rk + rv):].contiguous().view(torch.float16).view(cache.Hkv, -1, 16, 4)[:, :, row].double()
    s, z = (sz[..., 2 * int(is_value) + k:2 * int(is_value) + k + 1] for k in (0, 1))
    x, size = code * s + z, (code * s).abs() + z.abs()
    return x.reshape(cache.Hkv, -1, d)[:, :n], size.reshape(cache.Hkv, -1, d)[:, :n]
