"""A plain model of the paged cache for the tests: pages as bytes, written and
read token by token from the layout in include/kvq.h; attention in 64 bits."""

from __future__ import annotations

import math

import numpy as np
import torch

from oracle import kvq_oracle as O

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def key_row(i: int) -> int:
    return 2 * (i & 3) + ((i >> 2) & 1) + (i & 8)


def row_bytes(x: torch.Tensor) -> np.ndarray:
    """Bytes of a row of 16-bit values."""
    return x.contiguous().view(torch.uint8).numpy()


def pack(codes: np.ndarray, bits: int) -> np.ndarray:
    out = np.zeros(len(codes) * bits // 8, np.uint8)
    for c, v in enumerate(codes):
        out[c * bits // 8] |= int(v) << (c * bits % 8)
    return out


def unpack(data: np.ndarray, bits: int, d: int) -> np.ndarray:
    c = np.arange(d)
    return (data[c * bits // 8] >> (c * bits % 8)) & ((1 << bits) - 1)


class Pages:
    """One layer's pages, [num_pages][Hkv][P / 16][tile bytes]."""

    def __init__(self, kb, vb, hkv, d, page_size, num_pages, dtype):
        self.kb, self.vb, self.hkv, self.d, self.P, self.dtype = kb, vb, hkv, d, page_size, dtype
        self.rk, self.rv = d * kb // 8, d * vb // 8
        self.tile = 16 * (self.rk + self.rv) + (0 if kb == 16 else 128)
        self.data = np.zeros((num_pages, hkv, page_size // 16, self.tile), np.uint8)

    def _row(self, is_value, i):
        """(start of the code row, its length, XOR on the byte offset) in a tile."""
        if self.kb == 16:
            return (16 * self.rk if is_value else 0) + i * 2 * self.d, 2 * self.d, (i & 7) * 16
        if is_value:
            x = (i & 3) * 32 if self.rv == 128 else (i >> 1 & 1) * 32 if self.rv == 64 else 0
            return 16 * self.rk + i * self.rv, self.rv, x
        return key_row(i) * self.rk, self.rk, (key_row(i) & 1) * 64 if self.rk == 128 else 0

    def put(self, page, slot, head, is_value, x):
        """x: [d] values of the cache's type (values) or fp32 (turned keys)."""
        tile, i = self.data[page, head, slot // 16], slot % 16
        start, n, xor = self._row(is_value, i)
        at = start + (np.arange(n) ^ xor)
        if self.kb == 16:
            tile[at] = row_bytes(x.to(self.dtype))
            return
        bits = self.vb if is_value else self.kb
        h = x.float().clamp(-65504, 65504).half().numpy()[None]
        mn, mx = h.min(1), h.max(1)
        # the range times the reciprocal of the code range, as documented (kvq_append divides)
        s = ((mx.astype(np.float32) - mn.astype(np.float32)) * (np.float32(1) / np.float32(2 ** bits - 1))).astype(np.float16)
        codes = O.asym_codes(h, mn[:, None], s.astype(np.float32)[:, None], 2 ** bits - 1)[0]
        tile[at] = pack(codes, bits)
        off = 16 * (self.rk + self.rv) + key_row(i) * 8 + (4 if is_value else 0)
        tile[off:off + 4] = np.concatenate([s, mn]).astype(np.float16).view(np.uint8)

    def get(self, page, slot, head, is_value):
        """([d] values, [d] code * scale part, the scale or 1) in 64 bits."""
        tile, i = self.data[page, head, slot // 16], slot % 16
        start, n, xor = self._row(is_value, i)
        raw = tile[start + (np.arange(n) ^ xor)]
        if self.kb == 16:
            v = torch.from_numpy(raw.copy()).view(self.dtype).double().numpy()
            return v, v, 1.0
        bits = self.vb if is_value else self.kb
        off = 16 * (self.rk + self.rv) + key_row(i) * 8 + (4 if is_value else 0)
        s, z = tile[off:off + 4].view(np.float16).astype(np.float64)
        c = unpack(raw, bits, self.d) * s
        return c + z, c, s

    def rows(self, table_row, lo, hi, head, is_value):
        """Values and code parts of positions lo .. hi - 1, [n, d] each, and scales [n]."""
        got = [self.get(table_row[p // self.P], p % self.P, head, is_value) for p in range(lo, hi)]
        return np.stack([g[0] for g in got]), np.stack([g[1] for g in got]), np.array([g[2] for g in got])


def turn(x, pos, table, interleaved):
    """Rows [heads, d] turned in fp32, every operation rounded."""
    y = x.float().clone()
    dim = table.shape[1]
    c, s = table[pos, :dim // 2], table[pos, dim // 2:]
    a, b = (y[:, 0:dim:2], y[:, 1:dim:2]) if interleaved else (y[:, :dim // 2], y[:, dim // 2:dim])
    u, w = a * c - b * s, b * c + a * s
    if interleaved:
        y[:, 0:dim:2], y[:, 1:dim:2] = u, w
    else:
        y[:, :dim // 2], y[:, dim // 2:dim] = u, w
    return y


def attend(pages, table, lens, q, scale=0.0, window=0, dtype=torch.float16):
    """64-bit attention over the pages: (out, lse, tolerance of out, tolerance of lse).

    The tolerances count what the kernel may round, element by element, with
    u the half step of the 16-bit type the weights are held in for the product
    with the values (fp16 for codes):
      * the output's own rounding, u_out |o|;
      * each weight's rounding, u sum_j p_j |w_j| with w_j what it multiplies
        (the value, or scale * code: the zeros are summed in fp32).  An fp16
        weight of codes is p_j s_j over 2^m, m at most the largest log2(p s):
        below 2^-14 it is off by at most 2^-25, so the codes' sum by 2^-25 *
        max(p s) * sum_j c_j, and a 16-bit value's by 2^-25 * sum_j |v_j|;
      * the scores' fp32 sums over d channels, e = (d + 16) 2^-23 max_j |scale|
        sum_c |q_c| |k_jc| (both parts of a dequantized key counted), which
        moves every weight by at most a factor exp(2 e);
      * fp32 sums over n tokens, a thread's chain of n / 8 additions at the
        most and the merges' of a few dozen: (n / 8 + 64) 2^-23 of sum_j p_j |v_j|.
    """
    B, hq, d = q.shape
    g = hq // pages.hkv
    out, lse = np.zeros((B, hq, d)), np.full((B, hq), -math.inf)
    tol, ltol = np.zeros((B, hq, d)), np.zeros((B, hq))
    sc = scale or 1 / math.sqrt(d)
    quant = pages.kb != 16
    u_out = torch.finfo(dtype).eps / 2
    u = torch.finfo(torch.float16).eps / 2 if quant else u_out
    for b in range(B):
        n = int(lens[b])
        lo = max(0, n - window) if window else 0
        if n == 0:
            continue
        for h in range(pages.hkv):
            k, kc, _ = pages.rows(table[b], lo, n, h, False)
            v, vc, vs = pages.rows(table[b], lo, n, h, True)
            codes = np.abs(vc) / np.where(vs > 0, vs, 1.0)[:, None]
            for j in range(h * g, h * g + g):
                qq = q[b, j].double().numpy()
                t = k @ qq * sc
                p = np.exp(t - t.max())
                total = p.sum()
                out[b, j] = p @ v / total
                lse[b, j] = t.max() + np.log(total)
                e = (d + 16) * 2.0 ** -23 * abs(sc) * ((np.abs(kc) + np.abs(k - kc)) @ np.abs(qq)).max() + 2.0 ** -20
                f = ((n - lo) / 8 + 64) * 2.0 ** -23
                tol[b, j] = (u_out * np.abs(out[b, j])
                             + (u * (p @ np.abs(vc)) + 2.0 ** -25 * (p * vs).max() * codes.sum(0)) / total
                             + (2 * e + f) * (p @ (np.abs(v) + np.abs(v - vc))) / total + 2.0 ** -24)
                ltol[b, j] = 2 * e + f + 2.0 ** -20 * (1 + abs(lse[b, j]))
    return out, lse, tol, ltol
