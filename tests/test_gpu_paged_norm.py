"""Append with a norm of query and key heads and with keys out, against 64 bits;
the new operators run together."""

import math

import numpy as np
import pytest
import torch

import chunk_testutil as C
import paged_testutil as T
from mixed_precision_quantized_quant_gb300 import kvq as K
from test_gpu_paged import Case

pytestmark = pytest.mark.gpu


def _normed(x, w, eps, pos, table, interleaved):
    """[heads, d] rows normed and turned in 64 bits, and the sizes that its fp32 errors scale with."""
    y = x.double()
    y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt()
    if w is not None:
        y = y * w.double()
    size = y.abs()
    if table is None:
        return y, size
    dim = table.shape[1]
    c, s = table[pos, :dim // 2].double(), table[pos, dim // 2:].double()
    first, second = (slice(0, dim, 2), slice(1, dim, 2)) if interleaved else (slice(0, dim // 2), slice(dim // 2, dim))
    a, b = y[:, first].clone(), y[:, second].clone()
    y[:, first], y[:, second] = a * c - b * s, b * c + a * s
    a, b = size[:, first].clone(), size[:, second].clone()
    size[:, first] = size[:, second] = a + b
    return y, size


def _check(c, wq, wk, eps=1e-6, dim=None, interleaved=False, how="fused", extra=0, in_place=False, with_q=True):
    n = (len(c.lens) if c.news is None else sum(c.news)) + extra
    k, v, q = c.rows(n, c.hkv, how), c.rows(n, c.hkv, how), c.rows(n, c.hq, how)
    k0, q0 = k.clone(), q.clone()
    rot = table = None
    if dim:
        table = K.rotation_table(max(c.lens) + 1, dim)
        rot, table = K.Rotation(table, interleaved), table.cpu()
    fresh = lambda h: torch.full((n, h, c.d), 7.0, dtype=c.dtype, device="cuda")  # noqa: E731
    k_out, q_out = (k, q) if in_place else (fresh(c.hkv), fresh(c.hq))
    got = c.cache.append(c.layer, c.batch, k, v, q=q if with_q else None, rotation=rot, q_out=q_out if with_q else None,
                         norm=K.HeadNorm(wq, wk, eps), k_out=k_out)
    assert c.cache.device_error() == 0
    assert got is (q_out if with_q else None)
    pages = c.download()
    # rounded once (u |y|), from a root, a reciprocal (2 ulp of the function, 1 of the sum over d in fp32: d 2^-25
    # at most), two products and a rotation, each 2^-24 of the sizes that meet: 16 + d / 2 steps together
    u, f = torch.finfo(c.dtype).eps / 2, (16 + c.d / 2) * 2.0 ** -24
    tiny = 2.0 ** -25 if c.dtype == torch.float16 else 0.0
    owned = np.zeros(n, bool)
    for row, b, p in c.places():
        owned[row] = True
        for x0, out, w in ((k0, k_out, wk),) + (((q0, q_out, wq),) if with_q else ()):
            e, size = _normed(x0[row].cpu(), None if w is None else w.cpu(), eps, p, table, interleaved)
            err = (out[row].cpu().double() - e).abs()
            tol = u * e.abs() * (1 + 2 * f) + 2 * f * size + tiny
            assert bool((err <= tol).all()), (row, float((err / tol).max()))
        for h in range(c.hkv):
            page, slot = c.table[b, p // c.P], p % c.P
            m = T.Pages(c.model.kb, c.model.vb, c.hkv, c.d, c.P, 1, c.dtype)
            m.data[0] = pages[page]
            gv, _, sv = m.get(0, slot, h, True)
            gk, _, sk = m.get(0, slot, h, False)
            if c.model.kb == 16:
                # the pages hold the very keys that k_out has, and the values as they came
                assert np.array_equal(gk, k_out[row, h].cpu().double().numpy())
                assert np.array_equal(gv, v[row, h].cpu().double().numpy())
            else:
                e, size = _normed(k0[row].cpu(), None if wk is None else wk.cpu(), eps, p, table, interleaved)
                # half a step of the codes (the scale's own rounding at the far end: 2^-11 of the range), the
                # rounding to fp16 first, and fp32's
                rng = float(e[h].max() - e[h].min())
                tol = sk / 2 + rng * 2.0 ** -10 + 2.0 ** -10 * e[h].abs() + 4 * f * size[h] + 2.0 ** -24
                assert bool(((torch.from_numpy(gk) - e[h]).abs() <= tol).all())
    if not in_place:
        assert bool((k_out[~torch.from_numpy(owned).cuda()] == 7).all())
        if with_q:
            assert bool((q_out[~torch.from_numpy(owned).cuda()] == 7).all())


def _w(c, heads=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    shape = (c.d,) if heads is None else (heads, c.d)
    return (1 + 0.5 * torch.randn(shape, generator=g)).to(c.dtype).cuda()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 4), (2, 2)])
def test_norm_one_row_each(kb, vb, d, dtype):
    c = Case([1, 16, 17, 0, 32, 70], kb=kb, vb=vb, d=d, dtype=dtype, page=32, fill=False)
    _check(c, _w(c), _w(c, seed=1), dim=d)


@pytest.mark.parametrize("kb,vb", [(16, 16), (4, 8)])
@pytest.mark.parametrize("how", ["fused", "odd"])
def test_norm_prompts(kb, vb, how):
    # more rows than the few-row form takes, rows behind the last sequence, per-head weights, part of the head turned
    c = Case([300, 130, 9, 77, 1], [300, 33, 0, 77, 1], kb=kb, vb=vb, d=128, hq=4, fill=False)
    _check(c, _w(c, 4), _w(c, 2, seed=1), dim=64, interleaved=True, how=how, extra=3)
    _check(c, _w(c), None, eps=0.0, dim=128, how=how)


@pytest.mark.parametrize("hq,hkv", [(7, 1), (3, 3), (10, 2)])
def test_norm_heads(hq, hkv):
    # groups of rows that the last heads do not fill
    for d in (64, 128):
        c = Case([40, 11], [40, 11], d=d, hq=hq, hkv=hkv, fill=False)
        _check(c, _w(c, hq), _w(c, hkv, seed=2), dim=32)


def test_norm_without_rotation_or_queries_and_in_place():
    c = Case([40, 600], [40, 500], d=64, dtype="bf16", fill=False)
    _check(c, None, _w(c), with_q=False)
    _check(c, None, None)
    _check(c, _w(c), _w(c, 2), dim=64, in_place=True)


@pytest.mark.parametrize("kb,vb", [(16, 16), (4, 2)])
@pytest.mark.parametrize("n", [20, 700])
def test_keys_out_without_a_norm(kb, vb, n):
    # the turned keys bit for bit, and the pages that a plain append leaves
    c = Case([n], [n], kb=kb, vb=vb, d=128, fill=False)
    k, v = c.rows(n, 2), c.rows(n, 2)
    rot = K.Rotation(K.rotation_table(n, 128))
    k_out = torch.empty(n, 2, 128, dtype=c.dtype, device="cuda")
    c.cache.append(0, c.batch, k, v, rotation=rot, k_out=k_out)
    a = c.download().copy()
    table = rot.table.cpu()
    for p in range(n):
        assert torch.equal(k_out[p].cpu(), T.turn(k[p].cpu(), p, table, False).to(c.dtype))
    c.upload()
    c.cache.append(0, c.batch, k, v, rotation=rot)
    assert np.array_equal(a, c.download())


def test_norm_rows_of_zeros_and_large_rows():
    c = Case([3], [3], d=64, dtype="bf16", fill=False)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    k[1] = 1e15
    k[2] = 1e-15
    out = torch.empty_like(k)
    c.cache.append(0, c.batch, k, k, norm=K.HeadNorm(eps=1e-6), k_out=out)
    assert bool((out[0] == 0).all()) and bool((out[1] == 1).all())
    assert torch.allclose(out[2].double(), torch.tensor(1e-12, dtype=torch.float64).cuda(), rtol=2 ** -7, atol=0)
    c.cache.append(0, c.batch, k, k, norm=K.HeadNorm(eps=0.0), k_out=out)
    assert bool(torch.isnan(out[0].float()).all()) and bool((out[1:] == 1).all())


def test_norm_refusals():
    c = Case([20, 5], kb=4, vb=4, d=64, hq=4, hkv=2)
    q, k, v = c.rows(2, 4), c.rows(2, 2), c.rows(2, 2)
    before = c.download().copy()
    w = _w(c)
    a = c.cache.append
    for fn in (lambda: K.HeadNorm(w.cpu()), lambda: K.HeadNorm(w, eps=-1.0), lambda: K.HeadNorm(w, eps=math.nan), lambda: K.HeadNorm(eps=math.inf),
               lambda: K.HeadNorm(w[1:]), lambda: K.HeadNorm(None, w.view(1, 1, 64)), lambda: K.HeadNorm(_w(c, 2).t()),
               lambda: a(0, c.batch, k, v, norm=K.HeadNorm(w.float())), lambda: a(0, c.batch, k, v, norm=K.HeadNorm(None, w[:32])),
               lambda: a(0, c.batch, k, v, norm=K.HeadNorm(None, _w(c, 4))), lambda: a(0, c.batch, k, v, norm=K.HeadNorm(_w(c, 2))),
               lambda: a(0, c.batch, k, v, k_out=k[:1]), lambda: a(0, c.batch, k, v, k_out=q), lambda: a(0, c.batch, k, v, k_out=k[:1].expand(2, 2, 64)),
               lambda: a(0, c.batch, k, v, k_out=k.float())):
        with pytest.raises(ValueError):
            fn()
    with pytest.raises(K.KVQError):
        a(1, c.batch, k, v, norm=K.HeadNorm())
    L, h, b, s = K.load(), c.cache.h, c.batch.args, torch.cuda.current_stream().cuda_stream
    rk = c.cache._rows(k, "k", 2, 2)
    call = lambda norm, ko=None: L.kvq_paged_append_norm(h, 0, b, rk, rk, None, None, ko, norm, None, 2, s)  # noqa: E731
    p = w.data_ptr()
    assert call(K.HeadNormArgs(p, p, 0, 0, -1.0)) == 1 and call(K.HeadNormArgs(p, p, 0, 0, math.nan)) == 1
    assert call(K.HeadNormArgs(p, p, 4, 0, 0.0)) == 1 and call(K.HeadNormArgs(p, p, 0, 4, 0.0)) == 1
    assert call(K.HeadNormArgs(p + 2, p, 0, 0, 0.0)) == 3 and call(K.HeadNormArgs(p, p + 8, 0, 0, 0.0)) == 3
    assert call(None, K.Rows(None, 1, 1)) == 1 and call(None, K.Rows(rk.data + 1, 64, 64)) == 3
    assert np.array_equal(c.download(), before) and c.cache.device_error() == 0


def test_norm_of_one_cache_is_refused_by_another_that_it_does_not_fit():
    one = Case([20, 5], kb=4, vb=4, d=64, hq=4, hkv=2)
    norm = K.HeadNorm(_w(one, 4), _w(one, 2))
    for _ in range(2):  # fitting calls in between change nothing
        one.cache.append(0, one.batch, one.rows(2, 2), one.rows(2, 2), norm=norm)
        for kw in (dict(hq=4, hkv=4), dict(hq=8, hkv=2)):
            two = Case([20, 5], kb=4, vb=4, d=64, **kw)
            with pytest.raises(ValueError):
                two.cache.append(0, two.batch, two.rows(2, two.hkv), two.rows(2, two.hkv), norm=norm)
    assert one.cache.device_error() == 0


@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 4)])
def test_prompt_then_chunk_then_decode(kb, vb):
    # as a server runs them: prompts admitted, pieces appended and attended, then single tokens; the attention of every
    # call against 64 bits over the rows that it is to see
    c = Case([0, 0], [0, 0], kb=kb, vb=vb, d=128, page=16, dtype="bf16", fill=False, spare=40, width=12)
    order = torch.randperm(40, generator=c.g)[:24].view(2, 12).to(torch.int32)
    c.table = order.numpy()
    table, rot = order.cuda(), K.Rotation(K.rotation_table(200, 128))
    norm = K.HeadNorm(_w(c), _w(c, seed=4))
    lens = [0, 0]
    for step, news in enumerate(([50, 33], [20, 7], [1, 40], None, None)):
        lens = [n + (1 if news is None else m) for n, m in zip(lens, news or [1, 1])]
        cu = None if news is None else torch.tensor([0, news[0], sum(news)], dtype=torch.int32).cuda()
        batch = K.PagedBatch(table, torch.tensor(lens, dtype=torch.int32).cuda(), cu)
        n = 2 if news is None else sum(news)
        k, v, q = c.rows(n, 2), c.rows(n, 2), c.rows(n, 8)
        k_out = torch.empty(n, 2, 128, dtype=c.dtype, device="cuda")
        q = c.cache.append(0, batch, k, v, q=q, rotation=rot, norm=norm, k_out=k_out)
        if step == 0:
            got, lse = c.cache.prompt_attn(batch, q, k_out, v, return_lse=True)
        elif news is not None:
            got, lse = c.cache.chunk_attn(0, batch, q, return_lse=True)
        else:
            got, lse = c.cache.decode_attn(0, batch, q, return_lse=True)
        c.model.data = c.download().copy()
        a = 0
        for b, (L, m) in enumerate(zip(lens, news or [1, 1])):
            last = torch.arange(L - m, L)
            if step == 0:
                kk, vv, parts = *(x[a:a + m].cpu().double().transpose(0, 1) for x in (k_out, v)), None
            else:
                rows = [[c.model.rows(c.table[b], 0, L, h, x) for h in range(2)] for x in (False, True)]
                kk, vv = (torch.stack([torch.from_numpy(y[0]) for y in x]) for x in rows)
                parts = torch.stack([torch.from_numpy(np.abs(y[1]) + np.abs(y[0] - y[1])) for y in rows[0]])
            exp = C.attend(q[a:a + m].cpu(), kk, vv, torch.zeros_like(last), last, c.dtype, 0.0, kb != 16 and step > 0, parts)
            C.close(got[a:a + m], lse[a:a + m], exp)
            a += m
    assert c.cache.device_error() == 0
