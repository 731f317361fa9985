"""Attention of runs of new tokens, over the pages and over prompts' own rows,
against 64 bits (rows read from the plain model of the pages)."""

import math

import numpy as np
import pytest
import torch

import chunk_testutil as C
import paged_testutil as T
from mixed_precision_quantized_quant_gb300 import kvq as K
from test_gpu_paged import PAIRS, Case

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _fast_fill(c, seed=0, mu=1.0):
    """Random rows in every page that a sequence owns, a page at a time (Case fills token by token)."""
    g = torch.Generator().manual_seed(seed)
    m = c.model
    shift = torch.randn(c.hkv, 1, c.d, generator=g) * mu
    for b, n in enumerate(c.lens):
        for i in range(-(-n // c.P)):
            page = c.table[b, i]
            k, v = torch.randn(2, c.hkv, c.P, c.d, generator=g).to(c.dtype).float()
            k = (k + shift).to(c.dtype).float()
            for slot in range(min(c.P, n - i * c.P)):
                if m.kb == 16:
                    for h in range(c.hkv):
                        m.put(page, slot, h, False, k[h, slot])
                        m.put(page, slot, h, True, v[h, slot])
                else:  # any codes, and scales of a few steps
                    for h in range(c.hkv):
                        m.put(page, slot, h, False, k[h, slot])
                        m.put(page, slot, h, True, v[h, slot])
    c.upload()


def _dense(c, b, n):
    """Keys, values [hkv, n, d] of sequence b's positions and |scale code| + |zero| of its keys, in 64 bits."""
    ks, vs, ps = [], [], []
    for h in range(c.hkv):
        k, kc, _ = c.model.rows(c.table[b], 0, n, h, False)
        v, _, _ = c.model.rows(c.table[b], 0, n, h, True)
        ks.append(torch.from_numpy(k)), vs.append(torch.from_numpy(v))
        ps.append(torch.from_numpy(np.abs(kc) + np.abs(k - kc)))
    return torch.stack(ks), torch.stack(vs), torch.stack(ps)


def _check(c, q=None, scale=0.0, window=0, extra=0, how="fused", stream=None, tol_scale=1.0):
    n = sum(c.news) + extra if c.news is not None else len(c.lens)
    q = c.rows(n, c.hq, how) if q is None else q
    out = torch.full((n, c.hq, c.d), 7.0, dtype=c.dtype, device="cuda")
    got, lse = c.cache.chunk_attn(c.layer, c.batch, q, out=out, scale=scale, window=window, return_lse=True, stream=stream)
    assert got is out
    torch.cuda.synchronize()
    assert c.cache.device_error() == 0
    row = 0
    for b, L in enumerate(c.lens):
        m = 1 if c.news is None else c.news[b]
        if L and m:
            k, v, parts = _dense(c, b, L)
            last = torch.arange(L - m, L)
            first = (last - window + 1).clamp(min=0) if window else torch.zeros_like(last)
            exp = C.attend(q[row:row + m].cpu(), k, v, first, last, c.dtype, scale, c.model.kb != 16, parts)
            C.close(got[row:row + m], lse[row:row + m], exp)
        row += m
    assert bool((got[row:] == 7).all())
    return got, lse


# ---------------------------------------------------------------- over the pages

@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kb,vb", PAIRS)
def test_chunk_pairs(kb, vb, d, dtype):
    # one token, some, all of a sequence, none, a page's edge; rows behind the last sequence
    c = Case([1, 40, 33, 17, 70, 16], [1, 5, 33, 0, 37, 16], kb=kb, vb=vb, d=d, dtype=dtype, page=32)
    _check(c, extra=3)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 4), (4, 2)])
def test_chunk_pages(kb, vb, page):
    # sequences of several tiles, pages that end inside a tile
    c = Case([300, 129, 128, 257], [150, 129, 1, 40], kb=kb, vb=vb, d=128, page=page, dtype="bf16")
    _check(c)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (6, 2), (7, 1), (14, 2), (8, 1), (10, 2), (3, 1)])
@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 8)])
def test_chunk_heads(kb, vb, hq, hkv):
    c = Case([150, 20, 64], [40, 20, 33], kb=kb, vb=vb, hq=hq, hkv=hkv, d=64, page=16)
    _check(c)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 100, 127, 128, 129, 1000])
@pytest.mark.parametrize("kb,vb", [(16, 16), (4, 4)])
def test_chunk_window(kb, vb, window):
    c = Case([400, 30, 131], [300, 7, 131], kb=kb, vb=vb, hq=4, hkv=1, d=64, page=32)
    _check(c, window=window)


def test_chunk_window_reads_no_page_before_it():
    # pages wholly before every row's window are nobody's: bad numbers there are not read
    for kb, vb in ((16, 16), (8, 4)):
        c = Case([500], [10], kb=kb, vb=vb, d=64, page=16)
        table = c.table.copy()
        table[0, :(490 - 99) // 16] = -1
        c.batch = K.PagedBatch(torch.from_numpy(table).cuda(), _i32(c.lens), _i32([0, 10]))
        _check(c, window=100)


@pytest.mark.parametrize("how", ["fused", "odd"])
@pytest.mark.parametrize("kb,vb", [(16, 16), (4, 8)])
def test_chunk_scale_and_strides(kb, vb, how):
    for scale in (0.31, -0.2, 4.0):
        c = Case([77, 9], [20, 9], kb=kb, vb=vb, d=64)
        _check(c, scale=scale, how=how)


@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 4), (2, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_of_one_row_each_is_decode(kb, vb, d):
    # cu_tokens None, a padded place among the sequences; near decode_attn, which rounds less
    c = Case([300, 0, 1, 77], kb=kb, vb=vb, d=d, page=64)
    q = c.rows(4, 8)
    got, lse = _check(c, q=q)
    o, l = c.cache.decode_attn(0, c.batch, q, return_lse=True)
    keep = [0, 2, 3]
    assert float((got[keep].float() - o[keep].float()).norm() / o[keep].float().norm()) < 2e-3
    assert torch.allclose(lse[keep], l[keep], rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("kb,vb", [(16, 16), (4, 2)])
@pytest.mark.parametrize("seqs", [40, 130])
def test_chunk_of_many_sequences(kb, vb, seqs):
    g = torch.Generator().manual_seed(seqs)
    news = torch.randint(0, 4, (seqs,), generator=g)
    news[5:30:2] = 0
    lens = (news + torch.randint(0, 25, (seqs,), generator=g)).tolist()
    c = Case(lens, news.tolist(), kb=kb, vb=vb, d=64, hq=2, hkv=1, page=16)
    _check(c, extra=1)


@pytest.mark.parametrize("kb,vb,dtype", [(16, 16, "bf16"), (16, 16, "fp16"), (8, 4, "bf16"), (4, 2, "fp16")])
def test_chunk_long(kb, vb, dtype):
    # few rows over a long cache, cut among many CTAs, beside short ones
    c = Case([2500, 3, 700], [3, 2, 5], kb=kb, vb=vb, d=128, dtype=dtype, page=64, hkv=1, hq=8)
    _check(c)


def test_chunk_many_tiles_of_queries():
    # several tiles of queries a sequence, lengths that end inside them
    c = Case([600, 333], [600, 200], d=64, hq=8, hkv=1, page=16)
    _check(c)


@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 8)])
def test_chunk_is_deterministic(kb, vb):
    c = Case([900, 20, 300], [9, 20, 100], kb=kb, vb=vb, d=128, page=16, hkv=1, hq=4)
    q = c.rows(129, 4)
    a = c.cache.chunk_attn(0, c.batch, q)
    for _ in range(5):
        assert torch.equal(a, c.cache.chunk_attn(0, c.batch, q))


def test_chunk_empty_rows_and_infinite_scores():
    # keys of -infinity leave a row nothing: 0 and -infinity
    c = Case([30], [30], d=64, hq=2, hkv=1, dtype="bf16")
    for p in range(30):
        x = torch.full((64,), 0.0)
        x[0] = -math.inf if p < 20 else 1.0
        c.model.put(c.table[0, p // 16], p % 16, 0, False, x)
    c.upload()
    q = torch.ones(30, 2, 64, dtype=torch.bfloat16, device="cuda")
    got, lse = c.cache.chunk_attn(0, c.batch, q, return_lse=True)
    assert bool((got[:20] == 0).all()) and bool((lse[:20] == -math.inf).all())
    assert bool(torch.isfinite(got[20:].float()).all()) and bool(torch.isfinite(lse[20:]).all())
    # a score of +infinity is no number where it is seen, and not before
    q[:] = -1
    got = c.cache.chunk_attn(0, c.batch, q)
    assert bool(torch.isnan(got.float()).all())


@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 4), (4, 8)])
@pytest.mark.parametrize("what", ["nan", "inf"])
@pytest.mark.parametrize("window", [0, 40])
def test_chunk_keeps_what_is_not_seen_out(kb, vb, what, window):
    # NaN or infinite values (16 bits: in two channels; codes: a NaN row) in the middle of the new tokens:
    # rows before them, and rows whose window has left them behind, are as without them
    if kb != 16 and what == "inf":
        pytest.skip("rows are clamped when they are quantized")
    c = Case([200, 60], [150, 60], kb=kb, vb=vb, d=64, hq=4, hkv=2, dtype="bf16", page=32)
    q = c.rows(210, 4)
    clean, clse = _check(c, q=q, window=window)
    at = 120  # position: row 70 of sequence 0
    bad = math.nan if what == "nan" else math.inf
    for h in range(2):
        k, _, _ = c.model.get(c.table[0, at // 32], at % 32, h, False)
        v, _, _ = c.model.get(c.table[0, at // 32], at % 32, h, True)
        v = torch.from_numpy(v).float()
        v[5] = bad
        v[40] = -bad
        c.model.put(c.table[0, at // 32], at % 32, h, True, v)
    c.upload()
    got, lse = c.cache.chunk_attn(0, c.batch, q, window=window, return_lse=True)
    assert torch.equal(lse, clse)
    hit = torch.zeros(210, dtype=torch.bool)
    hit[70:150] = True
    if window:
        hit[70 + window:150] = False
    assert torch.equal(got[~hit], clean[~hit])
    g = got[hit].float()
    if kb == 16:
        assert not bool(torch.isfinite(g[..., [5, 40]]).any())
        rest = [x for x in range(64) if x not in (5, 40)]
        assert torch.equal(got[hit][..., rest], clean[hit][..., rest])
        if what == "inf":
            assert bool((g[..., 5] == math.inf).all()) and bool((g[..., 40] == -math.inf).all())
    else:
        assert bool(torch.isnan(g).all())
    # a NaN key: NaN from the row that sees it on, not before
    for h in range(2):
        k, _, _ = c.model.get(c.table[0, at // 32], at % 32, h, False)
        k = torch.from_numpy(k).float()
        k[7] = math.nan
        c.model.put(c.table[0, at // 32], at % 32, h, False, k)
    c.upload()
    got, lse = c.cache.chunk_attn(0, c.batch, q, window=window, return_lse=True)
    assert torch.equal(got[~hit], clean[~hit]) and torch.equal(lse[~hit], clse[~hit])
    assert bool(torch.isnan(got[hit].float()).all()) and bool(torch.isnan(lse[hit]).all())


def test_chunk_weights_far_below_the_greatest():
    # one token of weight 1 among many of 2^-20 whose values count together
    for dtype in ("fp16", "bf16"):
        c = Case([1025], [1], d=64, hq=1, hkv=1, dtype=dtype, page=64, fill=False)
        for p in range(1025):
            k, v = torch.zeros(64), torch.full((64,), 1.0 if p else 0.0)
            k[0] = 0.0 if p else 8.0 * 20 * math.log(2)
            c.model.put(c.table[0, p // 64], p % 64, 0, False, k)
            c.model.put(c.table[0, p // 64], p % 64, 0, True, v)
        c.upload()
        q = torch.zeros(1, 1, 64, dtype=c.dtype, device="cuda")
        q[..., 0] = 1
        _check(c, q=q)


def test_chunk_large_and_small_values():
    # values at both ends of the type, queries of any size
    for dtype, kb, vb in (("fp16", 16, 16), ("bf16", 16, 16), ("fp16", 8, 8), ("bf16", 4, 4)):
        for big in (1.0, 3e4, 2.0 ** -10):
            c = Case([90], [90], d=64, kb=kb, vb=vb, hq=2, hkv=1, dtype=dtype, page=16, fill=False)
            g = torch.Generator().manual_seed(1)
            for p in range(90):
                c.model.put(c.table[0, p // 16], p % 16, 0, False, torch.randn(64, generator=g).to(c.dtype).float())
                c.model.put(c.table[0, p // 16], p % 16, 0, True, (torch.rand(64, generator=g) * 2 - 1).mul(big).to(c.dtype).float())
            c.upload()
            q = (torch.randn(90, 2, 64, generator=g) * torch.logspace(-4, 1, 90)[:, None, None]).to(c.dtype).cuda()
            _check(c, q=q)


def test_chunk_bad_pages_lengths_and_ends():
    c = Case([40, 20], [3, 2], page=16)
    q = c.rows(5, 8)
    n = c.model.data.shape[0]

    def run(table, lens, cu):
        out = torch.full((5, 8, 64), 7.0, dtype=c.dtype, device="cuda")
        c.cache.chunk_attn(0, K.PagedBatch(_i32(table), _i32(lens), _i32(cu)), q, out=out)
        return c.cache.device_error(), (out != 7).flatten(1).any(1).tolist()

    good = [[0, 1, 2], [3, 4, 0]]
    assert run(good, [40, 20], [0, 3, 5]) == (0, [True] * 5)
    for bad in (-1, n, 2 ** 31 - 1):
        code, wrote = run([[0, bad, 2], [3, 4, 0]], [40, 20], [0, 3, 5])
        assert code == 4 and wrote[3:] == [True, True]
    for lens in ([49, 20], [-1, 20], [2 ** 31 - 1, 20], [2, 20]):
        code, wrote = run(good, lens, [0, 3, 5])
        assert code == 2 and wrote == [False] * 3 + [True] * 2
    code, wrote = run(good, [40, 20], [0, 3, 2])
    assert code == 2 and not any(wrote[3:])
    # rows that the tensors do not hold are not written; the others of that sequence are
    code, wrote = run(good, [40, 20], [0, 3, 9])
    assert code in (0, 2) and wrote[:3] == [True] * 3
    code, wrote = run(good, [40, 20], [-2, 3, 5])
    assert code in (0, 2) and wrote[3:] == [True, True]
    assert run(good, [40, 20], [0, 3, 5]) == (0, [True] * 5)
    # no rows, and sequences without tokens
    assert run(good, [0, 0], [0, 0, 0]) == (0, [False] * 5)


def test_chunk_captured_follows_its_tensors():
    # two captured calls side by side, replayed after lengths and rows changed
    c = Case([200, 90], [5, 3], kb=8, vb=4, d=128, page=16)
    d = Case([310, 64], [4, 4], kb=8, vb=4, d=128, page=16, seed=3)
    runs = []
    for x in (c, d):
        q = x.rows(8, 8).clone()
        lens, cu = _i32([0, 0]), _i32([0, 0, 0])
        batch = K.PagedBatch(torch.from_numpy(x.table).cuda(), lens, cu)
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        x.cache.chunk_attn(0, batch, q)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            out, lse = x.cache.chunk_attn(0, batch, q, return_lse=True)
        runs.append((x, q, lens, cu, batch, s, g, out, lse))
    for news in ([5, 3], [1, 7], [8, 0]):
        for x, q, lens, cu, batch, s, g, out, lse in runs:
            q.copy_(x.rows(8, 8))
            lens.copy_(_i32(x.lens))
            cu.copy_(_i32([0, news[0], sum(news)]))
        torch.cuda.synchronize()
        for x, *_, s, g, _, _ in runs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for x, q, lens, cu, batch, s, g, out, lse in runs:
            e, le = x.cache.chunk_attn(0, batch, q, return_lse=True)
            assert torch.equal(out, e) and torch.equal(lse, le)
            x.news, x.batch = news, batch
            _check(x, q=q)


def test_chunk_on_a_stream_of_its_own():
    c = Case([100, 30], [50, 2], kb=4, vb=4, d=128)
    s = torch.cuda.Stream()
    q = c.rows(52, 8)
    s.wait_stream(torch.cuda.current_stream())
    _check(c, q=q, stream=s)


# ---------------------------------------------------------------- prompts

def _prompt_case(news, hq, hkv, d, dtype, extra=0, seed=0, how="fused"):
    c = Case([1] * len(news), news, hq=hq, hkv=hkv, d=d, dtype=dtype, fill=False, seed=seed)
    n = sum(news) + extra
    return c, c.rows(n, hq, how), c.rows(n, hkv, how), c.rows(n, hkv, how)


def _check_prompt(c, q, k, v, scale=0.0, window=0, stream=None):
    out = torch.full(q.shape, 7.0, dtype=c.dtype, device="cuda")
    got, lse = c.cache.prompt_attn(c.batch, q, k, v, out=out, scale=scale, window=window, return_lse=True, stream=stream)
    assert got is out
    torch.cuda.synchronize()
    assert c.cache.device_error() == 0
    a = 0
    for m in c.news:
        if m:
            last = torch.arange(m)
            first = (last - window + 1).clamp(min=0) if window else torch.zeros_like(last)
            kk, vv = (x[a:a + m].cpu().double().transpose(0, 1) for x in (k, v))
            C.close(got[a:a + m], lse[a:a + m], C.attend(q[a:a + m].cpu(), kk, vv, first, last, c.dtype, scale))
        a += m
    assert bool((got[a:] == 7).all())
    return got, lse


@pytest.mark.parametrize("how", ["fused", "odd"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_packed(d, dtype, how):
    _check_prompt(*_prompt_case([1, 37, 0, 128, 129, 300, 2], 8, 2, d, dtype, extra=5, how=how))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (7, 1), (14, 2), (8, 1), (10, 2), (3, 1)])
def test_prompt_heads(hq, hkv):
    _check_prompt(*_prompt_case([200, 63], hq, hkv, 128, "bf16"))


@pytest.mark.parametrize("window", [1, 2, 100, 128, 129, 1000])
def test_prompt_window(window):
    _check_prompt(*_prompt_case([400, 30], 4, 1, 64, "fp16"), window=window)


def test_prompt_long():
    _check_prompt(*_prompt_case([2100, 900], 2, 1, 128, "bf16"), scale=0.2)


def test_prompt_one_row_each():
    # cu_tokens None: prompts of one token, which get their own values
    c, q, k, v = _prompt_case([1, 1, 1], 8, 2, 64, "fp16")
    batch = K.PagedBatch(torch.from_numpy(c.table).cuda(), _i32([0, 5, 9]))
    got, lse = c.cache.prompt_attn(batch, q, k, v, return_lse=True)
    assert torch.equal(got, v.repeat_interleave(4, 1))
    e = (q.double().view(3, 2, 4, 64) * k.double()[:, :, None]).sum(-1).view(3, 8) / 8
    assert torch.allclose(lse.double(), e, atol=1e-5)


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("how", ["fused", "odd"])
def test_prompt_keeps_others_rows_out(window, how):
    # NaN and infinities in later rows, in rows behind the window, in other prompts and behind them all
    c, q, k, v = _prompt_case([150, 90, 20], 4, 2, 64, "bf16", extra=40, how=how)
    k, v = k.clone(), v.clone()
    if how == "odd":
        pad = torch.zeros(300, 2 * 64 + 3, dtype=k.dtype, device="cuda")
        k, v = (pad.clone()[:, 3:].unflatten(1, (2, 64)).copy_(x) for x in (k, v))
    clean, clse = c.cache.prompt_attn(c.batch, q, k, v, window=window, return_lse=True)
    v[100, :, 5] = math.nan
    v[101, :, 6] = math.inf
    v[260:] = math.nan
    k[260:] = math.nan
    got, lse = c.cache.prompt_attn(c.batch, q, k, v, window=window, return_lse=True)
    hit = torch.zeros(300, 64, dtype=torch.bool)
    hit[100:150 if not window else 140, 5] = True
    hit[101:150 if not window else 141, 6] = True
    hit = hit[:260, None].expand(260, 4, 64)
    assert torch.equal(lse[:260], clse[:260])
    assert torch.equal(got[:260][~hit], clean[:260][~hit])
    assert not bool(torch.isfinite(got[:260][hit].float()).any())
    k[50] = math.nan
    got, lse = c.cache.prompt_attn(c.batch, q, k, v, window=window, return_lse=True)
    end = 150 if not window else 90
    rows = torch.zeros(260, dtype=torch.bool)
    rows[50:end] = True
    assert bool(torch.isnan(lse[:260][rows]).all()) and torch.equal(lse[:260][~rows], clse[:260][~rows])
    assert bool(torch.isnan(got[:260][rows].float()).all())
    assert torch.equal(got[:50], clean[:50]) and torch.equal(got[150:260], clean[150:260])


def test_prompt_ends():
    c, q, k, v = _prompt_case([3, 2], 8, 2, 64, "fp16")

    def run(cu):
        out = torch.full((5, 8, 64), 7.0, dtype=c.dtype, device="cuda")
        c.cache.prompt_attn(K.PagedBatch(torch.from_numpy(c.table).cuda(), _i32([-5, 2 ** 31 - 1]), _i32(cu)), q, k, v, out=out)
        return c.cache.device_error(), (out != 7).flatten(1).any(1).tolist()

    assert run([0, 3, 5]) == (0, [True] * 5)
    code, wrote = run([0, 3, 2])  # (row 2 lies between ends that do not ascend)
    assert code == 2 and wrote[:2] == [True] * 2 and wrote[3:] == [False] * 2
    assert run([0, 3, 9]) == (2, [True] * 3 + [False] * 2)
    assert run([-1, 3, 5]) == (2, [False] * 3 + [True] * 2)
    assert run([2, 2, 4]) == (0, [False, False, True, True, False])


def test_prompt_is_chunk_over_its_pages():
    # a prompt appended to an unquantized layer: the pages hold its rows
    c = Case([260, 31], [260, 31], d=128, page=32, dtype="bf16", fill=False)
    k, v, q = c.rows(291, 2), c.rows(291, 2), c.rows(291, 8)
    c.cache.append(0, c.batch, k, v)
    a, la = c.cache.chunk_attn(0, c.batch, q, return_lse=True)
    b, lb = c.cache.prompt_attn(c.batch, q, k, v, return_lse=True)
    assert float((a.float() - b.float()).abs().max()) < 1e-2 and torch.allclose(la, lb, rtol=1e-6, atol=1e-5)


# ---------------------------------------------------------------- refusals

def test_refusals():
    c = Case([20, 5], [2, 1], kb=4, vb=4, d=64, hq=4, hkv=2)
    q, k, v = c.rows(3, 4), c.rows(3, 2), c.rows(3, 2)
    t, u = c.cache.chunk_attn, c.cache.prompt_attn
    half, one = torch.float16, K.PagedBatch(*c.batch._keep[:2])
    for fn in (lambda: t(0, c.batch, q.bfloat16()), lambda: t(0, c.batch, k), lambda: t(0, c.batch, q.cpu()), lambda: t(0, one, q),
               lambda: t(0, c.batch, q, out=torch.empty(3, 4, 64, device="cuda")),
               lambda: t(0, c.batch, q, out=torch.empty(2, 4, 64, dtype=half, device="cuda")),
               lambda: t(0, c.batch, q, out=torch.empty(3, 64, 4, dtype=half, device="cuda").transpose(1, 2)),
               lambda: t(0, c.batch, q, scale=1e-39), lambda: u(c.batch, q, k[:2], v), lambda: u(c.batch, q, k, v.float()),
               lambda: u(one, q, k, v), lambda: u(c.batch, q, q, v), lambda: u(c.batch, q, k, v.cpu())):
        with pytest.raises(ValueError):
            fn()
    odd = torch.empty(3 * 4 * 64 + 1, dtype=half, device="cuda")[1:].view(3, 4, 64)
    for fn, code in ((lambda: t(1, c.batch, q), 1), (lambda: t(-1, c.batch, q), 1), (lambda: t(0, c.batch, q, window=-1), 1),
                     (lambda: t(0, c.batch, q, window=2 ** 31), 1), (lambda: t(0, c.batch, q, scale=math.nan), 1),
                     (lambda: t(0, c.batch, q, scale=3e38), 1), (lambda: t(0, c.batch, q, out=odd), 3),
                     (lambda: u(c.batch, q, k, v, window=-1), 1), (lambda: u(c.batch, q, k, v, scale=math.inf), 1),
                     (lambda: u(c.batch, q, k, v, out=odd), 3)):
        with pytest.raises(K.KVQError) as e:
            fn()
        assert e.value.status == code
    L, h, b, s = K.load(), c.cache.h, c.batch.args, torch.cuda.current_stream().cuda_stream
    rq, rk = c.cache._rows(q, "q", 3, 4), c.cache._rows(k, "k", 3, 2)
    nw = K.kvq_paged_chunk_workspace_bytes(h, 2, 3)
    out, ws = torch.empty(3, 4, 64, dtype=half, device="cuda"), torch.empty(nw + 256, dtype=torch.uint8, device="cuda")
    o, w = out.data_ptr(), ws.data_ptr()
    assert K.kvq_paged_chunk_workspace_bytes(h, 0, 3) == 0 and K.kvq_paged_chunk_workspace_bytes(h, 1, -1) == 0
    chunk = lambda *a: L.kvq_paged_chunk_attn(h, 0, *a, s)  # noqa: E731
    prompt = lambda *a: L.kvq_paged_prompt_attn(h, *a, s)  # noqa: E731
    assert chunk(b, rq, None, None, 0.0, 0, 3, w, nw) == 1
    assert chunk(b, None, o, None, 0.0, 0, 3, w, nw) == 1
    assert chunk(None, rq, o, None, 0.0, 0, 3, w, nw) == 1
    assert chunk(b, rq, o, None, 0.0, 0, -1, w, nw) == 1
    assert chunk(b, rq, o, None, 0.0, 0, 3, None, nw) == 1
    assert chunk(b, rq, o, None, 0.0, 0, 3, w + 16, nw) == 3
    assert chunk(b, rq, o, o + 2, 0.0, 0, 3, w, nw) == 3
    assert chunk(b, rq, o, None, 0.0, 0, 3, w, nw - 1) == 4
    assert chunk(b, K.Rows(rq.data + 1, 1, 1), o, None, 0.0, 0, 3, w, nw) == 3
    assert prompt(b, rq, None, rk, o, None, 0.0, 0, 3, w, nw) == 1
    assert prompt(b, rq, rk, K.Rows(None, 1, 1), o, None, 0.0, 0, 3, w, nw) == 1
    assert prompt(b, rq, rk, rk, o, None, 0.0, 0, 3, w, nw - 1) == 4
    assert chunk(b, rq, o, None, 0.0, 0, 0, w, nw) == 0  # nothing to do
    assert c.cache.device_error() == 0
    assert t(0, c.batch, q[:0]).shape == (0, 4, 64)
    c.cache.close()
    with pytest.raises(K.KVQError):
        t(0, c.batch, q)
