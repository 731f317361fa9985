"""Calls at the edges of what the paged cache documents."""

import math

import numpy as np
import pytest
import torch

from mixed_precision_quantized_quant_gb300 import kvq as K
from test_gpu_paged import Case, _check_append

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


# ---------------------------------------------------------------- rows of sequences

# a row a CTA, 2 rows a CTA, 31 rows a CTA
@pytest.mark.parametrize("n", [12, 612, 14_000])
def test_ends_that_do_not_ascend(n):
    # a row is written only where a sequence's two ends hold it, and only to its place there
    rng = np.random.default_rng(n)
    cases = [[0, 5, 1, 2, 9], [0, 9, 9, 9, 9, 1, 1, 2], [3, 4, 4, 1, 2, 7]]
    cases += [rng.integers(0, 13, rng.integers(3, 12)).tolist() for _ in range(20)]
    for ends in cases:
        S = len(ends) - 1
        c = Case([10] * S, page=16, fill=False)
        batch = K.PagedBatch(_i32(c.table), _i32(c.lens), _i32(ends))
        may = np.zeros(c.model.data.shape, bool)
        for s in range(S):
            for row in range(ends[s], min(ends[s + 1], n)):
                p = 10 - (ends[s + 1] - row)
                for is_v in (False, True):
                    start, m, xor = c.model._row(is_v, max(p, 0))
                    if p >= 0:
                        may[c.table[s, 0], :, 0, start + (np.arange(m) ^ xor)] = True
        c.cache.append(0, batch, c.rows(n, 2), c.rows(n, 2))
        assert (c.download()[~may] == 0xFF).all(), ends
        k, v = (torch.full((n, 2, 64), 7.0, dtype=c.dtype, device="cuda") for _ in range(2))
        code = c.cache.device_error()
        c.cache.read(0, batch, n, K=k, V=v)
        held = [any(ends[s] <= row < ends[s + 1] and ends[s + 1] - row <= 10 for s in range(S)) for row in range(n)]
        for x in (k, v):
            assert bool((x[~torch.tensor(held).cuda()] == 7).all()), ends
        assert c.cache.device_error() == code and code in (0, 2)
        if ends == [0, 9, 9, 9, 9, 1, 1, 2] and n == 12 or ends == [0, 5, 1, 2, 9] and n == 14_000:
            assert code == 2, ends  # row 3 counts as a sequence's whose ends are 1 and 2


@pytest.mark.parametrize("kb,vb", [(16, 16), (4, 2)])
@pytest.mark.parametrize("seqs", [33, 70, 200])
def test_append_and_read_of_many_sequences(seqs, kb, vb):
    # rows whose sequences' ends are found 32 at a time, runs of sequences without rows among them
    g = torch.Generator().manual_seed(seqs)
    news = torch.randint(0, 6, (seqs,), generator=g)
    news[3:3 + seqs // 2:2] = 0
    news[seqs // 3:seqs // 3 + 40] = 0
    news[-1] = 3
    lens = (news + torch.randint(0, 20, (seqs,), generator=g)).tolist()
    c = Case(lens, news.tolist(), kb=kb, vb=vb, d=64, hq=2, hkv=1, page=16, fill=False)
    _check_append(c, dim=64, extra=2)
    n = int(news.sum())
    k, v = c.cache.read(0, c.batch, n)
    for row, b, p in c.places():
        for x, is_v in ((k, False), (v, True)):
            e, _, _ = c.model.get(c.table[b, p // 16], p % 16, 0, is_v)
            assert torch.equal(x[row, 0].cpu(), torch.from_numpy(e).float().to(c.dtype))


@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 4)])
def test_append_and_read_on_a_stream_of_their_own(kb, vb):
    c = Case([40, 3], [30, 3], kb=kb, vb=vb, d=64, fill=False)
    s = torch.cuda.Stream()
    k, v, q = c.rows(33, 2), c.rows(33, 2), c.rows(33, 8)
    rot = K.Rotation(K.rotation_table(60, 64))
    s.wait_stream(torch.cuda.current_stream())
    got = c.cache.append(0, c.batch, k, v, q=q, rotation=rot, stream=s)
    rk, rv = c.cache.read(0, c.batch, 33, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    got, rk, rv = got.clone(), rk.clone(), rv.clone()
    again = c.cache.append(0, c.batch, k, v, q=q, rotation=rot)
    ak, av = c.cache.read(0, c.batch, 33)
    assert torch.equal(got, again) and torch.equal(rk, ak) and torch.equal(rv, av)
    assert float(rk.abs().max()) > 0 and c.cache.device_error(s) == 0


# ---------------------------------------------------------------- tables

def test_the_widest_table():
    # max_pages * page_size = 2^30 positions, the documented limit; one page more is refused
    P, pages = 128, 1 << 23
    c = Case([300], [300], d=64, hq=2, hkv=1, page=P, fill=False)
    table = torch.zeros(1, pages + 1, dtype=torch.int32, device="cuda")
    table[0, :3] = torch.from_numpy(c.table[0]).cuda()
    lens, cu = _i32([300]), _i32([0, 300])
    k, v, q = c.rows(300, 1), c.rows(300, 1), c.rows(1, 2)
    narrow = K.PagedBatch(table[:, :3].contiguous(), lens, cu)
    c.cache.append(0, narrow, k, v)
    expect = c.cache.decode_attn(0, narrow, q), *c.cache.read(0, narrow, 300)
    b = K.PagedBatch(table[:, :pages].contiguous(), lens, cu)
    c.cache.append(0, b, k, v)
    got = c.cache.decode_attn(0, b, q), *c.cache.read(0, b, 300)
    assert torch.equal(got[1], expect[1]) and torch.equal(got[2], expect[2])
    assert float((got[0].float() - expect[0].float()).abs().max()) <= 2 ** -11 * 2 * float(expect[0].abs().max())
    wide = K.PagedBatch(table, lens, cu)
    for fn in (lambda: c.cache.append(0, wide, k, v), lambda: c.cache.decode_attn(0, wide, q),
               lambda: c.cache.read(0, wide, 300)):
        with pytest.raises(K.KVQError) as e:
            fn()
        assert e.value.status == 1
    assert c.cache.device_error() == 0


# ---------------------------------------------------------------- scores

@pytest.mark.parametrize("width", [None, 200])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_scores_of_minus_infinity_have_no_weight(dtype, width):
    # keys of -infinity over whole chunks, ahead of and between others, and over all of a sequence
    c = Case([200, 200, 33], d=64, hq=4, hkv=1, dtype=dtype, width=width)
    dark = [(0, p) for p in range(0, 70)] + [(0, p) for p in range(128, 150)] + [(1, p) for p in range(199)] + \
           [(2, p) for p in range(33)]
    for b, p in dark:
        c.model.put(c.table[b, p // 16], p % 16, 0, False, torch.full((64,), -math.inf))
    c.upload()
    q = c.rows(3, 4).abs() + 0.1
    out, lse = c.cache.decode_attn(0, c.batch, q, return_lse=True)
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    gone = {b: [p for x, p in dark if x == b] for b in range(3)}
    for b, n in ((0, 200), (1, 200)):
        live = [p for p in range(n) if p not in gone[b]]
        k, _, _ = c.model.rows(c.table[b], 0, n, 0, False)
        v, _, _ = c.model.rows(c.table[b], 0, n, 0, True)
        for j in range(4):
            qq = q[b, j].double().cpu().numpy()
            t = k[live] @ qq / 8
            p = np.exp(t - t.max())
            e = 80 * 2.0 ** -23 / 8 * (np.abs(k[live]) @ np.abs(qq)).max() + 2.0 ** -20
            tol = torch.finfo(c.dtype).eps / 2 * np.abs(p @ v[live] / p.sum()) + \
                (2.0 ** -16 + 2 * e + 89 * 2.0 ** -23) * (p @ np.abs(v[live])) / p.sum() + 2.0 ** -24
            assert (np.abs(o[b, j] - p @ v[live] / p.sum()) <= tol).all()
            assert abs(l[b, j] - t.max() - np.log(p.sum())) <= 2 * e + 2.0 ** -16 + 2.0 ** -20 * abs(l[b, j])
    assert (o[2] == 0).all() and (l[2] == -math.inf).all()
    assert c.cache.device_error() == 0


@pytest.mark.parametrize("width", [None, 200])
def test_a_scale_that_leaves_fp32_is_refused(width):
    c = Case([40], d=64, width=width)
    q = c.rows(1, 8)
    for scale in (3e38, -3e38, 1e-46):
        with pytest.raises((K.KVQError, ValueError)):
            c.cache.decode_attn(0, c.batch, q, scale=scale)
    out, lse = c.cache.decode_attn(0, c.batch, q, scale=1e-30, return_lse=True)
    v = c.model.rows(c.table[0], 0, 40, 0, True)[0].mean(0)
    assert np.abs(out[0, 0].double().cpu().numpy() - v).max() <= 2 ** -11 * 4 and float((lse - math.log(40)).abs().max()) < 1e-5


# ---------------------------------------------------------------- what the binding takes

def test_numbers_that_do_not_fit_the_c_types_are_refused():
    c = Case([40, 20], [1, 1], kb=8, vb=4, d=64)
    q, k, v = c.rows(2, 8), c.rows(2, 2), c.rows(2, 2)
    before = c.download().copy()
    for layer in (2 ** 32, -2 ** 32, 2 ** 64):
        for fn in (lambda: c.cache.append(layer, c.batch, k, v), lambda: c.cache.decode_attn(layer, c.batch, q),
                   lambda: c.cache.read(layer, c.batch, 2), lambda: c.cache.view(layer)):
            with pytest.raises(K.KVQError) as e:
                fn()
            assert e.value.status == 1
    for window in (2 ** 32, 2 ** 32 + 5, 2 ** 31, -2 ** 32 + 7):
        with pytest.raises(K.KVQError) as e:
            c.cache.decode_attn(0, c.batch, q, window=window)
        assert e.value.status == 1
    wide = k[:1].expand(2 ** 32 + 2, 2, 64)
    for fn in (lambda: c.cache.append(0, c.batch, wide, wide),
               lambda: c.cache.read(0, c.batch, 2 ** 32 + 2, K=wide, V=wide)):
        with pytest.raises((K.KVQError, ValueError)):
            fn()
    assert np.array_equal(c.download(), before) and c.cache.device_error() == 0
    a = c.cache.decode_attn(0, c.batch, q, window=2 ** 31 - 1)
    assert torch.equal(a, c.cache.decode_attn(0, c.batch, q))


def test_outputs_that_overlap_themselves_are_refused():
    c = Case([40, 20, 9], [1, 1, 1], kb=8, vb=4, d=64, hq=4, hkv=2)
    q, k, v = c.rows(3, 4), c.rows(3, 2), c.rows(3, 2)
    before = c.download().copy()
    half = torch.float16
    flat = torch.zeros(3 * 4 * 64, dtype=half, device="cuda")
    for n, strides in ((4, (0, 64, 1)), (4, (4 * 64, 0, 1)), (4, (128, 64, 1)), (4, (64, 32, 1)), (2, (0, 64, 1)), (2, (64, 64, 1)),
                       (2, (128, 63, 1))):
        out = flat.as_strided((3, n, 64), strides)
        for fn in (lambda: c.cache.append(0, c.batch, k, v, q=q, q_out=out),) if n == 4 else (
                lambda: c.cache.read(0, c.batch, 3, K=out), lambda: c.cache.read(0, c.batch, 3, V=out)):
            with pytest.raises(ValueError):
                fn()
    assert np.array_equal(c.download(), before) and not bool(flat.any())
    # heads outside, tokens inside; inputs that repeat a row
    out = torch.zeros(4, 3, 64, dtype=half, device="cuda").transpose(0, 1)
    one = k[:1].expand(3, 2, 64)
    got = c.cache.append(0, c.batch, one, one, q=q, q_out=out)
    assert got is out and torch.equal(got, q)
    rk, _ = c.cache.read(0, c.batch, 3)
    assert torch.equal(rk[0], rk[2])


def test_the_functions_of_the_c_names():
    # the binding's functions by the names of the C entries do what the class does
    c = Case([40, 20], [3, 2], kb=8, vb=4, d=64, hq=4, hkv=2)
    h, s = c.cache.h, torch.cuda.current_stream().cuda_stream
    q, k, v = c.rows(5, 4), c.rows(5, 2), c.rows(5, 2)
    out, rk, rv = torch.empty(2, 4, 64, dtype=c.dtype, device="cuda"), torch.empty_like(k), torch.empty_like(v)
    qo = torch.empty(5, 4, 64, dtype=c.dtype, device="cuda")
    rot = K.Rotation(K.rotation_table(60, 64))

    def rows(x):
        return K.Rows(x.data_ptr(), x.stride(0), x.stride(1))

    K.kvq_paged_append(h, 0, c.batch.args, rows(k), rows(v), rows(q), rows(qo), rot.args, 5, s)
    mine = c.download().copy()
    K.kvq_paged_read(h, 0, c.batch.args, rows(rk), rows(rv), 5, s)
    ws = torch.empty(K.kvq_paged_workspace_bytes(h, 2), dtype=torch.uint8, device="cuda")
    K.kvq_paged_decode_attn(h, 0, c.batch.args, rows(qo), out.data_ptr(), None, 0.0, 0, ws.data_ptr(), ws.numel(), s)
    assert torch.equal(qo, c.cache.append(0, c.batch, k, v, q=q, rotation=rot))
    assert np.array_equal(mine, c.download())
    ek, ev = c.cache.read(0, c.batch, 5)
    assert torch.equal(rk, ek) and torch.equal(rv, ev)
    assert torch.equal(out, c.cache.decode_attn(0, c.batch, qo[:2]))
