"""The paged cache on the GPU: append, read and attention against a plain model
of the pages (bytes compared exactly, attention against 64 bits)."""

import math

import numpy as np
import pytest
import torch

import paged_testutil as T
from mixed_precision_quantized_quant_gb300 import kvq as K

pytestmark = pytest.mark.gpu

PAIRS = [(16, 16), (8, 8), (8, 4), (4, 8), (4, 4), (4, 2), (2, 4), (2, 2), (8, 2), (2, 8)]


class Case:
    """A cache with random pages, its plain model, and sequences of `lens` tokens."""

    def __init__(self, lens, news=None, kb=16, vb=16, hq=8, hkv=2, d=64, page=16, dtype="fp16", seed=0, layers=1,
                 spare=2, width=None, fill=True):
        g = torch.Generator().manual_seed(seed)
        self.g, self.lens, self.news = g, lens, news
        self.hq, self.hkv, self.d, self.P, self.dtype = hq, hkv, d, page, T.DTYPES[dtype]
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=g).tolist()
        width = width or max(need + [1])
        self.table = np.full((len(lens), width), -7, np.int32)
        for b, k in enumerate(need):
            self.table[b, :k] = [order.pop() for _ in range(k)]
        self.cache = K.KVQPagedCache([(kb, vb)] * layers, hq, hkv, d, page, pages, dtype=self.dtype)
        self.layer = layers - 1
        self.model = T.Pages(kb, vb, hkv, d, page, pages, self.dtype)
        # what no sequence owns is left as garbage: every byte 0xff (NaN as fp16, bf16 and as scales)
        self.model.data[:] = 0xFF
        if fill:
            mu = torch.randn(hkv, d, generator=g)
            for b, n in enumerate(lens):
                for p in range(n):
                    for h in range(hkv):
                        x = torch.randn(2, d, generator=g)
                        at = (self.table[b, p // page], p % page, h)
                        self.model.put(*at, False, (x[0] + mu[h]).to(self.dtype).float())
                        self.model.put(*at, True, x[1].to(self.dtype).float())
        self.upload()
        cu = None if news is None else torch.tensor([0] + news, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
        self.batch = K.PagedBatch(torch.from_numpy(self.table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), cu)

    def _layer_bytes(self):
        v = self.cache.view(self.layer)
        off = v["pages"] - self.cache.buf.data_ptr()
        return self.cache.buf[off:off + self.model.data.size]

    def upload(self):
        self._layer_bytes().copy_(torch.from_numpy(self.model.data.reshape(-1)).cuda())

    def download(self):
        torch.cuda.synchronize()
        return self._layer_bytes().cpu().numpy().reshape(self.model.data.shape)

    def rows(self, n, heads, how="fused"):
        """Random rows [n, heads, d] as a slice of a wider tensor: `fused` 16-byte aligned, `odd` not."""
        pad = 2 * self.d if how == "fused" else 3
        x = torch.randn(n, heads * self.d + pad, generator=self.g).to(self.dtype).cuda()
        return x[:, pad:].view(n, heads, self.d) if how == "fused" else x[:, pad:].unflatten(1, (heads, self.d))

    def places(self):
        """(row, sequence, position) of every new row."""
        row = 0
        for b, n in enumerate(self.lens):
            for i in range(1 if self.news is None else self.news[b]):
                m = 1 if self.news is None else self.news[b]
                if n:
                    yield row, b, n - m + i
                row += 1


def _check_append(c, how="fused", with_q=True, dim=None, interleaved=False, positions=None, extra=0, in_place=False):
    n = (len(c.lens) if c.news is None else sum(c.news)) + extra
    k, v = c.rows(n, c.hkv, how), c.rows(n, c.hkv, how)
    q = c.rows(n, c.hq, how) if with_q else None
    q0 = q.clone() if with_q else None
    rot = None
    if dim:
        table = K.rotation_table(max(c.lens) + 40, dim, 10000.0)
        rot = K.Rotation(table, interleaved, None if positions is None else positions.cuda())
        table = table.cpu()
    q_out = q if in_place else (torch.full((n, c.hq, c.d), 7.0, dtype=c.dtype, device="cuda") if with_q else None)
    got = c.cache.append(c.layer, c.batch, k, v, q=q, rotation=rot, q_out=q_out)
    owned = np.zeros(n, bool)
    exp_q = None if not with_q else (q0.cpu().clone() if in_place else torch.full((n, c.hq, c.d), 7.0, dtype=c.dtype))
    for row, b, p in c.places():
        owned[row] = True
        at = p if positions is None else int(positions[row])
        kr, qr = k[row].cpu().float(), q0[row].cpu().float() if with_q else None
        if dim:
            kr = T.turn(kr, at, table, interleaved)
            qr = T.turn(qr, at, table, interleaved) if with_q else None
        for h in range(c.hkv):
            place = (c.table[b, p // c.P], p % c.P, h)
            c.model.put(*place, False, kr[h])
            c.model.put(*place, True, v[row, h].cpu())
        if with_q:
            exp_q[row] = qr.to(c.dtype)
    assert np.array_equal(c.download(), c.model.data)
    assert c.cache.device_error() == 0
    if with_q:
        assert torch.equal(got.cpu(), exp_q)
    else:
        assert got is None


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kb,vb", PAIRS)
def test_append_one_row_each(kb, vb, d, dtype):
    # one new token a sequence: the first of a page, the last, one inside, and a padded place of the batch
    c = Case([1, 16, 17, 0, 32, 70], kb=kb, vb=vb, d=d, dtype=dtype, page=32, fill=False)
    _check_append(c, dim=d)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 4)])
def test_append_prompts_ragged(kb, vb, page):
    # prompts, a chunk after earlier tokens, no new token, and rows behind the last sequence
    c = Case([40, 130, 9, 77, 1], [40, 33, 0, 77, 1], kb=kb, vb=vb, d=128, page=page, fill=False)
    _check_append(c, dim=128, extra=3)


@pytest.mark.parametrize("dim,interleaved", [(16, False), (64, False), (64, True), (128, True), (32, True)])
@pytest.mark.parametrize("kb,vb", [(16, 16), (4, 2)])
def test_append_rotations(kb, vb, dim, interleaved):
    c = Case([5, 61], [5, 30], kb=kb, vb=vb, d=128, fill=False)
    pos = torch.randint(0, 100, (35,), generator=torch.Generator().manual_seed(5), dtype=torch.int32)
    _check_append(c, dim=dim, interleaved=interleaved, positions=pos)


@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 8)])
@pytest.mark.parametrize("d,hq,hkv", [(64, 7, 7), (128, 28, 4), (64, 3, 1), (128, 1, 1)])
def test_append_heads_and_odd_strides(d, hq, hkv, kb, vb):
    for how in ("fused", "odd"):
        c = Case([3, 20], [3, 18], kb=kb, vb=vb, d=d, hq=hq, hkv=hkv, fill=False)
        _check_append(c, how=how, dim=d // 2)


@pytest.mark.parametrize("how", ["fused", "odd"])
@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 4), (2, 2)])
@pytest.mark.parametrize("d,hq,hkv,interleaved", [(64, 6, 3, False), (128, 5, 1, True)])
def test_append_and_read_many_rows(d, hq, hkv, interleaved, kb, vb, how):
    # enough rows for several a CTA (the few-row form is left at 3 an SM): runs that cross tokens,
    # sequences and sequences without rows, then rows behind the last one
    lens = [300, 7, 0, 0, 260, 1, 90]
    c = Case(lens, [290, 7, 0, 0, 250, 1, 60], kb=kb, vb=vb, d=d, hq=hq, hkv=hkv, page=64, fill=False, dtype="bf16")
    _check_append(c, how=how, dim=d // 2, interleaved=interleaved, extra=9)
    k, v = (torch.full((617, hkv, d), 7.0, dtype=c.dtype, device="cuda") for _ in range(2))
    c.cache.read(0, c.batch, 617, K=k, V=v)
    exp = [torch.full((617, hkv, d), 7.0, dtype=c.dtype) for _ in range(2)]
    for row, b, p in c.places():
        for h in range(hkv):
            for is_v in (0, 1):
                x, _, _ = c.model.get(c.table[b, p // 64], p % 64, h, bool(is_v))
                exp[is_v][row, h] = torch.from_numpy(x).float().to(c.dtype)
    assert torch.equal(k.cpu(), exp[0]) and torch.equal(v.cpu(), exp[1])


@pytest.mark.parametrize("kb,vb", [(16, 16), (4, 2)])
def test_append_of_several_waves_is_that_of_its_parts(kb, vb):
    n, hq, hkv, d, P = 20_011, 4, 2, 64, 64
    pages = -(-n // P)
    g = torch.Generator(device="cuda").manual_seed(2)
    rows = torch.randn(n, hq + 2 * hkv, d, generator=g, device="cuda").half()
    q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
    rot = K.Rotation(K.rotation_table(n, d))
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None].contiguous()
    bufs = [torch.zeros(K.kvq_paged_bytes(K.make_paged_config([(kb, vb)], hq, hkv, d, P, pages)), dtype=torch.uint8, device="cuda")
            for _ in range(2)]
    whole, parts = (K.KVQPagedCache([(kb, vb)], hq, hkv, d, P, pages, buffer=x) for x in bufs)

    def batch(a, b):
        return K.PagedBatch(table, torch.tensor([b], dtype=torch.int32).cuda(), torch.tensor([0, b - a], dtype=torch.int32).cuda())

    qo = whole.append(0, batch(0, n), k, v, q=q, rotation=rot)
    for a in range(0, n, 400):
        b = min(n, a + 400)
        assert torch.equal(parts.append(0, batch(a, b), k[a:b], v[a:b], q=q[a:b], rotation=rot), qo[a:b])
    assert torch.equal(*bufs)
    rk, rv = whole.read(0, batch(0, n), n)
    for a in range(0, n, 400):
        b = min(n, a + 400)
        pk, pv = parts.read(0, batch(a, b), b - a)
        assert torch.equal(pk, rk[a:b]) and torch.equal(pv, rv[a:b])


def test_append_without_queries_or_rotation_and_in_place():
    _check_append(Case([33, 2], fill=False), with_q=False)
    _check_append(Case([33, 2], kb=4, vb=4, fill=False), with_q=False, dim=64)
    _check_append(Case([33, 2], fill=False), dim=64, in_place=True)
    _check_append(Case([33, 20], [30, 20], kb=4, vb=2, fill=False, layers=3), dim=32, in_place=True)


def test_append_values_at_the_borders():
    # constant rows, zeros, infinities, huge bf16 values, exact ties
    for dtype, big in (("fp16", math.inf), ("bf16", 1e30)):
        c = Case([1] * 6, kb=4, vb=2, d=64, dtype=dtype, fill=False)
        x = torch.zeros(6, 2, 64)
        x[1] = 3.25
        x[2, :, ::2] = 15.0
        x[2, 0, 1] = 7.5
        x[2, 1, 1] = 2.5
        x[3] = torch.arange(64) / 8
        x[4, :, 5] = big
        x[5, :, 7] = -big
        k = x.to(c.dtype).cuda()
        c.cache.append(0, c.batch, k, k)
        for row, b, p in c.places():
            for h in range(2):
                c.model.put(c.table[b, 0], 0, h, False, k[row, h].cpu())
                c.model.put(c.table[b, 0], 0, h, True, k[row, h].cpu())
        assert np.array_equal(c.download(), c.model.data)


def test_append_nan_row_gets_nan_scales():
    c = Case([1], kb=8, vb=4, d=64, fill=False)
    k = torch.ones(1, 2, 64, dtype=torch.float16, device="cuda")
    k[0, 1, 9] = math.nan
    c.cache.append(0, c.batch, k, k)
    kk, vv = (x.cpu() for x in c.cache.read(0, c.batch, 1))
    assert torch.equal(kk[0, 0], torch.ones(64).half()) and torch.equal(vv[0, 0], torch.ones(64).half())
    assert kk[0, 1].isnan().all() and vv[0, 1].isnan().all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kb,vb", PAIRS)
def test_read(kb, vb, d, dtype):
    c = Case([21, 0, 48], [21, 0, 17], kb=kb, vb=vb, d=d, dtype=dtype, layers=2)
    out = [torch.full((41, 2, d), 7.0, dtype=c.dtype, device="cuda") for _ in range(2)]
    k, v = c.cache.read(c.layer, c.batch, 41, K=out[0], V=out[1])
    exp = [torch.full((41, 2, d), 7.0, dtype=c.dtype) for _ in range(2)]
    for row, b, p in c.places():
        for h in range(2):
            for is_v in (0, 1):
                x, _, _ = c.model.get(c.table[b, p // 16], p % 16, h, bool(is_v))
                # code * scale + zero, rounded to fp32 and then to the type, as documented
                exp[is_v][row, h] = torch.from_numpy(x).float().to(c.dtype)
    assert torch.equal(k.cpu(), exp[0]) and torch.equal(v.cpu(), exp[1])
    assert c.cache.device_error() == 0
    # odd strides, and one of the two alone
    wide = torch.full((41, 2 * d + 3), 7.0, dtype=c.dtype, device="cuda")
    odd = wide[:, 3:].unflatten(1, (2, d))
    k2, _ = c.cache.read(c.layer, c.batch, 41, K=odd)
    assert torch.equal(k2.cpu(), exp[0]) and bool((wide[:, :3] == 7).all())


def _check_attn(c, scale=0.0, window=0, how="fused", q=None, stream=None):
    B = len(c.lens)
    q = c.rows(B, c.hq, how) if q is None else q
    out, lse = c.cache.decode_attn(c.layer, c.batch, q, scale=scale, window=window, return_lse=True, stream=stream)
    torch.cuda.synchronize()
    eo, el, tol, ltol = T.attend(c.model, c.table, c.lens, q.cpu(), scale, window, c.dtype)
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(o).all()
    assert (np.abs(o - eo) <= tol).all(), float((np.abs(o - eo) / np.maximum(tol, 1e-30)).max())
    live = np.isfinite(el)
    assert np.array_equal(live, np.isfinite(l)) and (l[~live] == -math.inf).all()
    assert (np.abs(l[live] - el[live]) <= ltol[live]).all()
    assert c.cache.device_error() == 0
    return out


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 64, 65, 129, 200]


# narrow tables give each (sequence, head) a CTA of its own, wide ones are split
@pytest.mark.parametrize("width", [None, 200])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kb,vb", PAIRS)
def test_attn_pairs(kb, vb, d, dtype, width):
    _check_attn(Case(LENS, kb=kb, vb=vb, d=d, dtype=dtype, page=32, width=width))


@pytest.mark.parametrize("width", [None, 100])
@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 8), (4, 2)])
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 1), (7, 1), (6, 2), (28, 4), (5, 5)])
def test_attn_heads_and_pages(hq, hkv, page, kb, vb, width):
    _check_attn(Case([70, 1, 130, 0, 19], kb=kb, vb=vb, d=128, hq=hq, hkv=hkv, page=page, width=width), how="odd")


@pytest.mark.parametrize("width", [None, 300])
@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 4), (2, 2)])
@pytest.mark.parametrize("window", [1, 5, 16, 50, 128, 4000])
def test_attn_window(window, kb, vb, width):
    c = Case(LENS, kb=kb, vb=vb, d=128, page=16, width=width)
    for b, n in enumerate(c.lens):  # pages wholly before the window may be gone
        c.table[b, :max(0, n - window) // 16] = -1
    c.batch = K.PagedBatch(torch.from_numpy(c.table).cuda(), torch.tensor(c.lens, dtype=torch.int32).cuda())
    _check_attn(c, window=window, scale=0.3)


@pytest.mark.parametrize("kb,vb", [(16, 16), (4, 4)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_attn_long_and_unequal(kb, vb, dtype):
    # one long sequence beside short ones: splits of one unit, and many units in one split
    _check_attn(Case([3000, 1, 40, 0, 700] + [3] * 20, kb=kb, vb=vb, d=64, hq=4, hkv=1, page=64, dtype=dtype))


@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 2)])
@pytest.mark.parametrize("width", [4, 80])
def test_attn_many_sequences(kb, vb, width):
    # more sequences than a CTA looks at together, runs of empty ones among them
    lens = [0] * 140 + [5, 0, 33] * 40 + [0] * 30 + [61, 2]
    _check_attn(Case(lens, kb=kb, vb=vb, d=64, hq=2, hkv=1, page=16, width=width))


@pytest.mark.parametrize("kb,vb", [(16, 16), (4, 2), (8, 8)])
def test_attn_very_long_over_repeated_pages(kb, vb):
    # 300,000 tokens made of 16 pages in random order: a weight counts as often as its page
    n, P = 300_000, 128
    c = Case([16 * P], kb=kb, vb=vb, d=128, hq=8, hkv=1, page=P)
    k, kc, _ = c.model.rows(c.table[0], 0, 16 * P, 0, False)
    v, vc, vs = c.model.rows(c.table[0], 0, 16 * P, 0, True)
    order = np.random.default_rng(3).integers(0, 16, -(-n // P))
    table = torch.from_numpy(c.table[0][order][None].astype(np.int32)).cuda()
    batch = K.PagedBatch(table, torch.tensor([n], dtype=torch.int32).cuda())
    q = c.rows(1, 8)
    out, lse = c.cache.decode_attn(0, batch, q, return_lse=True)
    count = np.zeros(16 * P)
    for i, o in enumerate(order):
        m = min(P, n - i * P)
        count[o * P:o * P + m] += 1
    qq = q[0].double().cpu().numpy()
    t = qq @ k.T / math.sqrt(128)
    p = np.exp(t - t.max(1, keepdims=True)) * count
    eo, el = p @ v / p.sum(1, keepdims=True), t.max(1) + np.log(p.sum(1))
    # as in paged_testutil.attend, with chains of n / 8 / 4 tiles' additions at the most in a warp of a full wave
    u = 2.0 ** -11
    e = 144 * 2.0 ** -23 / math.sqrt(128) * (np.abs(qq) @ (np.abs(kc) + np.abs(k - kc)).T).max(1)[:, None] + 2.0 ** -20
    f = (n / 400 + 64) * 2.0 ** -23
    codes = np.abs(vc) / np.where(vs > 0, vs, 1.0)[:, None]
    tol = (u * np.abs(eo) + (u * (p @ np.abs(vc)) + 2.0 ** -25 * (p / np.maximum(count, 1) * vs).max(1)[:, None]
                             * (count @ codes)) / p.sum(1, keepdims=True)
           + (2 * e + f) * (p @ (np.abs(v) + np.abs(v - vc))) / p.sum(1, keepdims=True))
    assert (np.abs(out[0].double().cpu().numpy() - eo) <= tol).all()
    assert (np.abs(lse[0].double().cpu().numpy() - el) <= 2 * e[:, 0] + f + 2.0 ** -19 * np.abs(el)).all()
    assert c.cache.device_error() == 0


@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 4)])
def test_pages_past_32_bits(kb, vb):
    # a pool of over 4 GiB: its last pages hold what its first ones do
    P, hkv, d = 128, 8, 128
    page = hkv * P * (512 if kb == 16 else 200)
    pages = (5 << 30) // page
    c = K.KVQPagedCache([(kb, vb)], 8, hkv, d, P, pages)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(300, hkv, d, generator=g, device="cuda").half() for _ in range(2))
    q = torch.randn(1, 8, d, generator=g, device="cuda").half()
    rot = K.Rotation(K.rotation_table(300, d))
    res = []
    for t in ([0, 1, 2], [pages - 1, pages - 3, pages - 2]):
        b = K.PagedBatch(torch.tensor([t], dtype=torch.int32).cuda(), torch.tensor([300], dtype=torch.int32).cuda(),
                         torch.tensor([0, 300], dtype=torch.int32).cuda())
        c.append(0, b, k, v, rotation=rot)
        res.append((c.decode_attn(0, b, q), *c.read(0, b, 300)))
    assert all(torch.equal(x, y) for x, y in zip(*res))
    assert c.device_error() == 0 and float(res[0][0].abs().max()) > 0


def test_nan_in_an_attended_row_shows():
    for kb in (16, 8):
        c = Case([40, 20], kb=kb, vb=kb, d=64)
        x = torch.ones(1, 2, 64, dtype=torch.float16, device="cuda")
        bad = x.clone()
        bad[0, 1, 3] = math.nan
        b = K.PagedBatch(c.batch._keep[0][:1].contiguous(), torch.tensor([12], dtype=torch.int32).cuda())
        c.cache.append(0, b, x, bad)
        out = c.cache.decode_attn(0, c.batch, c.rows(2, 8))
        assert out[0, 4:].isnan().any() and not out[0, :4].isnan().any() and not out[1].isnan().any()


def test_attn_rising_scores_and_large_ones():
    # the running maximum rises all along, in steps large and small
    for kb, vb in ((16, 16), (8, 8)):
        c = Case([500], kb=kb, vb=vb, d=64, hq=4, hkv=1, fill=False)
        for p in range(500):
            x = torch.full((64,), 0.02 * p if p % 50 else 0.03 * p)
            x[0] = 0.0
            at = (c.table[0, p // 16], p % 16, 0)
            c.model.put(*at, False, x.half().float())
            c.model.put(*at, True, torch.randn(64, generator=c.g).half().float())
        c.upload()
        q = torch.ones(1, 4, 64, dtype=torch.float16, device="cuda")
        q[0, 1] *= 8
        q[0, 2] *= -8
        q[0, 3] = 0
        _check_attn(c, q=q)


def test_attn_tiny_and_huge_values():
    # scales from fp16's smallest steps to its largest, side by side and apart
    for f in (2.0 ** -20, 2.0 ** -12, 500.0, None):
        c = Case([100], kb=8, vb=4, d=64, hq=8, hkv=2, fill=False)
        for p in range(100):
            for h in range(2):
                x = torch.randn(2, 64, generator=c.g)
                at = (c.table[0, p // 16], p % 16, h)
                s = (2.0 ** (p % 20 - 12)) if f is None else f
                c.model.put(*at, False, x[0].half().float())
                c.model.put(*at, True, (x[1] * s).half().float())
        c.upload()
        _check_attn(c)


def test_attn_shared_prefix_pages():
    c = Case([48, 48], page=16, kb=4, vb=4)
    c.table[1, :2] = c.table[0, :2]
    c.batch = K.PagedBatch(torch.from_numpy(c.table).cuda(), torch.tensor(c.lens, dtype=torch.int32).cuda())
    q = c.rows(1, 8).expand(2, 8, 64).contiguous()
    _check_attn(c, q=q)


def test_attn_is_deterministic():
    c = Case([300, 20, 900], kb=4, vb=2, d=128, page=16)
    q = c.rows(3, 8)
    a = c.cache.decode_attn(0, c.batch, q)
    for _ in range(5):
        assert torch.equal(a, c.cache.decode_attn(0, c.batch, q))


def _step_inputs(c, n):
    return c.rows(n, c.hq), c.rows(n, c.hkv), c.rows(n, c.hkv)


@pytest.mark.parametrize("kb,vb", [(16, 16), (4, 2)])
def test_prefill_then_decode_steps(kb, vb):
    # a prompt appended, read back and attended, then decode steps, as a server runs them
    c = Case([37, 60, 18], [30, 53, 11], kb=kb, vb=vb, d=128, page=16, fill=False)
    _check_append(c, dim=128)
    start, c.news = [7, 7, 7], None
    c.lens = [30, 53, 11]
    # the prompts again from position 0, so that every attended token is one of theirs
    c = Case([30, 53, 11], [30, 53, 11], kb=kb, vb=vb, d=128, page=16, fill=False, width=6, spare=8)
    _check_append(c, dim=128)
    free = sorted(set(range(c.model.data.shape[0])) - set(c.table[c.table >= 0].tolist()))
    lens = torch.tensor(c.lens, dtype=torch.int32).cuda()
    table = torch.from_numpy(c.table).cuda()
    c.batch, c.news = K.PagedBatch(table, lens), None
    for _ in range(5):
        lens += 1
        c.lens = [n + 1 for n in c.lens]
        for b, n in enumerate(c.lens):
            if (n - 1) % 16 == 0:
                c.table[b, (n - 1) // 16] = free.pop()
        table.copy_(torch.from_numpy(c.table))
        _check_append(c, dim=128)
        _check_attn(c)


@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 4)])
def test_captured_steps_on_two_streams(kb, vb):
    # two captured decode steps of one cache, replayed side by side and following
    # what their tensors hold at the replay
    c = Case([0, 0, 0], kb=kb, vb=vb, d=64, page=16, fill=False, spare=24)
    free = list(range(24))
    rot = K.Rotation(K.rotation_table(200, 64))
    steps = []
    for s in range(2):
        st = dict(table=torch.tensor([[free.pop() for _ in range(6)] for _ in range(2)], dtype=torch.int32).cuda(),
                  lens=torch.zeros(2, dtype=torch.int32, device="cuda"))
        st["batch"] = K.PagedBatch(st["table"], st["lens"])
        st["q"], st["k"], st["v"] = (x.clone() for x in _step_inputs(c, 2))
        st["stream"], st["graph"] = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        st["inputs"] = [tuple(x.clone() for x in _step_inputs(c, 2)) for _ in range(60)]
        steps.append(st)

    def step(st):
        q = c.cache.append(0, st["batch"], st["k"], st["v"], q=st["q"], rotation=rot)
        return c.cache.decode_attn(0, st["batch"], q)

    for st in steps:
        step(st)
    torch.cuda.synchronize()
    for st in steps:
        with torch.cuda.graph(st["graph"], stream=st["stream"]):
            st["out"] = step(st)
    outs = [[], []]
    for i in range(60):
        for s, st in enumerate(steps):
            with torch.cuda.stream(st["stream"]):
                for a, b in zip((st["q"], st["k"], st["v"]), st["inputs"][i]):
                    a.copy_(b)
                st["lens"].add_(1)
                st["graph"].replay()
                outs[s].append(st["out"].clone())
    torch.cuda.synchronize()
    for s, st in enumerate(steps):  # the same steps one after another, without graphs
        st["lens"].zero_()
        for i in range(60):
            for a, b in zip((st["q"], st["k"], st["v"]), st["inputs"][i]):
                a.copy_(b)
            st["lens"].add_(1)
            assert torch.equal(step(st), outs[s][i]), (s, i)
    assert c.cache.device_error() == 0


def test_work_on_a_stream_of_its_own():
    c = Case([100, 30], kb=4, vb=4, d=128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    _check_attn(c, stream=s)


def test_bad_pages_lengths_and_positions_are_reported_and_not_followed():
    c = Case([40, 20], [1, 1], page=16)
    before = c.download().copy()
    k, v, q = c.rows(2, 2), c.rows(2, 2), c.rows(2, 8)

    def batch(table, lens, cu=(0, 1, 2)):
        return K.PagedBatch(torch.tensor(table, dtype=torch.int32).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                            None if cu is None else torch.tensor(cu, dtype=torch.int32).cuda())

    n = c.model.data.shape[0]
    for bad in (-1, n, 2 ** 31 - 1):
        b = batch([[bad, bad, bad], [bad, bad, bad]], [40, 20])
        qo = torch.full((2, 8, 64), 7.0, dtype=torch.float16, device="cuda")
        c.cache.append(0, b, k, v, q=q, q_out=qo)
        assert c.cache.device_error() == 4 and bool((qo == 7).all())
        c.cache.read(0, b, 2)
        assert c.cache.device_error() == 4
        c.cache.decode_attn(0, b, q)
        assert c.cache.device_error() == 4
    for lens in ([49, 20], [-1, 20], [2 ** 31 - 1, 20]):
        b = batch([[0, 1, 2], [3, 4, 0]], lens)
        b2 = batch([[n, n, n], [n, n, n]], lens)
        c.cache.append(0, b2, k, v)
        assert c.cache.device_error() in (2, 4)
        c.cache.decode_attn(0, b, q)
        assert c.cache.device_error() == 2
    # more new rows than tokens, and ends that do not ascend
    c.cache.append(0, batch([[n] * 3, [n] * 3], [0, 0]), k, v)
    assert c.cache.device_error() == 2
    c.cache.append(0, batch([[n] * 3, [n] * 3], [40, 20], (0, 2, 1)), k, v)
    assert c.cache.device_error() in (0, 2, 4)
    rot = K.Rotation(K.rotation_table(10, 64))
    c.cache.append(0, batch([[0, 1, 2], [3, 4, 0]], [40, 20]), k, v, rotation=rot)
    assert c.cache.device_error() == 5
    rot = K.Rotation(K.rotation_table(10, 64), positions=torch.tensor([-1, 10], dtype=torch.int32).cuda())
    c.cache.append(0, batch([[0, 1, 2], [3, 4, 0]], [40, 20]), k, v, rotation=rot)
    assert c.cache.device_error() == 5
    assert np.array_equal(c.download(), before)
    assert c.cache.device_error() == 0


def test_refusals():
    c = Case([20, 5], kb=4, vb=4, d=64, hq=4, hkv=2)
    q, k, v = c.rows(2, 4), c.rows(2, 2), c.rows(2, 2)
    a, t, r = c.cache.append, c.cache.decode_attn, c.cache.read
    half, table, lens = torch.float16, c.batch._keep[0], c.batch._keep[1]
    cu = torch.tensor([0, 1, 2], dtype=torch.int32).cuda()
    before = c.download().copy()
    for fn in (lambda: a(0, c.batch, k[:1], v[:1]), lambda: a(0, c.batch, k, v[:1]), lambda: a(0, c.batch, k.float(), v),
               lambda: a(0, c.batch, k.cpu(), v), lambda: a(0, c.batch, k, v, q_out=q), lambda: a(0, c.batch, k, q),
               lambda: a(0, c.batch, k, v, q=k), lambda: a(0, c.batch, k.transpose(1, 2).contiguous().transpose(1, 2), v),
               lambda: a(0, c.batch, k, v, rotation=K.Rotation(K.rotation_table(40, 128))),
               lambda: a(0, c.batch, k, v, rotation=K.Rotation(K.rotation_table(40, 64), positions=cu[:1])),
               lambda: t(0, c.batch, q[:1]), lambda: t(0, c.batch, q.bfloat16()), lambda: t(0, c.batch, k),
               lambda: t(0, c.batch, q, out=torch.empty(2, 4, 64, device="cuda")),
               lambda: t(0, c.batch, q, out=torch.empty(2, 64, 4, dtype=half, device="cuda").transpose(1, 2)),
               lambda: r(0, c.batch, 3), lambda: r(0, c.batch, 2, K=torch.empty(2, 2, 64, device="cuda")),
               lambda: K.PagedBatch(table.long(), lens), lambda: K.PagedBatch(table, lens.cpu()),
               lambda: K.PagedBatch(table, lens[:1]), lambda: K.PagedBatch(table.t(), lens),
               lambda: K.PagedBatch(table, lens, lens), lambda: K.PagedBatch(table[:0], lens[:0]),
               lambda: K.Rotation(torch.zeros(4, 24, device="cuda")), lambda: K.Rotation(torch.zeros(4, 0, device="cuda")),
               lambda: K.Rotation(torch.zeros(4, 64, dtype=half, device="cuda")),
               lambda: K.KVQPagedCache([(4, 4)], 4, 2, 64, 16, 4, dtype=torch.float32),
               lambda: K.KVQPagedCache([(4, 4)], 4, 2, 64, 16, 4, buffer=torch.zeros(9, device="cuda"))):
        with pytest.raises(ValueError):
            fn()
    for fn, code in ((lambda: a(1, c.batch, k, v), 1), (lambda: a(-1, c.batch, k, v), 1), (lambda: t(1, c.batch, q), 1),
                     (lambda: t(0, c.batch, q, window=-1), 1), (lambda: t(0, c.batch, q, scale=math.nan), 1),
                     (lambda: t(0, c.batch, q, scale=math.inf), 1), (lambda: r(2, c.batch, 2), 1),
                     (lambda: t(0, c.batch, q, out=torch.empty(2 * 4 * 64 + 1, dtype=half, device="cuda")[1:].view(2, 4, 64)), 3),
                     (lambda: K.KVQPagedCache([(3, 3)], 4, 2, 64, 16, 4), 1),
                     (lambda: K.KVQPagedCache([(4, 4)], 4, 2, 64, 16, 4, buffer=torch.zeros(64, dtype=torch.uint8, device="cuda")), 4)):
        with pytest.raises(K.KVQError) as e:
            fn()
        assert e.value.status == code
    # the C entry itself: missing rows, workspaces and counts
    L, h, b, s = K.load(), c.cache.h, c.batch.args, torch.cuda.current_stream().cuda_stream
    rk, rq = c.cache._rows(k, "k", 2, 2), c.cache._rows(q, "q", 2, 4)
    out, ws = torch.empty(2, 4, 64, dtype=half, device="cuda"), torch.empty(K.kvq_paged_workspace_bytes(h, 2), dtype=torch.uint8, device="cuda")
    o, w, nw = out.data_ptr(), ws.data_ptr(), ws.numel()
    assert L.kvq_paged_append(h, 0, b, rk, None, None, None, None, 2, s) == 1
    assert L.kvq_paged_append(h, 0, b, rk, rk, rq, None, None, 2, s) == 1
    assert L.kvq_paged_append(h, 0, b, rk, rk, None, None, None, -1, s) == 1
    assert L.kvq_paged_append(h, 0, None, rk, rk, None, None, None, 2, s) == 1
    assert L.kvq_paged_append(h, 0, b, K.Rows(rk.data + 1, 1, 1), rk, None, None, None, 2, s) == 3
    assert L.kvq_paged_append(h, 0, b, K.Rows(None, 1, 1), rk, None, None, None, 2, s) == 1
    rot = K.RotationArgs(w + 4, None, 1, 64, 0)
    assert L.kvq_paged_append(h, 0, b, rk, rk, None, None, rot, 2, s) == 3
    for bad in (K.RotationArgs(w, None, 0, 64, 0), K.RotationArgs(w, None, 1, 24, 0), K.RotationArgs(w, None, 1, 80, 0),
                K.RotationArgs(w, None, 1, 64, 2), K.RotationArgs(None, None, 1, 64, 0)):
        assert L.kvq_paged_append(h, 0, b, rk, rk, None, None, bad, 2, s) == 1
    assert L.kvq_paged_read(h, 0, b, None, None, 2, s) == 1
    assert L.kvq_paged_decode_attn(h, 0, b, rq, None, None, 0.0, 0, w, nw, s) == 1
    assert L.kvq_paged_decode_attn(h, 0, b, rq, o, None, 0.0, 0, None, nw, s) == 1
    assert L.kvq_paged_decode_attn(h, 0, b, rq, o, None, 0.0, 0, w + 16, nw, s) == 3
    assert L.kvq_paged_decode_attn(h, 0, b, rq, o, o + 2, 0.0, 0, w, nw, s) == 3
    assert L.kvq_paged_decode_attn(h, 0, b, rq, o, None, 0.0, 0, w, nw - 1, s) == 4
    for field, value in (("num_seqs", 0), ("max_pages", 0), ("table_stride", 1), ("page_table", None), ("seq_lens", None),
                         ("max_pages", 2 ** 27)):
        x = K.PagedBatchArgs.from_buffer_copy(b)
        setattr(x, field, value)
        if field == "max_pages" and value:
            x.table_stride = value
        assert L.kvq_paged_decode_attn(h, 0, x, rq, o, None, 0.0, 0, w, nw, s) == 1, field
    assert np.array_equal(c.download(), before) and c.cache.device_error() == 0
    # nothing to do
    a(0, K.PagedBatch(table, lens, torch.zeros(3, dtype=torch.int32, device="cuda")), k[:0], v[:0])
    c.cache.close()
    with pytest.raises(K.KVQError):
        t(0, c.batch, q)
