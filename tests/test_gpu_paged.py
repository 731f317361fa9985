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


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kb,vb", PAIRS)
def test_attn_pairs(kb, vb, d, dtype):
    _check_attn(Case(LENS, kb=kb, vb=vb, d=d, dtype=dtype, page=32))


@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 8), (4, 2)])
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 1), (7, 1), (6, 2), (28, 4), (5, 5)])
def test_attn_heads_and_pages(hq, hkv, page, kb, vb):
    _check_attn(Case([70, 1, 130, 0, 19], kb=kb, vb=vb, d=128, hq=hq, hkv=hkv, page=page), how="odd")


@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 4), (2, 2)])
@pytest.mark.parametrize("window", [1, 5, 16, 50, 128, 4000])
def test_attn_window(window, kb, vb):
    _check_attn(Case(LENS, kb=kb, vb=vb, d=128, page=16), window=window, scale=0.3)


@pytest.mark.parametrize("kb,vb", [(16, 16), (4, 4)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_attn_long_and_unequal(kb, vb, dtype):
    # one long sequence beside short ones: splits of one unit, and many units in one split
    _check_attn(Case([3000, 1, 40, 0, 700] + [3] * 20, kb=kb, vb=vb, d=64, hq=4, hkv=1, page=64, dtype=dtype))


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
