"""Chunk and prompt attention over many tiles: items cut among many CTAs, rings that
wrap, both widths of a query tile, whatever the workspace holds; lengths that change
under a call; rows that are no plain tensors."""

import numpy as np
import pytest
import torch

import chunk_testutil as C
import paged_testutil as T
from mixed_precision_quantized_quant_gb300 import kvq as K

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


class Big:
    """A cache whose pages hold random rows (any codes, scales and zeros)."""

    def __init__(self, lens, news, kb, vb, hq, hkv, d, page, dtype, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 1
        self.cache = c = K.KVQPagedCache([(kb, vb)], hq, hkv, d, page, pages, dtype=T.DTYPES[dtype])
        v = c.view(0)
        body = c.buf[:pages * v["page_stride"]]
        if kb == 16:
            body.view(c.dtype).copy_(torch.randn(body.numel() // 2, generator=g, device="cuda"))
        else:
            body.copy_(torch.randint(0, 256, body.shape, generator=g, device="cuda", dtype=torch.int32).to(torch.uint8))
            sz = body.view(-1, v["tile_bytes"])[:, -128:].view(torch.float16).view(-1, 16, 4)
            for at, bits in ((0, kb), (2, vb)):  # rows of about two sizes, zeros that put them around 0.3
                s = torch.rand(sz.shape[:2], generator=g, device="cuda") * 2 / (2 ** bits - 1)
                sz[..., at] = s.half()
                sz[..., at + 1] = (0.3 - s * (2 ** bits - 1) / 2).half()
        order = torch.randperm(pages, generator=g, device="cuda").int()
        self.table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[at:at + k]
            at += k
        self.lens, self.news = lens, news
        self.batch = K.PagedBatch(self.table, _i32(lens), _i32(np.cumsum([0] + news).tolist()))
        self.q = torch.randn(sum(news), hq + 2 * hkv, d, generator=g, device="cuda").to(c.dtype)[:, :hq]

    def run(self, window=0):
        """The call, over a workspace that holds NaN."""
        n = K.kvq_paged_chunk_workspace_bytes(self.cache.h, len(self.lens), sum(self.news))
        dirt = torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
        del dirt
        out = self.cache.chunk_attn(0, self.batch, self.q, window=window, return_lse=True)
        assert self.cache.device_error() == 0
        return out

    def check(self, window=0, times=3):
        out, lse = self.run(window)
        row = 0
        for b, (n, m) in enumerate(zip(self.lens, self.news)):
            k, size = C.dense(self.cache, 0, self.table[b], n, False)
            v, _ = C.dense(self.cache, 0, self.table[b], n, True)
            last = torch.arange(n - m, n, device="cuda")
            first = (last - window + 1).clamp(min=0) if window else torch.zeros_like(last)
            for a in range(0, m, 256):  # (the scores in 64 bits)
                e = min(m, a + 256)
                exp = C.attend(self.q[row + a:row + e], k, v, first[a:e], last[a:e], self.cache.dtype, 0.0,
                               self.cache.layers[0][0] != 16, size)
                C.close(out[row + a:row + e], lse[row + a:row + e], exp)
            row += m
        for _ in range(times):
            o, l = self.run(window)
            assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kb,vb,dtype", [(16, 16, "bf16"), (16, 16, "fp16"), (8, 8, "bf16"), (8, 4, "fp16"), (4, 2, "fp16"), (2, 8, "bf16")])
def test_few_rows_over_long_caches(kb, vb, dtype, d):
    # one query tile, sequences cut among the CTAs, some of which get two or three pieces
    lens = [4096, 2830, 3612, 1, 129, 3911, 2645, 2048, 700, 4025]
    Big(lens, [5, 3, 4, 1, 2, 5, 1, 5, 3, 5], kb, vb, 32, 8, d, 64, dtype).check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kb,vb,dtype", [(16, 16, "bf16"), (16, 16, "fp16"), (8, 8, "bf16"), (8, 4, "fp16"), (4, 4, "bf16"), (2, 2, "fp16")])
def test_many_rows_over_long_caches(kb, vb, dtype, d):
    # two query tiles, of which the last items lack the second
    Big([3001, 1500, 2222], [700, 1023, 130], kb, vb, 8, 2, d, 16, dtype).check()


@pytest.mark.parametrize("window", [500, 4096])
@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 8)])
def test_windows_over_long_caches(kb, vb, window):
    Big([6000, 4500], [300, 1100], kb, vb, 14, 2, 128, 128, "bf16").check(window)
    Big([9000, 4500], [3, 7], kb, vb, 14, 2, 128, 128, "bf16").check(window)


@pytest.mark.parametrize("kb,vb", [(16, 16), (4, 2)])
def test_one_query_head_a_kv_head(kb, vb):
    # 256 tokens an item: the query tiles end in different tiles of keys
    Big([1900, 300], [900, 290], kb, vb, 4, 4, 128, 32, "fp16").check()
    Big([1900, 300, 5], [60, 90, 5], kb, vb, 4, 4, 64, 32, "fp16").check()


@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 4)])
def test_more_sequences_than_the_plan_has_entries(kb, vb):
    # 2,300 sequences, many without rows: three to an entry of the plan
    news = [(7 * i) % 4 for i in range(2300)]
    Big([n + (11 * i) % 40 + 1 for i, n in enumerate(news)], news, kb, vb, 2, 1, 64, 16, "fp16").check(times=1)


def test_prompts_of_many_tiles():
    c = K.KVQPagedCache([(16, 16)], 32, 8, 128, 64, 1, dtype=torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(0)
    news = [2047, 1300, 60, 1999, 513]
    n = sum(news)
    qkv = torch.randn(n, 48, 128, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = qkv[:, :32], qkv[:, 32:40], qkv[:, 40:]
    batch = K.PagedBatch(_i32([[0]] * 5), _i32([0] * 5), _i32(np.cumsum([0] + news).tolist()))
    out, lse = c.prompt_attn(batch, q, k, v, return_lse=True)
    assert c.device_error() == 0
    a = 0
    for m in news:
        kk, vv = (x[a:a + m].double().transpose(0, 1) for x in (k, v))
        for s in range(0, m, 512):
            e = min(m, s + 512)
            last = torch.arange(s, e, device="cuda")
            C.close(out[a + s:a + e], lse[a + s:a + e], C.attend(q[a + s:a + e], kk[:, :e], vv[:, :e], torch.zeros_like(last), last, c.dtype))
        a += m


@pytest.mark.parametrize("hq,hkv", [(8, 2), (4, 4)])
def test_rows_that_are_no_plain_tensors(hq, hkv):
    # heads that share their rows (a stride of 0), a step between tokens, an output on 16 bytes but not on 32
    c = K.KVQPagedCache([(16, 16), (8, 8)], hq, hkv, 64, 16, 8, dtype=torch.float16)
    g = torch.Generator(device="cuda").manual_seed(0)
    n = 100
    k = torch.randn(2 * n, 1, 64, generator=g, device="cuda").half()[::2].expand(n, hkv, 64)
    v = torch.randn(n, hkv, 64, generator=g, device="cuda").half().flip(0)
    q = torch.randn(n, 1, 64, generator=g, device="cuda").half().expand(n, hq, 64)
    batch = K.PagedBatch(torch.arange(8, dtype=torch.int32, device="cuda")[None], _i32([n]), _i32([0, n]))
    out = torch.empty(n * hq * 64 + 8, dtype=torch.float16, device="cuda")[8:].view(n, hq, 64)
    assert out.data_ptr() % 32 == 16
    last = torch.arange(n, device="cuda")
    exp = C.attend(q, k.double().transpose(0, 1), v.double().transpose(0, 1), 0 * last, last, c.dtype)
    got, lse = c.prompt_attn(batch, q, k, v, out=out, return_lse=True)
    C.close(got, lse, exp)
    for layer in (0, 1):
        c.append(layer, batch, k, v)
        kk, size = C.dense(c, layer, batch._keep[0][0], n, False)
        vv, _ = C.dense(c, layer, batch._keep[0][0], n, True)
        got, lse = c.chunk_attn(layer, batch, q, out=out, return_lse=True)
        C.close(got, lse, C.attend(q, kk, vv, 0 * last, last, c.dtype, 0.0, layer == 1, size))
    assert c.device_error() == 0


@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 4)])
def test_lengths_that_change_under_a_call(kb, vb):
    # results mean nothing then; every call ends, and the next one is right
    b = Big([3000, 2000, 900], [4, 300, 20], kb, vb, 8, 2, 128, 32, "bf16")
    good, want = b.batch._keep[1].clone(), b.run()[0]
    other, cu = torch.cuda.Stream(), b.batch._keep[2]
    ends = cu.clone()
    for i in range(30):
        with torch.cuda.stream(other):
            for j in range(20):
                b.batch._keep[1].copy_(good - (i * 37 + j * 101) % 800)
                cu[1:3].copy_(ends[1:3] - (i + j) % 4)
        for _ in range(3):
            b.cache.chunk_attn(0, b.batch, b.q)
    torch.cuda.synchronize()
    assert b.cache.device_error() in (0, 2, 4)
    b.batch._keep[1].copy_(good)
    cu.copy_(ends)
    assert torch.equal(b.run()[0], want)


def test_layers_of_one_cache():
    # every layer has its own widths and its own place in the buffer
    layers = [(16, 16), (4, 2), (16, 16), (8, 8)]
    c = K.KVQPagedCache(layers, 8, 2, 128, 32, 12, dtype=torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(0)
    batch = K.PagedBatch(torch.randperm(12, generator=g, device="cuda").int().view(2, 6), _i32([150, 190]), _i32([0, 150, 340]))
    rows = [[torch.randn(340, h, 128, generator=g, device="cuda").bfloat16() for h in (8, 2, 2)] for _ in layers]
    for layer, (q, k, v) in enumerate(rows):
        c.append(layer, batch, k, v)
    for layer, (q, k, v) in enumerate(rows):
        got, lse = c.chunk_attn(layer, batch, q, return_lse=True)
        for b, (a, n) in enumerate(((0, 150), (150, 190))):
            kk, size = C.dense(c, layer, batch._keep[0][b], n, False)
            vv, _ = C.dense(c, layer, batch._keep[0][b], n, True)
            last = torch.arange(n, device="cuda")
            C.close(got[a:a + n], lse[a:a + n], C.attend(q[a:a + n], kk, vv, 0 * last, last, c.dtype, 0.0, layers[layer][0] != 16, size))
    assert c.device_error() == 0


@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 8)])
def test_pages_past_four_gibibytes(kb, vb):
    pages = 20_000 if kb != 16 else 10_000  # of 8 heads: 0.26 and 0.5 MiB each
    c = K.KVQPagedCache([(kb, vb)], 8, 8, 128, 128, pages, dtype=torch.float16)
    assert c.nbytes > 4 << 30
    g = torch.Generator(device="cuda").manual_seed(0)
    batch = K.PagedBatch(_i32([[pages - 1, 0, pages - 2, pages // 2]]), _i32([450]), _i32([0, 450]))
    q, k, v = (torch.randn(450, 8, 128, generator=g, device="cuda").half() for _ in range(3))
    c.append(0, batch, k, v)
    got, lse = c.chunk_attn(0, batch, q, return_lse=True)
    few = K.KVQPagedCache([(kb, vb)], 8, 8, 128, 128, 4, dtype=torch.float16)
    near = K.PagedBatch(_i32([[0, 1, 2, 3]]), _i32([450]), _i32([0, 450]))
    few.append(0, near, k, v)
    e, le = few.chunk_attn(0, near, q, return_lse=True)
    assert torch.equal(got, e) and torch.equal(lse, le) and c.device_error() == 0


def test_calls_side_by_side():
    # one cache, calls on three streams at once: each as by itself
    big = [Big([2500, 700], [300, 9], 8, 4, 8, 2, 128, 32, "fp16", seed=1), Big([3000, 64, 900], [4, 2, 1], 16, 16, 8, 2, 128, 32, "fp16", seed=2)]
    alone = [b.run() for b in big]
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    torch.cuda.synchronize()
    for i in range(20):
        for s in streams:
            with torch.cuda.stream(s):
                got.append([b.cache.chunk_attn(0, b.batch, b.q, return_lse=True) for b in big])
    torch.cuda.synchronize()
    for pair in got:
        for (o, l), (e, le) in zip(pair, alone):
            assert torch.equal(o, e) and torch.equal(l, le)
