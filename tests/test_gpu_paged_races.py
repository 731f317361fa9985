"""The paged cache under what its caller does at the same time: lengths that
change while the attention reads them, errors of one stream read on another."""

import pytest
import torch

from mixed_precision_quantized_quant_gb300 import kvq as K
from test_gpu_paged import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 8), (4, 2)])
def test_lengths_that_change_under_the_attention(kb, vb):
    # every page and length is one of the pool's and the table's, so that only how the work is cut changes
    # under the calls: each of them ends without a wait that ran out, and the next one by itself is right
    S, P, width = 40, 16, 256
    c = Case([64] * S, kb=kb, vb=vb, d=64, hq=4, hkv=2, page=P)
    pages = c.model.data.shape[0]
    g = torch.Generator().manual_seed(4)
    table = torch.randint(0, pages - 2, (S, width), generator=g, dtype=torch.int32)
    table[:, :4] = torch.from_numpy(c.table)
    lens = torch.full((S,), 64, dtype=torch.int32, device="cuda")
    batch = K.PagedBatch(table.cuda(), lens)
    q = c.rows(S, c.hq)
    before = c.download().copy()
    alone = c.cache.decode_attn(0, batch, q)
    others = [torch.randint(0, width * P + 1, (S,), generator=g, dtype=torch.int32).cuda() for _ in range(4)]
    others += [torch.zeros_like(lens), torch.full_like(lens, width * P)]
    side, work = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(100):
        with torch.cuda.stream(side):
            for j in range(6):
                lens.copy_(others[(i + j) % 6])
        with torch.cuda.stream(work):
            for _ in range(3):
                c.cache.decode_attn(0, batch, q)
    torch.cuda.synchronize()
    assert c.cache.device_error() in (0, 2)
    lens.fill_(64)
    assert torch.equal(c.cache.decode_attn(0, batch, q), alone)
    assert (c.download() == before).all() and c.cache.device_error() == 0


def test_errors_of_another_stream_are_not_lost():
    # one bad call each time, whose report is taken while it runs or after it, but taken
    c = Case([40], d=64, hq=8, hkv=1, fill=False)
    bad = K.PagedBatch(torch.full((1, 3), -1, dtype=torch.int32, device="cuda"), torch.tensor([40], dtype=torch.int32).cuda())
    k, q = c.rows(1, 1), c.rows(1, 8)
    work, side = torch.cuda.Stream(), torch.cuda.Stream()
    a = torch.randn(256, 256, device="cuda")
    torch.cuda.synchronize()
    for i in range(400):
        with torch.cuda.stream(work):
            for _ in range(i % 5):
                a @ a
            c.cache.append(0, bad, k, k, q=q)
        first = c.cache.device_error(side)
        work.synchronize()
        assert 4 in (first, c.cache.device_error(side)), i
    assert c.cache.device_error() == 0
