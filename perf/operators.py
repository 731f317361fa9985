"""Cases that measure the paged-cache operators: append with rotation, one-token attention, read back.

Run with ``own`` false, every pass is the operators' plain form in elementary torch operations; with ``own`` true it is
the calls a user makes of ``mixed_precision_quantized_quant_gb300.kvq.KVQPagedCache``.

The page pool that both sides take is one uint8 buffer: ``[num_pages][kv heads][page_size / 16]`` tiles of 16 tokens,
then 256 bytes of the cache's own.  A tile of 16-bit rows holds 16 key rows, then 16 value rows, the 16-byte chunk c of
token i at chunk ``c ^ (i & 7)``.  A tile of k/v-bit codes holds 16 key code rows, 16 value code rows (least significant
field first) and 16 quadruples (key scale, key zero, value scale, value zero) in fp16; key rows and quadruples of token i
sit at row ``2 (i & 3) + (i >> 2 & 1) + (i & 8)``; a 128-byte key row at row r has its 64-byte halves exchanged when r is
odd; a 128-byte value row keeps its 32-byte block b at ``b ^ (i & 3)``, a 64-byte one at ``b ^ (i >> 1 & 1)``.
"""

import math

import torch

own = False

TAIL = 256  # bytes behind the pages that belong to the cache


# ------------------------------------------------------------------ cases

def _case(name, op, batch, hq, hkv, d, length, kb, vb, page, dtype, new=1, ragged=True, window=0, rot=0, interleaved=False):
    """`length`: longest sequence after the new tokens; `new`: new tokens a sequence (the longest prompt where it is
    a prefill); `rot`: rotary width (0: the whole head)."""
    c = dict(op=op, batch=batch, hq=hq, hkv=hkv, d=d, length=length, kb=kb, vb=vb, page=page, dtype=dtype, new=new,
             ragged=ragged, window=window, rot=rot or d, interleaved=interleaved)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one short chat on the smallest configuration: nothing but latency
        _case("attn-tiny-d64-fp16", "attn", 1, 8, 2, 64, 256, 16, 16, 32, "fp16", ragged=False),
        # a serving batch of an 8B-shaped model on an unquantized layer
        _case("attn-8b-4k-bf16", "attn", 16, 32, 8, 128, 4096, 16, 16, 64, "bf16"),
        # the same batch on a sensitive layer (K8V4), odd lengths in small pages
        _case("attn-8b-4k-k8v4", "attn", 16, 32, 8, 128, 4095, 8, 4, 16, "fp16"),
        # seven query heads a kv head, a layer that looks back over 4096 tokens only
        _case("attn-7b-8k-k8v8-window", "attn", 32, 28, 4, 128, 8192, 8, 8, 64, "bf16", window=4096),
        # long contexts on the common layers (K4V2), and on one left in 16 bits (the largest)
        _case("attn-70b-32k-k4v2", "attn", 8, 64, 8, 128, 32768, 4, 2, 128, "fp16"),
        _case("attn-70b-32k-fp16", "attn", 8, 64, 8, 128, 32768, 16, 16, 128, "fp16"),
        # a decode step's append for one sequence: nothing but latency
        _case("append-one-d64-fp16", "append", 1, 8, 2, 64, 257, 16, 16, 32, "fp16", ragged=False),
        # prompts of several requests admitted together
        _case("append-prefill-8b-bf16", "append", 5, 32, 8, 128, 2047, 16, 16, 64, "bf16", new=2047),
        # a short reused prefix, and long ones, brought back for a chunked prefill
        _case("read-prefix-k8v4", "read", 1, 32, 8, 128, 515, 8, 4, 16, "fp16", new=515, ragged=False),
        _case("read-prefix-70b-k4v2", "read", 8, 64, 8, 128, 8192, 4, 2, 128, "bf16", new=8192),
        # one layer's whole decode step: append, attend, and the new rows as the cache holds them
        _case("step-8b-k4v2", "step", 16, 32, 8, 128, 4096, 4, 2, 32, "fp16"),
        # prompts into a quantized layer, and their rows as the cache holds them for the prefill's attention
        _case("fill-70b-k4v2", "fill", 8, 64, 8, 128, 1500, 4, 2, 128, "bf16", new=1500),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    hq, hkv, d = rng.choice([(8, 2, 64), (16, 4, 64), (32, 8, 128), (28, 4, 128), (32, 32, 128), (64, 8, 128)])
    kb, vb = rng.choice([(16, 16), (16, 16), (8, 8), (8, 4), (4, 4), (4, 2), (2, 2), (2, 8)])
    op = rng.choice(["attn", "attn", "attn", "append", "read", "step", "fill"])
    if op == "append":
        kb = vb = 16  # quantized rows are seen through a read: "fill"
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["fp16", "bf16"])
    batch = _log(rng, 1, 48)
    ragged = rng.random() < 0.8
    if op in ("attn", "step"):
        length = _log(rng, 1, 32768)
        length = max(1, min(length, (8 * 32768 * 8) // (batch * hkv)))
        window = rng.choice([0, 0, 0, _log(rng, 1, 8192)])
        return _case(None, op, batch, hq, hkv, d, length, kb, vb, page, dtype, ragged=ragged, window=window)
    new = _log(rng, 1, 8192)
    new = max(1, min(new, 12000 // batch))
    length = new + rng.choice([0, _log(rng, 1, 4096)])
    rot = rng.choice([d, d, d // 2])
    return _case(None, op, batch, hq, hkv, d, length, kb, vb, page, dtype, new=new, ragged=ragged, rot=rot,
                 interleaved=rng.random() < 0.3)


_DTYPE = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _lengths(case):
    """Each sequence's tokens and new tokens, the same for every seed."""
    B, L, new = case["batch"], case["length"], case["new"]
    if not case["ragged"]:
        return [L] * B, [new] * B
    lens, news = [], []
    for b in range(B):
        f = 1.0 - 0.5 * ((b * 0.6180339887) % 1.0)  # between a half and the whole of the longest
        n = max(1, int(new * f))
        lens.append(max(n, int(L * f)))
        news.append(n)
    if B >= 6 and new == 1 and case["op"] == "attn":
        lens[3] = 0  # a padded place of the batch
    return lens, news


def _row_bytes(case):
    q = case["kb"] != 16
    return case["d"] * (case["kb"] + case["vb"]) / 8 + (8 if q else 0)


def work(case):
    lens, news = _lengths(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    n = sum(news)
    seen = sum(min(x, case["window"]) if case["window"] else x for x in lens)
    table = sum(-(-x // case["page"]) for x in lens) * 4 + 4 * len(lens)
    attn = seen * hkv * _row_bytes(case) + len(lens) * hq * (d * 4 + 4) + table
    append = n * (hq * 4 * d + hkv * (4 * d + _row_bytes(case)) + case["rot"] * 4)
    read = n * hkv * (_row_bytes(case) + 4 * d)
    rot = n * (hq + hkv) * case["rot"] * 3
    op = case["op"]
    if op == "attn":
        return {"bytes": attn, "flops": 4 * seen * hq * d}
    if op == "append":
        return {"bytes": append, "flops": rot}
    if op == "read":
        return {"bytes": read, "flops": 2 * n * hkv * 2 * d}
    if op == "step":
        return {"bytes": attn + append + read, "flops": 4 * seen * hq * d + rot}
    return {"bytes": append + read, "flops": rot}


# ------------------------------------------------------------------ the pool's layout, in torch

def _positions(device):
    i = torch.arange(16, device=device)
    return 2 * (i & 3) + ((i >> 2) & 1) + (i & 8)


def _sizes(case):
    d, kb, vb = case["d"], case["kb"], case["vb"]
    rk, rv = d * kb // 8, d * vb // 8
    return rk, rv, 16 * (rk + rv) + (0 if kb == 16 else 128)


def _key_byte(rk, pos, bits):
    """[len(pos), rk] place of every byte of the key rows stored at rows `pos` (the tokens themselves for 16 bits)."""
    b = torch.arange(rk, device=pos.device)
    p = pos[..., None]
    if bits == 16:
        return ((b >> 4) ^ (p & 7)) * 16 + (b & 15)
    return b ^ ((p & 1) * 64) if rk == 128 else b + 0 * p


def _value_byte(rv, tok, bits):
    b = torch.arange(rv, device=tok.device)
    t = tok[..., None]
    if bits == 16:
        return ((b >> 4) ^ (t & 7)) * 16 + (b & 15)
    if rv == 128:
        return b ^ ((t & 3) * 32)
    return b ^ (((t >> 1) & 1) * 32) if rv == 64 else b + 0 * t


def _fields(codes, bits):
    """[..., d] codes -> [..., d * bits / 8] bytes, least significant field first."""
    per = 8 // bits
    c = codes.to(torch.int32).reshape(*codes.shape[:-1], -1, per)
    sh = torch.arange(per, device=codes.device, dtype=torch.int32) * bits
    return (c << sh).sum(-1).to(torch.uint8)


def _codes(data, bits):
    per = 8 // bits
    sh = torch.arange(per, device=data.device, dtype=torch.int32) * bits
    return ((data.to(torch.int32)[..., None] >> sh) & (2 ** bits - 1)).reshape(*data.shape[:-1], -1)


def _quantize(x, bits):
    """Rows of fp16 values -> (codes, scale, zero), per row over its channels."""
    f = x.float()
    z, top = f.amin(-1, keepdim=True), f.amax(-1, keepdim=True)
    s = ((top - z) / (2 ** bits - 1)).half()
    c = torch.round((f - z) / s.float())
    c = torch.where(s > 0, c, torch.zeros_like(c)).clamp(0, 2 ** bits - 1)
    return c, s.squeeze(-1), z.half().squeeze(-1)


def _half(x):
    return x.float().clamp(-65504.0, 65504.0).half()


def _tiles_from_rows(case, k, v):
    """k, v [..., 16, d] in the cache's type -> the tiles' bytes [..., tile bytes]."""
    rk, rv, tb = _sizes(case)
    tok = torch.arange(16, device=k.device)
    lead = k.shape[:-2]
    if case["kb"] == 16:
        out = []
        for x, r in ((k, rk), (v, rv)):
            raw = x.contiguous().view(torch.uint8)
            dst = torch.empty_like(raw)
            dst.scatter_(-1, _key_byte(r, tok, 16).expand_as(raw), raw)
            out.append(dst.reshape(*lead, 16 * r))
        return torch.cat(out, -1)
    pos = _positions(k.device)
    ck, ks, kz = _quantize(_half(k), case["kb"])
    cv, vs, vz = _quantize(_half(v), case["vb"])
    bk, bv = _fields(ck, case["kb"]), _fields(cv, case["vb"])
    sk = torch.empty_like(bk)
    sk[..., pos, :] = torch.empty_like(bk).scatter_(-1, _key_byte(rk, pos, case["kb"]).expand_as(bk), bk)
    sv = torch.empty_like(bv).scatter_(-1, _value_byte(rv, tok, case["vb"]).expand_as(bv), bv)
    sz = torch.empty(*lead, 16, 4, dtype=torch.float16, device=k.device)
    sz[..., pos, :] = torch.stack([ks, kz, vs, vz], -1)
    return torch.cat([sk.reshape(*lead, 16 * rk), sv.reshape(*lead, 16 * rv), sz.view(torch.uint8).reshape(*lead, 128)], -1)


def _rows_from_tiles(case, tiles, dtype):
    """The tiles' bytes [..., tile bytes] -> keys and values [..., 16, d] in fp32."""
    rk, rv, tb = _sizes(case)
    tok = torch.arange(16, device=tiles.device)
    lead = tiles.shape[:-1]
    bk = tiles[..., :16 * rk].reshape(*lead, 16, rk)
    bv = tiles[..., 16 * rk:16 * (rk + rv)].reshape(*lead, 16, rv)
    if case["kb"] == 16:
        return [torch.gather(b, -1, _key_byte(r, tok, 16).expand_as(b)).contiguous().view(dtype).float()
                for b, r in ((bk, rk), (bv, rv))]
    pos = _positions(tiles.device)
    bk = bk[..., pos, :]
    bk = torch.gather(bk, -1, _key_byte(rk, pos, case["kb"]).expand_as(bk))
    bv = torch.gather(bv, -1, _value_byte(rv, tok, case["vb"]).expand_as(bv))
    sz = tiles[..., 16 * (rk + rv):].contiguous().view(torch.float16).reshape(*lead, 16, 4)[..., pos, :].float()
    k = _codes(bk, case["kb"]).float() * sz[..., 0:1] + sz[..., 1:2]
    v = _codes(bv, case["vb"]).float() * sz[..., 2:3] + sz[..., 3:4]
    return [k, v]


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev, dt = "cuda", _DTYPE[case["dtype"]]
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    lens, news = _lengths(case)
    B, hq, hkv, d, P = case["batch"], case["hq"], case["hkv"], case["d"], case["page"]
    rk, rv, tb = _sizes(case)
    need = [-(-x // P) for x in lens]
    width = max(max(need), 1)
    pages = sum(need) + 1
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = torch.arange(at, at + k, dtype=torch.int32)
        at += k
    table = table.to(dev)
    table = torch.where(table >= 0, order[table.clamp(min=0).long()], table).contiguous()
    # keys with a few strong channels, values that drift, as the caches of real models have them
    pool = torch.empty(pages * hkv * (P // 16) * tb + TAIL, dtype=torch.uint8, device=dev)
    body = pool[:-TAIL].view(pages, hkv, P // 16, tb)
    mu = torch.randn(hkv, 1, 1, d, generator=g, device=dev) * 0.5
    sigma = torch.exp(torch.randn(hkv, 1, 1, d, generator=g, device=dev) * 0.5)
    strong = torch.ones(hkv, 1, 1, d, device=dev)
    strong[..., torch.randperm(d, generator=g, device=dev)[:4]] = 10.0
    step = max(1, (1 << 26) // (hkv * P * d))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        z = torch.randn(n, hkv, P // 16, 16, d, generator=g, device=dev)
        k = (mu + sigma * z) * strong
        v = torch.randn(n, hkv, P // 16, 16, d, generator=g, device=dev) + 4.0 * a / pages
        body[a:a + n] = _tiles_from_rows(case, k.to(dt), v.to(dt))
    pool[-TAIL:] = 0
    n = sum(news)
    # the new rows as the model's projection leaves them: one tensor, q, k and v side by side
    qkv = torch.randn(n, hq + 2 * hkv, d, generator=g, device=dev)
    qkv[:, hq:hq + hkv] = (mu + sigma * qkv[:, hq:hq + hkv].transpose(0, 1)[:, None]).mul(strong).squeeze(1).transpose(0, 1)
    qkv = qkv.to(dt)
    rot = case["rot"]
    inv = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    ang = torch.arange(max(max(lens), 1), dtype=torch.float64, device=dev)[:, None] * inv
    rope = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
    cu = torch.tensor([0] + news, dtype=torch.int32).cumsum(0).to(torch.int32).to(dev) if case["new"] > 1 else None
    s = dict(case=case, dtype=dt, pool=pool, table=table, lens=torch.tensor(lens, dtype=torch.int32, device=dev), cu=cu,
             q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], rope=rope, n=n, pages=pages)
    if own:
        from mixed_precision_quantized_quant_gb300 import kvq
        s["cache"] = kvq.KVQPagedCache([(case["kb"], case["vb"])], num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                                       page_size=P, num_pages=pages, dtype=dt, device=dev, buffer=pool)
        s["batch"] = kvq.PagedBatch(table, s["lens"], cu)
        s["rotation"] = kvq.Rotation(rope, interleaved=case["interleaved"])
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        c, b, out = s["cache"], s["batch"], {}
        if op in ("append", "step", "fill"):
            out["q"] = c.append(0, b, s["k"], s["v"], q=s["q"], rotation=s["rotation"])
        if op in ("attn", "step"):
            q = out["q"] if op == "step" else s["q"]
            out["out"], out["lse"] = c.decode_attn(0, b, q, window=s["case"]["window"], return_lse=True)
        if op in ("read", "step", "fill"):
            out["k"], out["v"] = c.read(0, b, s["n"])
        if op == "append":
            out["pool"] = s["pool"][:-TAIL].view(s["dtype"])
        return out
    out = {}
    if op in ("append", "step", "fill"):
        out["q"] = _append(s)
    if op in ("attn", "step"):
        out["out"], out["lse"] = _attend(s, out["q"] if op == "step" else s["q"])
    if op in ("read", "step", "fill"):
        out["k"], out["v"] = _read(s)
    if op == "append":
        out["pool"] = s["pool"][:-TAIL].view(s["dtype"])
    return out


def _new_rows(s):
    """Position and (tile of kv head 0, token of the tile) of every new row, and the tiles from one head to the next."""
    c, lens = s["case"], s["lens"].long()
    if s["cu"] is None:
        seq = torch.arange(s["n"], device=lens.device)
        p = lens - 1
    else:
        cu = s["cu"].long()
        row = torch.arange(s["n"], device=lens.device)
        seq = torch.searchsorted(cu, row, right=True) - 1
        p = lens[seq] - (cu[seq + 1] - cu[seq]) + row - cu[seq]
    P = c["page"]
    page = s["table"][seq, p // P].long()
    return p, page * c["hkv"] * (P // 16) + (p % P) // 16, p % 16


def _rotate(s, x, p):
    """Rows [n, heads, d] rotated in fp32 (products and sums rounded one by one), rounded once."""
    r = s["case"]["rot"]
    cos, sin = s["rope"][p][:, None, :r // 2], s["rope"][p][:, None, r // 2:]
    f = x.float()
    t = f[..., :r]
    if s["case"]["interleaved"]:
        a, b = t[..., 0::2], t[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = t[..., :r // 2], t[..., r // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, f[..., r:]], -1)


def _row_places(s):
    """Flat byte places in the pool of the new rows' key bytes, value bytes and scale quadruples."""
    c = s["case"]
    rk, rv, tb = _sizes(c)
    _, tile, tok = _new_rows(s)
    head = torch.arange(c["hkv"], device=tile.device) * (c["page"] // 16)
    base = ((tile[:, None] + head) * tb)[..., None]
    pos = tok if c["kb"] == 16 else _positions(tile.device)[tok]
    k = base + (pos * rk)[:, None, None] + _key_byte(rk, pos, c["kb"])[:, None]
    v = base + 16 * rk + (tok * rv)[:, None, None] + _value_byte(rv, tok, c["vb"])[:, None]
    z = base + 16 * (rk + rv) + (pos * 8)[:, None, None] + torch.arange(8, device=tile.device)
    return k, v, z


def _append(s):
    c = s["case"]
    p, _, _ = _new_rows(s)
    kplace, vplace, zplace = _row_places(s)
    k = _rotate(s, s["k"], p)
    if c["kb"] == 16:
        s["pool"][kplace] = k.to(s["dtype"]).contiguous().view(torch.uint8)
        s["pool"][vplace] = s["v"].contiguous().view(torch.uint8)
    else:
        ck, ks, kz = _quantize(_half(k), c["kb"])
        cv, vs, vz = _quantize(_half(s["v"]), c["vb"])
        s["pool"][kplace] = _fields(ck, c["kb"])
        s["pool"][vplace] = _fields(cv, c["vb"])
        s["pool"][zplace] = torch.stack([ks, kz, vs, vz], -1).view(torch.uint8)
    return _rotate(s, s["q"], p).to(s["dtype"])


def _read(s):
    c = s["case"]
    kplace, vplace, zplace = _row_places(s)
    bk, bv = s["pool"][kplace], s["pool"][vplace]
    if c["kb"] == 16:
        return bk.view(s["dtype"]), bv.view(s["dtype"])
    sz = s["pool"][zplace].view(torch.float16).float()
    k = _codes(bk, c["kb"]).float() * sz[..., 0:1] + sz[..., 1:2]
    v = _codes(bv, c["vb"]).float() * sz[..., 2:3] + sz[..., 3:4]
    return k.to(s["dtype"]), v.to(s["dtype"])


def _attend(s, q):
    c = s["case"]
    B, hq, hkv, d, P = c["batch"], c["hq"], c["hkv"], c["d"], c["page"]
    rk, rv, tb = _sizes(c)
    body = s["pool"][:-TAIL].view(s["pages"], hkv, P // 16, tb)
    tiles = body[s["table"].clamp(min=0).long()].transpose(1, 2)  # [B, hkv, pages, tiles, bytes]
    k, v = _rows_from_tiles(c, tiles, s["dtype"])
    k, v = k.reshape(B, hkv, -1, d), v.reshape(B, hkv, -1, d)
    at, n = torch.arange(k.shape[2], device=k.device), s["lens"][:, None]
    seen = at < n
    if c["window"]:
        seen = seen & (at >= n - c["window"])
    seen = seen[:, None, None]
    t = torch.matmul(q.float().view(B, hkv, hq // hkv, d), k.transpose(2, 3)) / math.sqrt(d)
    t = torch.where(seen, t, torch.full_like(t, -math.inf))
    top = t.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    e = torch.exp(t - top)
    total = e.sum(-1, keepdim=True)
    v = torch.where(seen[:, :, 0, :, None], v, torch.zeros_like(v))
    o = torch.matmul(e, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (torch.log(total) + top).squeeze(-1)
    return o.view(B, hq, d).to(s["dtype"]), lse.reshape(B, hq)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, dev = case["op"], s["pool"].device
    hq, hkv, d, P, kb, vb, r = (case[x] for x in ("hq", "hkv", "d", "page", "kb", "vb", "rot"))
    lens, news = _lengths(case)
    table = s["table"].cpu()
    tile = 2 * 16 * d * 2 if kb == 16 else 2 * d * (kb + vb) + 128
    page_bytes = hkv * (P // 16) * tile
    pool, chan, heads = s["pool"], torch.arange(d, device=dev), torch.arange(hkv, device=dev)[:, None]

    def start(b, p):  # first byte of the tile of position p: [heads, tokens]
        page = table[b].to(dev).long()[p // P]
        return page * page_bytes + (heads * (P // 16) + (p % P) // 16) * tile

    def row_of(i):
        return i // 8 * 8 + i % 4 * 2 + i % 8 // 4

    def value_at(b, p, is_key):
        """[heads, tokens, d] stored values of positions p, in 64 bits."""
        i, base = p % 16, start(b, p)
        bits = kb if is_key else vb
        if bits == 16:
            off = (0 if is_key else 32 * d) + i[:, None] * 2 * d + ((chan // 8)[None] ^ (i % 8)[:, None]) * 16 + chan % 8 * 2
            at = (base[..., None] + off) // 2
            return pool.view(s["dtype"])[at].double()
        rb = d * bits // 8
        byte = (chan * bits // 8)[None].expand(len(i), d)
        if is_key:
            row = row_of(i)
            byte = torch.where((row % 2 == 1)[:, None] & torch.tensor(rb == 128, device=dev), (byte + 64) % 128, byte)
            off = row[:, None] * rb + byte
        else:
            flip = i % 4 if rb == 128 else i // 2 % 2 if rb == 64 else i * 0
            byte = ((byte // 32) ^ flip[:, None]) * 32 + byte % 32
            off = 2 * d * kb + i[:, None] * rb + byte
        code = (pool[base[..., None] + off].long() >> (chan * bits % 8)) % (1 << bits)
        sz = (base + 2 * d * (kb + vb) + row_of(i) * 8 + (0 if is_key else 4)) // 2
        h = pool.view(torch.float16)
        return code.double() * h[sz].double()[..., None] + h[sz + 1].double()[..., None]

    def turned(x, p):  # [tokens, heads, d]
        y = x.double().clone()
        cos, sin = (s["rope"][p].double()[:, None, j * (r // 2):(j + 1) * (r // 2)] for j in (0, 1))
        first, second = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
        a, b = x[..., first].double(), x[..., second].double()
        y[..., first], y[..., second] = a * cos - b * sin, a * sin + b * cos
        return y

    def stored(x, bits):  # rows as the cache holds them
        if bits == 16:
            return x
        h = x.clamp(-65504, 65504).half().double()
        low, high = h.min(-1, keepdim=True).values, h.max(-1, keepdim=True).values
        sc = ((high - low) / (2 ** bits - 1)).half().double()
        code = torch.where(sc > 0, ((h - low) / sc.clamp(min=1e-30)).round(), torch.zeros_like(h)).clamp(0, 2 ** bits - 1)
        return code * sc + low

    out = {k: [] for k in ("q", "out", "lse", "k", "v")}
    if op == "append":
        full = pool[:-TAIL].view(s["dtype"]).double()
    a = 0
    for b, (n, m) in enumerate(zip(lens, news)):
        p = torch.arange(n - m, n, device=dev) if op != "attn" else None
        if op in ("append", "step", "fill"):
            rows = slice(a, a + m)
            q, k, v = turned(s["q"][rows], p), turned(s["k"][rows], p), s["v"][rows].double()
            out["q"].append(q)
            if op == "append":
                i = p % 16
                off = i[:, None] * 2 * d + ((chan // 8)[None] ^ (i % 8)[:, None]) * 16 + chan % 8 * 2
                at = (start(b, p)[..., None] + off) // 2
                full[at], full[at + 16 * d] = k.transpose(0, 1), v.transpose(0, 1)
            else:
                k, v = (stored(x, y) for x, y in ((k, kb), (v, vb)))
                if op == "step" and kb == 16:  # the cache holds what was rounded
                    k = k.to(s["dtype"]).double()
        if op in ("read", "step", "fill"):
            if op == "read":
                k, v = value_at(b, p, True).transpose(0, 1), value_at(b, p, False).transpose(0, 1)
            out["k"].append(k)
            out["v"].append(v)
        if op in ("attn", "step"):
            lo = max(0, n - case["window"]) if case["window"] else 0
            if n == 0:
                out["out"].append(torch.zeros(1, hq, d, dtype=torch.float64, device=dev))
                out["lse"].append(torch.full((1, hq), -math.inf, dtype=torch.float64, device=dev))
            else:
                seen = torch.arange(lo, n, device=dev)
                kk, vv = value_at(b, seen, True), value_at(b, seen, False)
                if op == "step":  # the row that this pass appends
                    kk[:, -1], vv[:, -1] = k[0], v[0]
                    query = q[0].to(s["dtype"]).double()
                else:
                    query = s["q"][b].double()
                t = torch.einsum("hgd,htd->hgt", query.view(hkv, hq // hkv, d), kk) * d ** -0.5
                out["out"].append(torch.einsum("hgt,htd->hgd", t.softmax(-1), vv).reshape(1, hq, d))
                out["lse"].append(t.logsumexp(-1).reshape(1, hq))
        a += m
    got = {k: torch.cat(v) for k, v in out.items() if v}
    if op == "append":
        got["pool"] = full
    return got
