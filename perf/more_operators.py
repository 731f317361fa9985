"""Cases that measure the paged cache's operators for runs of new tokens: attention of a chunk of new tokens over the
pages, attention of whole prompts over their own rows, and append with a norm of every query and key head before the
rotation.

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
EPS = 1e-6


# ------------------------------------------------------------------ cases

def _case(name, op, batch, hq, hkv, d, length, new, kb, vb, page, dtype, ragged=True, window=0, rot=0, interleaved=False):
    """`op`: "chunk" (queries of the new tokens over the pages), "prompt" (over the prompts' own rows), "norm" (append
    with norms) or "admit" (append with norms, then the prompts' attention).  `length`: longest sequence after the new
    tokens; `new`: the longest run of new tokens; `rot`: rotary width (0: the whole head)."""
    c = dict(op=op, batch=batch, hq=hq, hkv=hkv, d=d, length=length, new=new, kb=kb, vb=vb, page=page, dtype=dtype,
             ragged=ragged, window=window, rot=rot or d, interleaved=interleaved)
    return dict(c, name=name) if name else c


def listed():
    return [
        # four drafted tokens of one short chat on the smallest configuration: nothing but latency
        _case("chunk-tiny-d64-fp16", "chunk", 1, 8, 2, 64, 257, 4, 16, 16, 32, "fp16", ragged=False),
        # drafted tokens of a serving batch checked against the cache, on an unquantized layer
        _case("chunk-verify-8b-bf16", "chunk", 16, 32, 8, 128, 4096, 5, 16, 16, 64, "bf16"),
        # the same over long contexts on the common layers (K4V2)
        _case("chunk-verify-70b-k4v2", "chunk", 8, 64, 8, 128, 32768, 8, 4, 2, 128, "fp16"),
        # a long prompt taken in pieces: 2048 new tokens behind 8192 cached ones
        _case("chunk-prefill-8b-bf16", "chunk", 1, 32, 8, 128, 10240, 2048, 16, 16, 64, "bf16", ragged=False),
        # pieces of several prompts on a sensitive layer (K8V4), odd lengths in small pages
        _case("chunk-prefill-8b-k8v4", "chunk", 4, 32, 8, 128, 5119, 1023, 8, 4, 16, "fp16"),
        # seven query heads a kv head, a layer that looks back over 4096 tokens only
        _case("chunk-7b-8k-k8v8-window", "chunk", 6, 28, 4, 128, 8192, 700, 8, 8, 64, "bf16", window=4096),
        # one short question on the smallest configuration
        _case("prompt-tiny-d64-fp16", "prompt", 1, 8, 2, 64, 37, 37, 16, 16, 32, "fp16", ragged=False),
        # prompts of several requests admitted together
        _case("prompt-packed-8b-bf16", "prompt", 12, 32, 8, 128, 2047, 2047, 16, 16, 64, "bf16"),
        # one long prompt, 64 query heads (the largest)
        _case("prompt-long-70b-fp16", "prompt", 1, 64, 8, 128, 8192, 8192, 16, 16, 128, "fp16", ragged=False),
        # a decode step's append for one sequence: nothing but latency
        _case("norm-one-d64-fp16", "norm", 1, 8, 2, 64, 257, 1, 16, 16, 32, "fp16", ragged=False),
        # prompts of several requests into an unquantized layer
        _case("norm-prefill-8b-bf16", "norm", 5, 32, 8, 128, 2047, 2047, 16, 16, 64, "bf16"),
        # prompts admitted to a quantized layer: append with norms, attention over the exact rows
        _case("admit-8b-k8v4", "admit", 6, 32, 8, 128, 1500, 1500, 8, 4, 64, "bf16", rot=64, interleaved=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    hq, hkv, d = rng.choice([(8, 2, 64), (16, 4, 64), (32, 8, 128), (28, 4, 128), (32, 32, 128), (64, 8, 128)])
    op = rng.choice(["chunk", "chunk", "chunk", "prompt", "prompt", "norm", "admit"])
    kb, vb = rng.choice([(16, 16), (16, 16), (8, 8), (8, 4), (4, 4), (4, 2), (2, 2), (2, 8)])
    if op in ("norm", "admit"):
        kb, vb = rng.choice([(16, 16), (8, 8), (8, 4)])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["fp16", "bf16"])
    batch = _log(rng, 1, 32)
    ragged = rng.random() < 0.8
    window = rng.choice([0, 0, 0, _log(rng, 1, 8192)])
    pairs = 64 * 8192 * 8192 // 2  # (query head, token) pairs of the largest case
    if op == "chunk":
        new = _log(rng, 1, 2048)
        new = max(1, min(new, 8192 // batch))
        length = new + _log(rng, 1, 32768)
        length = min(length, (8 * 32768 * 8) // (batch * hkv), pairs // (batch * hq * new))
        return _case(None, op, batch, hq, hkv, d, max(length, new), new, kb, vb, page, dtype, ragged=ragged, window=window)
    new = _log(rng, 1, 8192)
    new = max(1, min(new, 12000 // batch))
    if op != "norm":
        new = max(1, min(new, int(math.sqrt(pairs // (batch * hq)))))
    rot = rng.choice([d, d, d // 2])
    if op == "prompt":
        kb = vb = 16
    return _case(None, op, batch, hq, hkv, d, new, new, kb, vb, page, dtype, ragged=ragged,
                 window=0 if op == "norm" else window, rot=rot, interleaved=rng.random() < 0.3)


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
        lens.append(max(n, int(L * f)) if L > new else n)
        news.append(n)
    return lens, news


def _pairs(case):
    """(query token, token it sees) pairs of all sequences, and rows that any of them sees."""
    w, total, rows = case["window"], 0, 0
    for n, m in zip(*_lengths(case)):
        first, last = n - m + 1, n  # tokens that the first and the last new one could see
        if w:
            total += sum(min(w, x) for x in range(first, last + 1))
            rows += n - max(0, first - w)
        else:
            total += m * (first + last) // 2
            rows += n
    return total, rows


def _row_bytes(case):
    q = case["kb"] != 16
    return case["d"] * (case["kb"] + case["vb"]) / 8 + (8 if q else 0)


def work(case):
    lens, news = _lengths(case)
    hq, hkv, d, op = case["hq"], case["hkv"], case["d"], case["op"]
    n = sum(news)
    pairs, rows = _pairs(case)
    queries = n * hq * (4 * d + 4)  # rows in, rows and log-sum-exps out
    flops = 4 * pairs * hq * d
    if op == "chunk":
        table = sum(-(-x // case["page"]) for x in lens) * 4 + 8 * len(lens) + 4
        return {"bytes": rows * hkv * _row_bytes(case) + queries + table, "flops": flops}
    if op == "prompt":
        return {"bytes": rows * hkv * 4 * d + queries + 4 * len(lens) + 4, "flops": flops}
    append = n * (hq * 4 * d + hkv * (6 * d + _row_bytes(case)) + case["rot"] * 4) + 4 * d
    append_flops = n * (hq + hkv) * (case["rot"] * 3 + 4 * d)
    read = 0 if case["kb"] == 16 else n * hkv * (_row_bytes(case) + 4 * d)
    if op == "norm":
        return {"bytes": append + read, "flops": append_flops}
    return {"bytes": append + read + rows * hkv * 4 * d + queries, "flops": append_flops + flops}


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
        raw = torch.stack([k, v], -3).contiguous().view(torch.uint8)
        dst = torch.empty_like(raw)
        return dst.scatter_(-1, _key_byte(rk, tok, 16).expand_as(raw), raw).reshape(*lead, 32 * rk)
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
        return [torch.gather(b, -1, _key_byte(rk, tok, 16).expand_as(b)).contiguous().view(dtype).float() for b in (bk, bv)]
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
    width = max(need)
    # a prompt's attention reads no page
    pages = 1 if case["op"] == "prompt" else sum(need) + 1
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = torch.arange(at, at + k, dtype=torch.int32)
        at += k
    table = table.to(dev)
    table = torch.where(table >= 0, order[table.clamp(0, pages - 1).long()], table).contiguous()
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
    ang = torch.arange(max(lens), dtype=torch.float64, device=dev)[:, None] * inv
    rope = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
    cu = torch.tensor([0] + news, dtype=torch.int32).cumsum(0).to(torch.int32).to(dev)
    wq, wk = ((1.0 + 0.3 * torch.randn(d, generator=g, device=dev)).to(dt) for _ in range(2))
    s = dict(case=case, dtype=dt, pool=pool, table=table, lens=torch.tensor(lens, dtype=torch.int32, device=dev), cu=cu,
             q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], rope=rope, wq=wq, wk=wk, n=n, pages=pages,
             longest=max(lens), most=max(news))
    if own:
        from mixed_precision_quantized_quant_gb300 import kvq
        s["cache"] = kvq.KVQPagedCache([(case["kb"], case["vb"])], num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                                       page_size=P, num_pages=pages, dtype=dt, device=dev, buffer=pool)
        s["batch"] = kvq.PagedBatch(table, s["lens"], cu)
        s["rotation"] = kvq.Rotation(rope, interleaved=case["interleaved"])
        s["norm"] = kvq.HeadNorm(wq, wk, eps=EPS)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    op, out = c["op"], {}
    if own:
        cache, batch = s["cache"], s["batch"]
        if op == "chunk":
            out["out"], out["lse"] = cache.chunk_attn(0, batch, s["q"], window=c["window"], return_lse=True)
            return out
        q, k = s["q"], s["k"]
        if op != "prompt":
            k = out["k"] = torch.empty(k.shape, dtype=k.dtype, device=k.device)
            q = out["q"] = cache.append(0, batch, s["k"], s["v"], q=q, rotation=s["rotation"], norm=s["norm"], k_out=k)
            if c["kb"] == 16:
                out["pool"] = s["pool"][:-TAIL].view(s["dtype"])
            else:
                out["cached_k"], out["cached_v"] = cache.read(0, batch, s["n"])
        if op != "norm":
            out["out"], out["lse"] = cache.prompt_attn(batch, q, k, s["v"], window=c["window"], return_lse=True)
        return out
    if op == "chunk":
        out["out"], out["lse"] = _chunk(s)
        return out
    q, k = s["q"], s["k"]
    if op != "prompt":
        out["k"], out["q"] = _append(s)
        q, k = out["q"], out["k"]
        if c["kb"] == 16:
            out["pool"] = s["pool"][:-TAIL].view(s["dtype"])
        else:
            out["cached_k"], out["cached_v"] = _read(s)
    if op != "norm":
        out["out"], out["lse"] = _prompt(s, q, k)
    return out


def _new_rows(s):
    """Sequence, place in it and position of every new row."""
    cu, lens = s["cu"].long(), s["lens"].long()
    row = torch.arange(s["n"], device=lens.device)
    seq = torch.searchsorted(cu, row, right=True) - 1
    at = row - cu[seq]
    return seq, at, lens[seq] - (cu[seq + 1] - cu[seq]) + at


def _norm(x, w):
    """Every row over its channels, in fp32."""
    f = x.float()
    return f * (1.0 / torch.sqrt((f * f).mean(-1, keepdim=True) + EPS)) * w.float()


def _rotate(s, f, p):
    """fp32 rows [n, heads, d] turned by their positions."""
    r = s["case"]["rot"]
    cos, sin = s["rope"][p][:, None, :r // 2], s["rope"][p][:, None, r // 2:]
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
    seq, _, p = _new_rows(s)
    P = c["page"]
    tile, tok = s["table"][seq, p // P].long() * c["hkv"] * (P // 16) + (p % P) // 16, p % 16
    head = torch.arange(c["hkv"], device=tile.device) * (P // 16)
    base = ((tile[:, None] + head) * tb)[..., None]
    pos = tok if c["kb"] == 16 else _positions(tile.device)[tok]
    k = base + (pos * rk)[:, None, None] + _key_byte(rk, pos, c["kb"])[:, None]
    v = base + 16 * rk + (tok * rv)[:, None, None] + _value_byte(rv, tok, c["vb"])[:, None]
    z = base + 16 * (rk + rv) + (pos * 8)[:, None, None] + torch.arange(8, device=tile.device)
    return k, v, z


def _append(s):
    """Stores the rows; the turned keys and queries in the cache's type."""
    c = s["case"]
    _, _, p = _new_rows(s)
    kplace, vplace, zplace = _row_places(s)
    k = _rotate(s, _norm(s["k"], s["wk"]), p)
    q = _rotate(s, _norm(s["q"], s["wq"]), p).to(s["dtype"])
    if c["kb"] == 16:
        s["pool"][kplace] = k.to(s["dtype"]).contiguous().view(torch.uint8)
        s["pool"][vplace] = s["v"].contiguous().view(torch.uint8)
    else:
        ck, ks, kz = _quantize(_half(k), c["kb"])
        cv, vs, vz = _quantize(_half(s["v"]), c["vb"])
        s["pool"][kplace] = _fields(ck, c["kb"])
        s["pool"][vplace] = _fields(cv, c["vb"])
        s["pool"][zplace] = torch.stack([ks, kz, vs, vz], -1).view(torch.uint8)
    return k.to(s["dtype"]), q


def _read(s):
    c = s["case"]
    kplace, vplace, zplace = _row_places(s)
    sz = s["pool"][zplace].view(torch.float16).float()
    k = _codes(s["pool"][kplace], c["kb"]).float() * sz[..., 0:1] + sz[..., 1:2]
    v = _codes(s["pool"][vplace], c["vb"]).float() * sz[..., 2:3] + sz[..., 3:4]
    return k.to(s["dtype"]), v.to(s["dtype"])


def _attend(s, q, k, v, first, last):
    """q [B, m, hq, d] (one row's queries at a time see positions first .. last, [B, m]) over k, v [B, hkv, t, d] in fp32."""
    c = s["case"]
    B, m = q.shape[:2]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    at = torch.arange(k.shape[2], device=k.device)
    seen = ((at >= first[..., None]) & (at <= last[..., None]))[:, None, None]  # [B, 1, 1, m, t]
    x = q.float().view(B, m, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    t = torch.matmul(x.reshape(B, hkv, -1, d), k.transpose(2, 3)).view(B, hkv, hq // hkv, m, -1) / math.sqrt(d)
    t.masked_fill_(~seen, -math.inf)
    top = t.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    t = t.sub_(top).exp_()
    total = t.sum(-1, keepdim=True)
    o = torch.matmul(t.view(B, hkv, -1, t.shape[-1]), v).view(B, hkv, hq // hkv, m, d)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    lse = (torch.log(total) + top).squeeze(-1)
    return o.permute(0, 3, 1, 2, 4).reshape(B, m, hq, d), lse.permute(0, 3, 1, 2).reshape(B, m, hq)


def _padded(s, x):
    """Rows [n, heads, d] -> [B, the longest run, heads, d], zeros behind a run's end."""
    seq, at, _ = _new_rows(s)
    y = torch.zeros(s["case"]["batch"], s["most"], *x.shape[1:], dtype=x.dtype, device=x.device)
    y[seq, at] = x
    return y


def _chunk(s):
    c = s["case"]
    B, hkv, d, P = c["batch"], c["hkv"], c["d"], c["page"]
    body = s["pool"][:-TAIL].view(s["pages"], hkv, P // 16, -1)
    tiles = body[s["table"].clamp(min=0).long()].transpose(1, 2)  # [B, hkv, pages, tiles, bytes]
    k, v = (x.reshape(B, hkv, -1, d)[:, :, :s["longest"]] for x in _rows_from_tiles(c, tiles, s["dtype"]))
    seq, at, p = _new_rows(s)
    last = torch.full((B, s["most"]), -1, dtype=torch.int64, device=p.device)
    last[seq, at] = p
    first = (last - c["window"] + 1).clamp(min=0) if c["window"] else torch.zeros_like(last)
    # rows behind a sequence's end are another's, or nothing's
    v = torch.where((torch.arange(v.shape[2], device=v.device) < s["lens"][:, None])[:, None, :, None], v, torch.zeros_like(v))
    o, lse = _attend(s, _padded(s, s["q"]), k, v, first, last)
    return o[seq, at].to(s["dtype"]), lse[seq, at]


def _prompt(s, q, k):
    c = s["case"]
    seq, at, _ = _new_rows(s)
    last = torch.full((c["batch"], s["most"]), -1, dtype=torch.int64, device=at.device)
    last[seq, at] = at
    first = (last - c["window"] + 1).clamp(min=0) if c["window"] else torch.zeros_like(last)
    k, v = (_padded(s, x).float().transpose(1, 2).contiguous() for x in (k, s["v"]))
    o, lse = _attend(s, _padded(s, q), k, v, first, last)
    return o[seq, at].to(s["dtype"]), lse[seq, at]


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, dev = case["op"], s["pool"].device
    hq, hkv, d, P, kb, vb, r = (case[x] for x in ("hq", "hkv", "d", "page", "kb", "vb", "rot"))
    lens, news = _lengths(case)
    table = s["table"].cpu()
    tile = 64 * d if kb == 16 else 2 * d * (kb + vb) + 128
    pool, chan, heads = s["pool"], torch.arange(d, device=dev), torch.arange(hkv, device=dev)[:, None]

    def start(b, p):  # first byte of the tile of position p: [heads, tokens]
        page = table[b].to(dev).long()[p // P]
        return page * (hkv * (P // 16) * tile) + (heads * (P // 16) + (p % P) // 16) * tile

    def value_at(b, p, is_key):
        """[heads, tokens, d] stored values of positions p, in 64 bits."""
        i, base = p % 16, start(b, p)
        bits = kb if is_key else vb
        if bits == 16:
            off = (0 if is_key else 32 * d) + i[:, None] * 2 * d + ((chan // 8)[None] ^ (i % 8)[:, None]) * 16 + chan % 8 * 2
            return pool.view(s["dtype"])[(base[..., None] + off) // 2].double()
        rb = d * bits // 8
        row = i // 8 * 8 + i % 4 * 2 + i % 8 // 4
        byte = (chan * bits // 8)[None].expand(len(i), d)
        if is_key:
            if rb == 128:
                byte = torch.where((row % 2 == 1)[:, None], (byte + 64) % 128, byte)
            off = row[:, None] * rb + byte
        else:
            flip = i % 4 if rb == 128 else i // 2 % 2 if rb == 64 else i * 0
            off = 2 * d * kb + i[:, None] * rb + ((byte // 32) ^ flip[:, None]) * 32 + byte % 32
        code = (pool[base[..., None] + off].long() >> (chan * bits % 8)) % (1 << bits)
        sz = (base + 2 * d * (kb + vb) + row * 8 + (0 if is_key else 4)) // 2
        h = pool.view(torch.float16)
        return code.double() * h[sz].double()[..., None] + h[sz + 1].double()[..., None]

    def turned(x, w, p):  # [tokens, heads, d]
        y = x.double()
        y = y / ((y * y).mean(-1, keepdim=True) + EPS).sqrt() * w.double()
        cos, sin = (s["rope"][p].double()[:, None, j * (r // 2):(j + 1) * (r // 2)] for j in (0, 1))
        first, second = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
        a, b = y[..., first].clone(), y[..., second].clone()
        y[..., first], y[..., second] = a * cos - b * sin, a * sin + b * cos
        return y

    def stored(x, bits):  # rows as a quantized cache holds them
        h = x.clamp(-65504, 65504).half().double()
        low, high = h.min(-1, keepdim=True).values, h.max(-1, keepdim=True).values
        sc = ((high - low) / (2 ** bits - 1)).half().double()
        code = torch.where(sc > 0, ((h - low) / sc.clamp(min=1e-30)).round(), torch.zeros_like(h)).clamp(0, 2 ** bits - 1)
        return code * sc + low

    def attend(q, k, v, p0):
        """q [m, hq, d] at positions p0 .., k, v [hkv, t, d] of positions 0 ..: out [m, hq, d], lse [m, hq]."""
        m, n = q.shape[0], k.shape[1]
        o = torch.empty(m, hq, d, dtype=torch.float64, device=dev)
        lse = torch.empty(m, hq, dtype=torch.float64, device=dev)
        block = 512
        for h in range(hq):
            for a in range(0, m, block):
                e = min(m, a + block)
                lo = max(0, p0 + a - case["window"] + 1) if case["window"] else 0
                hi = p0 + e
                kk, vv = k[h * hkv // hq, lo:hi].double(), v[h * hkv // hq, lo:hi].double()
                t = q[a:e, h].double() @ kk.T * d ** -0.5
                dist = torch.arange(p0 + a, p0 + e, device=dev)[:, None] - torch.arange(lo, hi, device=dev)
                t[(dist < 0) | ((dist >= case["window"]) if case["window"] else (dist < 0))] = -math.inf
                o[a:e, h], lse[a:e, h] = t.softmax(-1) @ vv, t.logsumexp(-1)
        return o, lse

    names = {"chunk": ("out", "lse"), "prompt": ("out", "lse")}.get(op) or \
        ("k", "q") + (("pool",) if kb == 16 else ("cached_k", "cached_v")) + (() if op == "norm" else ("out", "lse"))
    out = {k: [] for k in names}
    full = pool[:-TAIL].view(s["dtype"]).double() if "pool" in out else None
    a = 0
    for b, (n, m) in enumerate(zip(lens, news)):
        rows = slice(a, a + m)
        a += m
        q, k, v = s["q"][rows], s["k"][rows], s["v"][rows]
        if op == "chunk":
            p = torch.arange(n, device=dev)
            o, lse = attend(q, value_at(b, p, True), value_at(b, p, False), n - m)
        else:
            if op != "prompt":
                p = torch.arange(n - m, n, device=dev)
                q, k = turned(q, s["wq"], p), turned(k, s["wk"], p)
                out["q"].append(q)
                out["k"].append(k)
                if kb == 16:
                    i = p % 16
                    off = i[:, None] * 2 * d + ((chan // 8)[None] ^ (i % 8)[:, None]) * 16 + chan % 8 * 2
                    at = (start(b, p)[..., None] + off) // 2
                    full[at], full[at + 16 * d] = k.transpose(0, 1), v.double().transpose(0, 1)
                else:
                    out["cached_k"].append(stored(k, kb))
                    out["cached_v"].append(stored(v.double(), vb))
                q, k = q.to(s["dtype"]), k.to(s["dtype"])  # what the attention is given
            if op != "norm":
                o, lse = attend(q, k.transpose(0, 1), v.transpose(0, 1), 0)
        if op != "norm":
            out["out"].append(o)
            out["lse"].append(lse)
    got = {k: torch.cat(v) for k, v in out.items() if v}
    if full is not None:
        got["pool"] = full
    return {k: got[k] for k in out}
