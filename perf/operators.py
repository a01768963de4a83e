"""Cases of the 4-bit KV cache operators (append, read, attention, evict), their plain forms in elementary
torch operations, and their definition in 64 bits.

The cache is a pool of pages, uint8 [num_pages][n_layers][n_kv_heads][page / 32][block]: a block holds 32
rows of one KV head, as K codes [32][d / 2] (element 2b in the low half of byte b), K parameters
[32][d / 64] of fp16 (scale, lo), the same for V, and in a tracked pool the rows' positions (int32 [32])
and accumulated attention weights (fp32 [32]).  A group of 64 elements x has lo = fp16(min x) and
scale = fp16((max x - min x) / 15); code = (x - lo) / scale rounded to nearest even, in 0 .. 15; value = lo + scale * code.
"""
import math

import torch

own = False

BLOCK_ROWS = 32


# ------------------------------------------------------------------ the cases
def _case(op, **kw):
    c = dict(op=op, dtype="float32", heads=9, kv=3, d=64, layers=2, page=64, seqs=1, rows=128, count=1, ragged=False,
             track=False, cap=0.0, bias=False, window=0, accumulate=False, keep=0, recent=0)
    c.update(kw)
    return c


def listed():
    return [
        # one token of a short chat with the 135M shape: latency
        _case("append", name="append one token", rows=117, track=True),
        # prompts of several users enter the cache together, ragged, bf16 activations, head dim 128
        _case("append", name="append prompts", dtype="bfloat16", heads=32, kv=8, d=128, seqs=16, rows=1500, count=1000, ragged=True),
        # one sequence is taken out of the cache, to be looked at or moved
        _case("read", name="read one sequence", heads=14, kv=2, rows=1501, count=1501),
        # a whole batch is taken out of the cache (as many KV heads as query heads)
        _case("read", name="read a batch", dtype="bfloat16", heads=32, kv=32, seqs=24, rows=2048, count=2048, page=128),
        # the smallest decode step: one sequence, a short context
        _case("attention", name="decode short", rows=120),
        # one sequence with a very long context, odd length
        _case("attention", name="decode long", rows=130001, page=128),
        # serving: 64 sequences of all lengths, bf16, capped scores
        _case("attention", name="decode batch capped", dtype="bfloat16", heads=32, kv=8, d=128, seqs=64, rows=16384, ragged=True, cap=30.0),
        # serving with eviction: rows carry positions and weights, distance bias, weights added up
        _case("attention", name="decode tracked", heads=14, kv=2, seqs=48, rows=8191, ragged=True, track=True, bias=True, accumulate=True),
        # the last chunk of a long prompt, fp32 activations
        _case("attention", name="prompt chunk", rows=8192, count=2048),
        # chunks of several prompts, bf16, sliding window and cap
        _case("attention", name="prompt batch window", dtype="bfloat16", heads=32, kv=8, d=128, seqs=4, rows=4096, count=1024, ragged=True,
              cap=50.0, window=2000),
        # one short sequence reaches its budget
        _case("evict", name="evict one sequence", layers=1, rows=300, keep=201, recent=32, track=True),
        # a batch is cut to its budget in several layers
        _case("evict", name="evict a batch", heads=32, kv=8, d=128, layers=4, seqs=16, rows=8192, ragged=True, keep=2048, recent=256, track=True),
    ]


#: the most that a drawn case may cost, in rows x KV heads x d (cache work) and query-row pairs x d (prompt work)
_MOST = {"append": 16 * 1000 * 8 * 128, "read": 24 * 2048 * 32 * 64, "attention": 64 * 16384 * 8 * 128, "evict": 4 * 16 * 8192 * 8 * 128}
_MOST_PAIRS = 2048 * 8192 * 9 * 64


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attention", "attention", "attention", "evict"])
    heads, kv, d = rng.choice([(9, 3, 64), (14, 2, 64), (4, 2, 64), (32, 32, 64), (32, 8, 128), (16, 1, 64), (8, 1, 128), (12, 4, 128), (5, 5, 128)])
    c = _case(op, dtype=rng.choice(["float32", "bfloat16"]), heads=heads, kv=kv, d=d, layers=rng.choice([1, 2, 3]), page=rng.choice([32, 64, 128]),
              seqs=_log(rng, 1, 64), ragged=rng.random() < 0.7, track=rng.random() < 0.4)
    if op == "evict":
        c["track"] = True
        c["rows"] = _log(rng, 40, 40000)
        c["keep"] = max(1, int(c["rows"] * rng.uniform(0.1, 0.9)))
        c["recent"] = int(c["keep"] * rng.uniform(0, 0.5))
    elif op == "attention":
        prompt = rng.random() < 0.4
        c["rows"] = _log(rng, 1, 8192 if prompt else 130001)
        c["count"] = min(c["rows"], _log(rng, 2, 2048)) if prompt else min(c["rows"], rng.choice([1, 1, 1, 2, 5]))
        c["cap"] = rng.choice([0.0, 0.0, 30.0, 50.0])
        c["bias"] = rng.random() < 0.3
        c["window"] = rng.choice([0, 0, 1, 100, 1000, 4096])
        c["accumulate"] = c["track"] and rng.random() < 0.6
    else:
        c["rows"] = _log(rng, 1, 8192)
        c["count"] = c["rows"] if op == "read" and rng.random() < 0.5 else _log(rng, 1, c["rows"])
    while c["seqs"] > 1 and _cost(c) > 1:
        c["seqs"] = max(1, c["seqs"] * 2 // 3)
    while _cost(c) > 1 and c["rows"] > 1:
        c["rows"] = max(1, c["rows"] * 3 // 4)
        c["count"] = min(c["rows"], c["count"])
        c["keep"] = min(c["rows"], c["keep"])
        c["recent"] = min(c["recent"], c["keep"])
    return c


def _cost(c):
    at_once = c["layers"] if c["op"] == "evict" else 1
    per = c["count"] if c["op"] in ("append", "read") else c["rows"]
    cost = at_once * c["seqs"] * per * c["kv"] * c["d"] / _MOST[c["op"]]
    if c["op"] == "attention" and c["count"] > 1:
        cost = max(cost, c["seqs"] * c["count"] * c["rows"] * c["heads"] * c["d"] / _MOST_PAIRS)
    return cost


def _lengths(c):
    """Rows and new tokens of each sequence: sequence 0 has the most, the others spread down to a fifth; every eighth slot of a ragged
    batch is idle (no new token)."""
    rows, counts = [], []
    for s in range(c["seqs"]):
        f = 1.0 if s == 0 or not c["ragged"] else 0.2 + 0.8 * ((s * 0.6180339887) % 1.0)
        r = max(1, int(c["rows"] * f))
        n = max(1, int(c["count"] * f))
        rows.append(r)
        counts.append(0 if c["ragged"] and s % 8 == 7 else min(n, r))
    return rows, counts


def _block_bytes(c):
    return BLOCK_ROWS * (c["d"] + c["d"] // 64 * 8 + (8 if c["track"] else 0))


def _row_bytes(c):
    return c["d"] + c["d"] // 64 * 8  # K and V codes and parameters of a row and KV head


def _visible(c, r, n, i):
    """How many rows query i of n sees of a cache of r rows (rows in the order of their positions)."""
    upto = r - n + i + 1
    return min(upto, c["window"]) if c["window"] else upto


def work(case):
    c = dict(case)
    size = 4 if c["dtype"] == "float32" else 2
    rows, counts = _lengths(c)
    n = sum(counts)
    pages = sum(-(-r // c["page"]) for r in rows) * 4
    if c["op"] in ("append", "read"):
        b = n * c["kv"] * (2 * c["d"] * size + _row_bytes(c)) + pages + (n * c["kv"] * 8 if c["op"] == "append" and c["track"] else 0)
        if c["op"] == "append":  # the appended rows come back through a read in bf16
            b += n * c["kv"] * (2 * c["d"] * 2 + _row_bytes(c))
        return {"bytes": b, "flops": 8 * n * c["kv"] * 2 * c["d"]}
    if c["op"] == "evict":
        b, f = pages, 0
        for r in rows:
            kept = min(r, c["keep"])
            b += c["layers"] * c["kv"] * (8 * r + kept * 2 * (_row_bytes(c) + 8))
            f += c["layers"] * c["kv"] * 8 * r
        return {"bytes": b, "flops": f}
    b, pairs = pages + 2 * n * c["heads"] * c["d"] * size, 0
    for r, k in zip(rows, counts):
        if k == 0:
            continue
        read = r if c["track"] or not c["window"] else min(r, c["window"] + k - 1)
        b += read * c["kv"] * (_row_bytes(c) + (4 if c["track"] and (c["bias"] or c["window"]) else 0) + (8 if c["accumulate"] else 0))
        pairs += sum(_visible(c, r, k, i) for i in range(k))
    return {"bytes": b, "flops": 4 * c["d"] * c["heads"] * pairs + (2 * c["d"] * c["heads"] * pairs if c["accumulate"] else 0)}


# ------------------------------------------------------------------ the pool in elementary torch operations
def _quantize(x):
    """x fp32 [..., d] -> codes uint8 [..., d / 2], parameters fp16 [..., d / 64, 2]."""
    g = x.clamp(-65504.0, 65504.0).unflatten(-1, (-1, 64))
    lo32, hi32 = g.amin(-1), g.amax(-1)
    lo, scale = lo32.half(), ((hi32 - lo32) / 15.0).half()
    sf = scale.float()[..., None]
    code = torch.where(sf > 0, (g - lo.float()[..., None]) / sf, 0.0).round().clamp(0, 15).nan_to_num(0.0).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.stack([scale, lo], -1)


def _dequantize(codes, params):
    """codes uint8 [..., d / 2], parameters fp16 [..., d / 64, 2] -> fp32 [..., d]."""
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (-1, 64))
    p = params.float()
    return (p[..., 1:2] + p[..., 0:1] * code).flatten(-2)


def _fields(c):
    """(first byte, bytes of a row) of a block's fields: K codes, K parameters, V codes, V parameters, positions, weights."""
    code, par, at, f = c["d"] // 2, c["d"] // 64 * 4, 0, []
    for n in (code, par, code, par) + ((4, 4) if c["track"] else ()):
        f.append((at, n))
        at += n * BLOCK_ROWS
    return f


def _field(c, blocks, k):
    """Field k of blocks [..., block bytes] as bytes [..., 32, bytes of a row] (a view)."""
    at, n = _fields(c)[k]
    return blocks[..., at:at + n * BLOCK_ROWS].unflatten(-1, (BLOCK_ROWS, n))


def _gather(c, pool, layer, tables):
    """The blocks of sequences [S, KV heads, blocks, block bytes] (a copy)."""
    x = pool[tables.long(), layer]  # [S, pages, kv, page / 32, bytes]
    return x.transpose(1, 2).flatten(2, 3)


def _values(c, blocks, k):
    """K (k = 0) or V (k = 2) rows [S, kv, rows, d] in fp32."""
    codes = _field(c, blocks, k).flatten(2, 3)
    params = _field(c, blocks, k + 1).contiguous().view(torch.float16).flatten(2, 3).unflatten(-1, (-1, 2))
    return _dequantize(codes, params)


def _token_rows(c, st):
    """Of each new token its sequence, and the row that it has in the cache."""
    counts = st["offsets"].long().diff()
    seq = torch.repeat_interleave(torch.arange(c["seqs"], device=counts.device), counts, output_size=st["n"])
    i = torch.arange(st["n"], device=counts.device) - st["offsets"].long()[seq]
    return seq, st["rows"].long()[seq] - counts[seq] + i, i


def _store(c, pool, layer, tables, seq, row, field, x):
    """Bytes x [n, kv, bytes] become field `field` of rows `row` of sequences `seq`."""
    page = tables.long()[seq, row // c["page"]]
    view = _field(c, pool, field)  # [pages, layers, kv, page / 32, 32, bytes]
    view[page, layer, :, row % c["page"] // BLOCK_ROWS, row % BLOCK_ROWS] = x


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rows, counts = _lengths(c)
    per = -(-max(rows) // c["page"])
    keep_pages = -(-c["keep"] // c["page"]) if c["op"] == "evict" else 0
    need = [-(-r // c["page"]) for r in rows]
    total = sum(need) + c["seqs"] * keep_pages
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    slot = torch.zeros(c["seqs"], per, dtype=torch.long)
    at = 0
    for s, k in enumerate(need):
        slot[s, :k] = torch.arange(at, at + k)
        at += k
    tables = order[slot.to(dev)]  # entries past a sequence's last page name a page that is not read
    st = {"case": c, "tables": tables.contiguous(), "rows": torch.tensor(rows, dtype=torch.int32, device=dev),
          "offsets": torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device=dev), "n": sum(counts),
          "max_rows": max(rows), "max_count": max(counts)}
    # the cache: K with offsets and sizes that differ by channel, V nearly normal, in the rows' own scales
    pool = torch.zeros(total, c["layers"], c["kv"], c["page"] // BLOCK_ROWS, _block_bytes(c), dtype=torch.uint8, device=dev)
    st["layer"] = c["layers"] - 1
    shift = torch.randn(2, c["kv"], 1, 1, c["d"], generator=g, device=dev) * torch.tensor([1.0, 0.1], device=dev).view(2, 1, 1, 1, 1)
    for layer in range(c["layers"]) if c["op"] == "evict" else [st["layer"]]:
        for a in range(0, total, 2048):  # pages by parts: the fp32 values are eight times the pool
            part = pool[a:a + 2048, layer]
            for k in (0, 1):
                x = torch.randn(part.shape[0], c["kv"], c["page"] // BLOCK_ROWS, BLOCK_ROWS, c["d"], generator=g, device=dev) + shift[k]
                codes, params = _quantize(x)
                _field(c, part, 2 * k).copy_(codes)
                _field(c, part, 2 * k + 1).copy_(params.flatten(-2).contiguous().view(torch.uint8))
            if c["track"]:
                # weights as attention leaves them: a few rows have most
                w = torch.rand(part.shape[:-1] + (BLOCK_ROWS,), generator=g, device=dev).pow(8) * 20
                _field(c, part, 5).copy_(w[..., None].contiguous().view(torch.uint8))
    if c["track"]:
        # a tracked cache has been cut before: its rows' positions have gaps, the new tokens follow on
        pos = torch.arange(per * c["page"], device=dev, dtype=torch.int32) * 2
        last = st["rows"] - st["offsets"].diff()
        st["positions"] = 2 * last
        seq = torch.arange(c["seqs"], device=dev)[:, None].expand(-1, per * c["page"])
        row = torch.arange(per * c["page"], device=dev)[None].expand(c["seqs"], -1)
        new = row - last[:, None]
        p = torch.where(new >= 0, 2 * last[:, None] + new, pos[None]).to(torch.int32)
        ok = row < st["rows"][:, None]
        for layer in range(c["layers"]) if c["op"] == "evict" else [st["layer"]]:
            _store(c, pool, layer, st["tables"], seq[ok], row[ok], 4, p[ok][:, None, None].expand(-1, c["kv"], 1).contiguous().view(torch.uint8))
        st["next"] = (2 * last + st["offsets"].diff()).to(torch.int32)
        st["weights"] = _field(c, pool, 5).view(torch.float32)[..., 0]
    st["pool"] = pool
    dt = getattr(torch, c["dtype"])
    if c["op"] == "append":
        st["k"] = (torch.randn(st["n"], c["kv"], c["d"], generator=g, device=dev) + shift[0, :, 0, 0]).to(dt)
        st["v"] = (torch.randn(st["n"], c["kv"], c["d"], generator=g, device=dev) + shift[1, :, 0, 0]).to(dt)
    if c["op"] == "attention":
        st["q"] = (torch.randn(st["n"], c["heads"], c["d"], generator=g, device=dev) * 1.5).to(dt)
        if c["bias"]:
            st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / c["heads"]) for h in range(c["heads"])], device=dev)
    if c["op"] == "evict":
        st["out_tables"] = order[sum(need) + torch.arange(c["seqs"] * keep_pages, device=dev)].view(c["seqs"], keep_pages).contiguous()
    if own:
        from persistent_decode_megakernel_gb300.kv4 import Kv4Cache
        st["cache"] = Kv4Cache(n_layers=c["layers"], n_heads=c["heads"], n_kv_heads=c["kv"], head_dim=c["d"], num_pages=total, page_size=c["page"],
                               max_pages=per, track=c["track"], pool=pool)
        st["batch"] = st["cache"].batch(st["offsets"], st["rows"], st["tables"], positions=st.get("positions"), n_tokens=st["n"],
                                        max_count=st["max_count"], max_rows=st["max_rows"])
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    c = st["case"]
    if own:
        return _own(c, st)
    if c["op"] == "append":
        _plain_append(c, st)
        return _plain_read(c, st, torch.bfloat16)
    if c["op"] == "read":
        return _plain_read(c, st, getattr(torch, c["dtype"]))
    if c["op"] == "attention":
        return _plain_attention(c, st)
    return _plain_evict(c, st)


def _own(c, st):
    cache, b = st["cache"], st["batch"]
    if c["op"] == "append":
        cache.append(st["layer"], b, st["k"], st["v"])
        k, v = cache.read(st["layer"], b, torch.bfloat16)
        return {"k": k, "v": v}
    if c["op"] == "read":
        k, v = cache.read(st["layer"], b, getattr(torch, c["dtype"]))
        return {"k": k, "v": v}
    if c["op"] == "attention":
        out = cache.attention(st["layer"], b, st["q"], cap=c["cap"], slopes=st.get("slopes"), window=c["window"], accumulate=c["accumulate"])
        return {"out": out, "weights": st["weights"][:, st["layer"]]} if c["accumulate"] else {"out": out}
    rows = cache.evict(st["rows"], st["tables"], st["next"], c["keep"], recent=c["recent"], out_tables=st["out_tables"], max_rows=st["max_rows"])
    return {"rows": rows, "weights": st["weights"], "pool": st["pool"]}


def _plain_append(c, st):
    seq, row, i = _token_rows(c, st)
    for k, x in ((0, st["k"]), (2, st["v"])):
        codes, params = _quantize(x.float())
        _store(c, st["pool"], st["layer"], st["tables"], seq, row, k, codes)
        _store(c, st["pool"], st["layer"], st["tables"], seq, row, k + 1, params.flatten(-2).contiguous().view(torch.uint8))
    if c["track"]:
        pos = (st["positions"].long()[seq] + i).to(torch.int32)[:, None, None].expand(-1, c["kv"], 1).contiguous()
        _store(c, st["pool"], st["layer"], st["tables"], seq, row, 4, pos.view(torch.uint8))
        _store(c, st["pool"], st["layer"], st["tables"], seq, row, 5, torch.zeros_like(pos).view(torch.uint8))


def _plain_read(c, st, dtype):
    seq, row, _ = _token_rows(c, st)
    page = st["tables"].long()[seq, row // c["page"]]
    out = []
    for k in (0, 2):
        at = (page, st["layer"], slice(None), row % c["page"] // BLOCK_ROWS, row % BLOCK_ROWS)
        params = _field(c, st["pool"], k + 1)[at].contiguous().view(torch.float16).unflatten(-1, (-1, 2))
        out.append(_dequantize(_field(c, st["pool"], k)[at], params).to(dtype))
    return {"k": out[0], "v": out[1]}


def _plain_attention(c, st):
    dev, S, R, C, G = st["q"].device, c["seqs"], st["max_rows"], st["max_count"], c["heads"] // c["kv"]
    blocks = _gather(c, st["pool"], st["layer"], st["tables"])
    k = _values(c, blocks, 0)[:, :, :R]
    counts = st["offsets"].long().diff()
    i = torch.arange(C, device=dev)
    at = (st["offsets"].long()[:-1, None] + i).clamp(max=st["n"] - 1)  # [S, C]
    real = i < counts[:, None]
    q = st["q"].float()[at].unflatten(2, (c["kv"], G)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [S, kv, G * C, d]
    s = ((q @ k.transpose(-1, -2)) * c["d"] ** -0.5).unflatten(2, (G, C))  # [S, kv, G, C, R]
    del k
    if c["cap"]:
        s = c["cap"] * torch.tanh(s / c["cap"])
    row = torch.arange(R, device=dev)
    last = st["rows"].long()[:, None] - counts[:, None] + i  # [S, C]: the query's own row
    see = real[..., None] & (row <= last[..., None])  # [S, C, R]
    if c["track"]:
        kpos = _field(c, blocks, 4).contiguous().view(torch.int32).flatten(2, 4)[:, :, :R].long()  # [S, kv, R]
        qpos = st["positions"].long()[:, None] + i
    else:
        kpos, qpos = row.expand(S, 1, R), last
    gap = kpos[:, :, None, :] - qpos[:, None, :, None]  # [S, kv or 1, C, R]
    if c["bias"]:
        s = s + st["slopes"].view(1, c["kv"], G, 1, 1) * gap[:, :, None]
    see = see[:, None] & (gap > -c["window"]) if c["window"] else see[:, None].expand_as(gap)
    s = s.masked_fill(~see[:, :, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    del s
    o = (p.flatten(2, 3) @ _values(c, blocks, 2)[:, :, :R].masked_fill((row >= st["rows"][:, None])[:, None, :, None], 0.0)).unflatten(2, (G, C))
    out = torch.zeros_like(st["q"])
    keep = real.flatten()
    out[at.flatten()[keep]] = o.permute(0, 3, 1, 2, 4).flatten(2, 3).flatten(0, 1)[keep].to(out.dtype)
    if not c["accumulate"]:
        return {"out": out}
    seq, r = (x.flatten() for x in torch.broadcast_tensors(torch.arange(S, device=dev)[:, None], row[None]))
    ok = (r < st["rows"][seq]) & (counts[seq] > 0)
    seq, r = seq[ok], r[ok]
    page, w = st["tables"].long()[seq, r // c["page"]], st["weights"]
    w[page, st["layer"], :, r % c["page"] // BLOCK_ROWS, r % BLOCK_ROWS] += p.sum((2, 3)).transpose(1, 2)[seq, r]
    return {"out": out, "weights": w[:, st["layer"]]}


def _plain_evict(c, st):
    pool, keep, page = st["pool"], c["keep"], c["page"]
    S, R, L = c["seqs"], st["max_rows"], c["layers"]
    x = pool[st["tables"].long()].permute(0, 2, 3, 1, 4, 5).flatten(3, 4)  # [S, L, kv, blocks, bytes]
    field = [_field(c, x, k).flatten(3, 4) for k in range(6)]  # [S, L, kv, rows, bytes]
    w = field[5].contiguous().view(torch.float32)[..., :R, 0]
    pos = field[4].contiguous().view(torch.int32)[..., :R, 0]
    row = torch.arange(R, device=pool.device)
    held = st["rows"].long().view(S, 1, 1, 1)
    key = torch.where(pos >= (st["next"].view(S, 1, 1, 1) - c["recent"]), math.inf, w.nan_to_num(0.0, posinf=math.inf))
    key = torch.where(row < held, key, -math.inf)
    rank = key.sort(dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(key, dtype=torch.bool).scatter_(-1, rank[..., :keep], True) & (row < held)
    low, high = kept[..., :keep], kept[..., keep:]
    holes = low.to(torch.uint8).sort(dim=-1, stable=True).indices  # free rows first, ascending
    movers = (~high).to(torch.uint8).sort(dim=-1, stable=True).indices + keep  # kept rows above first, ascending
    m = min(holes.shape[-1], movers.shape[-1])
    n = high.sum(-1, keepdim=True)
    src = torch.arange(min(keep, R), device=pool.device).expand(low.shape).clone()
    j = torch.arange(m, device=pool.device)
    src.scatter_(-1, holes[..., :m], torch.where(j < n, movers[..., :m], holes[..., :m]))
    new = torch.minimum(st["rows"], torch.tensor(keep, device=pool.device, dtype=torch.int32))
    seq, r = (t.flatten() for t in torch.broadcast_tensors(torch.arange(S, device=pool.device)[:, None], torch.arange(src.shape[-1], device=pool.device)[None]))
    ok = r < new[seq]
    seq, r = seq[ok], r[ok]
    to = st["out_tables"].long()[seq, r // page]
    for k in range(6):
        moved = field[k].gather(3, src[..., None].expand(-1, -1, -1, -1, field[k].shape[-1]))  # [S, L, kv, keep, bytes]
        _field(c, pool, k)[to, :, :, r % page // BLOCK_ROWS, r % BLOCK_ROWS] = moved.permute(0, 3, 1, 2, 4)[seq, r]
    return {"rows": new, "weights": st["weights"], "pool": pool}


# ------------------------------------------------------------------ the definition in 64 bits, sequence by sequence
def _row_of(c, st, s, r0, r1, layer, k):
    """Values of rows r0 .. r1 - 1 of sequence s in 64 bits, [kv, rows, d], k = 0 for K and 1 for V, from the block's layout."""
    r = torch.arange(r0, r1, device=st["pool"].device)
    blocks = st["pool"][st["tables"][s].long()[r // c["page"]], layer, :, r % c["page"] // 32]  # [rows, kv, bytes]
    half, par = 16 * c["d"], 32 * (c["d"] // 64) * 4
    base, lane = k * (half + par), (r % 32)[:, None, None]
    byte = blocks.gather(2, (base + lane * (c["d"] // 2) + torch.arange(c["d"] // 2, device=r.device)).expand(-1, c["kv"], -1)).long()
    code = torch.empty(len(r), c["kv"], c["d"], dtype=torch.float64, device=r.device)
    code[..., 0::2], code[..., 1::2] = (byte % 16).double(), (byte // 16).double()
    n = c["d"] // 64
    pb = blocks.gather(2, (base + half + lane * (4 * n) + torch.arange(4 * n, device=r.device)).expand(-1, c["kv"], -1)).contiguous()
    p = pb.view(torch.float16).double().view(len(r), c["kv"], n, 2).repeat_interleave(64, dim=2)
    return (p[..., 1] + p[..., 0] * code).transpose(0, 1)


def _evicted_weights(c, st, rows):
    """The weights after the eviction, segment by segment."""
    w = st["weights"].double()
    every = _field(c, st["pool"], 4).view(torch.int32)[..., 0]
    for s, r in enumerate(rows):
        mine = torch.arange(r, device=w.device)
        at = (st["tables"][s].long()[mine // c["page"]], slice(None), slice(None), mine % c["page"] // 32, mine % 32)
        new = mine[:c["keep"]]
        to = (st["out_tables"][s].long()[new // c["page"]], new % c["page"] // 32, new % 32)
        held, young = w[at], every[at] >= int(st["next"][s]) - c["recent"]  # [r, L, kv]
        for layer in range(c["layers"]):
            for h in range(c["kv"]):
                x = held[:, layer, h]
                first = torch.argsort(x + 1e9 * young[:, layer, h], descending=True, stable=True) if r > c["keep"] else mine
                stay = torch.zeros(r, dtype=torch.bool, device=w.device)
                stay[first[young[:, layer, h][first]][:c["keep"]]] = True  # the recent rows, whatever their weight
                old = first[~young[:, layer, h][first]]
                stay[old[:max(0, c["keep"] - int(stay.sum()))]] = True
                src = new.clone()
                src[~stay[:len(new)]] = mine[len(new):][stay[len(new):]]
                w[to[0], layer, h, to[1], to[2]] = x[src]
    return w


def exact(case, seed):
    c = dict(case)
    st = prepare(case, seed)
    rows, counts = _lengths(c)
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    if c["op"] == "append":
        out = {}
        for name in ("k", "v"):
            x = st[name].double().view(-1, c["kv"], c["d"] // 64, 64)
            lo = x.amin(-1, keepdim=True)
            scale = ((x.amax(-1, keepdim=True) - lo) / 15).half().double()
            lo = lo.half().double()
            code = torch.where(scale > 0, torch.round((x - lo) / scale), 0.0).clamp(0, 15)
            out[name] = (lo + scale * code).view(-1, c["kv"], c["d"])
        return out
    if c["op"] == "read":
        parts = [[_row_of(c, st, s, r - n, r, st["layer"], k).transpose(0, 1) for s, (r, n) in enumerate(zip(rows, counts))] for k in (0, 1)]
        return {"k": torch.cat(parts[0]), "v": torch.cat(parts[1])}
    if c["op"] == "evict":
        return {"rows": None, "weights": _evicted_weights(c, st, rows), "pool": None}  # bytes are moved, none is computed
    G = c["heads"] // c["kv"]
    out = torch.zeros(st["n"], c["heads"], c["d"], dtype=torch.float64, device=st["pool"].device)
    w = st["weights"].double() if c["accumulate"] else None
    for s, (r, n) in enumerate(zip(rows, counts)):
        if n == 0:
            continue
        k, v = (_row_of(c, st, s, 0, r, st["layer"], j) for j in (0, 1))  # [kv, r, d]
        mine = torch.arange(r, device=k.device)
        pages, blk, lane = st["tables"][s].long()[mine // c["page"]], mine % c["page"] // 32, mine % 32
        if c["track"]:
            raw = _field(c, st["pool"], 4).view(torch.int32)[..., 0]
            kpos = raw[pages, st["layer"], :, blk, lane].double().t()  # [kv, r]
            first = float(st["positions"][s])
        else:
            kpos, first = mine.double().expand(c["kv"], r), float(r - n)
        for a in range(0, n, 256):
            b = min(n, a + 256)
            i = torch.arange(a, b, device=k.device)
            gap = kpos[:, None, :] - (first + i.double())[None, :, None]  # [kv, b - a, r]
            see = (mine[None, None, :] <= (r - n + i)[None, :, None]).expand_as(gap)
            if c["window"]:
                see = see & (-gap < c["window"])
            for h in range(c["heads"]):
                x = st["q"][at[s] + a:at[s] + b, h].double() @ k[h // G].t() / math.sqrt(c["d"])
                if c["cap"]:
                    x = c["cap"] * torch.tanh(x / c["cap"])
                if c["bias"]:
                    x = x + st["slopes"][h].double() * gap[h // G]
                x = x.masked_fill(~see[h // G], -math.inf)
                p = torch.softmax(x, -1).nan_to_num(0.0)
                out[at[s] + a:at[s] + b, h] = p @ v[h // G]
                if w is not None:
                    w[pages, st["layer"], h // G, blk, lane] += p.sum(0)
    return {"out": out, "weights": w[:, st["layer"]]} if w is not None else {"out": out}
