"""The measured cases of two more groups of operators of the paged-KV attention
step.  A cache of 4-bit codes: its write (and the read back), and attention over
it for decodes and prompts.  Attention over the pages that a score selects: the
bounds of each page's keys, the selection, and attention over the selected pages.

``own = False`` computes them with elementary torch operations in 32 bits (the
selection's scores in 64); ``own = True`` makes the library's calls.  ``exact``
computes the same from the definition in 64 bits."""
import math

import torch

own = False

D = 128      # head size
BS = 16      # tokens of a cache page
CODES = 2 * BS * (D // 2)      # bytes of a page's codes of one KV head: keys, then values
PAGE4 = CODES + 2 * BS * 4     # and a (scale, zero) pair of bf16 for each row
TINY = 2.0 ** -36              # a row whose spread is below this has scale 0
TOP = 2.0 ** 126               # values are clamped to +-TOP


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _named(name, c):
    return dict(c, name=name) if name else c


def _write(name, tokens, hkv, pad=0, std=1.0):
    return _named(name, {"op": "write", "tokens": tokens, "pad": pad, "hkv": hkv, "std": std})


def _batch(op, hq, hkv, decodes=0, dec_lo=0, dec_hi=0, dec_q=1, chunks=0, chunk_q=0, chunk_step=0,
           chunk_ctx=0, pad=0):
    return {"op": op, "hq": hq, "hkv": hkv, "decodes": decodes, "dec_lo": dec_lo,
            "dec_hi": dec_hi, "dec_q": dec_q, "chunks": chunks, "chunk_q": chunk_q,
            "chunk_step": chunk_step, "chunk_ctx": chunk_ctx, "pad": pad}


def _attention(name, hq, hkv, **kw):
    return _named(name, _batch("attention", hq, hkv, **kw))


def _bounds(name, hkv, **kw):
    return _named(name, _batch("bounds", hkv, hkv, **kw))


def _select(name, hq, hkv, budget, first=0, last=1, **kw):
    return _named(name, dict(_batch("select", hq, hkv, **kw), budget=budget, first=first,
                             last=last))


def _selected(name, hq, hkv, rows, budget, lo, pad=0):
    return _named(name, {"op": "selected", "hq": hq, "hkv": hkv, "rows": rows, "budget": budget,
                         "lo": lo, "pad": pad})


def listed():
    return [
        # a step of 64 decodes writes its tokens, padded to a capture size
        _write("int4_write_step", 64, 8, pad=3),
        # a prompt of an odd length, every head with its own K and V
        _write("int4_write_prompt", 8191, 32),
        # a mixed step of two decodes and a short prompt
        _attention("int4_trace_step", 32, 8, decodes=2, dec_lo=129, dec_hi=540, chunks=1,
                   chunk_q=298, pad=4),
        # a batch of long decodes
        _attention("int4_gqa_decode", 32, 8, decodes=128, dec_lo=8192, dec_hi=8192),
        # few very long sequences that share one KV head
        _attention("int4_mqa_decode", 32, 1, decodes=32, dec_lo=32768, dec_hi=32768),
        # long prompts in chunks: one that continues, one that starts, odd lengths
        _attention("int4_chunks", 64, 8, chunks=4, chunk_q=2047, chunk_step=37, chunk_ctx=4099),
        # the page bounds after a step of decodes
        _bounds("bounds_step", 8, decodes=128, dec_lo=1024, dec_hi=8192),
        # the page bounds after a large prefill
        _bounds("bounds_prefill", 8, chunks=8, chunk_q=2047, chunk_step=3, chunk_ctx=500),
        # one sequence generating far into its context: 64 of its 2050 pages
        _select("select_one", 32, 8, 64, first=1, last=2, decodes=1, dec_lo=32791, dec_hi=32791),
        # a batch of long decodes: 64 of 513 pages
        _select("select_batch", 32, 8, 64, decodes=128, dec_lo=8192, dec_hi=8192),
        # the attention of one sequence's row over its selected pages
        _selected("selected_one", 32, 8, 1, 64, 64),
        # the attention of a batch, some rows with fewer pages
        _selected("selected_batch", 32, 8, 128, 128, 97, pad=3),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    hq, hkv = rng.choice([(32, 8), (32, 32), (64, 8), (8, 8), (32, 1), (16, 2), (24, 8), (12, 4)])
    op = rng.choice(["write", "attention", "attention", "attention", "bounds", "select", "select",
                     "selected"])
    pad = rng.choice([0, 0, 3])
    if op == "write":
        return _write(None, _log(rng, 1, 8000), hkv, pad, rng.choice([1.0, 0.02, 30.0]))
    if op == "bounds":
        if rng.random() < 0.5:
            hi = _log(rng, 16, 8192)
            return _bounds(None, hkv, decodes=_log(rng, 1, 200), dec_lo=_log(rng, 1, hi), dec_hi=hi,
                           dec_q=rng.choice([1, 1, 2, 5]), pad=pad)
        q = _log(rng, 17, 2048)
        return _bounds(None, hkv, chunks=rng.randint(1, 4), chunk_q=q, chunk_step=rng.randint(0, q // 8),
                       chunk_ctx=_log(rng, 1, 1024), pad=pad)
    if op == "select":
        hi = _log(rng, 64, 16384)
        return _select(None, hq, hkv, _log(rng, 4, 256), rng.choice([0, 1]), rng.choice([1, 2]),
                       decodes=_log(rng, 1, 64), dec_lo=_log(rng, 16, hi), dec_hi=hi,
                       dec_q=rng.choice([1, 1, 2, 3]), pad=pad)
    if op == "selected":
        budget = _log(rng, 4, 256)
        rows = _log(rng, 1, min(96, 1800000 // (hkv * budget * BS)))
        return _selected(None, hq, hkv, rows, budget, _log(rng, 1, budget), pad)
    kind = rng.choice(["decode", "decode", "prompt", "mixed"])
    if kind == "decode":
        hi = _log(rng, 16, 8192)
        dq = rng.choice([1, 1, 2, 3]) if hq // hkv <= 4 else 1
        n = _log(rng, 1, min(96, 8000000 // (hkv * hi)))
        return _attention(None, hq, hkv, decodes=n, dec_lo=_log(rng, 1, hi), dec_hi=hi, dec_q=dq,
                          pad=pad)
    if kind == "prompt":
        q = _log(rng, 17, 2048)
        return _attention(None, hq, hkv, chunks=rng.randint(1, 4), chunk_q=q,
                          chunk_step=rng.randint(0, q // 8),
                          chunk_ctx=rng.choice([0, _log(rng, 1, 4096)]), pad=pad)
    hi, q = _log(rng, 16, 2048), _log(rng, 17, 512)
    return _attention(None, hq, hkv, decodes=_log(rng, 1, 48), dec_lo=_log(rng, 1, hi), dec_hi=hi,
                      chunks=rng.randint(1, 2), chunk_q=q, chunk_step=rng.randint(0, q // 4),
                      chunk_ctx=rng.choice([0, _log(rng, 1, 1024)]), pad=pad)


def _requests(c):
    """(cached tokens, scheduled tokens) of every request, from the case alone:
    decodes with lengths spread over their range in a mixed order, then chunks,
    every other one continuing a cached prompt."""
    reqs = []
    n = c["decodes"]
    step = next(s for s in (7, 11, 13, 17, 1) if math.gcd(s, max(n, 1)) == 1)
    for i in range(n):
        j = (i * step) % n
        reqs.append((c["dec_lo"] + ((c["dec_hi"] - c["dec_lo"]) * j // (n - 1) if n > 1 else 0),
                     c["dec_q"]))
    for i in range(c["chunks"]):
        reqs.append((c["chunk_ctx"] if i % 2 == 0 else 0,
                     max(1, c["chunk_q"] - i * c["chunk_step"])))
    return reqs


def _counts(c):
    """Pages listed for every row of a "selected" case: from lo to budget."""
    n, span = c["rows"], c["budget"] - c["lo"]
    return [c["lo"] + (span * ((7 * i) % n) // (n - 1) if n > 1 else 0) for i in range(n)]


def work(case):
    c = case
    if c["op"] == "write":  # written, and read back into bf16 rows
        n, pool = c["tokens"], _pool_blocks(c["tokens"]) * BS
        b = n * (c["hkv"] * (4 * D + PAGE4 // BS) + 8) + pool * (c["hkv"] * (4 * D + PAGE4 // BS) + 8)
        return {"bytes": b, "flops": 2 * D * c["hkv"] * (4 * n + 2 * pool)}
    if c["op"] == "selected":
        keys = sum(16 * n - 8 for n in _counts(c))
        return {"bytes": c["hkv"] * keys * 4 * D + c["rows"] * (4 * c["hq"] * D + 4) +
                4 * c["hkv"] * sum(_counts(c)),
                "flops": 4 * D * keys * c["hq"]}
    reqs = _requests(c)
    rows = sum(n for _, n in reqs)
    if c["op"] == "bounds":
        pages = sum((x + n - 1) // BS - x // BS + 1 for x, n in reqs)
        keys = sum(x + n - x // BS * BS for x, n in reqs)
        return {"bytes": c["hkv"] * (keys * 2 * D + pages * 4 * D) + 8 * rows,
                "flops": 2 * D * c["hkv"] * keys}
    if c["op"] == "select":
        scored = listed_pages = 0
        for x, n in reqs:
            for p in range(x, x + n):
                k = p // BS + 1
                scored += k if k > c["budget"] else 0
                listed_pages += min(k, c["budget"])
        # (the rows of one request share the bounds that they read)
        read = sum((x + n - 1) // BS + 1 for x, n in reqs if (x + n - 1) // BS + 1 > c["budget"])
        return {"bytes": c["hkv"] * (read * 4 * D + 4 * listed_pages) + rows * c["hq"] * D * 2,
                "flops": 4 * D * c["hkv"] * scored}
    pairs = sum(n * x + n * (n + 1) // 2 for x, n in reqs)
    keys = sum(x + n for x, n in reqs)
    return {"bytes": 2 * rows * c["hq"] * D * 2 + keys * c["hkv"] * (PAGE4 // BS),
            "flops": 4 * D * pairs * c["hq"]}


# --------------------------------------------------------------------------
# the 4-bit pages, with torch operations
# --------------------------------------------------------------------------

LOW, HIGH = [0, 4, 1, 5], [2, 6, 3, 7]   # dims of the low and high half of a word's four bytes


def _quantise(x):
    """Codes (uint8, 0..15), scale and zero (bf16) of head rows [..., D]."""
    x = torch.where(x.isnan(), torch.zeros_like(x), x).float().clamp_(-TOP, TOP)
    zero = x.amin(-1, keepdim=True)
    spread = x.amax(-1, keepdim=True) - zero
    scale = torch.where(spread < TINY, torch.zeros_like(spread), spread / 15).to(torch.bfloat16)
    f = scale.float()
    q = torch.round((x - zero) / torch.where(f == 0, torch.ones_like(f), f))
    q = torch.where(f == 0, torch.zeros_like(q), q.clamp_(0, 15))
    return q.to(torch.uint8), scale, zero.to(torch.bfloat16)


def _bytes(codes):
    """[..., D] codes as the [..., D / 2] bytes of a row."""
    w = codes.view(*codes.shape[:-1], D // 8, 8)
    return (w[..., LOW] | (w[..., HIGH] << 4)).reshape(*codes.shape[:-1], D // 2)


def _values(cache):
    """Keys and values ([..., 2, BS, D] in fp32) of pages [..., PAGE4]."""
    lead = cache.shape[:-1]
    b = cache[..., :CODES].reshape(*lead, 2, BS, D // 8, 4)
    x = torch.empty(*lead, 2, BS, D // 8, 8, device=cache.device)
    x[..., LOW] = (b & 15).float()
    x[..., HIGH] = (b >> 4).float()
    pair = cache[..., CODES:].contiguous().view(torch.bfloat16).view(*lead, 2, BS, 2).float()
    return x.view(*lead, 2, BS, D).mul_(pair[..., :1]).add_(pair[..., 1:])


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, g, std=1.0):
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, 1.0, generator=g)
    return x if std == 1.0 else x * std


def _pool_blocks(tokens):
    return -(-tokens // BS) + 3


def _cache4(blocks, hkv, g):
    """A pool of pages whose rows are quantised normal values."""
    cache = torch.empty(blocks, hkv, PAGE4, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (hkv * 2 * BS * D))
    for at in range(0, blocks, step):
        n = min(step, blocks - at)
        codes, scale, zero = _quantise(_randn((n, hkv, 2, BS, D), g))
        cache[at:at + n, :, :CODES] = _bytes(codes).view(n, hkv, CODES)
        cache[at:at + n, :, CODES:] = torch.cat([scale, zero], -1).view(torch.uint8).view(n, hkv, -1)
    return cache


def _metadata(c, g):
    reqs = _requests(c)
    ctx = torch.tensor([r[0] for r in reqs], dtype=torch.int32)
    n = torch.tensor([r[1] for r in reqs], dtype=torch.int32)
    seq = ctx + n
    used = [-(-int(x) // BS) for x in seq]
    pool = sum(used) + 5
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32).cpu()
    bt = torch.full((len(reqs), max(used)), -1, dtype=torch.int32)
    at = 0
    for r, u in enumerate(used):
        bt[r, :u] = perm[at:at + u]
        at += u
    rows = int(n.sum())
    qsl = torch.zeros(len(reqs) + 1, dtype=torch.int32)
    qsl[1:] = n.cumsum(0)
    req_of = torch.repeat_interleave(torch.arange(len(reqs)), n.long())
    off = torch.arange(rows) - qsl[:-1].long()[req_of]
    pos = ctx.long()[req_of] + off
    slots = torch.full((rows + c["pad"],), -1, dtype=torch.int64)
    slots[:rows] = bt[req_of, pos // BS].long() * BS + pos % BS
    return {"c": c, "reqs": len(reqs), "rows": rows, "pool": pool, "nmax": int(n.max()),
            "qsl": qsl.cuda(), "seq": seq.cuda(), "bt": bt.cuda(), "req_of": req_of.cuda(),
            "off": off.cuda(), "pos": pos.cuda(), "slots": slots.cuda()}


def prepare(case, seed):
    c, g = case, _gen(seed)
    hkv = c["hkv"]
    if c["op"] == "write":
        n, rows, blocks = c["tokens"], c["tokens"] + c["pad"], _pool_blocks(c["tokens"])
        kv = _randn((rows, 2 * hkv * D), g, c["std"])     # column slices of a fused projection
        slots = torch.full((rows,), -1, dtype=torch.int64, device="cuda")
        slots[:n] = torch.randperm(blocks * BS, generator=g, device="cuda")[:n]
        out = torch.zeros(2, blocks * BS, hkv, D, dtype=torch.bfloat16, device="cuda")
        return {"c": c, "n": n, "k": kv[:, :hkv * D].view(rows, hkv, D),
                "v": kv[:, hkv * D:].view(rows, hkv, D), "slots": slots,
                "cache": _cache4(blocks, hkv, g), "all": torch.arange(blocks * BS, device="cuda"),
                "k_out": out[0], "v_out": out[1]}
    if c["op"] == "selected":
        rows, counts = c["rows"], _counts(c)
        n = torch.tensor(counts, device="cuda")
        pool = sum(counts) + 5
        ids = torch.rand(hkv, pool, generator=g, device="cuda").argsort(-1)
        at = (n.cumsum(0) - n)[:, None] + torch.arange(c["budget"], device="cuda")
        table = torch.full((rows + c["pad"], hkv, c["budget"]), -1, dtype=torch.int32, device="cuda")
        table[:rows] = ids[:, at.clamp(max=pool - 1)].transpose(0, 1).int()
        unused = torch.arange(c["budget"], device="cuda")[None] >= n[:, None]
        table[:rows].masked_fill_(unused[:, None], -1)
        last = torch.randint(1, BS + 1, (rows,), generator=g, device="cuda")
        lens = torch.zeros(rows + c["pad"], dtype=torch.int32, device="cuda")
        lens[:rows] = ((n - 1) * BS + last).int()
        q = _randn((rows + c["pad"], c["hq"], D), g)
        return {"c": c, "q": q, "kc": _randn((pool, BS, hkv, D), g),
                "vc": _randn((pool, BS, hkv, D), g), "table": table, "lens": lens,
                "rows": rows, "scale": D ** -0.5, "out": torch.zeros_like(q)}
    s = _metadata(c, g)
    rows = s["rows"] + c["pad"]
    if c["op"] == "bounds":
        s["kc"] = _randn((s["pool"], BS, hkv, D), g)
        s["bounds"] = torch.zeros(s["pool"], hkv, 2, D, dtype=torch.bfloat16, device="cuda")
        return s
    s["q"] = _randn((rows, (c["hq"] + 2 * hkv) * D), g)[:, :c["hq"] * D].view(rows, c["hq"], D)
    if c["op"] == "select":
        # pages of keys that lie about a centre of their own
        lo = _randn((s["pool"], hkv, D), g)
        half = 1 + _randn((s["pool"], hkv, D), g).abs()
        s["bounds"] = torch.stack([lo - half, lo + half], 2)
        s["table"] = torch.zeros(rows, hkv, c["budget"], dtype=torch.int32, device="cuda")
        s["lens"] = torch.zeros(rows, dtype=torch.int32, device="cuda")
        return s
    s["cache"] = _cache4(s["pool"], hkv, g)
    s["scale"] = D ** -0.5
    s["out"] = torch.zeros(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    return s


# --------------------------------------------------------------------------
# plain forms (32 bits)
# --------------------------------------------------------------------------

def _plain_write(s):
    n, hkv = s["n"], s["c"]["hkv"]
    slots = s["slots"][:n]
    block, slot = slots // BS, slots % BS
    cache = s["cache"]
    codes = cache[..., :CODES].view(-1, hkv, 2, BS, D // 2)
    pairs = cache[..., CODES:].view(-1, hkv, 2, BS, 4)
    for side, x in enumerate((s["k"], s["v"])):
        q, scale, zero = _quantise(x[:n])
        codes[block, :, side, slot] = _bytes(q)
        pairs[block, :, side, slot] = torch.cat([scale, zero], -1).view(torch.uint8)
    x = _values(cache).permute(2, 0, 3, 1, 4).reshape(2, -1, hkv, D)
    s["k_out"].copy_(x[0])
    s["v_out"].copy_(x[1])


def _plain_attention(s):
    c = s["c"]
    hq, hkv, R, N = c["hq"], c["hkv"], s["reqs"], s["nmax"]
    G = hq // hkv
    bt = s["bt"].clamp(min=0).long()
    L = bt.shape[1] * BS
    kv = _values(s["cache"][bt])                                   # [R, W, hkv, 2, BS, D]
    k = kv[:, :, :, 0].permute(0, 2, 1, 3, 4).reshape(R, hkv, L, D)
    v = kv[:, :, :, 1].permute(0, 2, 1, 3, 4).reshape(R, hkv, L, D)
    q = torch.zeros(R, N, hq, D, device="cuda")
    q[s["req_of"], s["off"]] = s["q"][:s["rows"]].float()
    q = q.view(R, N, hkv, G, D).permute(0, 2, 3, 1, 4).reshape(R, hkv, G * N, D)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(R, hkv, G, N, L)
    ctx = s["seq"].long() - (s["qsl"][1:] - s["qsl"][:-1]).long()
    pos = (ctx[:, None] + torch.arange(N, device="cuda"))[:, :, None]        # [R, N, 1]
    seen = torch.arange(L, device="cuda")[None, None, :] <= pos
    x = x.masked_fill_(~seen[:, None, None], float("-inf"))
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    total = x.sum(-1, keepdim=True).view(R, hkv, G * N, 1)
    o = torch.matmul(x.view(R, hkv, G * N, L), v).div_(total)
    o = o.view(R, hkv, G, N, D).permute(0, 3, 1, 2, 4).reshape(R, N, hq, D)
    s["out"][:s["rows"]] = o[s["req_of"], s["off"]].to(torch.bfloat16)


def _plain_bounds(s):
    slots = s["slots"][:s["rows"]]
    block, last = slots // BS, slots % BS
    ends = torch.ones(s["rows"], dtype=torch.bool, device="cuda")
    ends[:-1] = block[1:] != block[:-1]          # the last token of its page in this step
    block, last = block[ends], last[ends]
    k = s["kc"][block].float()                    # [pages, BS, hkv, D]
    held = (torch.arange(BS, device="cuda")[None] <= last[:, None])[:, :, None, None]
    s["bounds"][block, :, 0] = torch.where(held, k, math.inf).amin(1).to(torch.bfloat16)
    s["bounds"][block, :, 1] = torch.where(held, k, -math.inf).amax(1).to(torch.bfloat16)


def _plain_select(s):
    c = s["c"]
    hkv, budget, rows, R, N = c["hkv"], c["budget"], s["rows"], s["reqs"], s["nmax"]
    bt = s["bt"].long()
    W = bt.shape[1]
    b = s["bounds"][bt.clamp(min=0)].double()                       # [R, W, hkv, 2, D]
    q = torch.zeros(R, N, c["hq"], D, dtype=torch.float64, device="cuda")
    q[s["req_of"], s["off"]] = s["q"][:rows].double()
    q = q.view(R, N, hkv, -1, D)
    up, down = q.clamp(min=0).sum(3), q.clamp(max=0).sum(3)         # [R, N, hkv, D]
    score = (torch.einsum("rnhd,rwhd->rnhw", up, b[..., 1, :]) +
             torch.einsum("rnhd,rwhd->rnhw", down, b[..., 0, :]))[s["req_of"], s["off"]]
    w = torch.arange(W, device="cuda")
    n = (s["pos"] // BS + 1)[:, None, None]
    forced = (w < c["first"]) | (w >= n - c["last"])
    score = torch.where(forced, math.inf, score).masked_fill(w >= n, -math.inf)
    order = score.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    count = n.clamp(max=budget)
    order = torch.where(torch.arange(order.shape[-1], device="cuda") < count, order, W)
    order = order.sort(-1).values                                   # [rows, hkv, <= budget]
    ids = torch.cat([bt, bt.new_full((R, 1), -1)], 1)[s["req_of"]]
    ids = ids.gather(1, order.flatten(1)).view(order.shape).int()
    s["table"][:rows, :, :ids.shape[-1]] = ids
    s["table"][:rows, :, ids.shape[-1]:] = -1
    s["lens"][:rows] = ((count[:, 0, 0] - 1) * BS + s["pos"] % BS + 1).int()


def _plain_selected(s):
    c, rows = s["c"], s["rows"]
    hq, hkv = c["hq"], c["hkv"]
    table = s["table"][:rows].clamp(min=0).long()                   # [rows, hkv, budget]
    head = torch.arange(hkv, device="cuda")[None, :, None]
    k = s["kc"][table, :, head].float().reshape(rows, hkv, -1, D)    # [rows, hkv, keys, D]
    v = s["vc"][table, :, head].float().reshape(rows, hkv, -1, D)
    q = s["q"][:rows].float().view(rows, hkv, hq // hkv, D)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"])
    seen = torch.arange(x.shape[-1], device="cuda") < s["lens"][:rows, None].long()
    x = x.masked_fill_(~seen[:, None, None], float("-inf"))
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(x, v).div_(x.sum(-1, keepdim=True))
    s["out"][:rows] = o.reshape(rows, hq, D).to(torch.bfloat16)


def run(state):
    s = state
    c = s["c"]
    op = c["op"]
    if own:
        import paged_kv_attention_05_gb300 as pkv
    if op == "write":
        if own:
            pkv.pkv_write_int4(s["k"], s["v"], s["cache"], s["slots"])
            pkv.pkv_read_int4(s["cache"], s["all"], s["k_out"], s["v_out"])
        else:
            _plain_write(s)
        return {"k": s["k_out"], "v": s["v_out"]}
    if op == "attention":
        if own:
            pkv.pkv_attention_int4(s["q"], s["cache"], s["qsl"], s["seq"], s["bt"], s["reqs"],
                                   s["scale"], s["out"])
        else:
            _plain_attention(s)
        return s["out"]
    if op == "bounds":
        if own:
            pkv.pkv_page_bounds(s["kc"], s["bounds"], s["slots"])
        else:
            _plain_bounds(s)
        return s["bounds"]
    if op == "select":
        if own:
            pkv.pkv_select_pages(s["q"], s["bounds"], s["qsl"], s["seq"], s["bt"], s["reqs"],
                                 s["table"], s["lens"], first_pages=c["first"],
                                 last_pages=c["last"])
        else:
            _plain_select(s)
        return {"table": s["table"], "lens": s["lens"]}
    if own:
        pkv.pkv_attention_selected(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["scale"],
                                   s["out"])
    else:
        _plain_selected(s)
    return s["out"]


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_page(page, side):
    """[..., BS, D] values of pages [..., PAGE4], nibble by nibble."""
    rows = page[..., side * (CODES // 2):(side + 1) * (CODES // 2)]
    word = rows.reshape(*page.shape[:-1], BS, D // 8, 4).long()
    word = (word * torch.tensor([1, 1 << 8, 1 << 16, 1 << 24], device=page.device)).sum(-1)
    d = torch.arange(8, device=page.device)
    code = (word[..., None] >> (4 * (d // 2) + 16 * (d % 2))) & 15
    pair = page[..., CODES + side * 64:CODES + (side + 1) * 64].contiguous().view(torch.bfloat16)
    pair = pair.reshape(*page.shape[:-1], BS, 2).double()
    return code.reshape(*page.shape[:-1], BS, D).double() * pair[..., :1] + pair[..., 1:]


def _exact_softmax(q, k, v, scale, seen):
    x = (q @ k.T) * scale
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    return torch.exp(x - torch.logsumexp(x, -1, keepdim=True)) @ v


def exact(case, seed):
    c, s = case, prepare(case, seed)
    op, hkv = c["op"], c["hkv"]
    if op == "write":
        out = {}
        at = s["slots"][:s["n"]]
        for side, name in enumerate(("k", "v")):
            x = s[name][:s["n"]].double().clamp(-TOP, TOP)
            low = x.min(-1, keepdim=True).values
            spread = x.max(-1, keepdim=True).values - low
            step = (spread / 15).to(torch.bfloat16).double()
            code = torch.round((x - low) / step).clamp(0, 15)
            full = _exact_page(s["cache"], side).permute(0, 2, 1, 3).reshape(-1, hkv, D)
            full[at] = low + code * step
            out[name] = full
        return out
    if op == "bounds":
        out = s["bounds"].double()
        for r, (x, n) in enumerate(_requests(c)):
            for j in range(x // BS, (x + n - 1) // BS + 1):
                b = int(s["bt"][r, j])
                k = s["kc"][b, :min(BS, x + n - j * BS)].double()
                out[b, :, 0], out[b, :, 1] = k.min(0).values, k.max(0).values
        return out
    if op == "select":
        table, lens, at = s["table"].clone(), s["lens"].clone(), 0
        G = c["hq"] // hkv
        for r, (x, n) in enumerate(_requests(c)):
            for p in range(x, x + n):
                k = p // BS + 1
                pages = s["bt"][r, :k].long()
                b = s["bounds"][pages].double()                    # [k, hkv, 2, D]
                q = s["q"][at].double().view(hkv, G, 1, D)
                m = torch.maximum(q * b[:, :, 0].transpose(0, 1)[:, None],
                                  q * b[:, :, 1].transpose(0, 1)[:, None]).sum((1, 3))   # [hkv, k]
                keep = torch.ones(hkv, k, dtype=torch.bool, device="cuda")
                if k > c["budget"]:
                    mid = k - c["first"] - c["last"]
                    best = torch.argsort(-m[:, c["first"]:c["first"] + mid], dim=-1, stable=True)
                    keep[:, c["first"]:c["first"] + mid] = False
                    keep.scatter_(1, best[:, :c["budget"] - c["first"] - c["last"]] + c["first"], True)
                table[at] = -1
                for g in range(hkv):
                    ids = pages[keep[g]].int()
                    table[at, g, :len(ids)] = ids
                lens[at] = (min(k, c["budget"]) - 1) * BS + p % BS + 1
                at += 1
        return {"table": table, "lens": lens}
    out = s["out"].double()
    G = c["hq"] // hkv
    if op == "selected":
        for t, n in enumerate(_counts(c)):
            L = int(s["lens"][t])
            for g in range(hkv):
                ids = s["table"][t, g, :n].long()
                k = s["kc"][ids, :, g].double().reshape(-1, D)[:L]
                v = s["vc"][ids, :, g].double().reshape(-1, D)[:L]
                q = s["q"][t, g * G:(g + 1) * G].double()
                out[t, g * G:(g + 1) * G] = _exact_softmax(q, k, v, s["scale"],
                                                          torch.ones(L, dtype=torch.bool, device="cuda"))
        return out
    at = 0
    for r, (x, n) in enumerate(_requests(c)):
        L = x + n
        pages = s["cache"][s["bt"][r, :-(-L // BS)].long()]        # [W, hkv, PAGE4]
        seen = torch.arange(L, device="cuda")[None] <= torch.arange(x, L, device="cuda")[:, None]
        for g in range(hkv):
            k = _exact_page(pages[:, g], 0).reshape(-1, D)[:L]
            v = _exact_page(pages[:, g], 1).reshape(-1, D)[:L]
            q = s["q"][at:at + n, g * G:(g + 1) * G].double().transpose(0, 1)
            out[at:at + n, g * G:(g + 1) * G] = _exact_softmax(q, k, v, s["scale"], seen).transpose(0, 1)
        at += n
    return out
