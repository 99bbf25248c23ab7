"""The measured cases of two operators of the paged-KV attention step: the cache
write that rotates (and normalises) queries and keys on the way, and attention
with modified scores (tanh cap, distance bias, sliding window, prefix mask).

``own = False`` computes them with elementary torch operations in 32 bits;
``own = True`` makes the library's calls.  ``exact`` computes the same from the
definition in 64 bits."""
import math

import torch

own = False

D = 128      # head size
BS = 16      # tokens of a cache page


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _write(name, tokens, hq, hkv, rot=D, interleaved=False, norm=False, int8=False, pad=0,
           far=32768):
    c = {"op": "write", "tokens": tokens, "pad": pad, "hq": hq, "hkv": hkv, "rot": rot,
         "interleaved": interleaved, "norm": norm, "int8": int8, "far": far}
    return dict(c, name=name) if name else c


def _attention(name, hq, hkv, decodes=0, dec_lo=0, dec_hi=0, dec_q=1, chunks=0, chunk_q=0,
               chunk_step=0, chunk_ctx=0, softcap=0.0, window=0, alibi=False, prefix=0, pad=0,
               std=1.0):
    c = {"op": "attention", "hq": hq, "hkv": hkv, "decodes": decodes, "dec_lo": dec_lo,
         "dec_hi": dec_hi, "dec_q": dec_q, "chunks": chunks, "chunk_q": chunk_q,
         "chunk_step": chunk_step, "chunk_ctx": chunk_ctx, "softcap": softcap, "window": window,
         "alibi": alibi, "prefix": prefix, "pad": pad, "std": std}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one sequence generating: a single token per step, with query and key norms
        _write("rope_1_token", 1, 32, 8, norm=True),
        # a mixed step of two decodes and a short prompt, padded to a capture size
        _write("rope_trace_step", 300, 32, 8, pad=4),
        # a chunk of an odd length, a model that rotates half of each head in interleaved pairs
        _write("rope_chunk_interleaved", 4097, 32, 8, rot=64, interleaved=True),
        # a large prefill of eight prompts, with norms
        _write("rope_norm_prefill", 16384, 64, 8, norm=True),
        # a prompt written into the int8 cache, every head with its own K and V
        _write("rope_int8_prompt", 2048, 32, 32, int8=True),
        # the mixed step again: two decodes and a short prompt under a score cap
        _attention("cap_trace_step", 32, 8, decodes=2, dec_lo=129, dec_hi=540, chunks=1,
                   chunk_q=298, softcap=30.0, pad=4, std=3.0),
        # a batch of long decodes in a local layer: a window, and capped scores
        _attention("window_cap_decode", 32, 8, decodes=128, dec_lo=8192, dec_hi=8192,
                   softcap=50.0, window=4096, std=3.0),
        # decodes of a model without rotation: a distance bias, one KV head per head
        _attention("bias_decode", 32, 32, decodes=64, dec_lo=512, dec_hi=4096, alibi=True),
        # few long sequences that share one KV head, capped, over the whole length
        _attention("cap_long_decode", 32, 1, decodes=32, dec_lo=32768, dec_hi=32768,
                   softcap=50.0, std=3.0),
        # decodes beside prompt chunks whose prefix is seen by every row (prefix mask)
        _attention("prefix_mixed", 32, 8, decodes=64, dec_lo=256, dec_hi=2048, chunks=2,
                   chunk_q=224, chunk_ctx=1024, prefix=1150),
        # a large prefill under a score cap
        _attention("cap_prefill", 64, 8, chunks=8, chunk_q=2048, softcap=50.0, std=3.0),
        # one long prompt of an odd length in a local layer, with a distance bias
        _attention("window_bias_prompt", 32, 8, chunks=1, chunk_q=8191, window=1024, alibi=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    heads = [(32, 8), (32, 32), (64, 8), (8, 8), (32, 1), (16, 2), (24, 8), (12, 4)]
    hq, hkv = rng.choice(heads)
    if rng.random() < 0.4:
        rot = rng.choice([128, 128, 128, 64, 32, 96])
        return _write(None, _log(rng, 1, 12000), hq, hkv, rot, rng.random() < 0.4,
                      rng.random() < 0.5, rng.random() < 0.3, rng.choice([0, 0, 1, 7]))
    cap = rng.choice([0.0, 20.0, 30.0, 50.0])
    opt = {"softcap": cap, "alibi": rng.random() < 0.35,
           "window": _log(rng, 1, 4096) if rng.random() < 0.5 else 0,
           "std": rng.choice([1.0, 3.0]) if cap else 1.0, "pad": rng.choice([0, 0, 3])}
    if cap == 0.0 and not opt["alibi"] and not opt["window"]:
        opt["prefix"] = _log(rng, 16, 2048)
    kind = rng.choice(["decode", "decode", "prompt", "mixed"])
    if kind == "decode":
        n, hi = _log(rng, 1, 96), _log(rng, 16, 8192)
        dq = rng.choice([1, 1, 2, 3]) if hq // hkv <= 4 else 1
        return _attention(None, hq, hkv, decodes=n, dec_lo=_log(rng, 1, hi), dec_hi=hi, dec_q=dq,
                          **opt)
    if kind == "prompt":
        n, q = rng.randint(1, 4), _log(rng, 17, 2048)
        return _attention(None, hq, hkv, chunks=n, chunk_q=q, chunk_step=rng.randint(0, q // 8),
                          chunk_ctx=rng.choice([0, _log(rng, 1, 1024)]), **opt)
    hi = _log(rng, 16, 2048)
    q = _log(rng, 17, 512)
    return _attention(None, hq, hkv, decodes=_log(rng, 1, 48), dec_lo=_log(rng, 1, hi), dec_hi=hi,
                      chunks=rng.randint(1, 2), chunk_q=q, chunk_step=rng.randint(0, q // 4),
                      chunk_ctx=rng.choice([0, _log(rng, 1, 1024)]), **opt)


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


def _visible(c):
    """(visible (row, key) pairs, keys visible to some row) of the batch."""
    pairs = keys = 0
    for ctx, n in _requests(c):
        L = ctx + n
        lows = [max(0, p - c["window"] + 1) if c["window"] else 0 for p in (ctx, L - 1)]
        pre = min(c["prefix"], L)
        if not c["window"] and not pre:
            pairs += n * ctx + n * (n + 1) // 2
        else:
            for p in range(ctx, L):
                lo = max(0, p - c["window"] + 1) if c["window"] else 0
                pairs += max(p + 1, pre) - lo
        keys += L - lows[0]
    return pairs, keys


def work(case):
    c = case
    if c["op"] == "write":
        n, hq, hkv = c["tokens"], c["hq"], c["hkv"]
        b = n * ((hq + 2 * hkv) * D * 2 + hq * D * 2 + 2 * hkv * D * (1 if c["int8"] else 2) +
                 c["rot"] * 4 + 16)
        return {"bytes": b, "flops": n * (hq + hkv) * (3 * c["rot"] + (4 * D if c["norm"] else 0))}
    pairs, keys = _visible(c)
    rows = sum(n for _, n in _requests(c))
    return {"bytes": 2 * rows * c["hq"] * D * 2 + 2 * keys * c["hkv"] * D * 2,
            "flops": 4 * D * pairs * c["hq"]}


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


def _split(qkv, hq, hkv):
    """q, k, v as column slices of the fused projection's rows."""
    t = qkv.shape[0]
    return (qkv[:, :hq * D].view(t, hq, D), qkv[:, hq * D:(hq + hkv) * D].view(t, hkv, D),
            qkv[:, (hq + hkv) * D:].view(t, hkv, D))


def _table(far, rot):
    """cos | sin of position times frequency, angles in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(far, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def prepare(case, seed):
    c, g = case, _gen(seed)
    hq, hkv = c["hq"], c["hkv"]
    if c["op"] == "write":
        n, rows = c["tokens"], c["tokens"] + c["pad"]
        blocks = -(-n // BS) + 3
        q, k, v = _split(_randn((rows, (hq + 2 * hkv) * D), g), hq, hkv)
        slots = torch.randperm(blocks * BS, generator=g, device="cuda")[:rows].contiguous()
        slots[n:] = -1
        shape = (blocks, BS, hkv, D)
        if c["int8"]:
            kc = torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)
            vc = torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)
        else:
            kc, vc = _randn(shape, g), _randn(shape, g)
        s = {"c": c, "n": n, "q": q, "k": k, "v": v, "slots": slots, "kc": kc, "vc": vc,
             "positions": torch.randint(0, c["far"], (rows,), generator=g, device="cuda"),
             "table": _table(c["far"], c["rot"]),
             "q_out": torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda"),
             "qw": None, "kw": None, "eps": 1e-6}
        if c["norm"]:
            s["qw"], s["kw"] = 1 + 0.1 * _randn((D,), g), 1 + 0.1 * _randn((D,), g)
        if c["int8"]:
            # scales that a calibration would give: 4.5 standard deviations at code 127
            s["ks"], s["vs"] = 0.035400390625, 0.035400390625
            s["kst"] = torch.tensor(s["ks"], dtype=torch.bfloat16, device="cuda")
            s["vst"] = torch.tensor(s["vs"], dtype=torch.bfloat16, device="cuda")
        return s
    reqs = _requests(c)
    ctx = torch.tensor([r[0] for r in reqs], dtype=torch.int32)
    n = torch.tensor([r[1] for r in reqs], dtype=torch.int32)
    seq = ctx + n
    width = -(-int(seq.max()) // BS)
    used = [-(-int(x) // BS) for x in seq]
    pool = sum(used) + 5
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32).cpu()
    bt = torch.full((len(reqs), width), -1, dtype=torch.int32)
    at = 0
    for r, u in enumerate(used):
        bt[r, :u] = perm[at:at + u]
        at += u
    rows = int(n.sum())
    qsl = torch.zeros(len(reqs) + 1, dtype=torch.int32)
    qsl[1:] = n.cumsum(0)
    req_of = torch.repeat_interleave(torch.arange(len(reqs)), n.long())
    off = torch.arange(rows) - qsl[:-1].long()[req_of]
    q = _split(_randn((rows + c["pad"], (hq + 2 * hkv) * D), g, c["std"]), hq, hkv)[0]
    slopes = None
    if c["alibi"]:
        slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)]).cuda()
    prefix = None
    if c["prefix"]:
        # prompts see their prefix from every row; decodes have theirs behind them
        prefix = torch.full((len(reqs),), c["prefix"], dtype=torch.int32, device="cuda")
    return {"c": c, "q": q, "kc": _randn((pool, BS, hkv, D), g), "vc": _randn((pool, BS, hkv, D), g),
            "qsl": qsl.cuda(), "seq": seq.cuda(), "bt": bt.cuda(), "reqs": len(reqs), "rows": rows,
            "nmax": int(n.max()), "req_of": req_of.cuda(), "off": off.cuda(), "slopes": slopes,
            "prefix": prefix, "scale": D ** -0.5,
            "out": torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda")}


# --------------------------------------------------------------------------
# plain forms (32 bits)
# --------------------------------------------------------------------------

def _turned(x, w, s, cos, sin):
    c = s["c"]
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * w.float()
    rot, half = c["rot"], c["rot"] // 2
    z = y.clone()
    if c["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        z[..., 0:rot:2] = a * cos - b * sin
        z[..., 1:rot:2] = b * cos + a * sin
    else:
        a, b = y[..., :half], y[..., half:rot]
        z[..., :half] = a * cos - b * sin
        z[..., half:rot] = b * cos + a * sin
    return z


def _plain_write(s):
    c, n = s["c"], s["n"]
    t = s["table"][s["positions"][:n]]
    half = c["rot"] // 2
    cos, sin = t[:, None, :half], t[:, None, half:]
    q = _turned(s["q"][:n], s["qw"], s, cos, sin)
    k = _turned(s["k"][:n], s["kw"], s, cos, sin)
    v = s["v"][:n].float()
    slots = s["slots"][:n]
    kc, vc = s["kc"].view(-1, c["hkv"], D), s["vc"].view(-1, c["hkv"], D)
    if c["int8"]:
        k = torch.round(k / s["kst"].float()).clamp(-127, 127)
        v = torch.round(v / s["vst"].float()).clamp(-127, 127)
    s["q_out"][:n] = q.to(torch.bfloat16)
    kc[slots] = k.to(kc.dtype)
    vc[slots] = v.to(vc.dtype)


def _plain_attention(s):
    c = s["c"]
    hq, hkv, R, N = c["hq"], c["hkv"], s["reqs"], s["nmax"]
    G = hq // hkv
    bt = s["bt"].clamp(min=0).long()
    L = bt.shape[1] * BS
    k = s["kc"][bt].view(R, L, hkv, D).permute(0, 2, 1, 3).float()
    v = s["vc"][bt].view(R, L, hkv, D).permute(0, 2, 1, 3).float()
    q = torch.zeros(R, N, hq, D, device="cuda")
    q[s["req_of"], s["off"]] = s["q"][:s["rows"]].float()
    q = q.view(R, N, hkv, G, D).permute(0, 2, 3, 1, 4).reshape(R, hkv, G * N, D)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(R, hkv, G, N, L)
    if c["softcap"]:
        x = x.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    seq, ctx = s["seq"].long(), s["seq"].long() - (s["qsl"][1:] - s["qsl"][:-1]).long()
    pos = (ctx[:, None] + torch.arange(N, device="cuda"))[:, :, None]        # [R, N, 1]
    key = torch.arange(L, device="cuda")[None, None, :]
    if s["slopes"] is not None:
        dist = (pos - key).abs().float()[:, None, None]
        x = x.sub_(s["slopes"].view(1, hkv, G, 1, 1) * dist)
    hi = torch.minimum(pos + 1, seq[:, None, None])
    if s["prefix"] is not None:
        hi = torch.maximum(hi, torch.minimum(s["prefix"].long(), seq)[:, None, None])
    seen = key < hi
    if c["window"]:
        seen = seen & (key > pos - c["window"])
    x = x.masked_fill_(~seen[:, None, None], float("-inf"))
    # (rows past a request's own are computed and dropped)
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    total = x.sum(-1, keepdim=True).view(R, hkv, G * N, 1)
    o = torch.matmul(x.view(R, hkv, G * N, L), v).div_(total)
    o = o.view(R, hkv, G, N, D).permute(0, 3, 1, 2, 4).reshape(R, N, hq, D)
    s["out"][:s["rows"]] = o[s["req_of"], s["off"]].to(torch.bfloat16)


def run(state):
    s = state
    c = s["c"]
    if c["op"] == "write":
        if own:
            import paged_kv_attention_05_gb300 as pkv
            opt = {"interleaved": c["interleaved"], "q_weight": s["qw"], "k_weight": s["kw"],
                   "eps": s["eps"]}
            if c["int8"]:
                pkv.pkv_write_rope_int8(s["q"], s["k"], s["v"], s["positions"], s["table"],
                                        s["kc"], s["vc"], s["slots"], s["ks"], s["vs"],
                                        s["q_out"], **opt)
            else:
                pkv.pkv_write_rope(s["q"], s["k"], s["v"], s["positions"], s["table"], s["kc"],
                                   s["vc"], s["slots"], s["q_out"], **opt)
        else:
            _plain_write(s)
        if c["int8"]:  # the values that the codes stand for
            return {"q": s["q_out"], "k": torch.mul(s["kc"], s["kst"]),
                    "v": torch.mul(s["vc"], s["vst"])}
        return {"q": s["q_out"], "k": s["kc"], "v": s["vc"]}
    if own:
        import paged_kv_attention_05_gb300 as pkv
        pkv.pkv_attention_scored(s["q"], s["kc"], s["vc"], s["qsl"], s["seq"], s["bt"], s["reqs"],
                                 s["scale"], s["out"], softcap=c["softcap"], window=c["window"],
                                 alibi_slopes=s["slopes"], prefix_lens=s["prefix"])
    else:
        _plain_attention(s)
    return s["out"]


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_head_rows(x, w, eps, offset_rot, angles, interleaved):
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / D + eps).sqrt() * w.double()
    half = offset_rot // 2
    i = torch.arange(half, device=x.device)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    pair = torch.complex(x[..., first], x[..., second]) * angles[:, None, :]
    x[..., first], x[..., second] = pair.real, pair.imag
    return x


def exact(case, seed):
    c, s = case, prepare(case, seed)
    hq, hkv = c["hq"], c["hkv"]
    G = hq // hkv
    if c["op"] == "write":
        n, half = s["n"], c["rot"] // 2
        t = s["table"][s["positions"][:n]].double()
        angles = torch.complex(t[:, :half], t[:, half:])
        q = s["q_out"].double()
        q[:n] = _exact_head_rows(s["q"][:n].clone(), s["qw"], s["eps"], c["rot"], angles,
                                 c["interleaved"])
        k = _exact_head_rows(s["k"][:n].clone(), s["kw"], s["eps"], c["rot"], angles,
                             c["interleaved"])
        v = s["v"][:n].double()
        kc, vc = s["kc"].double(), s["vc"].double()
        if c["int8"]:
            k = torch.round(k / s["ks"]).clamp(-127, 127)
            v = torch.round(v / s["vs"]).clamp(-127, 127)
        at = (s["slots"][:n] // BS, s["slots"][:n] % BS)
        kc[at], vc[at] = k, v
        if c["int8"]:
            kc, vc = kc * s["ks"], vc * s["vs"]
        return {"q": q, "k": kc, "v": vc}
    out = s["out"].double()
    at = 0
    for r, (ctx, n) in enumerate(_requests(c)):
        L = ctx + n
        low = max(0, ctx - c["window"] + 1) if c["window"] else 0   # no row sees keys below
        j = torch.arange(low, L, device="cuda")
        block, slot = s["bt"][r].long()[j // BS], j % BS
        p = torch.arange(ctx, L, device="cuda")[:, None]
        seen = j[None] <= p
        if s["prefix"] is not None:
            seen = seen | (j[None] < c["prefix"])
        if c["window"]:
            seen = seen & (p - j[None] < c["window"])
        far = (p - j[None]).abs().double()
        for g in range(hkv):
            k, v = s["kc"][block, slot, g].double(), s["vc"][block, slot, g].double()
            q = s["q"][at:at + n, g * G:(g + 1) * G].double().transpose(0, 1)
            x = (q @ k.T) * s["scale"]
            if c["softcap"]:
                x = c["softcap"] * torch.tanh(x / c["softcap"])
            if s["slopes"] is not None:
                x = x - s["slopes"][g * G:(g + 1) * G].double()[:, None, None] * far
            x = torch.where(seen, x, torch.full_like(x, -math.inf))
            x = torch.exp(x - torch.logsumexp(x, -1, keepdim=True))
            out[at:at + n, g * G:(g + 1) * G] = (x @ v).transpose(0, 1)
        at += n
    return out
