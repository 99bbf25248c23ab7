"""Plain 64-bit forms that the tests of the 4-bit cache compare with: the
quantiser, the page record, and attention with a bound on what the kernels'
roundings may add.  Torch operations on any device; nothing of the library."""
import torch

D, BS, PAGE = 128, 16, 2176
TOP, TINY = 2.0 ** 126, 2.0 ** -36


def quantise(x):
    """Codes (int64), scale and zero (float64) of bf16 head rows [..., 128]."""
    x = x.double()
    x = torch.where(x.isnan(), torch.zeros_like(x), x).clamp(-TOP, TOP)
    z = x.amin(-1, keepdim=True)
    w = x.amax(-1, keepdim=True) - z
    s = torch.where(w < TINY, torch.zeros_like(w), (w / 15).to(torch.bfloat16).double())
    q = torch.round((x - z) / torch.where(s == 0, torch.ones_like(s), s)).clamp(0, 15)
    return torch.where(s == 0, torch.zeros_like(q), q).long(), s[..., 0], z[..., 0]


def pack_row(codes):
    """[..., 128] codes -> [..., 64] bytes: word i holds dimensions 8 i .. 8 i + 7,
    dimension 8 i + 2 a + b in bits 4 a + 16 b."""
    c = codes.reshape(*codes.shape[:-1], 16, 8)
    d = torch.arange(8, device=codes.device)
    word = (c << (4 * (d // 2) + 16 * (d % 2))).sum(-1)
    b = torch.stack([(word >> (8 * i)) & 255 for i in range(4)], -1)
    return b.reshape(*codes.shape[:-1], 64).to(torch.uint8)


def write(k, v, cache, slots):
    """The write, in place, row by row as the record is laid out."""
    keep = slots >= 0
    blk, off = slots[keep] // BS, slots[keep] % BS
    for side, x in enumerate((k, v)):
        q, s, z = quantise(x[:slots.shape[0]][keep])
        hkv = q.shape[1]
        rows = cache[:, :, side * 1024:(side + 1) * 1024].view(-1, hkv, BS, 64)
        rows[blk, :, off] = pack_row(q)
        meta = cache[:, :, 2048 + 64 * side:2112 + 64 * side].view(-1, hkv, BS, 4)
        pair = torch.stack([s, z], -1).to(torch.bfloat16).contiguous()
        meta[blk, :, off] = pair.view(torch.uint8).reshape(*s.shape, 4)


def unpack(pages, side):
    """Codes [..., 16, 128] and (scale, zero) [..., 16] of pages [..., 2176]."""
    b = pages[..., side * 1024:(side + 1) * 1024].reshape(*pages.shape[:-1], BS, 16, 4).long()
    word = b[..., 0] | b[..., 1] << 8 | b[..., 2] << 16 | b[..., 3] << 24
    d = torch.arange(8, device=pages.device)
    c = (word[..., None] >> (4 * (d // 2) + 16 * (d % 2))) & 15
    m = pages[..., 2048 + 64 * side:2112 + 64 * side].contiguous().view(torch.bfloat16)
    m = m.reshape(*pages.shape[:-1], BS, 2).double()
    return c.reshape(*pages.shape[:-1], BS, D).double(), m[..., 0], m[..., 1]


def attention(q, cache, qsl, seq_lens, block_table, scale):
    """(out, bound) in float64, [rows, hq, 128]; NaN in rows of no request.  The
    bound on |kernel - out| counts, for decode-path requests:
      the output's own rounding to bf16, 2^-8 |out|;
      the weights' rounding to fp16, 2^-11 of each weight's share of the codes' sum
      (times 1 + 2^-8 for the output's rounding on top: 1.01 below), and for weights below
      fp16's normal range 2^-25 of the largest weight seen so far a key, times codes up
      to 15;
      the logits, formed in fp32: each within 2^-17 of the sizes that cancel in them
      (17 additions and 4 other operations of 2^-24, the MMA's own sums of 2^-22),
      where they turn a weight by that much;
    for prefill requests:
      the same rounding of the output; of the weights to fp16 (2^-11, and below fp16's
      normal range 2^-24 of the largest weight a key); of keys and values to fp16 (2^-11,
      and for those far below the largest of their tile 2^-18 of that), the keys' in the
      products of a logit."""
    rows, hq, _ = q.shape
    hkv = cache.shape[1]
    G = hq // hkv
    out = torch.full((rows, hq, D), float("nan"), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    for r in range(len(seq_lens)):
        a, b, L = int(qsl[r]), int(qsl[r + 1]), int(seq_lens[r])
        n = b - a
        if n == 0:
            continue
        pages = cache[block_table[r, :-(-L // BS)].long()]
        prefill = n * G > (16 if G <= 16 else 32)
        pos = torch.arange(L - n, L, device=q.device)
        hidden = torch.arange(L, device=q.device)[None] > pos[:, None]
        for g in range(hkv):
            (kc, ks, kz), (vc, vs, vz) = (tuple(t.reshape(-1, *t.shape[2:])[:L]
                                                for t in unpack(pages[:, g], side))
                                          for side in (0, 1))
            k, v = kc * ks[:, None] + kz[:, None], vc * vs[:, None] + vz[:, None]
            for h in range(g * G, (g + 1) * G):
                qd = q[a:b, h].double()
                x = (qd @ k.T * scale).masked_fill(hidden, -torch.inf)
                size = abs(scale)
                p = torch.softmax(x, -1)
                o = p @ v
                av = p @ v.abs()
                if prefill:
                    dx = size * (2.0 ** -11 * (qd.abs() @ k.abs().T) + 2.0 ** -18 * k.abs().max() *
                                  qd.abs().sum(-1, keepdim=True))
                    t = 2 * 2.0 ** -11 * av + 2.0 ** -18 * v.abs().max() + \
                        2.0 ** -24 * L * p.amax(-1, keepdim=True) * v.abs().amax(0)
                else:
                    dx = 2.0 ** -17 * size * (qd.abs() @ (kc * ks[:, None]).T +
                                               qd.abs().sum(-1, keepdim=True) * kz.abs())
                    w = p * vs
                    t = 2.0 ** -11 * (w @ vc) + \
                        2.0 ** -25 * 15 * L * w.amax(-1, keepdim=True)
                dx = dx.masked_fill(hidden, 0.)
                turn = (p * dx) @ v.abs() + (p * dx).sum(-1, keepdim=True) * av
                out[a:b, h] = o
                bound[a:b, h] = 2.0 ** -8 * o.abs() + 1.01 * (t + 1.1 * turn) + 2.0 ** -20 * av
    return out, bound
