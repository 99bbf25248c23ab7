"""4-bit caches at the ends of their range: values whose size changes along the context,
constant rows, very large queries, queries whose dimensions differ widely."""
import math

import pytest
import torch

import paged_kv_attention_05_gb300 as pkv

pytestmark = pytest.mark.gpu

import int4_ref as R  # noqa: E402
import test_gpu_int4 as I  # noqa: E402

TILE = 128


@pytest.mark.parametrize("hq,hkv", [(8, 2), (12, 1), (32, 1)])
@pytest.mark.parametrize("scale", [I.R.D ** -0.5, -1.0])
@pytest.mark.parametrize("e", [60, 100, 108])
def test_decodes_with_very_large_queries(e, hq, hkv, scale):
    """Queries of up to 2^110, the documented limit.  Over keys of 2^-e, constant rows, the logits are small and
    outputs those of the formula; over keys of 1 one key has all of the weight."""
    s = I.Step([(300, 1), (33, 2 if hq == 8 else 1), (2000, 1)], hq, hkv, e)
    s.scale = scale
    s.q[:] = (s.q.clamp(-3, 3).double() * 2.0 ** e).to(torch.bfloat16)
    small = s.k[:, :, :1].double() * 2.0 ** -e / 8
    keys = s.k.clone()
    s.k[:] = small.to(torch.bfloat16)
    s.write()
    s.attention()
    assert pkv.pkv_get_error() == 0
    s.check("small keys")
    s.k[:] = keys / 64      # (sums below 2^128)
    s.write()
    s.attention()
    assert pkv.pkv_get_error() == 0
    assert bool(s.out[:s.rows].isfinite().all())
    clear = 0
    for r in range(len(s.reqs)):
        for t in range(int(s.qsl[r]), int(s.qsl[r + 1])):
            L = int(s.seq[r]) - (int(s.qsl[r + 1]) - 1 - t)
            pages = s.cache[s.bt[r, :-(-L // R.BS)].long()]
            for h in range(hq):
                (kc, ks, kz), (vc, vs, vz) = (tuple(x.reshape(-1, *x.shape[2:])[:L]
                                                    for x in R.unpack(pages[:, h // (hq // hkv)], i))
                                              for i in (0, 1))
                q = s.q[t, h].double()
                x = (kc * ks[:, None] + kz[:, None]) @ q * scale
                size = abs(scale) * ((kc * ks[:, None]) @ q.abs() + q.abs().sum() * kz.abs())
                top = x.topk(2)
                # (logits are formed within 2^-17 of what cancels in them)
                if float(top.values[0] - top.values[1]) < 2 * 2.0 ** -17 * float(size.max()):
                    continue
                clear += 1
                j = int(top.indices[0])
                v = vc[j] * vs[j] + vz[j]
                # the weight's rounding to fp16, the output's
                assert bool(((s.out[t, h].double() - v).abs() <=
                             2.0 ** -8 * v.abs() + 1.01 * 2.0 ** -11 * vs[j] * vc[j] + 2.0 ** -20).all())
    assert clear > s.rows * hq // 2


@pytest.mark.parametrize("hq,hkv", [(8, 2), (12, 1), (32, 1)])
def test_queries_whose_dimensions_differ_widely(hq, hkv):
    """Dimensions of a query row that differ by 2^30: the small ones meet keys that are as
    much larger."""
    s = I.Step([(300, 1), (33, 2 if hq == 8 else 1), (2000, 1)], hq, hkv, 5)
    e = torch.linspace(0, 30, R.D, device="cuda").round().double()
    e = e[torch.randperm(R.D, generator=I.gen(4), device="cuda")]
    s.q[:] = (s.q.double() * 2.0 ** -e).to(torch.bfloat16)
    s.write()
    s.attention()
    assert pkv.pkv_get_error() == 0
    s.check("wide queries")


@pytest.mark.parametrize("hq,hkv", [(8, 2), (12, 1), (32, 1)])
@pytest.mark.parametrize("grow", [0.0, 0.4])
def test_large_constant_value_rows(grow, hq, hkv):
    """Value rows without spread have the scale 0: their size, up to 2^60, is in the zeros
    alone.  With logits that grow by `grow` (log2) a key the reference stays 2^13 behind."""
    s = I.Step([(300, 1), (33, 2 if hq == 8 else 1), (2000, 1), (40, 1)], hq, hkv, 60)
    s.v[:] = (s.v[:, :, :1].clamp(-1, 1).double() * 2.0 ** 60).to(torch.bfloat16)
    s.v[::7] *= 2.0 ** -60
    if grow:
        at = torch.cat([torch.arange(c + n, device="cuda") for c, n in s.reqs]).double()
        s.q[:] = 1
        s.k[:] = (at * grow / math.log2(math.e) / (R.D * s.scale))[:, None, None].to(torch.bfloat16)
    s.write()
    s.attention()
    assert pkv.pkv_get_error() == 0
    s.check("constant rows")


def prompt_bound(s, r):
    """Attention of request r of a step in 64 bits and what a prompt's kernel may be off by:
    the output's rounding (2^-8); weights rounded to fp16, twice where the reference moved
    within a tile (2^-11 each); keys and values rounded to fp16 (2^-11), and what lies far
    below the largest of its own tile of 128 keys by 2^-18 of that (tiles 2^60 below the
    largest before them count as 2^-60 of it); and weights below fp16's normal range, of
    which the reference keeps the largest weight times its tile's size above 2^7: half of
    2^-24 a rounding, 2^-31 of the largest of weight times the tile's largest value, per key."""
    a, b, L = int(s.qsl[r]), int(s.qsl[r + 1]), int(s.seq[r])
    pages = s.cache[s.bt[r, :-(-L // R.BS)].long()]
    pos = torch.arange(L - (b - a), L, device="cuda")
    hidden = torch.arange(L, device="cuda")[None] > pos[:, None]
    G = s.hq // s.hkv
    pad = -L % TILE

    def largest(x):    # of each key's tile
        t = torch.nn.functional.pad(x.abs().amax(-1), (0, pad)).view(-1, TILE).amax(-1)
        return t

    outs, bounds = [], []
    for h in range(s.hq):
        g = h // G
        (kc, ks, kz), (vc, vs, vz) = (tuple(t.reshape(-1, *t.shape[2:])[:L]
                                            for t in R.unpack(pages[:, g], side))
                                      for side in (0, 1))
        k, v = kc * ks[:, None] + kz[:, None], vc * vs[:, None] + vz[:, None]
        kt = largest(k).repeat_interleave(TILE)[:L]
        vt = largest(v)
        vt = torch.maximum(vt, 2.0 ** -60 * vt.cummax(0).values).repeat_interleave(TILE)[:L]
        q = s.q[a:b, h].double()
        p = torch.softmax((q @ k.T * s.scale).masked_fill(hidden, -torch.inf), -1)
        o, av = p @ v, p @ v.abs()
        dx = abs(s.scale) * (2.0 ** -11 * (q.abs() @ k.abs().T) +
                             2.0 ** -18 * q.abs().sum(-1, keepdim=True) * kt)
        dx = dx.masked_fill(hidden, 0.)
        t = 2 * 2.0 ** -11 * av + 2.0 ** -18 * (p @ vt)[:, None] + \
            2 * 2.0 ** -31 * L * (p * vt).amax(-1, keepdim=True)
        turn = (p * dx) @ v.abs() + (p * dx).sum(-1, keepdim=True) * av
        outs.append(o)
        bounds.append(2.0 ** -8 * o.abs() + 1.01 * (t + 1.1 * turn) + 2.0 ** -20 * av)
    return torch.stack(outs, 1), torch.stack(bounds, 1)


def check_prompts(s, what):
    for r in range(len(s.reqs)):
        ref, bound = prompt_bound(s, r)
        got = s.out[int(s.qsl[r]):int(s.qsl[r + 1])].double()
        err = (got - ref).abs()
        assert bool((err <= bound).all()), "%s, request %d: error up to %g of the bound" % (
            what, r, float((err / bound).nan_to_num(9e9).max()))


@pytest.mark.parametrize("hq,hkv", [(8, 2), (3, 1)])
@pytest.mark.parametrize("kind", ["one large row", "larger by and by", "smaller by and by",
                                  "by turns", "zero first", "zero tiles", "far apart"])
def test_values_whose_size_changes_from_tile_to_tile(kind, hq, hkv):
    s = I.Step([(700, 150), (0, 777), (1300, 33)], hq, hkv, 17)
    g = I.gen(3)
    s.q[:] = (1 + 0.3 * s.q.float()).to(torch.bfloat16)
    at = torch.cat([torch.arange(c + n, device="cuda") for c, n in s.reqs])
    tile = (at // TILE).double()
    if kind == "one large row":        # of which no weight is left
        s.k[at == 0] = -4
        s.v[at == 0] *= 2.0 ** 20
    else:
        e = {"larger by and by": 5 * tile, "smaller by and by": 20 - 7 * tile,
             "by turns": 30 * (tile % 2), "zero first": 5 - 4 * tile, "zero tiles": 3 * tile,
             "far apart": torch.where(tile % 3 == 1, 60., -20. * (tile % 3))}[kind]
        s.v[:] = (s.v.double() * (2.0 ** e)[:, None, None]).to(torch.bfloat16)
        if kind == "zero first":
            s.v[tile == 0] = 0
        if kind == "zero tiles":
            s.v[tile % 2 == 1] = 0
        if kind in ("smaller by and by", "by turns", "far apart"):
            # the small ones' keys have nearly all of the weight
            s.k[:] = (s.k.double() - (e - e.min())[:, None, None] / 16).to(torch.bfloat16)
    s.write()
    s.attention()
    assert pkv.pkv_get_error() == 0
    check_prompts(s, kind)
