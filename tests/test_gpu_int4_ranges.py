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
