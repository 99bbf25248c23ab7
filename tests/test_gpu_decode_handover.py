"""Decodes of groups above 16 heads in units of one or two pages, many to a warp
pair: the pair's first warp hands a unit to its second as fast as units come.

(No input can force the order of two warps, so the hand-over's wait is argued in
the kernel; this runs the shape that leans on it, in both of its instances.)
Tolerance: as in test_gpu_scored, for scores without options."""
import pytest
import torch

import paged_kv_attention_05_gb300 as pkv

pytestmark = pytest.mark.gpu

D = 128


@pytest.mark.parametrize("heads", [24, 32])
def test_many_units_of_one_step(heads):
    n, top = 5000, 40          # 912 warp pairs: five or six units each
    g = torch.Generator(device="cuda").manual_seed(heads)
    q = torch.randn(n, heads, D, generator=g, device="cuda").to(torch.bfloat16)
    pages = -(-top // 16)
    kc = torch.randn(n * pages, 16, 1, D, generator=g, device="cuda").to(torch.bfloat16)
    vc = torch.randn(n * pages, 16, 1, D, generator=g, device="cuda").to(torch.bfloat16)
    bt = torch.randperm(n * pages, generator=g, device="cuda").to(torch.int32).view(n, pages)
    lens = torch.randint(1, top + 1, (n,), generator=g, device="cuda").to(torch.int32)
    lens[:n // 2].clamp_(max=32)
    qsl = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    scale = D ** -0.5

    k = kc[bt.long()].view(n, pages * 16, D).double()
    v = vc[bt.long()].view(n, pages * 16, D).double()
    s = scale * torch.einsum("nhd,nkd->nhk", q.double(), k)
    d = 2.0 ** -16 * scale * torch.einsum("nhd,nkd->nhk", q.double().abs(), k.abs()).amax(-1)
    seen = torch.arange(pages * 16, device="cuda")[None, None] < lens[:, None, None]
    w = torch.softmax(s.masked_fill(~seen, float("-inf")), -1)
    ref, size = w @ v, w @ v.abs()
    tol = 2.0 ** -7 * ref.abs() + size * (2.0 ** -8 + 2.0 ** -14 + 2 * d[..., None])

    plain, scored = torch.empty_like(q), torch.empty_like(q)
    pkv.pkv_attention(q, kc, vc, qsl, lens, bt, n, scale, plain)
    pkv.pkv_attention_scored(q, kc, vc, qsl, lens, bt, n, scale, scored)
    assert pkv.pkv_get_error() == 0
    for out in (plain, scored):
        assert ((out.double() - ref).abs() <= tol).all()
    again = torch.empty_like(q)
    for turn in range(30):
        if turn % 2:
            pkv.pkv_attention(q, kc, vc, qsl, lens, bt, n, scale, again)
        else:
            pkv.pkv_attention_scored(q, kc, vc, qsl, lens, bt, n, scale, again)
        assert torch.equal(again, plain if turn % 2 else scored)
    assert pkv.pkv_get_error() == 0
