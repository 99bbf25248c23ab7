"""Views of one head and of one row, as transposes give them, through the calls:
the bits of the contiguous tensors' calls."""
import pytest
import torch

import paged_kv_attention_05_gb300 as pkv

pytestmark = pytest.mark.gpu

D = 128


@pytest.mark.parametrize("n,hq,hkv", [(40, 8, 1), (40, 1, 1), (1, 8, 2), (1, 4, 1)])
def test_views_of_one_head_and_of_one_row(n, hq, hkv):
    g = torch.Generator(device="cuda").manual_seed(n + hq)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v = rand(n, hq, D), rand(n, hkv, D), rand(n, hkv, D)
    def view(t):   # [heads, n, 128] transposed, where that differs in strides alone
        if n > 1 and t.shape[1] > 1:
            return t
        return t.permute(1, 0, 2).clone(memory_format=torch.contiguous_format).transpose(0, 1)

    assert any(view(t).stride() != t.stride() for t in (q, k))
    slots = torch.arange(n, device="cuda")
    pos = torch.arange(n, device="cuda")
    tab = torch.rand(n + 1, D, generator=g, device="cuda")
    bt = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    qsl = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    seq = torch.tensor([n], dtype=torch.int32, device="cuda")
    got = []
    for f in (lambda t: t, view):
        a, b, c = f(q), f(k), f(v)
        kc, vc = (torch.zeros(4, 16, hkv, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        qo, o1, o2 = (f(torch.zeros_like(q)) for _ in range(3))
        pkv.pkv_write(b, c, kc, vc, slots)
        pkv.pkv_attention(a, kc, vc, qsl, seq, bt, 1, 0.1, o1)
        pkv.pkv_write_rope(a, b, c, pos, tab, kc, vc, slots, qo)
        pkv.pkv_attention_scored(qo, kc, vc, qsl, seq, bt, 1, 0.1, o2, softcap=20.0)
        got.append([t.contiguous() for t in (kc, vc, qo, o1, o2)])
    assert pkv.pkv_get_error() == 0
    for x, y in zip(*got):
        assert torch.equal(x, y) and x.float().abs().sum() > 0
