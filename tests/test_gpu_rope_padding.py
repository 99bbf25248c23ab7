"""pkv_write_rope: nothing of a padding token (negative slot) is read, in the
streaming form as in the straight one.

A read has no effect that a test could see, so what is tested is the calls that
rely on it: positions for the real tokens only, and padding rows between the real
ones, whose every other value is garbage."""
import pytest
import torch

import paged_kv_attention_05_gb300 as pkv
from paged_kv_attention_05_gb300 import _binding

pytestmark = pytest.mark.gpu

from test_gpu_rope import Case, D  # noqa: E402


def c_call(c, n, slots, positions):
    """The call of plain arguments: n tokens, whatever the tensors' lengths."""
    t = [x.data_ptr() for x in (c.q, c.k, c.v, c.dev[1], positions, c.q_out, c.kc, c.vc, slots)]
    stream = torch.cuda.current_stream().cuda_stream
    return _binding.load().pkv_write_rope(
        t[0], c.q.stride(0), c.hq, t[1], c.k.stride(0), t[2], c.v.stride(0), None, None, 0.0, 1e-6,
        t[3], c.table.shape[0], c.rot, 0, t[4], t[5], c.q_out.stride(0), t[6], t[7],
        c.kc.shape[0], 16, c.hkv, D, t[8], n, stream)


@pytest.mark.parametrize("n,pad,hq,hkv", [(3, 20, 8, 2), (40, 900, 32, 8), (700, 2000, 32, 8),
                                          (1500, 1, 64, 8), (2000, 3000, 2, 1)])
def test_positions_of_the_real_tokens_only(n, pad, hq, hkv):
    c = Case(n, hq, hkv, pad=pad)
    # (the rest of the buffer is not part of the argument)
    positions = torch.full((n + pad,), -(1 << 60), dtype=torch.int64, device="cuda")
    positions[:n] = c.dev[0][:n]
    slots = torch.full((n + pad,), -1, dtype=torch.int64, device="cuda")
    slots[:n] = c.dev[2][:n]
    assert c_call(c, n + pad, slots, positions[:n]) == 0
    assert pkv.pkv_get_error() == 0
    c.check()
    assert torch.isnan(c.q_out[n:].float()).all()


@pytest.mark.parametrize("n,hq,hkv", [(50, 8, 2), (2500, 32, 8)])
def test_padding_between_the_tokens(n, hq, hkv):
    """Every third token is padding, the last ones too: runs of padding of one
    and of many in a warp's units."""
    c = Case(n, hq, hkv)
    slots, pos = c.dev[2].clone(), c.dev[0].clone()
    gone = torch.arange(n, device="cuda")
    gone = (gone % 3 == 1) | (gone > n - n // 4)
    slots[gone] = -1
    pos[gone] = 1 << 50
    c.q[gone] = float("nan")
    before = [c.kc.clone(), c.vc.clone()]
    keep = (~gone).cpu()
    pkv.pkv_write_rope(c.q, c.k, c.v, pos, c.dev[1], c.kc, c.vc, slots, c.q_out)
    assert pkv.pkv_get_error() == 0
    qr, qm = c.turned(c.host[0], None)
    kr, km = c.turned(c.host[1], None)
    got = c.q_out.cpu()
    c.near(got[keep], qr[keep], qm[keep], "q_out")
    assert torch.isnan(got[~keep].float()).all()
    at, was = c.slots[keep], c.slots[~keep]
    flat = lambda t: t.cpu().view(-1, hkv, D)  # noqa: E731
    c.near(flat(c.kc)[at], kr[keep], km[keep], "key cache")
    assert torch.equal(flat(c.vc)[at], c.host[2][keep])
    assert torch.equal(flat(c.kc)[was], flat(before[0])[was])
    assert torch.equal(flat(c.vc)[was], flat(before[1])[was])
