"""A call on the same inputs gives the same bits each time: work is handed out by atomics,
whose order no result follows."""
import pytest
import torch

import paged_kv_attention_05_gb300 as pkv

pytestmark = pytest.mark.gpu

import test_gpu_int4 as I  # noqa: E402
import test_gpu_pages as P  # noqa: E402


@pytest.mark.parametrize("hq,hkv", [(32, 8), (32, 1), (8, 8)])
@pytest.mark.parametrize("reqs", [[(9000, 1), (129, 1), (4000, 1)] * 5,
                                  [(540, 1), (0, 298), (3000, 2), (64, 170), (9000, 1), (1500, 700)]])
def test_4_bit_attention(reqs, hq, hkv):
    s = I.Step(reqs, hq, hkv, 13)
    s.write()
    s.attention()
    want = s.out.clone()
    for _ in range(20):
        s.out.fill_(float("nan"))
        s.attention()
        assert torch.equal(s.out[:s.rows], want[:s.rows])
    assert pkv.pkv_get_error() == 0


@pytest.mark.parametrize("ctx", [[33000], [2000 + 61 * i for i in range(60)]])
@pytest.mark.parametrize("hq,hkv", [(32, 8), (16, 1)])
def test_selection_and_attention_over_it(ctx, hq, hkv):
    d = P.Decode(ctx, 1, hq, hkv, 48, 7)
    d.next()
    d.step()
    want = [t.clone() for t in (d.table, d.lens, d.out, d.bounds)]
    for _ in range(20):
        d.table.fill_(-1), d.lens.zero_(), d.out.fill_(float("nan"))
        d.step()
        for t, w in zip((d.table, d.lens, d.out[:d.rows], d.bounds),
                        (want[0], want[1], want[2][:d.rows], want[3])):
            assert torch.equal(t, w)
    assert pkv.pkv_get_error() == 0
