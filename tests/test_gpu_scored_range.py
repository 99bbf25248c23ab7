"""pkv_attention_scored at the ends of its range: scores saturated at either end
of a cap, caps at the largest that takes the fixed reference and beyond, values of
V far from one, steep slopes.

Tolerance: that of test_gpu_scored (derived there); it is proportional to the
softmax average of |V|, so that it holds for V of any size."""
import pytest
import torch

import paged_kv_attention_05_gb300 as pkv
from paged_kv_attention_05_gb300 import workloads as W

pytestmark = pytest.mark.gpu

from gpu_util import DeviceStep  # noqa: E402
from test_gpu_scored import assert_near, call, reference  # noqa: E402

D = 128


def saturated(ctx, n, hq, hkv, signs, v_scale=1.0, seed=0):
    """A step whose raw scores are signs(L)[j] times 220, 110 or 55 (by the head):
    q = a u, K_j = s_j b u with u of signs, so that every product is exact.
    V falls from 1 to -1 along the keys, with noise of a tenth."""
    ds = DeviceStep(W.build(W.custom(ctx, n, hq, hkv, seed=seed)))
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    u = torch.randint(0, 2, (D,), generator=g, device="cuda").to(torch.bfloat16) * 2 - 1
    size = torch.tensor([(16.0, 8.0, 4.0)[h % 3] for h in range(hq)], device="cuda").bfloat16()
    ds.q[:] = size[:, None] * u
    for r, (c, m) in enumerate(zip(ctx, n)):
        L = c + m
        j = torch.arange(L, device="cuda")
        blk = ds.block_table[r].long()[j // 16]
        s = signs(L).to(torch.bfloat16)
        ds.key_cache[blk, j % 16] = (1.21875 * s[:, None, None] * u).expand(L, hkv, D)
        v = (1 - 2 * j.float() / L)[:, None, None] + 0.1 * torch.randn(
            L, hkv, D, generator=g, device="cuda")
        ds.value_cache[blk, j % 16] = (v * v_scale).to(torch.bfloat16)
    return ds


def check(ds, what, **opt):
    ref, tol = reference(ds, **opt)
    ds.out.fill_(float("nan"))
    call(ds, **opt)
    assert pkv.pkv_get_error() == 0
    assert_near(ds.out[:ref.shape[0]], ref, tol, what)


SIGNS = {
    "minus": lambda L: -torch.ones(L, device="cuda"),
    "plus": lambda L: torch.ones(L, device="cuda"),
    # (with a bias that falls with distance, keys a full cap up against keys near by)
    "far": lambda L: torch.where(torch.arange(L, device="cuda") < L // 4, 1.0, -1.0),
}
# a prompt, a chunk and decodes of several tokens and of one, some of them split
STEP = ([0, 5900, 6500, 800, 63], [700, 150, 1, 2, 1])


@pytest.mark.parametrize("signs", SIGNS)
@pytest.mark.parametrize("cap", [50.0, 54.0, 55.0, 55.4, 55.5, 60.0])
@pytest.mark.parametrize("hq,hkv", [(6, 2), (32, 1)])
def test_saturated_scores_with_a_bias(hq, hkv, cap, signs):
    """No weight that counts is lost where a bias lies below a score at the
    cap's lower end, up to the largest cap of the fixed reference (55.45) and
    past it; with a prefix too."""
    n = STEP[1] if hkv == 2 else [700, 150, 1, 1, 1]
    ds = saturated(STEP[0], n, hq, hkv, SIGNS[signs], seed=hq)
    slopes = torch.tensor([(0.02, -0.02, 0.004, 0.3)[h % 4] for h in range(hq)])
    check(ds, "bias", softcap=cap, slopes=slopes)
    check(ds, "bias, prefix", softcap=cap, slopes=slopes, prefix=[600, 6000, 0, 802, 40])


@pytest.mark.parametrize("signs", ["minus", "plus"])
@pytest.mark.parametrize("v_scale", [2.0 ** -30, 2.0 ** -20, 2.0 ** 20])
@pytest.mark.parametrize("cap", [50.0, 55.4])
@pytest.mark.parametrize("hq,hkv", [(6, 2), (32, 1)])
def test_saturated_scores_with_small_and_large_values(hq, hkv, cap, v_scale, signs):
    """The unnormalised sums keep V's bits whichever end of the cap the row's
    scores lie at (the first row of a prompt has one key)."""
    n = STEP[1] if hkv == 2 else [700, 150, 1, 1, 1]
    ds = saturated(STEP[0], n, hq, hkv, SIGNS[signs], v_scale=v_scale, seed=hq)
    check(ds, "no bias", softcap=cap)
    check(ds, "window", softcap=cap, window=100)


@pytest.mark.parametrize("opt", [dict(), dict(softcap=20.0), dict(softcap=55.0),
                                 dict(softcap=200.0)], ids=str)
@pytest.mark.parametrize("slope", [1e4, 1e8, 1e30, -1e4, -1e8, -1e30])
@pytest.mark.parametrize("hq,hkv", [(6, 2), (32, 1)])
def test_slopes_steep_enough_to_leave_one_key(hq, hkv, slope, opt):
    """The next key lies 1e4 below or more, scores differ by 400 at most: the row's
    one key is its own, or the farthest that it sees, with weight one, and the
    output that key's V to the bit (a bf16 value times a weight, divided by that
    weight in fp32, rounds back to it)."""
    ctx, n = [0, 300, 5000, 64, 300], [300, 140, 1, 3 if hkv == 2 else 1, 1]
    ds = DeviceStep(W.build(W.custom(ctx, n, hq, hkv, seed=77)))
    ds.write()
    slopes = torch.full((hq,), slope)
    # an even prefix: no row is as far from its last key as from key 0
    for window, prefix in ((0, None), (50, None), (0, [250, 400, 0, 66, 40])):
        ds.out.fill_(float("nan"))
        call(ds, slopes=slopes, window=window, prefix=prefix, **opt)
        assert pkv.pkv_get_error() == 0
        at = 0
        for r, (c, m) in enumerate(zip(ctx, n)):
            keys = []
            for p in range(c, c + m):
                hi = max(p + 1, min(prefix[r], c + m)) if prefix else p + 1
                lo = max(0, p - window + 1) if window else 0
                keys.append(p if slope > 0 else (lo if p - lo > hi - 1 - p else hi - 1))
            j = torch.tensor(keys, device="cuda")
            want = ds.value_cache[ds.block_table[r].long()[j // 16], j % 16]
            want = want.repeat_interleave(hq // hkv, dim=1)
            assert torch.equal(ds.out[at:at + m], want), (window, prefix, r)
            at += m
