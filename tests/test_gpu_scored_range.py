"""pkv_attention_scored at the ends of its range: scores saturated at either end
of a cap, caps at the largest that takes the fixed reference and beyond, values of
V far from one, steep slopes.

Tolerance: that of test_gpu_scored (derived there); it is proportional to the
softmax average of |V|, so that it holds for V of any size.  Where the products
q . K are whole numbers below 2^24 they are exact in fp32 and their term goes."""
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


def definition(ds, softcap, window=0, slopes=None, prefix=None):
    """(out, tolerance) in 64 bits for exact products q . K."""
    st = ds.step
    hq, hkv = st.spec.hq, st.spec.hkv
    G = hq // hkv
    rows = int(st.query_start_loc[-1])
    out = torch.empty(rows, hq, D, dtype=torch.float64, device="cuda")
    tol = torch.empty_like(out)
    scale = float(torch.tensor(st.scale, dtype=torch.float32))
    for r in range(st.num_reqs):
        a, b = int(st.query_start_loc[r]), int(st.query_start_loc[r + 1])
        L = int(st.seq_lens[r])
        p = torch.arange(L - (b - a), L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")[None]
        hi = torch.maximum(p + 1, torch.tensor(min(prefix[r], L) if prefix else 0, device="cuda"))
        seen = (j < hi) & (p - j < (window or L + 1))
        blk = ds.block_table[r].long()[j[0] // 16]
        for h in range(hq):
            k, v = (t[blk, j[0] % 16, h // G].double() for t in (ds.key_cache, ds.value_cache))
            x = scale * (ds.q[a:b, h].double() @ k.T)
            x = softcap * torch.tanh(x / softcap)
            d = torch.full_like(x[:, 0], 2.0 ** -20 * softcap)
            if slopes is not None:
                bias = float(slopes[h]) * (p - j).abs().double()
                x = x - bias
                d = d + 2.0 ** -20 * (bias.abs() * seen).amax(-1)
            w = torch.softmax(x.masked_fill(~seen, float("-inf")), -1)
            out[a:b, h] = w @ v
            tol[a:b, h] = (2.0 ** -7 * out[a:b, h].abs() + (w @ v.abs()) *
                           (2.0 ** -8 + 2.0 ** -14 + 2 * d[:, None]))
    return out, tol


CAP_OPTIONS = {
    "alone": dict(),
    "bias": dict(slopes="falling"),
    "bias of either sign": dict(slopes="either"),
    "window": dict(window=150),
    "prefix": dict(prefix=True),
    "all": dict(slopes="either", window=150, prefix=True),
}
# (heads, KV heads): cached tokens, tokens: prompts and chunks, decodes of one token
# and of several, whole and split; the second in warp pairs
CAP_STEPS = {
    (8, 2): ([0, 130, 2000, 500, 9000, 20000], [300, 129, 200, 4, 2, 1],
             [250, 200, 2100, 503, 0, 20001]),
    (32, 1): ([0, 15, 99, 700, 9000, 0, 300], [1, 1, 1, 1, 1, 70, 40],
              [1, 16, 50, 0, 9001, 65, 310]),
}


def cap_options(name, hq, prefix):
    o = dict(CAP_OPTIONS[name])
    if "slopes" in o:
        o["slopes"] = (torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)])
                       if o["slopes"] == "falling" else torch.linspace(-0.05, 0.05, hq))
    if "prefix" in o:
        o["prefix"] = prefix
    return o


@pytest.mark.parametrize("name", CAP_OPTIONS)
@pytest.mark.parametrize("cap,std", [(55.45, 8.0), (55.46, 8.0), (60.0, 2.0), (60.0, 8.0),
                                     (200.0, 13.0)])
@pytest.mark.parametrize("heads", CAP_STEPS, ids=str)
def test_caps_about_and_past_the_fixed_reference(heads, cap, std, name):
    """The running reference under a cap with every other option, on every path;
    scores of a small part of the cap, and past half of it."""
    ctx, n, prefix = CAP_STEPS[heads]
    ds = DeviceStep(W.build(W.custom(ctx, n, *heads, seed=int(cap), std=std)))
    ds.write()
    check(ds, "%s, cap %g" % (name, cap), softcap=cap, **cap_options(name, heads[0], prefix))


@pytest.mark.parametrize("name", CAP_OPTIONS)
@pytest.mark.parametrize("a,b", [(96, 92), (200, 132)])    # scores about 50,000 and 149,000
@pytest.mark.parametrize("heads", CAP_STEPS, ids=str)
def test_a_cap_of_a_hundred_thousand(heads, a, b, name):
    """Scores of half of the cap and of one and a half, a few units apart: half of
    the dimensions give every key the same large product, the others a small one
    of its own, all whole numbers."""
    hq, hkv = heads
    ctx, n, prefix = CAP_STEPS[heads]
    ds = DeviceStep(W.build(W.custom(ctx, n, hq, hkv, seed=9)))
    ds.write()
    g = torch.Generator(device="cuda").manual_seed(b)
    ds.q[..., :64] = a
    ds.q[..., 64:] = (torch.randint(0, 2, ds.q[..., 64:].shape, generator=g, device="cuda") *
                      2 - 1).bfloat16()
    ds.key_cache[..., :64] = b
    ds.key_cache[..., 64:] = torch.randint(-12, 13, ds.key_cache[..., 64:].shape, generator=g,
                                           device="cuda").bfloat16()
    opt = dict(softcap=1e5, **cap_options(name, hq, prefix))
    ref, tol = definition(ds, **opt)
    ds.out.fill_(float("nan"))
    call(ds, **opt)
    assert pkv.pkv_get_error() == 0
    assert_near(ds.out[:ref.shape[0]], ref, tol, name)
