"""pkv_attention_scored on the GPU against its formula in 64 bits: cap, bias,
window, prefix and their combinations, on the decode path (every group size,
several tokens, split keys) and the prefill path (ragged tiles, chunks), with
NaN in every cache slot that no request holds.

Tolerance, per output value o, with A = sum_j softmax_j |V_j| of its row and
column: the bf16 output is off by half a step (2^-8 |o|); each probability w_j
is rounded to bf16, w_j (1 + e_j) with |e_j| <= 2^-8, before it meets V and
before it enters the sum that divides, so that to first order
  sum w_j (1 + e_j) V_j / sum w_j (1 + e_j) - o = sum w_j e_j (V_j - o),
at most 2^-8 (A + |o|) (the second order, 2^-16 A, is inside the next term); the
fp32 sums over keys are off by less than 2^-14 A; and a logit off by d changes
the average by at most 2 d A.  d: the product of 128 terms in fp32, 128 * 2^-24 times scale *
sum |q||K| (2^-16 with the scaling and the exponent's argument), plus 2^-20 of
the cap and of the largest visible bias (identities in fp32 with two
approximations of 2^-22 each)."""
import numpy as np
import pytest
import torch

import paged_kv_attention_05_gb300 as pkv
from paged_kv_attention_05_gb300 import workloads as W

pytestmark = pytest.mark.gpu

from gpu_util import DeviceStep  # noqa: E402

D = 128


def reference(ds, softcap=0.0, window=0, slopes=None, prefix=None):
    """(out, tolerance) of the first query_start_loc[-1] rows, in float64."""
    st = ds.step
    hq, hkv = st.spec.hq, st.spec.hkv
    G = hq // hkv
    n_all = int(st.query_start_loc[-1])
    out = torch.empty(n_all, hq, D, dtype=torch.float64, device="cuda")
    tol = torch.empty_like(out)
    scale = float(np.float32(st.scale))
    for r in range(st.num_reqs):
        a, b = int(st.query_start_loc[r]), int(st.query_start_loc[r + 1])
        L = int(st.seq_lens[r])
        ctx = L - (b - a)
        if a == b:
            continue
        j = torch.arange(max(0, ctx - window + 1) if window else 0, L, device="cuda")
        p = torch.arange(ctx, L, device="cuda")[:, None]
        seen = j[None] <= p
        if prefix is not None:
            seen = seen | (j[None] < int(prefix[r]))
        if window:
            seen = seen & (j[None] > p - window)
        blk = ds.block_table[r].long()[j // 16]
        dist = (p - j[None]).abs().double()
        for g in range(hkv):
            k, v = ds.key_cache[blk, j % 16, g].double(), ds.value_cache[blk, j % 16, g].double()
            q = ds.q[a:b, g * G:(g + 1) * G].double().transpose(0, 1)
            s = scale * (q @ k.T)
            d = 2.0 ** -16 * scale * (q.abs() @ k.abs().T).where(seen, torch.zeros(()).cuda().double()).amax(-1)
            if softcap:
                s = softcap * torch.tanh(s / softcap)
                d = d + 2.0 ** -20 * softcap
            if slopes is not None:
                bias = slopes[g * G:(g + 1) * G].double().cuda()[:, None, None] * dist
                s = s - bias
                d = d + 2.0 ** -20 * (bias.abs() * seen).amax(-1)
            s = s.masked_fill(~seen, float("-inf"))
            w = torch.softmax(s, -1)
            o, A = w @ v, w @ v.abs()
            out[a:b, g * G:(g + 1) * G] = o.transpose(0, 1)
            tol[a:b, g * G:(g + 1) * G] = (2.0 ** -7 * o.abs() + A *
                                           (2.0 ** -8 + 2.0 ** -14 + 2 * d[..., None])).transpose(0, 1)
    return out, tol


def call(ds, out=None, softcap=0.0, window=0, slopes=None, prefix=None, **kw):
    pkv.pkv_attention_scored(
        ds.q, ds.key_cache, ds.value_cache, ds.qsl, ds.seq_lens, ds.block_table, ds.step.num_reqs,
        ds.step.scale, ds.out if out is None else out, softcap=softcap, window=window,
        alibi_slopes=None if slopes is None else slopes.float().cuda(),
        prefix_lens=None if prefix is None else torch.tensor(prefix, dtype=torch.int32).cuda(),
        **kw)


def assert_near(got, ref, tol, what=""):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    if bad.any():
        at = bad.nonzero()[0].tolist()
        raise AssertionError("%s: %d of %d values outside the tolerance, first at %s: %g for %g "
                             "(tolerance %g)" % (what, int(bad.sum()), bad.numel(), at,
                                                 float(got[tuple(at)]), float(ref[tuple(at)]),
                                                 float(tol[tuple(at)])))


def run_and_check(step, what="", pre=None, **opt):
    ds = step if isinstance(step, DeviceStep) else DeviceStep(step)
    if not isinstance(step, DeviceStep):
        ds.write()
    ref, tol = reference(ds, **opt)
    if pre:
        pre(ds)
    call(ds, **opt)
    assert pkv.pkv_get_error() == 0
    n = ref.shape[0]
    assert_near(ds.out[:n], ref, tol, what)
    assert torch.isnan(ds.out[n:].float()).all(), "rows past the last request must not be written"
    return ds


def slopes_for(hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)])


OPTIONS = {
    "off": dict(),
    "cap": dict(softcap=30.0),
    "bias": dict(slopes=True),
    "window": dict(window=100),
    "prefix": dict(prefix=True),
    "cap+bias": dict(softcap=20.0, slopes=True),
    "cap+window": dict(softcap=50.0, window=37),
    "bias+window": dict(slopes=True, window=200),
    "cap+bias+window+prefix": dict(softcap=15.0, slopes=True, window=150, prefix=True),
}


def options(name, hq, reqs, prefix=90):
    o = dict(OPTIONS[name])
    if o.get("slopes"):
        o["slopes"] = slopes_for(hq)
    if o.get("prefix"):
        o["prefix"] = [prefix + 7 * r for r in range(reqs)]
    return o


@pytest.mark.parametrize("name", OPTIONS)
@pytest.mark.parametrize("hq,hkv", [(8, 8), (8, 2), (16, 1), (32, 1), (24, 1)])
def test_decode(hq, hkv, name):
    """Single-token decodes of 1 to 700 keys, page edges among them."""
    ctx = [0, 1, 14, 15, 16, 99, 100, 101, 255, 699]
    run_and_check(W.build(W.custom(ctx, [1] * 10, hq, hkv, seed=hq + hkv, std=1.5, pad_tokens=2)),
                  name, **options(name, hq, 10))


@pytest.mark.parametrize("name", OPTIONS)
def test_prefill(name):
    """Prompts and chunks of ragged lengths through the tensor-core path."""
    ctx, n = [0, 0, 0, 130, 1000, 37], [17, 128, 300, 129, 200, 530]
    run_and_check(W.build(W.custom(ctx, n, 8, 2, seed=5, std=1.5, pad_tokens=3)), name,
                  **options(name, 8, 6, prefix=150))


@pytest.mark.parametrize("name", OPTIONS)
def test_mixed_step_odd_group(name):
    """Decodes, several-token decodes and chunks together, three heads a group."""
    ctx, n = [540, 0, 129, 700, 0, 61], [1, 298, 1, 3, 70, 5]
    run_and_check(W.build(W.custom(ctx, n, 12, 4, seed=6, pad_tokens=4)), name,
                  **options(name, 12, 6, prefix=200))


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 127, 128, 129, 300, 2 ** 31 - 1])
@pytest.mark.parametrize("group", [1, 4, 32])
def test_windows(window, group):
    """Windows of one key to more than the sequence, at page and tile edges;
    the pages before each request's window hold NaN, their table entries
    garbage that must not be read."""
    ctx, n = [0, 299, 1000, 40, 300, 0], [1, 1, 1, 1, 257, 400]
    hkv = 1 if group == 32 else 2
    step = W.build(W.custom(ctx, n, group * hkv, hkv, seed=window % 97, std=1.5))

    def free_pages(ds):
        for r, (c, _) in enumerate(zip(ctx, n)):
            gone = max(0, c - window + 1) // 16
            for b in range(gone):
                blk = int(ds.block_table[r, b])
                ds.key_cache[blk] = float("nan")
                ds.value_cache[blk] = float("nan")
                ds.block_table[r, b] = (-1, 10 ** 9, -10 ** 9)[b % 3]
            first = max(0, c - window + 1)
            if first % 16:   # the keys before the window in its first page
                blk = int(ds.block_table[r, first // 16])
                ds.key_cache[blk, :first % 16] = float("nan")
                ds.value_cache[blk, :first % 16] = float("inf")

    run_and_check(step, "window %d" % window, pre=free_pages, window=window)


@pytest.mark.parametrize("softcap,std", [(0.25, 3.0), (5.0, 6.0), (30.0, 3.0), (50.0, 8.0),
                                         (1e3, 3.0), (1e6, 1.0), (1e30, 1.0), (1e-20, 1.0)])
def test_caps_and_logit_sizes(softcap, std):
    """From caps that flatten every score to caps far above them; logits of a
    few units to a few hundred."""
    ctx, n = [0, 300, 500, 64], [200, 130, 1, 2]
    # (an identity through 1 - 2 / (1 + e^2x) keeps 2^-22 of the cap; a cap far
    # above the logits keeps the logits' own precision, which the bound asks for)
    step = W.build(W.custom(ctx, n, 8, 2, seed=11, std=std))
    ds = DeviceStep(step)
    ds.write()
    ref, tol = reference(ds, softcap=min(softcap, 1e12))
    if softcap > 1e4:    # the bound for the uncapped logits alone
        _, tol = reference(ds)
    call(ds, softcap=softcap)
    assert pkv.pkv_get_error() == 0
    assert_near(ds.out[:ref.shape[0]], ref, tol, "cap %g" % softcap)


@pytest.mark.parametrize("kind", ["steep", "zero", "negative", "mixed"])
def test_slopes(kind):
    s = {"steep": torch.full((8,), 8.0), "zero": torch.zeros(8),
         "negative": -slopes_for(8) * 0.05,
         "mixed": torch.tensor([4.0, 0.0, -0.01, 0.5, 0.001, 2.0, 0.0625, 1.0])}[kind]
    ctx, n = [0, 700, 1500, 3], [300, 150, 1, 1]
    run_and_check(W.build(W.custom(ctx, n, 8, 2, seed=21)), kind, slopes=s)


@pytest.mark.parametrize("hq,hkv", [(8, 2), (32, 1)])
def test_slopes_of_either_sign_under_a_cap(hq, hkv):
    """The fixed reference covers a bias that grows with distance: long rows,
    prefixes up to the largest integer, windows, steep slopes of both signs."""
    slopes = torch.linspace(-0.5, 0.5, hq)
    for pre, window in ((None, 0), ([2 ** 31 - 1, 5, 2 ** 31 - 1, 700, 0], 0), (None, 90)):
        ctx, n = [900, 300, 0, 200, 3000], [1, 1, 150, 140, 1]
        run_and_check(W.build(W.custom(ctx, n, hq, hkv, seed=22)), "prefix %s" % pre,
                      softcap=20.0, slopes=slopes, prefix=pre, window=window)


def test_prefixes():
    """No prefix, negative, a part, the whole request, more than it: prompts,
    a chunk whose prefix runs past it, and decodes."""
    ctx, n = [0, 0, 0, 100, 0, 50, 20], [200, 200, 200, 300, 129, 1, 3]
    pre = [0, -5, 77, 350, 10 ** 9, 40, 2 ** 31 - 1]
    run_and_check(W.build(W.custom(ctx, n, 8, 2, seed=31)), "prefixes", prefix=pre)
    run_and_check(W.build(W.custom(ctx, n, 8, 2, seed=32)), "prefixes, window", prefix=pre,
                  window=60)


def test_long_decodes_are_split_and_merged():
    for hq, hkv, opt in ((8, 2, dict(softcap=30.0)), (8, 2, dict(window=5000)),
                         (32, 1, dict(softcap=30.0, window=9001)),
                         (8, 8, dict(slopes=slopes_for(8)))):
        run_and_check(W.build(W.custom([20000, 777, 12345], [1, 1, 1], hq, hkv, seed=41)),
                      str(opt.keys()), **opt)


@pytest.mark.parametrize("opt", [dict(window=4), dict(window=40, prefix=[3, 500, 20]),
                                 dict(softcap=10.0, window=700), dict(slopes=slopes_for(4))])
def test_several_token_decodes(opt):
    """Up to 16 query rows a unit, so that a row's window starts after the
    unit's first page, and in a split without a key of the row."""
    for hq, hkv in ((4, 4), (4, 1)):
        run_and_check(W.build(W.custom([500, 90, 3000], [4, 2, 4], hq, hkv, seed=51)), "tokens",
                      **opt)


def test_masked_keys_of_any_kind():
    """K of masked keys (causal future, before a row's window) may be NaN or
    infinite, whether or not another row of the tile sees them."""
    step = W.build(W.custom([0, 64], [150, 40], 4, 2, seed=61))
    ds = DeviceStep(step)
    ds.write()
    ref, tol = reference(ds, window=30)
    blk = int(ds.block_table[0, 60 // 16])
    ds.key_cache[blk, 60 % 16] = float("nan")      # rows 60..89 of request 0 see it
    ds.key_cache[int(ds.block_table[0, 100 // 16]), 100 % 16] = float("inf")
    call(ds, window=30)
    assert pkv.pkv_get_error() == 0
    clean = [i for i in range(190) if i >= 150 or not (60 <= i < 90 or 100 <= i < 130)]
    assert_near(ds.out[clean], ref[clean], tol[clean], "rows that do not see the key")


def test_queries_beyond_the_request_may_hold_anything():
    """Rows behind the last sequence hold NaN; they are neither read into a
    result nor written."""
    step = W.build(W.custom([0, 300], [130, 100], 8, 2, seed=71, pad_tokens=40))
    ds = DeviceStep(step)
    ds.write()
    ds.q[230:] = float("nan")
    for opt in (dict(softcap=20.0), dict(window=50), dict(slopes=slopes_for(8))):
        ds.out.fill_(float("nan"))
        run_and_check(ds, "NaN behind", **opt)


def test_bad_requests_are_skipped_and_reported():
    """A bad length, a table row too short and a bad block id: reported, the
    other requests' rows as they should be."""
    ctx, n = [100, 50, 200, 0], [1, 40, 1, 33]
    step = W.build(W.custom(ctx, n, 8, 2, seed=81))
    ds = DeviceStep(step)
    ds.write()
    ref, tol = reference(ds, softcap=30.0, window=64)
    ds.seq_lens[1] = 20                        # below its query length
    ds.block_table[2, 200 // 16] = 10 ** 6     # outside the pool
    call(ds, softcap=30.0, window=64)
    assert pkv.pkv_get_error() == (pkv.DEV_ERR_BITS["SEQ_LEN"] | pkv.DEV_ERR_BITS["BLOCK_ID"])
    keep = [0] + list(range(42, 75))
    assert_near(ds.out[keep], ref[keep], tol[keep], "the other requests")
    assert torch.isnan(ds.out[1:41].float()).all()


def test_without_options_it_is_plain_attention():
    step = W.build(W.custom([0, 700, 33, 1500], [300, 1, 130, 1], 16, 4, seed=91))
    ds = DeviceStep(step)
    ds.write()
    ds.attention()
    plain = ds.out.clone()
    _, tol = reference(ds)
    call(ds)
    assert pkv.pkv_get_error() == 0
    n = tol.shape[0]
    assert_near(ds.out[:n], plain[:n].double(), 2 * tol, "plain")


def test_a_scored_plan_serves_no_planned_call():
    step = W.build(W.custom([100], [1], 8, 2, seed=92))
    ds = DeviceStep(step)
    ds.write()
    pkv.pkv_plan(1, 8, 2, ds.qsl, ds.seq_lens, ds.block_table.shape[1], 1)
    call(ds, window=16)
    with pytest.raises(pkv.PkvError):
        pkv.pkv_attention_planned(ds.q, ds.key_cache, ds.value_cache, ds.block_table,
                                  step.scale, ds.out)
    ds.attention()    # and the plain call plans for itself
    assert pkv.pkv_get_error() == 0


def test_refusals():
    step = W.build(W.custom([100, 5], [1, 2], 8, 2, seed=93))
    ds = DeviceStep(step)
    f = lambda **kw: pkv.pkv_attention_scored(**dict(dict(  # noqa: E731
        q=ds.q, key_cache=ds.key_cache, value_cache=ds.value_cache, query_start_loc=ds.qsl,
        seq_lens=ds.seq_lens, block_table=ds.block_table, num_reqs=2, scale=0.1, out=ds.out), **kw))
    for bad in (dict(alibi_slopes=torch.ones(7, device="cuda")),
                dict(alibi_slopes=torch.ones(0, device="cuda")),
                dict(alibi_slopes=torch.ones(16, device="cuda")[::2]),
                dict(prefix_lens=torch.ones(1, dtype=torch.int32, device="cuda")),
                dict(alibi_slopes=torch.ones(8)), dict(window=2 ** 31), dict(num_reqs=3),
                dict(out=ds.out[:2]), dict(out=ds.out[:, :4]), dict(q=ds.q[0]),
                dict(block_table=ds.block_table[0]), dict(value_cache=ds.value_cache[:2])):
        with pytest.raises(ValueError):
            f(**bad)
    for bad in (dict(alibi_slopes=torch.ones(8, device="cuda").double()), dict(q=ds.q.half()),
                dict(prefix_lens=torch.ones(2, device="cuda")),
                dict(seq_lens=ds.seq_lens.long())):
        with pytest.raises(TypeError):
            f(**bad)
    for bad in (dict(window=-1), dict(softcap=-1.0), dict(softcap=float("nan")), dict(scale=0.0)):
        with pytest.raises(pkv.PkvError) as e:
            f(**bad)
        assert e.value.code == -1
    torch.cuda.synchronize()
    assert torch.isnan(ds.out.float()).all() and pkv.pkv_get_error() == 0


def test_tensors_of_another_device_are_refused(monkeypatch):
    """With another device current (made up: the tests have one), the call's
    tensors are not on it, and nothing is enqueued."""
    from paged_kv_attention_05_gb300 import _binding
    ds = DeviceStep(W.build(W.custom([10], [1], 4, 2, seed=94)))
    call(ds)
    torch.cuda.synchronize()
    launches = pkv.pkv_launch_count()
    monkeypatch.setattr(_binding, "_get_device", lambda: 1)
    with pytest.raises(ValueError, match="cuda:0.*current device is cuda:1"):
        call(ds)
    with pytest.raises(ValueError, match="cuda:0.*current device is cuda:1"):
        pkv.pkv_write_rope(ds.q, ds.k, ds.v, ds.slot_mapping, torch.zeros(20, 128, device="cuda"),
                           ds.key_cache, ds.value_cache, ds.slot_mapping, ds.q)
    assert pkv.pkv_launch_count() == launches


def test_another_stream_and_a_replayed_graph():
    """Captured after a reservation, replayed on changed inputs."""
    ctx, n = [0, 700, 3000, 61], [200, 1, 1, 4]
    step = W.build(W.custom(ctx, n, 8, 2, seed=95))
    ds = DeviceStep(step)
    ds.write()
    opt = dict(softcap=30.0, window=500, slopes=slopes_for(8), prefix=[50, 0, 0, 0])
    slopes, prefix = opt["slopes"].cuda(), torch.tensor(opt["prefix"], dtype=torch.int32).cuda()
    pkv.pkv_reserve_workspace(4, ds.q.shape[0], ds.block_table.shape[1], 8, 2)
    go = lambda stream=None: pkv.pkv_attention_scored(  # noqa: E731
        ds.q, ds.key_cache, ds.value_cache, ds.qsl, ds.seq_lens, ds.block_table, 4, step.scale,
        ds.out, softcap=30.0, window=500, alibi_slopes=slopes, prefix_lens=prefix, stream=stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    go(side)
    side.synchronize()
    ref, tol = reference(ds, **opt)
    assert_near(ds.out[:206], ref, tol, "side stream")
    first = ds.out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    ds.out.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(ds.out[:206], first[:206])
    ds.q.mul_(-0.5)
    prefix.fill_(120)
    opt["prefix"] = [120] * 4
    ref, tol = reference(ds, **opt)
    g.replay()
    torch.cuda.synchronize()
    assert pkv.pkv_get_error() == 0
    assert_near(ds.out[:206], ref, tol, "replayed")


def test_calls_back_to_back_without_a_wait():
    """Each call's plan starts while the one before still runs; different steps
    (decodes that are split and merged, prompts, both), the cache write, the
    plain call and metadata changed by ordinary kernels in between, enqueued
    without a synchronisation, give the bits that they give alone."""
    specs = [([20000, 300], [1, 1]), ([0, 129, 540], [298, 1, 1]), ([40], [1]),
             ([0, 700], [400, 130])]
    steps = [DeviceStep(W.build(W.custom(c, n, 8, 2, seed=100 + i)))
             for i, (c, n) in enumerate(specs)]
    alone = []
    for ds in steps:
        ds.write()
        call(ds, softcap=30.0)
        torch.cuda.synchronize()
        alone.append(ds.out.clone())
    torch.cuda.synchronize()
    got = []
    for turn in range(40):
        ds = steps[turn % 4]
        if turn % 3 == 1:
            ds.write()
        if turn % 5 == 2:
            ds.attention()
        if turn % 7 == 3:      # the lengths are gone and come back, in stream order
            keep = ds.seq_lens.clone()
            ds.seq_lens.zero_()
            ds.seq_lens.copy_(keep)
        call(ds, softcap=30.0)
        if turn % 4 == 1:
            call(ds, softcap=30.0)
        got.append(ds.out.clone())
    assert pkv.pkv_get_error() == 0
    for turn, out in enumerate(got):
        n = int(steps[turn % 4].step.query_start_loc[-1])
        assert torch.equal(out[:n], alone[turn % 4][:n]), "turn %d" % turn


def test_a_graph_outlives_a_larger_workspace():
    """A graph captured on one workspace is replayed after a later call needed a
    larger one: the old one is still there, and the results are the graph's."""
    ds = DeviceStep(W.build(W.custom([700, 0], [1, 200], 8, 2, seed=98)))
    ds.write()
    ref, tol = reference(ds, softcap=30.0)
    call(ds, softcap=30.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(ds, softcap=30.0)
    size = lambda r: pkv.pkv_workspace_size(r, 4096, 2048, 32, 8, pkv.pkv_num_sms())["bytes"]  # noqa: E731
    reqs = 64
    while size(reqs) < 1 << 28:
        reqs *= 2
    pkv.pkv_reserve_workspace(reqs, 4096, 2048, 32, 8)
    filler = torch.full((1 << 28,), 255, dtype=torch.uint8, device="cuda")  # takes freed memory
    ds.out.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    assert pkv.pkv_get_error() == 0
    assert_near(ds.out[:201], ref, tol, "replayed")
    assert int(filler.min()) == 255
    call(ds, softcap=30.0)
    assert_near(ds.out[:201], ref, tol, "on the larger workspace")


def test_the_same_bits_every_time():
    ctx, n = [0, 700, 3000, 61], [300, 1, 1, 4]
    ds = DeviceStep(W.build(W.custom(ctx, n, 8, 2, seed=96)))
    ds.write()
    outs = []
    for _ in range(3):
        call(ds, softcap=30.0, slopes=slopes_for(8))
        outs.append(ds.out[:306].clone())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_layers_of_a_step_together():
    """Rotated write, then attention, layer by layer as a model alternates
    them: a window with a cap, the whole length with a cap, plain."""
    step = W.build(W.custom([540, 129, 0], [1, 1, 298], 16, 4, seed=97, pad_tokens=4))
    pos = torch.full((304,), -1, dtype=torch.int64)
    for r in range(3):
        a, b = int(step.query_start_loc[r]), int(step.query_start_loc[r + 1])
        pos[a:b] = torch.arange(int(step.seq_lens[r]) - (b - a), int(step.seq_lens[r]))
    pos = pos.cuda()
    inv = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    ang = torch.arange(600, dtype=torch.float64)[:, None] * inv
    tab = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    w = torch.full((D,), 1.25, dtype=torch.bfloat16, device="cuda")
    layers = [DeviceStep(step) for _ in range(3)]
    opts = [dict(softcap=50.0, window=128), dict(softcap=50.0), dict()]
    for ds, opt in zip(layers, opts):     # enqueued back to back, no synchronisation
        pkv.pkv_write_rope(ds.q, ds.k, ds.v, pos, tab, ds.key_cache, ds.value_cache,
                           ds.slot_mapping, ds.q, q_weight=w, k_weight=w)
        if opt:
            call(ds, **opt)
        else:
            ds.attention()
    assert pkv.pkv_get_error() == 0
    for ds, opt in zip(layers, opts):
        ref, tol = reference(ds, **opt)
        assert_near(ds.out[:300], ref, tol, str(opt))
        assert torch.isnan(ds.out[300:].float()).all()


def test_the_call_of_plain_arguments():
    """pkv_attention_scored itself (the binding passes a struct): the same bits,
    with all four options and a row stride of its own for out."""
    from paged_kv_attention_05_gb300 import _binding
    ds = DeviceStep(W.build(W.custom([300, 0, 77, 500], [1, 140, 3, 1], 8, 2, seed=12)))
    ds.write()
    opt = dict(softcap=20.0, window=90, slopes=slopes_for(8), prefix=[10, 100, 0, 501])
    call(ds, **opt)
    n = int(ds.step.query_start_loc[-1])
    sl = opt["slopes"].cuda()
    px = torch.tensor(opt["prefix"], dtype=torch.int32).cuda()
    wide = torch.full((ds.out.shape[0], 9, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    t = [x.data_ptr() for x in (ds.q, ds.key_cache, ds.value_cache, ds.qsl, ds.seq_lens,
                                ds.block_table, sl, px, wide)]
    rc = _binding.load().pkv_attention_scored(
        t[0], ds.q.stride(0), ds.q.shape[0], 8, t[1], t[2], ds.key_cache.shape[0], 16, 2, D, t[3],
        t[4], t[5], ds.block_table.shape[1], ds.step.num_reqs, ds.step.scale, 20.0, 90, t[6], t[7],
        t[8], wide.stride(0), torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and pkv.pkv_get_error() == 0
    assert torch.isnan(wide[:, 8].float()).all()
    assert torch.equal(wide[:n, :8].contiguous().view(torch.int16), ds.out[:n].view(torch.int16))


@pytest.mark.parametrize("name", ["off", "cap", "cap+bias+window+prefix"])
@pytest.mark.parametrize("hq,hkv", [(16, 8), (32, 1), (9, 3)])
def test_long_decodes_beside_a_short_prompt(hq, hkv, name):
    """Many keys to decode and few to prefill: the SMs left to the prefill are a
    few, which take several items each."""
    n_dec = 24 * 8 // hkv if hkv > 1 else 40
    ctx = [4000 + 3 * i for i in range(n_dec)] + [0, 60]
    run_and_check(W.build(W.custom(ctx, [1] * n_dec + [300, 130], hq, hkv, seed=hq)), name,
                  **options(name, hq, n_dec + 2, prefix=250))
