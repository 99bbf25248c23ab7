"""pkv_attention_scored on batches of more than 1024 requests: the plan's lists are
made in rounds of its 1024 threads, the second with offsets carried over from the
first.  Tolerance: that of test_gpu_scored."""
import pytest
import torch

import paged_kv_attention_05_gb300 as pkv

pytestmark = pytest.mark.gpu

D, SCALE = 128, 128 ** -0.5


def batch(reqs, hq, hkv, prompts, seed):
    """Decodes of 1 to 90 keys; every 7th request nothing, every `prompts`-th a
    prompt or a chunk of 17 to 140 rows."""
    g = torch.Generator().manual_seed(seed)
    n = torch.ones(reqs, dtype=torch.int64)
    ctx = torch.randint(0, 90, (reqs,), generator=g)
    i = torch.arange(reqs)
    pre = i % prompts == prompts - 1
    n[pre] = torch.randint(17, 141, (int(pre.sum()),), generator=g)
    n[i % 7 == 3] = 0
    return n, n + ctx


@pytest.mark.parametrize("opt", ["prefix", "window", "all"])
@pytest.mark.parametrize("reqs,hq,hkv", [(1024, 8, 2), (1025, 8, 2), (2600, 8, 2), (2100, 32, 1)])
def test_more_requests_than_plan_threads(reqs, hq, hkv, opt):
    G = hq // hkv
    n, seq = batch(reqs, hq, hkv, 20, reqs)
    rows, top = int(n.sum()), int(seq.max())
    pages = -(-top // 16)
    g = torch.Generator(device="cuda").manual_seed(reqs)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, kc, vc = rand(rows + 5, hq, D), rand(reqs * pages, 16, hkv, D), rand(reqs * pages, 16, hkv, D)
    bt = torch.randperm(reqs * pages, generator=g, device="cuda").to(torch.int32).view(reqs, pages)
    qsl = torch.zeros(reqs + 1, dtype=torch.int32)
    qsl[1:] = n.cumsum(0)
    kw, window, prefix, slopes = {}, 0, None, None
    if opt in ("prefix", "all"):
        # (each request's own: an index that is off by a round shows)
        prefix = torch.randint(0, 200, (reqs,), generator=torch.Generator().manual_seed(1))
        kw["prefix_lens"] = prefix.to(torch.int32).cuda()
    if opt in ("window", "all"):
        window = kw["window"] = 33
    if opt == "all":
        slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)])
        kw["alibi_slopes"], kw["softcap"] = slopes.cuda(), 20.0

    out = torch.full_like(q, float("nan"))
    pkv.pkv_attention_scored(q, kc, vc, qsl.cuda(), seq.to(torch.int32).cuda(), bt, reqs, SCALE,
                             out, **kw)
    assert pkv.pkv_get_error() == 0
    assert torch.isnan(out[rows:].float()).all()

    # the definition, a few hundred rows at a time
    req = torch.repeat_interleave(torch.arange(reqs), n)
    pos = torch.arange(rows) - qsl[:-1].long()[req] + (seq - n)[req]
    j = torch.arange(pages * 16, device="cuda")
    for a in range(0, rows, 512):
        b = min(a + 512, rows)
        r, p = req[a:b].cuda(), pos[a:b].cuda()[:, None]
        k = kc[bt[r].long()].view(len(r), -1, hkv, D).double()
        v = vc[bt[r].long()].view(len(r), -1, hkv, D).double()
        x = q[a:b].double().view(len(r), hkv, G, D)
        s = SCALE * torch.einsum("rghd,rkgd->rghk", x, k)
        d = 2.0 ** -16 * SCALE * torch.einsum("rghd,rkgd->rghk", x.abs(), k.abs())
        hi = p + 1
        if prefix is not None:
            hi = torch.maximum(hi, torch.minimum(prefix, seq).cuda()[r][:, None])
        seen = (j < hi) & (p - j < (window or 10 ** 6))
        seen = seen[:, None, None]
        d = (d * seen).amax(-1)
        if slopes is not None:
            s = 20.0 * torch.tanh(s / 20.0)
            bias = slopes.double().cuda().view(hkv, G)[:, :, None] * (p - j).abs()[:, None, None]
            s = s - bias
            d = d + 2.0 ** -20 * (20.0 + (bias * seen).amax(-1))
        w = torch.softmax(s.masked_fill(~seen, float("-inf")), -1)
        ref, size = (torch.einsum("rghk,rkgd->rghd", w, t).reshape(len(r), hq, D)
                     for t in (v, v.abs()))
        tol = 2.0 ** -7 * ref.abs() + size * (2.0 ** -8 + 2.0 ** -14 +
                                              2 * d.reshape(len(r), hq, 1))
        bad = ~((out[a:b].double() - ref).abs() <= tol)
        assert not bad.any(), "rows from %d: %d values off" % (a, int(bad.sum()))
