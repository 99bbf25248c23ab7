"""The page calls as a step makes them: reservations of exact sizes before a capture, two
graphs over one workspace, prompts, lists of one width used for another."""
import os
import subprocess
import sys

import pytest
import torch

import paged_kv_attention_05_gb300 as pkv

pytestmark = pytest.mark.gpu

import test_gpu_pages as P  # noqa: E402

HERE = os.path.dirname(os.path.abspath(__file__))

SCRIPT = r"""
import sys
sys.path[:0] = [%(root)r, %(here)r]
import torch
import paged_kv_attention_05_gb300 as pkv
import test_gpu_pages as P

ctx, hq, hkv = eval(sys.argv[1])
steps = [P.Decode(ctx, 1, hq, hkv, 64, 3), P.Decode(ctx[:1], 1, hq, hkv, 64, 4)]
d = steps[0]
pkv.pkv_reserve_workspace(d.rows + 2, d.rows + 2, 64, hq, hkv)
pkv.pkv_reserve_select(d.rows + 2, d.bt.shape[1], hkv)
graphs = []
for s in steps:
    s.next()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.step()
    graphs.append(g)
for turn in range(4):
    for s, g in zip(steps, graphs):
        g.replay()
    torch.cuda.synchronize()
    for s in steps:
        s.check()
        s.next()
assert pkv.pkv_get_error() == 0
print("as it should be")
"""


@pytest.mark.parametrize("case", ["([33000], 32, 8)", "([5000] * 9, 16, 1)", "([700, 3, 9000], 8, 8)"])
def test_two_graphs_on_reservations_of_exact_sizes(case):
    r = subprocess.run([sys.executable, "-c",
                        SCRIPT % {"root": os.path.dirname(HERE), "here": HERE}, case],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "as it should be" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("hq,hkv", [(8, 2), (16, 1)])
def test_rows_of_prompts(hq, hkv):
    """Rows of prompts choose and attend each for itself, whatever their request's length."""
    g = P.gen(hq)
    reqs = [(0, 257), (1000, 65), (4000, 1), (0, 1), (37, 0)]
    bt, qsl, seq, slots, nb = P.metadata(reqs, g, extra_width=3)
    kc, vc = P.randn((nb, 16, hkv, P.D), g), P.randn((nb, 16, hkv, P.D), g)
    every = torch.cat([bt[r, torch.arange(c + n, device="cuda") // 16].long() * 16 +
                       torch.arange(c + n, device="cuda") % 16 for r, (c, n) in enumerate(reqs)])
    bounds = torch.zeros((nb, hkv, 2, P.D), dtype=torch.bfloat16, device="cuda")
    pkv.pkv_page_bounds(kc, bounds, every)
    rows = sum(n for _, n in reqs)
    q = P.randn((rows, hq, P.D), g)
    table = torch.full((rows, hkv, 20), -5, dtype=torch.int32, device="cuda")
    lens = torch.full((rows,), -5, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, float("nan"))
    pkv.pkv_select_pages(q, bounds, qsl, seq, bt, len(reqs), table, lens, 1, 3)
    pkv.pkv_attention_selected(q, kc, vc, table, lens, P.D ** -0.5, out)
    assert pkv.pkv_get_error() == 0
    want, wlens = P.select_ref(q, bounds, reqs, bt, 20, 1, 3)
    assert torch.equal(table, want) and torch.equal(lens, wlens)
    P.close(out, P.attention_ref(q, kc, vc, want, wlens, P.D ** -0.5))


def list_bound(q, kc, vc, table, lens, scale):
    """Attention over the lists in 64 bits and what the kernel may be off by: the output's
    rounding to bf16 (2^-8), that of each weight (2^-8 of its share, in the sum of the values
    and, once more, where the row is divided by the weights' sum), and logits formed in
    fp32, each within 2^-17 of the sizes that cancel in them (128 products and the MMA's own
    sums), where they turn a weight by that much; references and sums 2^-18 of the shares."""
    rows, hq, _ = q.shape
    hkv = kc.shape[2]
    G = hq // hkv
    out = torch.zeros(rows, hq, P.D, dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(out)
    for t in range(rows):
        L = int(lens[t])
        for g in range(hkv):
            ids = table[t, g, :-(-L // 16)].long()
            k = kc[ids, :, g].double().reshape(-1, P.D)[:L]
            v = vc[ids, :, g].double().reshape(-1, P.D)[:L]
            qd = q[t, g * G:(g + 1) * G].double()
            p = torch.softmax(qd @ k.T * scale, -1)
            dx = 2.0 ** -17 * abs(scale) * (qd.abs() @ k.abs().T)
            o, av = p @ v, p @ v.abs()
            turn = (p * dx) @ v.abs() + (p * dx).sum(-1, keepdim=True) * av
            out[t, g * G:(g + 1) * G] = o
            bound[t, g * G:(g + 1) * G] = 2.0 ** -8 * o.abs() + \
                1.01 * (2.0 ** -8 * (av + o.abs()) + 1.1 * turn) + 2.0 ** -18 * av
    return out, bound


@pytest.mark.parametrize("std,qstd", [(1.0, 1.0), (1.0, 6.0), (0.02, 1.0), (30.0, 0.1)])
@pytest.mark.parametrize("hq,hkv", [(8, 8), (32, 8), (16, 1), (32, 1), (9, 3)])
def test_attention_over_lists_within_its_roundings(hq, hkv, std, qstd):
    g = P.gen(hq + hkv)
    nb, width = 300, 160
    lens = torch.tensor([1, 15, 16, 17, 300, 160 * 16, 33, 1000], dtype=torch.int32, device="cuda")
    rows = len(lens)
    kc, vc = P.randn((nb, 16, hkv, P.D), g, std), P.randn((nb, 16, hkv, P.D), g, std)
    table = torch.stack([torch.stack([torch.randperm(nb, generator=g, device="cuda")[:width]
                                      for _ in range(hkv)]) for _ in range(rows)]).int()
    q = P.randn((rows, hq, P.D), g, qstd)
    out = torch.full_like(q, float("nan"))
    pkv.pkv_attention_selected(q, kc, vc, table, lens, P.D ** -0.5, out)
    assert pkv.pkv_get_error() == 0
    ref, bound = list_bound(q, kc, vc, table, lens, P.D ** -0.5)
    err = (out.double() - ref).abs()
    assert bool((err <= bound).all()), "error up to %g of the bound" % float((err / bound).max())
