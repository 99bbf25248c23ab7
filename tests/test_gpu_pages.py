"""Page bounds, the selection of pages, and attention over selected pages on the
GPU, against plain 64-bit forms: bounds and lists have to be equal, outputs within
the tolerance of the other attention tests."""
import pytest
import torch

import paged_kv_attention_05_gb300 as pkv

pytestmark = pytest.mark.gpu

from gpu_util import ATOL, RTOL  # noqa: E402

BITS = pkv.DEV_ERR_BITS
D, BS = 128, 16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(shape, g, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def metadata(reqs, g, extra_width=0, spare=3):
    """Block table (random pages), query_start_loc, seq_lens, slots of the
    scheduled tokens, and the pool's size."""
    seq = [c + n for c, n in reqs]
    used = [-(-s // BS) for s in seq]
    nb = sum(used) + spare
    perm = torch.randperm(nb, generator=g, device="cuda")
    bt = torch.full((len(reqs), max(max(used), 1) + extra_width), -1, dtype=torch.int32,
                    device="cuda")
    at, slots = 0, []
    for r, u in enumerate(used):
        bt[r, :u] = perm[at:at + u].int()
        at += u
        p = torch.arange(reqs[r][0], seq[r], device="cuda")
        slots.append(bt[r, p // BS].long() * BS + p % BS)
    qsl = torch.tensor([0] + [n for _, n in reqs], device="cuda").cumsum(0).int()
    return bt, qsl, torch.tensor(seq, dtype=torch.int32, device="cuda"), torch.cat(slots), nb


# ------------------------------------------------------------------- bounds

@pytest.mark.parametrize("hkv", [1, 3, 8, 32])
@pytest.mark.parametrize("reqs", [[(c, 1) for c in (0, 1, 14, 15, 16, 31, 32, 100)],
                                  [(0, 5), (3, 40), (15, 1), (16, 200), (100, 17), (0, 16)],
                                  [(i % 37, 1 + i % 3) for i in range(400)],
                                  [(0, 6000), (7, 5001)]])
def test_bounds(hkv, reqs):
    g = gen(hkv + len(reqs))
    bt, qsl, seq, slots, nb = metadata(reqs, g)
    kc = randn((nb, BS, hkv, D), g)
    for r, (c, n) in enumerate(reqs):         # slots behind the last token: NaN
        if (c + n) % BS and n:
            kc[bt[r, (c + n) // BS], (c + n) % BS:] = float("nan")
    bounds = torch.full((nb, hkv, 2, D), 777.0, dtype=torch.bfloat16, device="cuda")
    want = bounds.clone()
    for r, (c, n) in enumerate(reqs):
        for j in range(c // BS, (c + n - 1) // BS + 1 if n else 0):
            k = kc[bt[r, j], :min(BS, c + n - j * BS)].float()
            want[bt[r, j], :, 0], want[bt[r, j], :, 1] = k.amin(0), k.amax(0)
    padded = torch.cat([slots, slots.new_full((5,), -1)])
    pkv.pkv_page_bounds(kc, bounds, padded)
    assert pkv.pkv_get_error() == 0
    assert torch.equal(bounds, want)


def test_bounds_padding_between_and_slots_past_the_pool():
    g = gen(4)
    kc = randn((5, BS, 2, D), g)
    bounds = torch.zeros((5, 2, 2, D), dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([0, 1, -1, 2 * BS + 5, 5 * BS, -7, 3 * BS + 15, 1 << 40], device="cuda")
    pkv.pkv_page_bounds(kc, bounds, slots)
    assert pkv.pkv_get_error() == BITS["SLOT_RANGE"]
    for blk, last in ((0, 1), (2, 5), (3, 15)):
        k = kc[blk, :last + 1].float()
        assert torch.equal(bounds[blk, :, 0].float(), k.amin(0))
        assert torch.equal(bounds[blk, :, 1].float(), k.amax(0))
    assert not bool(bounds[1].any()) and not bool(bounds[4].any())


# ---------------------------------------------------------------- selection

def select_ref(q, bounds, reqs, bt, budget, first, last):
    rows, hq, _ = q.shape
    hkv = bounds.shape[1]
    G = hq // hkv
    table = torch.full((rows, hkv, budget), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    at = 0
    for r, (c, n) in enumerate(reqs):
        for p in range(c, c + n):
            pages = p // BS + 1
            ids = bt[r, :pages]
            lens[at] = (min(pages, budget) - 1) * BS + p % BS + 1
            b = bounds[ids.long()].double()
            qd = q[at].double().view(hkv, G, D)
            score = (qd.clamp(min=0).sum(1)[:, None] * b[:, :, 1].transpose(0, 1) +
                     qd.clamp(max=0).sum(1)[:, None] * b[:, :, 0].transpose(0, 1)).sum(-1)
            for g in range(hkv):
                if pages <= budget:
                    keep = list(range(pages))
                else:
                    s = score[g].tolist()
                    mid = sorted(range(first, pages - last), key=lambda j: (-s[j], j))
                    keep = sorted(list(range(first)) + mid[:budget - first - last] +
                                  list(range(pages - last, pages)))
                table[at, g, :len(keep)] = ids[keep]
            at += 1
    return table, lens


def run_select(q, bounds, reqs, bt, qsl, seq, budget, first, last):
    rows, hkv = q.shape[0], bounds.shape[1]
    table = torch.full((rows, hkv, budget), -5, dtype=torch.int32, device="cuda")
    lens = torch.full((rows,), -5, dtype=torch.int32, device="cuda")
    pkv.pkv_select_pages(q, bounds, qsl, seq, bt, len(reqs), table, lens, first, last)
    return table, lens


def check_select(q, bounds, reqs, bt, qsl, seq, budget, first=0, last=1):
    table, lens = run_select(q, bounds, reqs, bt, qsl, seq, budget, first, last)
    want, wlens = select_ref(q, bounds, reqs, bt, budget, first, last)
    n = sum(m for _, m in reqs)
    assert torch.equal(lens, wlens)
    assert torch.equal(table[:n], want[:n]), \
        "%d of %d entries differ" % (int((table[:n] != want[:n]).sum()), want[:n].numel())
    assert bool((table[n:] == -5).all()), "lists behind the last request written"


REQS = [(700, 1), (0, 1), (5, 3), (16 * 40 - 1, 1), (16 * 40, 1), (3000, 2), (255, 1), (256, 1),
        (10000, 1)]


def a_case(hq, hkv, reqs, seed, std=1.0):
    g = gen(seed)
    bt, qsl, seq, _, nb = metadata(reqs, g, extra_width=2)
    lo = randn((nb, hkv, D), g, std)
    bounds = torch.stack([lo, lo + randn((nb, hkv, D), g, std).abs()], 2).contiguous()
    rows = sum(n for _, n in reqs) + 2
    q = randn((rows, (hq + 1) * D), g)[:, :hq * D].view(rows, hq, D)
    return q, bounds, reqs, bt, qsl, seq


@pytest.mark.parametrize("hq,hkv", [(8, 8), (32, 8), (32, 1), (24, 2), (9, 3), (64, 8)])
@pytest.mark.parametrize("budget,first,last", [(16, 0, 1), (40, 1, 2), (1, 0, 1), (3, 1, 2),
                                               (200, 4, 4), (700, 0, 1)])
def test_select(hq, hkv, budget, first, last):
    check_select(*a_case(hq, hkv, REQS, hq + 100 * hkv), budget, first, last)
    assert pkv.pkv_get_error() == 0


@pytest.mark.parametrize("kind", ["zero queries", "zero bounds", "few values", "twins",
                                  "near ties", "huge", "tiny", "all equal"])
def test_select_ties_and_ranges(kind):
    q, bounds, reqs, bt, qsl, seq = a_case(16, 4, REQS, 55)
    g = gen(8)
    nb = bounds.shape[0]
    if kind == "zero queries":
        q.zero_()
    elif kind == "zero bounds":
        bounds.zero_()
    elif kind == "few values":        # whole numbers: many exact ties
        q[:] = torch.randint(-1, 2, q.shape, generator=g, device="cuda").to(torch.bfloat16)
        bounds[:] = 0
        bounds[..., :3] = torch.randint(0, 2, (nb, 4, 2, 3), generator=g, device="cuda").float()
    elif kind == "twins":             # every page twice or more
        bounds[:] = bounds[torch.arange(nb, device="cuda") // 7 * 7]
    elif kind == "near ties":         # pages that differ in one dimension's last bits
        bounds[:] = bounds[:1]
        bounds[:, :, 1, 5] = 1 + torch.randint(0, 8, (nb, 4), generator=g, device="cuda") * 2.0 ** -7
        q[..., 5] = q[..., 5] * 2.0 ** -12
    elif kind == "huge":              # products past fp32's range
        q *= 2.0 ** 80
        bounds *= 2.0 ** 70
    elif kind == "tiny":              # products below it
        q *= 2.0 ** -80
        bounds *= 2.0 ** -72
    elif kind == "all equal":
        bounds[:] = bounds[:1]
    check_select(q, bounds, reqs, bt, qsl, seq, 16, 1, 2)
    assert pkv.pkv_get_error() == 0


@pytest.mark.parametrize("width", [513, 200, 40])
@pytest.mark.parametrize("kind", ["random", "few values", "twins", "near ties"])
def test_select_of_many_rows_with_narrow_tables(kind, width):
    """Enough rows and KV heads that one CTA of four warps takes all of a row's pages."""
    top = 16 * width - 1
    reqs = [(min(c, top), 1) for c in (top, top - 15, top - 16, 0, 15, 16, 255, 256, 400, 1000,
                                       2047, 2048, 3333, 4096, 5000, 6100, 7001, 8000)] * 2
    q, bounds, reqs, bt, qsl, seq = a_case(48, 24, reqs, width)
    g, nb = gen(5), bounds.shape[0]
    if kind == "few values":
        q[:] = torch.randint(-1, 2, q.shape, generator=g, device="cuda").to(torch.bfloat16)
        bounds[:] = 0
        bounds[..., :3] = torch.randint(0, 2, (nb, 24, 2, 3), generator=g, device="cuda").float()
    elif kind == "twins":
        bounds[:] = bounds[torch.arange(nb, device="cuda") // 7 * 7]
    elif kind == "near ties":
        bounds[:] = bounds[:1]
        bounds[:, :, 1, 5] = 1 + torch.randint(0, 8, (nb, 24), generator=g, device="cuda") * 2.0 ** -7
        q[..., 5] = q[..., 5] * 2.0 ** -12
    check_select(q, bounds, reqs, bt[:, :width].contiguous(), qsl, seq, 16, 1, 2)
    assert pkv.pkv_get_error() == 0


def test_select_launches_of_many_rows():
    """More rows times table entries than one launch takes, and a table of the
    largest width."""
    reqs = [(50 * i % 2500, 1) for i in range(130)]
    q, bounds, reqs, bt, qsl, seq = a_case(16, 8, reqs, 3)
    wide = torch.full((130, 32768), -1, dtype=torch.int32, device="cuda")
    wide[:, :bt.shape[1]] = bt
    check_select(q, bounds, reqs, wide, qsl, seq, 24, 1, 1)
    assert pkv.pkv_get_error() == 0


def test_select_one_very_long_request():
    reqs = [(32768 * 16 - 1, 1)]
    q, bounds, reqs, bt, qsl, seq = a_case(8, 2, reqs, 12)
    check_select(q, bounds, reqs, bt[:, :32768].contiguous(), qsl, seq, 1000, 2, 3)
    assert pkv.pkv_get_error() == 0


def test_select_bad_requests():
    reqs = [(600, 1), (500, 2), (700, 1), (90, 1)]
    q, bounds, reqs, bt, qsl, seq = a_case(8, 2, reqs, 9)
    good, lens = run_select(q, bounds, reqs, bt, qsl, seq, 8, 0, 1)
    bad = seq.clone()
    bad[1] = 1                                   # two rows, one key
    bad[2] = 16 * bt.shape[1] + 1
    t, l = run_select(q, bounds, reqs, bt, qsl, bad, 8, 0, 1)
    assert pkv.pkv_get_error() == BITS["SEQ_LEN"] | BITS["BT_WIDTH"]
    assert l.tolist() == [lens[0], 0, 0, 0, lens[4], 0, 0]
    assert torch.equal(t[[0, 4]], good[[0, 4]]) and bool((t[[1, 2, 3, 5, 6]] == -5).all())
    kept = bt.clone()
    bt[0, 3] = bounds.shape[0]
    run_select(q, bounds, reqs, bt, qsl, seq, 8, 0, 1)
    assert pkv.pkv_get_error() == BITS["BLOCK_ID"]
    bt.copy_(kept)
    qsl2 = qsl.clone()
    qsl2[2] = 0                                  # decreasing
    run_select(q, bounds, reqs, bt, qsl2, seq, 8, 0, 1)
    assert pkv.pkv_get_error() & BITS["QSL"]
    # no request: every row's length is zero
    t, l = run_select(q, bounds, [], bt, qsl, seq, 8, 0, 1)
    assert not bool(l.any()) and bool((t == -5).all())


# ------------------------------------------------------- attention over lists

def attention_ref(q, kc, vc, table, lens, scale):
    rows, hq, _ = q.shape
    hkv = kc.shape[2]
    G = hq // hkv
    out = torch.full((rows, hq, D), float("nan"), dtype=torch.float64, device="cuda")
    for t in range(rows):
        L = int(lens[t])
        if L == 0:
            continue
        for g in range(hkv):
            ids = table[t, g, :-(-L // BS)].long()
            k = kc[ids, :, g].double().reshape(-1, D)[:L]
            v = vc[ids, :, g].double().reshape(-1, D)[:L]
            x = q[t, g * G:(g + 1) * G].double() @ k.T * scale
            out[t, g * G:(g + 1) * G] = torch.softmax(x, -1) @ v
    return out


def close(got, ref):
    err = (got.double() - ref).abs()
    ok = (err <= ATOL + RTOL * ref.abs()) | (got.isnan() & ref.isnan())
    assert bool(ok.all()), "max error %g" % float(err.nan_to_num(0).max())


@pytest.mark.parametrize("hq,hkv", [(8, 8), (32, 8), (16, 1), (32, 1), (20, 1), (9, 3)])
def test_attention_over_lists(hq, hkv):
    g = gen(hq + hkv)
    nb, width = 300, 160
    lens = torch.tensor([1, 15, 16, 17, 0, 300, 160 * 16, 33, 1000, 0], dtype=torch.int32,
                        device="cuda")
    rows = len(lens)
    kc, vc = randn((nb, BS, hkv, D), g), randn((nb, BS, hkv, D), g)
    kc[:3], vc[:3] = float("nan"), float("nan")    # pages of nobody
    table = torch.stack([torch.stack([3 + torch.randperm(nb - 3, generator=g, device="cuda")[:width]
                                      for _ in range(hkv)]) for _ in range(rows)]).int()
    for t in range(rows):
        table[t, :, -(-int(lens[t]) // BS):] = -1
    q = randn((rows, (hq + 1) * D), g)[:, D:].view(rows, hq, D)
    out = torch.full((rows, hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    pkv.pkv_attention_selected(q, kc, vc, table, lens, D ** -0.5, out)
    assert pkv.pkv_get_error() == 0
    close(out, attention_ref(q, kc, vc, table, lens, D ** -0.5))


def test_attention_over_bad_lists():
    g = gen(2)
    kc, vc = randn((40, BS, 2, D), g), randn((40, BS, 2, D), g)
    table = torch.randint(0, 40, (5, 2, 8), generator=g, device="cuda", dtype=torch.int32)
    lens = torch.tensor([100, -1, 128, 129, 50], dtype=torch.int32, device="cuda")
    q = randn((5, 8, D), g)
    out = torch.full_like(q, float("nan"))
    pkv.pkv_attention_selected(q, kc, vc, table, lens, 0.1, out)
    assert pkv.pkv_get_error() == BITS["SEQ_LEN"] | BITS["BT_WIDTH"]
    ok = lens.clone()
    ok[1] = ok[3] = 0
    close(out, attention_ref(q, kc, vc, table, ok, 0.1))
    table[0, 1, 2] = 40
    pkv.pkv_attention_selected(q, kc, vc, table, ok, 0.1, out)
    assert pkv.pkv_get_error() == BITS["BLOCK_ID"]


class Decode:
    """Sequences that grow a token (or two) a step, through the four calls."""

    def __init__(self, ctx, qn, hq, hkv, budget, seed):
        self.g = gen(seed)
        self.reqs = [(c, qn) for c in ctx]
        self.hq, self.hkv, self.budget, self.qn = hq, hkv, budget, qn
        room = [(c, 80) for c in ctx]
        self.bt, _, _, _, nb = metadata(room, self.g)
        self.kc = randn((nb, BS, hkv, D), self.g)
        self.vc = randn((nb, BS, hkv, D), self.g)
        self.bounds = torch.zeros((nb, hkv, 2, D), dtype=torch.bfloat16, device="cuda")
        for r, c in enumerate(ctx):           # what the prompts' steps have left
            for j in range(-(-c // BS)):
                k = self.kc[self.bt[r, j], :min(BS, c - j * BS)].float()
                self.bounds[self.bt[r, j], :, 0] = k.amin(0)
                self.bounds[self.bt[r, j], :, 1] = k.amax(0)
        R = len(ctx)
        rows = R * qn + 2
        self.R, self.rows = R, R * qn
        self.qsl = (torch.arange(R + 1, device="cuda") * qn).int()
        self.done = torch.tensor(ctx, device="cuda")
        self.qkv = randn((rows, (hq + 2 * hkv) * D), self.g)
        self.q = self.qkv[:, :hq * D].view(rows, hq, D)
        self.k = self.qkv[:, hq * D:(hq + hkv) * D].view(rows, hkv, D)
        self.v = self.qkv[:, (hq + hkv) * D:].view(rows, hkv, D)
        self.slots = torch.full((rows,), -1, dtype=torch.int64, device="cuda")
        self.seq = torch.zeros(R, dtype=torch.int32, device="cuda")
        self.table = torch.full((rows, hkv, budget), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.out = torch.full((rows, hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")

    def next(self):
        self.qkv.copy_(randn(self.qkv.shape, self.g))
        p = (self.done[:, None] + torch.arange(self.qn, device="cuda")).view(-1)
        r = torch.arange(self.R, device="cuda").repeat_interleave(self.qn)
        self.slots[:self.rows] = self.bt[r, p // BS].long() * BS + p % BS
        self.done = self.done + self.qn
        self.seq.copy_(self.done.int())

    def step(self):
        pkv.pkv_write(self.k, self.v, self.kc, self.vc, self.slots)
        pkv.pkv_page_bounds(self.kc, self.bounds, self.slots)
        pkv.pkv_select_pages(self.q, self.bounds, self.qsl, self.seq, self.bt, self.R, self.table,
                             self.lens, 1, 2)
        pkv.pkv_attention_selected(self.q, self.kc, self.vc, self.table, self.lens, D ** -0.5,
                                   self.out)

    def check(self):
        reqs = [(int(c) - self.qn, self.qn) for c in self.done]
        table, lens = select_ref(self.q, self.bounds, reqs, self.bt, self.budget, 1, 2)
        assert torch.equal(self.lens, lens)
        assert torch.equal(self.table[:self.rows], table[:self.rows])
        close(self.out, attention_ref(self.q, self.kc, self.vc, table, lens, D ** -0.5))


@pytest.mark.parametrize("hq,hkv,qn", [(16, 4, 1), (8, 2, 2), (32, 1, 1)])
def test_decoding_over_selected_pages(hq, hkv, qn):
    """Steps back to back, with nothing between them that waits; bounds of every
    page stay those of its keys."""
    d = Decode([900, 5, 333, 2000, 62], qn, hq, hkv, 12, hq + qn)
    for i in range(36):
        d.next()
        d.step()
        if i % 9 == 8:
            d.check()
    assert pkv.pkv_get_error() == 0
    for r in range(d.R):
        L = int(d.seq[r])
        for j in range(-(-L // BS)):
            k = d.kc[d.bt[r, j], :min(BS, L - j * BS)].float()
            assert torch.equal(d.bounds[d.bt[r, j], :, 0].float(), k.amin(0))
            assert torch.equal(d.bounds[d.bt[r, j], :, 1].float(), k.amax(0))


def test_a_captured_step():
    d = Decode([900, 5, 333, 2000], 1, 16, 4, 12, 4)
    pkv.pkv_reserve_workspace(16, 16, 12, 16, 4)
    pkv.pkv_reserve_select(16, d.bt.shape[1], 4)
    d.next()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.step()
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        d.check()
        # a larger call in between grows the workspaces, the graph keeps its own
        q, bounds, reqs, bt, qsl, seq = a_case(16, 8, REQS, 3)
        check_select(q, bounds, reqs, bt, qsl, seq, 30, 1, 1)
        d.next()
    assert pkv.pkv_get_error() == 0


def test_a_capture_that_would_need_to_allocate_is_refused():
    import subprocess
    import sys
    import os
    here = os.path.dirname(os.path.abspath(__file__))
    code = r"""
import sys
sys.path[:0] = [%r, %r]
import torch, test_gpu_pages as T, paged_kv_attention_05_gb300 as pkv
q, bounds, reqs, bt, qsl, seq = T.a_case(8, 2, T.REQS, 1)
pkv.pkv_num_sms()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
said = None
with torch.cuda.graph(g):
    q.add_(0)
    try:
        T.run_select(q, bounds, reqs, bt, qsl, seq, 8, 0, 1)
    except pkv.PkvError as e:
        said = str(e)
assert said and "pkv_reserve_select" in said, said
pkv.pkv_reserve_select(64, bt.shape[1], 2)
T.check_select(q, bounds, reqs, bt, qsl, seq, 8)
print("as it should be")
""" % (os.path.dirname(here), here)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "as it should be" in r.stdout, r.stdout + r.stderr


def test_all_pages_within_the_budget_is_plain_attention():
    d = Decode([900, 5, 333, 100], 1, 16, 4, 64, 5)
    d.next()
    d.step()
    out = torch.full_like(d.out, float("nan"))
    pkv.pkv_attention(d.q, d.kc, d.vc, d.qsl, d.seq, d.bt, d.R, D ** -0.5, out)
    assert pkv.pkv_get_error() == 0
    close(d.out, out.double())


def test_other_stream_and_lists_from_it():
    d = Decode([900, 5, 333, 2000], 1, 16, 4, 12, 6)
    side = torch.cuda.Stream()
    d.next()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        d.step()
    torch.cuda.current_stream().wait_stream(side)
    d.check()
    assert pkv.pkv_get_error() == 0


def test_a_step_plan_and_the_page_calls():
    """The write, the bounds and the selection leave a step plan as it is (their workspace
    is another); the attention over selected pages replaces it with its own, which serves
    no planned call."""
    d = Decode([900, 5, 333, 2000], 1, 16, 4, 12, 6)
    d.next()
    want = torch.full_like(d.out, float("nan"))
    plain = (d.qsl, d.seq, d.bt, d.R, D ** -0.5)
    pkv.pkv_write(d.k, d.v, d.kc, d.vc, d.slots)
    pkv.pkv_attention(d.q, d.kc, d.vc, *plain, want)
    pkv.pkv_plan(d.q.shape[0], 16, 4, d.qsl, d.seq, d.bt.shape[1], d.R)
    pkv.pkv_write(d.k, d.v, d.kc, d.vc, d.slots)
    pkv.pkv_page_bounds(d.kc, d.bounds, d.slots)
    pkv.pkv_select_pages(d.q, d.bounds, d.qsl, d.seq, d.bt, d.R, d.table, d.lens, 1, 2)
    got = torch.full_like(d.out, float("nan"))
    pkv.pkv_attention_planned(d.q, d.kc, d.vc, d.bt, D ** -0.5, got)
    assert torch.equal(got[:d.rows], want[:d.rows])
    pkv.pkv_attention_selected(d.q, d.kc, d.vc, d.table, d.lens, D ** -0.5, d.out)
    d.check()
    with pytest.raises(pkv.PkvError):
        pkv.pkv_attention_planned(d.q, d.kc, d.vc, d.bt, D ** -0.5, got)
    assert pkv.pkv_get_error() == 0


def test_selected_lists_as_a_block_table():
    """With one KV head the lists are a block table and the keys in them sequence lengths:
    attention over the lists is pkv_attention over those, whose plan must see the selection
    finished."""
    d = Decode([900, 5, 333, 2000], 1, 8, 1, 12, 9)
    other = torch.full_like(d.out, float("nan"))
    for _ in range(8):
        d.next()
        pkv.pkv_write(d.k, d.v, d.kc, d.vc, d.slots)
        pkv.pkv_page_bounds(d.kc, d.bounds, d.slots)
        pkv.pkv_select_pages(d.q, d.bounds, d.qsl, d.seq, d.bt, d.R, d.table, d.lens, 1, 2)
        pkv.pkv_attention(d.q, d.kc, d.vc, d.qsl, d.lens, d.table.view(-1, 12), d.R, D ** -0.5,
                          other)
        pkv.pkv_attention_selected(d.q, d.kc, d.vc, d.table, d.lens, D ** -0.5, d.out)
        d.check()
        d.out.copy_(other)
        d.check()
    assert pkv.pkv_get_error() == 0
