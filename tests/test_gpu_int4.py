"""The cache of 4-bit codes on the GPU: the write byte for byte against a 64-bit
quantiser, the read back, and attention over it (decodes and prompts) within a
bound that counts the kernels' roundings (int4_ref.attention)."""
import math

import pytest
import torch

import paged_kv_attention_05_gb300 as pkv

pytestmark = pytest.mark.gpu

import int4_ref as R  # noqa: E402

BITS = pkv.DEV_ERR_BITS


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(shape, g, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def fill(nb, hkv, g, std=1.0):
    """A pool whose rows are quantised normal values (by the reference)."""
    cache = torch.full((nb, hkv, R.PAGE), 255, dtype=torch.uint8, device="cuda")
    n = nb * R.BS
    R.write(randn((n, hkv, R.D), g, std), randn((n, hkv, R.D), g, std), cache,
            torch.arange(n, device="cuda"))
    return cache


class Step:
    """Requests (cached, scheduled tokens) over a pool in random page order; the
    slots past each request's last token, and the pages of nobody, hold 0xFF bytes
    (NaN scales)."""

    def __init__(self, reqs, hq, hkv, seed, pad=2, std=1.0, qstd=1.0, extra_width=1):
        g = gen(seed)
        self.reqs, self.hq, self.hkv = reqs, hq, hkv
        seq = [c + n for c, n in reqs]
        used = [-(-s // R.BS) for s in seq]
        nb = sum(used) + 3
        perm = torch.randperm(nb, generator=g, device="cuda")
        self.bt = torch.full((len(reqs), max(used) + extra_width), -1, dtype=torch.int32,
                             device="cuda")
        slots, at = [], 0
        for r, u in enumerate(used):
            self.bt[r, :u] = perm[at:at + u].int()
            p = torch.arange(seq[r], device="cuda")
            slots.append(self.bt[r, p // R.BS].long() * R.BS + p % R.BS)
            at += u
        self.slots = torch.cat(slots)
        self.cache = torch.full((nb, hkv, R.PAGE), 255, dtype=torch.uint8, device="cuda")
        n = self.slots.shape[0]
        self.k, self.v = randn((n, hkv, R.D), g, std), randn((n, hkv, R.D), g, std)
        rows = sum(n for _, n in reqs)
        self.rows = rows
        wide = randn((rows + pad, (hq + 2) * R.D), g, qstd)
        self.q = wide[:, R.D:(hq + 1) * R.D].view(rows + pad, hq, R.D)   # strided rows
        self.out = torch.full((rows + pad, hq, R.D), float("nan"), dtype=torch.bfloat16,
                              device="cuda")
        self.qsl = torch.tensor([0] + [n for _, n in reqs], device="cuda").cumsum(0).int()
        self.seq = torch.tensor(seq, dtype=torch.int32, device="cuda")
        self.scale = R.D ** -0.5

    def write(self):
        pkv.pkv_write_int4(self.k, self.v, self.cache, self.slots)

    def attention(self, **kw):
        pkv.pkv_attention_int4(self.q, self.cache, self.qsl, self.seq, self.bt, len(self.reqs),
                               self.scale, self.out, **kw)

    def check(self, what="", rows=None):
        ref, bound = R.attention(self.q, self.cache, self.qsl, self.seq, self.bt, self.scale)
        sel = slice(0, self.rows) if rows is None else rows
        err = (self.out[sel].double() - ref[sel]).abs()
        assert bool((err <= bound[sel]).all()), \
            "%s: error up to %g of the bound" % (what, float((err / bound[sel]).nan_to_num(9e9).max()))
        assert bool(self.out[self.rows:].isnan().all()), "rows behind the last request written"


@pytest.mark.parametrize("hkv", [1, 2, 3, 8, 32, 5])
@pytest.mark.parametrize("n", [1, 17, 700])
def test_write_bytes(hkv, n):
    g = gen(hkv * 1000 + n)
    nb = -(-n // R.BS) + 2
    cache = torch.randint(0, 256, (nb, hkv, R.PAGE), generator=g, device="cuda").to(torch.uint8)
    wide = randn((n + 3, 2 * hkv * R.D + 64), g)
    k = wide[:, :hkv * R.D].view(n + 3, hkv, R.D)
    v = wide[:, hkv * R.D:2 * hkv * R.D].view(n + 3, hkv, R.D)
    slots = torch.randperm(nb * R.BS, generator=g, device="cuda")[:n + 3].contiguous()
    slots[n // 2] = -1
    slots[n:] = -1
    want = cache.clone()
    R.write(k, v, want, slots)
    pkv.pkv_write_int4(k, v, cache, slots)
    assert pkv.pkv_get_error() == 0
    assert torch.equal(cache, want)


def test_write_odd_rows():
    """Constant rows, rows of halves of a step, tiny and huge spreads, NaN and
    infinities, signed zeros, subnormals."""
    g = gen(5)
    rows = [torch.full((R.D,), 3.25), torch.zeros(R.D), -torch.zeros(R.D),
            torch.arange(R.D) % 31 / 2.0,                      # halves of a step of 1
            (torch.arange(R.D) % 31 / 2.0 - 7) * 2.0 ** 40,
            torch.randn(R.D) * 2.0 ** -37, torch.randn(R.D) * 2.0 ** -33,
            torch.randn(R.D) * 1e38, torch.randn(R.D) * 1e-40,
            torch.randn(R.D).index_fill(0, torch.tensor([3, 77]), float("nan")),
            torch.randn(R.D).index_fill(0, torch.tensor([0]), float("inf")),
            torch.randn(R.D).index_fill(0, torch.tensor([127]), float("-inf")),
            torch.full((R.D,), float("nan")), torch.full((R.D,), float("inf")),
            torch.randn(R.D) + 1000.0, torch.linspace(0, 15, R.D)]
    x = torch.stack(rows).to(torch.bfloat16).cuda()[:, None].contiguous()
    y = x.flip(0).contiguous()
    cache = torch.zeros((1, 1, R.PAGE), dtype=torch.uint8, device="cuda")
    want = cache.clone()
    slots = torch.arange(R.BS, device="cuda")
    R.write(x, y, want, slots)
    pkv.pkv_write_int4(x, y, cache, slots)
    # (a zero's sign is not part of the format)
    for a, b in zip(R.unpack(cache, 0) + R.unpack(cache, 1), R.unpack(want, 0) + R.unpack(want, 1)):
        assert torch.equal(a, b)
    ko, vo = torch.empty_like(x), torch.empty_like(y)
    pkv.pkv_read_int4(cache, slots, ko, vo)
    assert pkv.pkv_get_error() == 0
    assert bool(ko.isfinite().all()) and bool(vo.isfinite().all())
    good = x.float().isfinite().all(-1)[:, 0] & (x.float().abs().amax(-1)[:, 0] < 1e37)
    xs, ks = x[good].double(), ko[good].double()
    step = (xs.amax(-1, keepdim=True) - xs.amin(-1, keepdim=True)) / 15
    # half a step (of one rounded to bf16), the bf16 rounding of the value, and a spread
    # that counts as none
    assert bool(((xs - ks).abs() <= step * (0.5 + 16 * 2.0 ** -8) + 2.0 ** -8 * xs.abs() +
                 2.0 ** -36).all())


@pytest.mark.parametrize("hkv", [1, 6, 8])
def test_read_back(hkv):
    g = gen(hkv)
    cache = fill(9, hkv, g)
    n = 200
    slots = torch.randint(0, 9 * R.BS, (n,), generator=g, device="cuda")   # some twice
    slots[7] = -1
    out = torch.full((n, 2 * hkv * R.D + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    ko = out[:, :hkv * R.D].view(n, hkv, R.D)
    vo = out[:, hkv * R.D:2 * hkv * R.D].view(n, hkv, R.D)
    pkv.pkv_read_int4(cache, slots, ko, vo)
    assert pkv.pkv_get_error() == 0
    keep = torch.arange(n, device="cuda") != 7
    for side, o in enumerate((ko, vo)):
        c, s, z = R.unpack(cache, side)
        val = (c * s[..., None] + z[..., None]).permute(0, 2, 1, 3).reshape(-1, hkv, R.D)
        # (the fp32 sum s * c + z is rounded before the bf16 rounding: at most one
        # fp32 half-step beside a tie)
        err = (o[keep].double() - val[slots[keep]]).abs()
        assert bool((err <= val[slots[keep]].abs() * (2.0 ** -8 + 2.0 ** -23)).all())
        assert bool(o[7].isnan().all())
    assert bool(out[:, 2 * hkv * R.D:].isnan().all())


def test_slots_past_the_pool():
    g = gen(1)
    cache = fill(2, 2, g)
    before = cache.clone()
    x = randn((3, 2, R.D), g)
    slots = torch.tensor([-1, 2 * R.BS, 1 << 40], device="cuda")
    pkv.pkv_write_int4(x, x, cache, slots)
    assert pkv.pkv_get_error() == BITS["SLOT_RANGE"]
    assert torch.equal(cache, before)
    y = torch.full_like(x, float("nan"))
    pkv.pkv_read_int4(cache, slots, y, y.clone())
    assert pkv.pkv_get_error() == BITS["SLOT_RANGE"]
    assert bool(y.isnan().all())


LENS = [0, 1, 15, 16, 63, 200, 1023, 2100, 5000]


@pytest.mark.parametrize("hq,hkv,qn", [(8, 8, 1), (32, 8, 1), (64, 8, 1), (12, 4, 1), (24, 2, 1),
                                       (32, 2, 1), (17, 1, 1), (24, 1, 1), (32, 1, 1), (8, 8, 16),
                                       (16, 4, 2), (16, 4, 3), (16, 4, 4), (8, 1, 2), (9, 3, 5)])
def test_decode(hq, hkv, qn):
    s = Step([(c, qn) for c in LENS], hq, hkv, hq * 7 + hkv + qn)
    s.write()
    s.attention()
    assert pkv.pkv_get_error() == 0
    s.check("decode")


@pytest.mark.parametrize("hq,hkv", [(8, 8), (32, 8), (6, 2), (9, 3), (32, 1), (20, 1)])
def test_prompts_and_chunks(hq, hkv):
    s = Step([(0, 33), (0, 128), (5, 129), (250, 300), (0, 511), (777, 97), (0, 1)], hq, hkv,
             hq + 3 * hkv)
    s.write()
    s.attention()
    assert pkv.pkv_get_error() == 0
    s.check("prompts")


@pytest.mark.parametrize("hq,hkv", [(32, 8), (32, 1), (8, 8)])
def test_mixed(hq, hkv):
    """Decodes, multi-token decodes, prompts, and requests without a token."""
    s = Step([(540, 1), (129, 1), (0, 298), (40, 0), (3000, 2), (0, 1), (64, 70), (9000, 1)], hq,
             hkv, 11 * hq + hkv)
    s.write()
    s.attention()
    assert pkv.pkv_get_error() == 0
    s.check("mixed")


def test_many_short_requests():
    """Every warp takes several units in turn: the ring's phases carry over."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(1, 120, (2300,), generator=g).tolist()
    s = Step([(c, 1 + (i % 3 == 0)) for i, c in enumerate(lens)], 8, 2, 77)
    s.write()
    s.attention()
    assert pkv.pkv_get_error() == 0
    s.check("many")


@pytest.mark.parametrize("hq,hkv", [(16, 4), (32, 1)])
@pytest.mark.parametrize("kind", ["value rows of all sizes", "one huge value row", "sharp scores",
                                  "constant rows", "large queries", "tiny queries", "zero queries",
                                  "offset rows", "all zero", "tiny everything"])
def test_ranges(hq, hkv, kind):
    s = Step([(1500, 1), (70, 1), (0, 1), (700, 150 if hkv == 4 else 1), (33, 2 if hkv == 4 else 1)],
             hq, hkv, 4242)
    g = gen(9)
    n = s.k.shape[0]
    if kind == "value rows of all sizes":   # 2^-20 .. 2^20
        s.v *= 2.0 ** torch.randint(-20, 21, (n, hkv, 1), generator=g, device="cuda").float()
    elif kind == "one huge value row":
        s.v[0] *= 2.0 ** 60
        s.v[::97] *= 2.0 ** 30
    elif kind == "sharp scores":
        s.q *= 12
    elif kind == "constant rows":
        s.k[::3] = 0.5
        s.v[::2] = s.v[::2, :, :1]
    elif kind == "large queries":
        s.q *= 2.0 ** 15
        s.k *= 2.0 ** -15
    elif kind == "tiny queries":
        s.q *= 2.0 ** -40
    elif kind == "zero queries":
        s.q.zero_()
    elif kind == "all zero":
        s.q.zero_(), s.k.zero_(), s.v.zero_()
    elif kind == "tiny everything":
        s.q *= 2.0 ** -60
        s.k *= 2.0 ** -30
        s.v *= 2.0 ** -30
    elif kind == "offset rows":
        s.k += 4
        s.v -= 3
    s.write()
    s.attention()
    assert pkv.pkv_get_error() == 0
    s.check(kind)


def test_a_reference_that_keeps_moving():
    """Scores that grow along the context, and value scales that grow with them:
    the reference moves again and again."""
    s = Step([(2000, 1), (500, 2)], 8, 2, 31)
    base = s.q[:s.rows].float().mean((0, 1))
    grow = torch.cat([torch.linspace(0, 3, 2001), torch.linspace(0, 4, 502)]).cuda()
    s.k[:] = (s.k.float() * 0.1 + grow[:, None, None] * base.sign() * 2).to(torch.bfloat16)
    s.v[:] = (s.v.float() * (2.0 ** (3 * grow))[:, None, None]).to(torch.bfloat16)
    s.q[:s.rows] += (base.sign() * 3).to(torch.bfloat16)
    s.write()
    s.attention()
    assert pkv.pkv_get_error() == 0
    s.check("moving")


def test_bad_requests_are_skipped():
    s = Step([(40, 1), (0, 20), (300, 1), (7, 9), (50, 1)], 8, 2, 321)
    s.write()
    s.attention()
    s.check("good")
    good = s.out.clone()
    s.out.fill_(float("nan"))
    s.seq[1] = 5                              # 20 rows, 5 keys
    s.seq[2] = 16 * s.bt.shape[1] + 1         # a row of the table too short
    s.attention()
    assert pkv.pkv_get_error() == BITS["SEQ_LEN"] | BITS["BT_WIDTH"]
    q = s.qsl.tolist()
    for r in range(5):
        rows = slice(q[r], q[r + 1])
        if r in (1, 2):
            assert bool(s.out[rows].isnan().all())
        else:
            assert torch.equal(s.out[rows], good[rows])
    s.seq[1], s.seq[2] = 20, 301
    for r, bad in ((2, s.cache.shape[0]), (1, -7), (0, 1 << 30)):
        kept = s.bt.clone()
        s.bt[r, 0] = bad
        s.attention()
        assert pkv.pkv_get_error() == BITS["BLOCK_ID"]
        s.bt.copy_(kept)


def test_strides_streams_and_graphs():
    s = Step([(700, 1), (3000, 2), (0, 200)], 8, 2, 98)
    s.write()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.attention()
    torch.cuda.current_stream().wait_stream(side)
    s.check("other stream")
    want = s.out.clone()
    # out as a column slice, q of one token as a lone row of odd stride
    wide = torch.full((s.out.shape[0], 10 * R.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    s.out = wide[:, R.D:9 * R.D].view(-1, 8, R.D)
    s.attention()
    assert torch.equal(s.out[:s.rows], want[:s.rows])
    assert bool(wide[:, :R.D].isnan().all()) and bool(wide[:, 9 * R.D:].isnan().all())
    s.out = torch.full_like(want, float("nan"))
    pkv.pkv_reserve_workspace(8, 512, 512, 8, 2)
    torch.cuda.synchronize()
    blank = s.cache.clone().fill_(255)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.write()
        s.attention()
    for _ in range(3):
        s.out.fill_(float("nan"))
        s.cache.copy_(blank)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s.out[:s.rows], want[:s.rows])
    assert pkv.pkv_get_error() == 0


@pytest.mark.parametrize("scale", [-0.11, 0.0, 1.0])
def test_scales(scale):
    s = Step([(700, 1), (1500, 2), (0, 200), (300, 140)], 8, 2, 77)
    s.scale = scale
    s.write()
    s.attention()
    assert pkv.pkv_get_error() == 0
    s.check("scale %g" % scale)


SCRIPT = r"""
import sys
sys.path[:0] = [%r, %r]
import torch, test_gpu_int4 as T, paged_kv_attention_05_gb300 as pkv
# one decode: its plan's one-wave split has more units than the bound for its lengths
s = T.Step([(5000, 1)], %d, %d, 3, pad=0)
pkv.pkv_reserve_workspace(1, 1, s.bt.shape[1], s.hq, s.hkv)
s.write()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    s.attention()
for _ in range(3):
    s.out.fill_(float("nan"))
    g.replay()
torch.cuda.synchronize()
assert pkv.pkv_get_error() == 0
s.check("captured first")
print("as it should be")
"""


@pytest.mark.parametrize("hq,hkv", [(8, 1), (16, 1), (32, 1), (8, 8)])
def test_a_reservation_of_exact_sizes_serves_a_capture(hq, hkv):
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", SCRIPT % (os.path.dirname(here), here, hq, hkv)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "as it should be" in r.stdout, r.stdout + r.stderr


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes: pages at its end."""
    hkv = 32
    nb = (1 << 32) // (hkv * R.PAGE) + 40
    cache = torch.empty((nb, hkv, R.PAGE), dtype=torch.uint8, device="cuda")
    g = gen(6)
    n = 30
    k, v = randn((n, hkv, R.D), g), randn((n, hkv, R.D), g)
    slots = (nb - 2) * R.BS + torch.arange(n, device="cuda")
    pkv.pkv_write_int4(k, v, cache, slots)
    want = torch.zeros((2, hkv, R.PAGE), dtype=torch.uint8, device="cuda")
    R.write(k, v, want, slots - (nb - 2) * R.BS)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    pkv.pkv_read_int4(cache, slots, ko, vo)
    wk, wv = torch.empty_like(k), torch.empty_like(v)
    pkv.pkv_read_int4(want, slots - (nb - 2) * R.BS, wk, wv)
    assert torch.equal(ko, wk) and torch.equal(vo, wv)
    q = randn((n, hkv, R.D), g)
    for qn in (1, n):   # a decode, a prompt
        out, ref = torch.empty_like(q[:qn]), torch.empty_like(q[:qn])
        qsl = torch.tensor([0, qn], dtype=torch.int32, device="cuda")
        seq = torch.tensor([n], dtype=torch.int32, device="cuda")
        bt = torch.tensor([[nb - 2, nb - 1]], dtype=torch.int32, device="cuda")
        pkv.pkv_attention_int4(q[:qn], cache, qsl, seq, bt, 1, 0.1, out)
        pkv.pkv_attention_int4(q[:qn], want, qsl, seq, bt - (nb - 2), 1, 0.1, ref)
        assert torch.equal(out, ref)
    assert pkv.pkv_get_error() == 0


def test_the_other_caches_after_an_int4_call():
    """An int4 call's plan does not serve pkv_attention_planned."""
    s = Step([(300, 1)], 8, 2, 5)
    s.write()
    s.attention()
    kc = torch.zeros((4, 16, 2, R.D), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pkv.PkvError):
        pkv.pkv_attention_planned(s.q, kc, kc, s.bt, s.scale, s.out)


def test_many_keys_of_little_weight():
    """A first key that takes nearly all of the weight, and 2^17 others of 2^-23 each:
    their share of the output stays, although a weight of theirs alone would be below
    fp16's normal numbers.  Keys are constant rows (cached exactly), values 0 and 150 by
    turns."""
    n_keys, n, hq = 1 << 17, 300, 2
    k = torch.full((n_keys, 1, R.D), 0.03125, dtype=torch.bfloat16, device="cuda")
    k[0] = 1.4375
    v = torch.zeros(n_keys, 1, R.D, dtype=torch.bfloat16, device="cuda")
    v[1:, :, 1::2] = 150.0
    cache = torch.empty(n_keys // R.BS, 1, R.PAGE, dtype=torch.uint8, device="cuda")
    pkv.pkv_write_int4(k, v, cache, torch.arange(n_keys, device="cuda"))
    q = torch.ones(n, hq, R.D, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, float("nan"))
    scale = R.D ** -0.5
    i32 = dict(dtype=torch.int32, device="cuda")
    pkv.pkv_attention_int4(q, cache, torch.tensor([0, n], **i32), torch.tensor([n_keys], **i32),
                           torch.arange(n_keys // R.BS, **i32).view(1, -1), 1, scale, out)
    assert pkv.pkv_get_error() == 0
    w = math.exp(-128 * (1.4375 - 0.03125) * scale)
    others = torch.arange(n_keys - n, n_keys, device="cuda").double()
    want = 150.0 * others * w / (1 + others * w)
    # bf16's rounding of the output; of each weight fp16's, half of 2^-24 where the largest
    # is at least 2^7; logits of up to 2^5 in fp32 (2^-19 of a weight), exp2 and the sums
    tol = want * (2.0 ** -8 + 2.0 ** -17) + 150.0 * others * 2.0 ** -32
    assert bool(((out[:, :, 1::2].double() - want[:, None, None]).abs() <= tol[:, None, None]).all())
    assert not out[:, :, 0::2].any()
