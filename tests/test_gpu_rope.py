"""pkv_write_rope and pkv_write_rope_int8 on the GPU against the formula in 64
bits: both pair styles, partial rotation, norms, padding, bad slots and
positions, strides, in place, streams and graphs.

Tolerance.  A bf16 output is off by half a step, eps / 2 = 2^-8 of the value
(2^-8 bounds it: bf16 keeps 8 bits), plus the fp32 arithmetic before it: for a
pair with magnitudes M = |y_a| + |y_b| the rotation makes three roundings of
terms of at most M (3 * 2^-24 M); the norm's factor is a sum of 128 squares (16
in a thread, three exchanges), a reciprocal root (2 units) and two products: at
most 26 roundings, 26 * 2^-24 M.  29 * 2^-24 < 2^-19."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_attention_05_gb300 as pkv
from paged_kv_attention_05_gb300 import workloads as W

pytestmark = pytest.mark.gpu

from gpu_util import assert_close, to_host_bits  # noqa: E402

D = 128


def table(far, rot, base=10000.0):
    inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(far, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


class Case:
    def __init__(self, n, hq, hkv, rot=128, interleaved=False, qn=False, kn=False, offset=0.0,
                 pad=0, int8=False, seed=0, far=5000, std=1.0, fused=True):
        g = torch.Generator().manual_seed(seed * 7919 + n * 31 + hq)
        rows = n + pad
        width = (hq + 2 * hkv) * D
        qkv = (torch.randn(rows, width, generator=g) * std).to(torch.bfloat16)
        self.n, self.rows, self.hq, self.hkv, self.rot = n, rows, hq, hkv, rot
        self.interleaved, self.offset, self.int8 = interleaved, offset, int8
        blocks = -(-max(n, 1) // 16) + 2
        slots = torch.randperm(blocks * 16, generator=g)[:rows].contiguous()
        slots[n:] = -1
        pos = torch.randint(0, far, (rows,), generator=g)
        pos[n:] = 1 << 40   # positions of padding rows are never written: garbage here
        shape = (blocks, 16, hkv, D)
        if int8:
            kc = torch.randint(-127, 128, shape, generator=g, dtype=torch.int8)
        else:
            kc = torch.randn(shape, generator=g).to(torch.bfloat16)
        self.kc0, self.vc0 = kc, kc.flip(0).contiguous()
        self.qw = (1 + 0.3 * torch.randn(D, generator=g)).to(torch.bfloat16) if qn else None
        self.kw = (1 + 0.3 * torch.randn(D, generator=g)).to(torch.bfloat16) if kn else None
        self.table, self.pos, self.slots = table(far, rot), pos, slots
        self.qkv = qkv.cuda()
        self.q = self.qkv[:, :hq * D].view(rows, hq, D)
        self.k = self.qkv[:, hq * D:(hq + hkv) * D].view(rows, hkv, D)
        self.v = self.qkv[:, (hq + hkv) * D:].view(rows, hkv, D)
        if not fused:
            self.q, self.k, self.v = (t.contiguous() for t in (self.q, self.k, self.v))
        self.host = [t.cpu() for t in (self.q, self.k, self.v)]
        self.ks, self.vs = 0.03 * std, 0.02 * std
        self.kc, self.vc = self.kc0.cuda(), self.vc0.cuda()
        self.q_out = torch.full((rows, hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.dev = [t.cuda() for t in (self.pos, self.table, self.slots)]
        self.w = [None if t is None else t.cuda() for t in (self.qw, self.kw)]

    def run(self, q_out=None, **kw):
        pos, tab, slots = self.dev
        opt = dict(interleaved=self.interleaved, q_weight=self.w[0], k_weight=self.w[1],
                   weight_offset=self.offset, eps=1e-6, **kw)
        q_out = self.q_out if q_out is None else q_out
        if self.int8:
            pkv.pkv_write_rope_int8(self.q, self.k, self.v, pos, tab, self.kc, self.vc, slots,
                                    self.ks, self.vs, q_out, **opt)
        else:
            pkv.pkv_write_rope(self.q, self.k, self.v, pos, tab, self.kc, self.vc, slots, q_out,
                               **opt)

    def turned(self, x, w):
        """(value, M) of the formula in 64 bits for the first n rows of x."""
        y = x[:self.n].double()
        if w is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + float(np.float32(1e-6)))
            y = y * (w.double() + self.offset)
        half = self.rot // 2
        t = self.table[self.pos[:self.n]].double()
        c, s = t[:, None, :half], t[:, None, half:]
        i = torch.arange(half)
        a, b = (2 * i, 2 * i + 1) if self.interleaved else (i, i + half)
        z, m = y.clone(), y.abs()
        z[..., a] = y[..., a] * c - y[..., b] * s
        z[..., b] = y[..., b] * c + y[..., a] * s
        m[..., a] = m[..., b] = y[..., a].abs() + y[..., b].abs()
        return z, m

    def check(self, q_out=None):
        got = (self.q_out if q_out is None else q_out).cpu()
        qr, qm = self.turned(self.host[0], self.qw)
        kr, km = self.turned(self.host[1], self.kw)
        self.near(got[:self.n], qr, qm, "q_out")
        slots = self.slots[:self.n]
        kc, vc = (t.cpu().view(-1, self.hkv, D) for t in (self.kc, self.vc))
        k0, v0 = (t.view(-1, self.hkv, D) for t in (self.kc0, self.vc0))
        if self.int8:
            vr = self.host[2][:self.n].double()
            for codes, ref, m, sc, name in ((kc[slots], kr, km, self.ks, "key codes"),
                                            (vc[slots], vr, vr.abs(), self.vs, "value codes")):
                sc = float(np.float32(sc))
                want = (ref / sc).clamp(-127, 127)
                # half a code, the fp32 value's own error and the division's rounding
                off = (codes.double() - want).abs()
                assert (off <= 0.5 + (2.0 ** -19 * m + 2.0 ** -24 * ref.abs()) / sc).all(), name
        else:
            self.near(kc[slots], kr, km, "key cache")
            assert torch.equal(vc[slots], self.host[2][:self.n]), "value cache"
        rest = torch.ones(kc.shape[0], dtype=torch.bool)
        rest[slots] = False
        assert torch.equal(kc[rest], k0[rest]) and torch.equal(vc[rest], v0[rest])

    @staticmethod
    def near(got, ref, m, what):
        err = (got.double() - ref).abs()
        bad = ~(err <= 2.0 ** -8 * ref.abs() + 2.0 ** -19 * m)
        assert not bad.any(), "%s: %d values off, worst %g" % (what, int(bad.sum()),
                                                               float(err[bad].max()))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [128, 112, 96, 64, 32, 16])
def test_rotation(rot, interleaved):
    c = Case(37, 8, 2, rot, interleaved, pad=3, seed=rot)
    c.run()
    assert pkv.pkv_get_error() == 0
    c.check()
    assert torch.isnan(c.q_out[37:].float()).all()   # padding rows of q_out are left alone


@pytest.mark.parametrize("n,hq,hkv", [(1, 32, 8), (1, 1, 1), (2, 3, 1), (5, 64, 8), (33, 7, 7),
                                      (300, 32, 8), (1000, 32, 1), (4097, 12, 4), (257, 5, 3)])
@pytest.mark.parametrize("int8", [False, True])
def test_shapes(n, hq, hkv, int8):
    c = Case(n, hq, hkv, int8=int8, qn=n % 2 == 1, kn=n % 2 == 1, pad=n % 4)
    c.run()
    assert pkv.pkv_get_error() == 0
    c.check()


@pytest.mark.parametrize("qn,kn,offset", [(True, True, 0.0), (True, False, 0.0),
                                          (False, True, 0.0), (True, True, 1.0)])
@pytest.mark.parametrize("rot,interleaved,std", [(128, False, 1.0), (64, True, 300.0),
                                                 (32, False, 1e-3)])
def test_norms(qn, kn, offset, rot, interleaved, std):
    for int8 in (False, True):
        c = Case(70, 16, 4, rot, interleaved, qn, kn, offset, int8=int8, std=std, seed=5)
        if int8:   # (normalised keys are of size one whatever the input's)
            c.ks = 0.03 * (1.0 + offset) if kn else c.ks
        c.run()
        assert pkv.pkv_get_error() == 0
        c.check()


def test_contiguous_inputs_and_fewer_tokens_than_rows():
    c = Case(50, 8, 2, fused=False)
    c.run(n_tokens=20)
    assert pkv.pkv_get_error() == 0
    assert torch.isnan(c.q_out[20:].float()).all()
    c.n = 20
    c.check()


def test_in_place():
    for fused in (True, False):
        c = Case(90, 8, 2, 128, qn=True, kn=True, pad=2, fused=fused)
        c.run(q_out=c.q)
        assert pkv.pkv_get_error() == 0
        c.check(q_out=c.q)
        assert torch.equal(c.q[90:].cpu(), c.host[0][90:])
        if fused:   # k and v of the fused rows are read only
            assert torch.equal(c.k.cpu(), c.host[1]) and torch.equal(c.v.cpu(), c.host[2])


def test_zero_rows_and_specials():
    """An all-zero head row stays zero through the norm; an infinity or NaN
    stays in its own head row; the largest values keep their rotation."""
    c = Case(6, 4, 2, qn=True, kn=True)
    c.q[0] = 0
    c.q[1, 1, 5] = float("inf")
    c.k[2, 0, 7] = float("nan")
    c.host = [t.cpu() for t in (c.q, c.k, c.v)]
    c.run()
    assert pkv.pkv_get_error() == 0
    got = c.q_out.float().cpu()
    assert (got[0] == 0).all()
    assert torch.isfinite(got[1, [0, 2, 3]]).all()
    kc = c.kc.view(-1, 2, D).float().cpu()[c.slots]
    assert torch.isfinite(kc[2, 1]).all() and torch.isnan(kc[2, 0]).any()
    assert torch.isfinite(kc[[0, 1, 3, 4, 5]]).all()


def test_bad_slots_and_positions_are_skipped_and_reported():
    c = Case(8, 4, 2)
    far, total = c.table.shape[0], c.kc0.shape[0] * 16
    c.dev[2][1] = total            # a slot past the pool
    c.dev[0][3] = far              # a position past the table
    c.dev[0][5] = -1
    c.dev[2][6] = -7               # padding, with a position that would be bad
    c.dev[0][6] = far + 9
    c.run()
    assert pkv.pkv_get_error() == (pkv.DEV_ERR_BITS["SLOT_RANGE"] | pkv.DEV_ERR_BITS["POSITION"])
    assert pkv.pkv_get_error() == 0
    skipped = [1, 3, 5, 6]
    assert torch.isnan(c.q_out[skipped].float()).all()
    keep = torch.tensor([0, 2, 4, 7])
    c.q_out, c.n = c.q_out[keep.cuda()], 4
    c.host = [t[keep] for t in c.host]
    c.pos, c.slots = c.pos[keep], c.slots[keep]
    c.check()


@pytest.mark.parametrize("scale", [0.03125, 1 / 3, 0.0123, 127.0, 3.0, 1e-3, 2.0 ** -40, 5e-25,
                                   1e25, 1e-37])
def test_value_codes_are_those_of_write_int8(scale):
    """Every bf16 bit pattern as a value, at scales with and without exact
    halves between codes: the same codes as pkv_write_int8's, bit for bit
    (ties, infinities, NaN and tiny values among them)."""
    hkv, n = 4, 128
    v = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v.view(n, hkv, D).cuda()
    q = torch.zeros((n, 4, D), dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(n, device="cuda")
    pos, tab = torch.zeros(n, dtype=torch.int64, device="cuda"), table(1, 64).cuda()
    caches = [torch.full((n // 16, 16, hkv, D), 99, dtype=torch.int8, device="cuda")
              for _ in range(4)]
    pkv.pkv_write_int8(v, v, caches[0], caches[1], slots, scale, scale)
    # (position 0 rotates by nothing: the keys' codes are the plain ones too,
    # but for an infinity times a sine of zero, which is no number)
    pkv.pkv_write_rope_int8(q, v, v, pos, tab, caches[2], caches[3], slots, scale, scale, q)
    assert pkv.pkv_get_error() == 0
    assert torch.equal(caches[1], caches[3])
    finite = v.float().isfinite()
    pair = finite.clone()
    pair[..., :32] &= finite[..., 32:64]
    pair[..., 32:64] &= finite[..., :32]
    assert torch.equal(caches[0].view(n, hkv, D)[pair], caches[2].view(n, hkv, D)[pair])


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("hq,hkv,rot,il", [(64, 8, 128, False), (32, 8, 64, True), (7, 5, 96, False),
                                           (32, 32, 128, True), (1, 1, 16, False)])
def test_larger_steps(hq, hkv, rot, il, int8):
    """Steps long enough for the streaming form, whose warps take many units of
    one token after another, with padding and bad tokens in between."""
    n = 9000 if hq + hkv < 20 else 4500
    c = Case(n, hq, hkv, rot, il, qn=True, kn=True, int8=int8, seed=n)
    c.dev[2][7::13] = -1                     # padding inside the batch
    c.dev[0][5::101] = c.table.shape[0]      # positions past the table
    c.run()
    assert pkv.pkv_get_error() == pkv.DEV_ERR_BITS["POSITION"]
    left_out = torch.zeros(n, dtype=torch.bool)
    left_out[7::13] = True
    left_out[5::101] = True
    assert torch.isnan(c.q_out[left_out.cuda()].float()).all()
    keep = (~left_out).nonzero().view(-1)
    c.q_out, c.n = c.q_out[keep.cuda()], keep.numel()
    c.host = [t[keep] for t in c.host]
    c.pos, c.slots = c.pos[keep], c.slots[keep]
    c.check()


def test_no_tokens():
    c = Case(4, 4, 2)
    c.run(n_tokens=0)
    torch.cuda.synchronize()
    assert torch.isnan(c.q_out.float()).all() and torch.equal(c.kc.cpu(), c.kc0)


def test_refusals():
    c = Case(4, 4, 2)
    pos, tab, slots = c.dev
    args = lambda **kw: dict(dict(q=c.q, k=c.k, v=c.v, positions=pos, cos_sin=tab, key_cache=c.kc,  # noqa: E731
                                  value_cache=c.vc, slot_mapping=slots, q_out=c.q_out), **kw)
    for bad in (dict(q_out=c.q_out[:, :2]), dict(q_out=c.q_out[:3]), dict(k=c.k[:, :1]),
                dict(k=c.k[:3]), dict(positions=pos[:3]), dict(cos_sin=tab[0]),
                dict(cos_sin=tab[:, ::2]), dict(q_weight=torch.ones(64, dtype=torch.bfloat16,
                                                                    device="cuda")),
                dict(n_tokens=5), dict(q=c.q[0]), dict(q=c.q.transpose(0, 1)),
                dict(positions=torch.zeros(8, dtype=torch.int64, device="cuda")[::2]),
                dict(positions=pos.cpu()), dict(value_cache=c.vc[:1])):
        with pytest.raises(ValueError):
            pkv.pkv_write_rope(**args(**bad))
    for bad in (dict(positions=pos.int()), dict(cos_sin=tab.double()), dict(q=c.q.half()),
                dict(key_cache=c.kc.float()), dict(q_weight=torch.ones(128, device="cuda"))):
        with pytest.raises(TypeError):
            pkv.pkv_write_rope(**args(**bad))
    with pytest.raises(pkv.PkvError) as e:
        pkv.pkv_write_rope(**args(cos_sin=tab[:, :40].contiguous()))
    assert e.value.code == -2
    with pytest.raises(pkv.PkvError) as e:   # 8 bytes off a 16-byte boundary
        pkv.pkv_write_rope(**args(q_out=torch.zeros(4 * 4 * D + 8, dtype=torch.bfloat16,
                                                    device="cuda")[4:-4].view(4, 4, D)))
    assert e.value.code == -3
    torch.cuda.synchronize()
    assert torch.isnan(c.q_out.float()).all()


def test_another_stream_and_a_replayed_graph():
    c = Case(130, 8, 2, qn=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.run(stream=side)
    side.synchronize()
    c.check()
    c.kc.copy_(c.kc0)
    c.vc.copy_(c.vc0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    c.q_out.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    c.check()
    # new inputs in the same buffers: the graph reads them again
    c.qkv.copy_((torch.randn(c.qkv.shape, device="cuda") * 2).to(torch.bfloat16))
    c.host = [t.cpu() for t in (c.q, c.k, c.v)]
    g.replay()
    torch.cuda.synchronize()
    c.check()
    assert pkv.pkv_get_error() == 0


def test_slots_past_32_bits_of_elements():
    """A pool whose last slots lie past 2^31 elements (and 2^32 bytes)."""
    hkv, blocks = 32, 2 ** 31 // (16 * 32 * D) + 40
    c = Case(40, 32, hkv)
    kc = torch.zeros((blocks, 16, hkv, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    c.kc, c.vc = kc, vc
    c.slots = torch.arange(blocks * 16 - 40, blocks * 16)
    c.dev[2].copy_(c.slots)
    c.run()
    assert pkv.pkv_get_error() == 0
    kr, km = c.turned(c.host[1], None)
    last = kc.view(-1, hkv, D)[-40:]
    c.near(last.cpu(), kr, km, "far keys")
    assert torch.equal(vc.view(-1, hkv, D)[-40:].cpu(), c.host[2])
    assert int(kc.view(-1, hkv, D)[:-40].count_nonzero()) == 0


def test_rotated_step_then_attention_matches_the_oracle():
    """write_rope and attention together, as a layer runs them: two decodes and
    a prompt with padding rows; the oracle attends over the rotated rows."""
    step = W.build(W.custom([540, 129, 0], [1, 1, 298], 16, 4, seed=33, pad_tokens=4))
    dev = lambda b: torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).view(torch.bfloat16).cuda()  # noqa: E731
    rows = step.qkv.shape[0]
    qkv = dev(step.qkv)
    q = qkv[:, :16 * D].view(rows, 16, D)
    k = qkv[:, 16 * D:20 * D].view(rows, 4, D)
    v = qkv[:, 20 * D:].view(rows, 4, D)
    kc, vc = dev(step.key_cache), dev(step.value_cache)
    qsl, sl = (torch.from_numpy(x).cuda() for x in (step.query_start_loc, step.seq_lens))
    bt, sm = torch.from_numpy(step.block_table).cuda(), torch.from_numpy(step.slot_mapping).cuda()
    pos = torch.full((rows,), -5, dtype=torch.int64)
    for r in range(step.num_reqs):
        a, b = int(step.query_start_loc[r]), int(step.query_start_loc[r + 1])
        pos[a:b] = torch.arange(int(step.seq_lens[r]) - (b - a), int(step.seq_lens[r]))
    tab = table(1024, D).cuda()
    out = torch.full((rows, 16, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    pkv.pkv_write_rope(q, k, v, pos.cuda(), tab, kc, vc, sm, q)
    pkv.pkv_attention(q, kc, vc, qsl, sl, bt, step.num_reqs, step.scale, out)
    assert pkv.pkv_get_error() == 0
    ref, err = oracle.attention(to_host_bits(q), to_host_bits(kc), to_host_bits(vc),
                                step.query_start_loc, step.seq_lens, step.block_table,
                                step.num_reqs, step.scale)
    assert err == 0
    got = out.float().cpu().numpy().astype(np.float64)
    assert_close(got[:300], ref[:300], "rotated step")
    assert np.isnan(got[300:]).all()


@pytest.mark.parametrize("int8", [False, True])
def test_the_calls_of_plain_arguments(int8):
    """pkv_write_rope and pkv_write_rope_int8 themselves (the binding passes a
    struct): the same bits, two different weights and every stride its own."""
    from paged_kv_attention_05_gb300 import _binding
    c = Case(40, 6, 3, rot=96, interleaved=True, qn=True, kn=True, offset=1.0, pad=2, int8=int8)
    c.run()
    c.check()
    want = [t.clone() for t in (c.q_out, c.kc, c.vc)]
    wide = torch.full((c.rows, c.hq + 1, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    kc, vc = c.kc0.cuda(), c.vc0.cuda()
    k = torch.nn.functional.pad(c.k, (0, 0, 0, 2)).contiguous()
    p = [t.data_ptr() for t in (c.q, k, c.v, *c.w, c.dev[1], c.dev[0], wide, kc, vc, c.dev[2])]
    head = (p[0], c.q.stride(0), c.hq, p[1], k.stride(0), p[2], c.v.stride(0), p[3], p[4], 1.0,
            1e-6, p[5], c.table.shape[0], c.rot, 1, p[6], p[7], wide.stride(0), p[8], p[9])
    tail = (kc.shape[0], 16, c.hkv, D, p[10], c.rows, torch.cuda.current_stream().cuda_stream)
    lib = _binding.load()
    if int8:
        assert lib.pkv_write_rope_int8(*head, c.ks, c.vs, *tail) == 0
    else:
        assert lib.pkv_write_rope(*head, *tail) == 0
    assert pkv.pkv_get_error() == 0
    assert torch.isnan(wide[:, c.hq].float()).all()
    for got, ref in zip((wide[:, :c.hq].contiguous(), kc, vc), want):
        assert torch.equal(got.view(torch.int8), ref.contiguous().view(torch.int8))
