"""pkv_select_pages where its 32-bit scores cannot be trusted, beside bad requests and
next to other requests' bounds, against the 64-bit definition."""
import pytest
import torch

import paged_kv_attention_05_gb300 as pkv

pytestmark = pytest.mark.gpu

import test_gpu_pages as P  # noqa: E402

BITS = pkv.DEV_ERR_BITS


@pytest.mark.parametrize("e", [50, 58, 60, 61, 62, 64, 66, 68, 71, 75])
@pytest.mark.parametrize("hq,hkv,width", [(16, 4, None), (2, 2, None), (48, 24, 513)])
def test_scores_past_32_bits(e, hq, hkv, width):
    """Sums of products past fp32's largest number (2^128) that cancel, or do not, over pages
    whose bounds differ in size: q and bounds of about 2^e, queries of both signs."""
    if width:
        top = 16 * width - 1
        reqs = [(min(c, top), 1) for c in (top, 0, 400, 1000, 2048, 3333, 5000, 7001, 8000)] * 4
    else:
        reqs = P.REQS
    q, bounds, reqs, bt, qsl, seq = P.a_case(hq, hkv, reqs, 100 + e)
    g = P.gen(e)
    size = torch.randint(-12, 1, (bounds.shape[0], hkv, 1, 1), generator=g, device="cuda")
    bounds *= 2.0 ** (e + size).double()
    q *= 2.0 ** e
    if width:
        bt = bt[:, :width].contiguous()
    P.check_select(q, bounds, reqs, bt, qsl, seq, 16, 1, 2)
    assert pkv.pkv_get_error() == 0


def test_a_page_whose_sums_overflow_to_both_sides():
    """Its score is 0, its fp32 sums are inf - inf; eleven small pages are larger."""
    q = torch.full((1, 1, P.D), 2.0 ** 62, dtype=torch.bfloat16, device="cuda")
    q[..., 64:] *= -1
    bounds = torch.zeros(13, 1, 2, P.D, dtype=torch.bfloat16, device="cuda")
    bounds[0] = 2.0 ** 62
    for j in range(1, 12):
        bounds[j, :, :, :64] = 2.0 ** 50 * (1 + j / 16)
    i32 = dict(dtype=torch.int32, device="cuda")
    table, lens = P.run_select(q, bounds, [(12 * 16 + 3, 1)], torch.arange(13, **i32).view(1, -1),
                               torch.tensor([0, 1], **i32), torch.tensor([12 * 16 + 4], **i32),
                               4, 0, 1)
    assert pkv.pkv_get_error() == 0
    assert table.flatten().tolist() == [9, 10, 11, 12] and lens.tolist() == [3 * 16 + 4]


def test_bounds_of_a_page_of_nobody_cost_nothing():
    """Block 0 belongs to no row here, and its bounds are infinite: the lists are those of
    the definition, and no row's pages are scored again in 64 bits for its sake (all were)."""
    reqs = [(16 * 2047 - 5 - 16 * r, 1) for r in range(8)]
    q, bounds, reqs, bt, qsl, seq = P.a_case(16, 4, reqs, 7)
    bounds = torch.cat([bounds[:1], bounds]).contiguous()
    bt = torch.where(bt >= 0, bt + 1, bt)

    def once():
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(10):
            got = P.run_select(q, bounds, reqs, bt, qsl, seq, 64, 0, 1)
        b.record()
        b.synchronize()
        return a.elapsed_time(b), got

    times = {}
    for value in (0.5, float("inf")):
        bounds[0] = value
        once()
        times[value] = sorted(once()[0] for _ in range(9))[4]
        P.check_select(q, bounds, reqs, bt, qsl, seq, 64, 0, 1)
    assert pkv.pkv_get_error() == 0
    assert times[float("inf")] < 1.5 * times[0.5], times


def test_rows_of_valid_requests_beside_bad_ones():
    """A request of decreasing or negative query_start_loc is skipped; the others keep
    their rows, as in pkv_attention."""
    reqs = [(100 + 90 * r, 2) for r in range(12)]
    q, bounds, reqs, bt, qsl, seq = P.a_case(8, 2, reqs, 21)
    good, lens = P.run_select(q, bounds, reqs, bt, qsl, seq, 8, 0, 1)
    assert pkv.pkv_get_error() == 0
    for at, value in ((3, -5), (6, -1), (5, 999), (6, 999), (9, 1000), (1, 30)):
        bad = qsl.clone()
        bad[at] = value
        t, n = P.run_select(q, bounds, reqs, bt, bad, seq, 8, 0, 1)
        assert pkv.pkv_get_error() & BITS["QSL"]
        for r in range(12):
            rows = slice(2 * r, 2 * r + 2)
            if r in (at - 1, at):       # the two requests that the entry belongs to
                assert not n[rows].any() and bool((t[rows] == -5).all()), (at, value, r)
            else:
                assert torch.equal(n[rows], lens[rows]) and torch.equal(t[rows], good[rows]), \
                    (at, value, r)
        assert not n[24:].any()
