"""Refusals of the page bounds, the selection and the attention over selected
pages on the host (no GPU is touched)."""
import pytest
import torch

import paged_kv_attention_05_gb300 as pkv

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    from paged_kv_attention_05_gb300 import build
    build.build()
    return pkv.load()


def test_bounds(lib):
    def b(kc=FAKE, nb=10, bs=16, hkv=8, d=128, out=FAKE, sm=FAKE, n=4):
        return lib.pkv_page_bounds(kc, nb, bs, hkv, d, out, sm, n, None)

    assert b(bs=8) == -2 and b(d=64) == -2 and b(hkv=40000) == -2
    assert b(hkv=0) == -1 and b(n=-1) == -1 and b(nb=0) == -1
    assert b(kc=None) == -1 and b(out=None) == -1 and b(sm=None) == -1
    assert b(kc=FAKE + 8) == -3 and b(out=FAKE + 2) == -3
    assert b(n=0, kc=None, out=None, sm=None) == 0


def test_select(lib):
    def s(q=FAKE, qs=4096, rows=4, hq=32, bd=FAKE, nb=10, bs=16, hkv=8, d=128, qsl=FAKE, sl=FAKE,
          bt=FAKE, w=40, R=2, budget=8, first=1, last=2, tab=FAKE, lens=FAKE):
        return lib.pkv_select_pages(q, qs, rows, hq, bd, nb, bs, hkv, d, qsl, sl, bt, w, R, budget,
                                    first, last, tab, lens, None)

    assert s(hq=30) == -2 and s(hq=512, qs=65536) == -2 and s(bs=32) == -2 and s(w=40000) == -2
    assert s(rows=1 << 31) == -2
    assert s(budget=0) == -1 and s(budget=40000) == -1 and s(first=-1) == -1 and s(last=0) == -1
    assert s(first=7, last=2) == -1 and s(first=2 ** 31 - 1, last=2 ** 31 - 1) == -1
    assert s(q=None) == -1 and s(bd=None) == -1 and s(bt=None) == -1 and s(qsl=None) == -1
    assert s(tab=None) == -1 and s(lens=None) == -1 and s(R=-1) == -1 and s(qs=100) == -1
    assert s(q=FAKE + 8) == -3 and s(bd=FAKE + 8) == -3 and s(qs=4100) == -3
    assert s(rows=0) == 0


def test_attention(lib):
    def a(q=FAKE, qs=4096, rows=4, hq=32, kc=FAKE, vc=FAKE, nb=10, bs=16, hkv=8, d=128, tab=FAKE,
          w=4, lens=FAKE, scale=0.088, out=FAKE, os=4096):
        return lib.pkv_attention_selected(q, qs, rows, hq, kc, vc, nb, bs, hkv, d, tab, w, lens,
                                          scale, out, os, None)

    assert a(hq=30) == -2 and a(bs=32) == -2 and a(w=40000) == -2 and a(rows=1 << 31) == -2
    assert a(qs=100) == -1 and a(kc=None) == -1 and a(tab=None) == -1 and a(lens=None) == -1
    assert a(w=0) == -1 and a(nb=0) == -1 and a(scale=float("nan")) == -1
    assert a(vc=FAKE + 8) == -3 and a(out=FAKE + 8) == -3
    assert a(rows=0) == 0
    assert lib.pkv_reserve_select(-1, 10, 8) == -1 and lib.pkv_reserve_select(1, 40000, 8) == -1
    assert lib.pkv_reserve_select(1, 10, 0) == -1


def test_binding():
    bf = torch.bfloat16
    kc = torch.zeros(4, 16, 8, 128, dtype=bf)
    b = torch.zeros(4, 8, 2, 128, dtype=bf)
    sm = torch.zeros(2, dtype=torch.int64)
    i = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 32, 128, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.pkv_page_bounds(kc, b, sm)
    with pytest.raises((TypeError, ValueError)):
        pkv.pkv_select_pages(q, b.float(), i, i, i, 1, i, i)
    with pytest.raises((TypeError, ValueError)):
        pkv.pkv_attention_selected(q, kc, kc, None, i, 1.0, q)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.pkv_attention_selected(q, kc, kc, i, i, 1.0, q)
