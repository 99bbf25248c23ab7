"""Refusals of the 4-bit cache's calls on the host (no GPU is touched)."""
import pytest
import torch

import paged_kv_attention_05_gb300 as pkv

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    from paged_kv_attention_05_gb300 import build
    build.build()
    return pkv.load()


def test_write_and_read(lib):
    def w(k=FAKE, ks=1024, v=FAKE, vs=1024, c=FAKE, nb=10, bs=16, hkv=8, d=128, sm=FAKE, n=4):
        return lib.pkv_write_int4(k, ks, v, vs, c, nb, bs, hkv, d, sm, n, None)

    def r(k=FAKE, ks=1024, v=FAKE, vs=1024, c=FAKE, nb=10, bs=16, hkv=8, d=128, sm=FAKE, n=4):
        return lib.pkv_read_int4(c, nb, bs, hkv, d, sm, n, k, ks, v, vs, None)

    for f in (w, r):
        assert f(bs=8) == -2 and f(d=64) == -2 and f(hkv=40000) == -2
        assert f(hkv=0) == -1 and f(n=-1) == -1 and f(nb=0) == -1
        assert f(k=None) == -1 and f(v=None) == -1 and f(c=None) == -1 and f(sm=None) == -1
        assert f(ks=1000) == -1 and f(vs=1016) == -1
        assert f(ks=1028) == -3 and f(k=FAKE + 8) == -3 and f(c=FAKE + 4) == -3
        assert f(n=0, k=None, v=None, c=None, sm=None) == 0


def test_attention(lib):
    def a(q=FAKE, qs=4096, rows=4, hq=32, c=FAKE, nb=10, bs=16, hkv=8, d=128, qsl=FAKE, sl=FAKE,
          bt=FAKE, w=4, R=2, scale=0.088, out=FAKE, os=4096):
        return lib.pkv_attention_int4(q, qs, rows, hq, c, nb, bs, hkv, d, qsl, sl, bt, w, R, scale,
                                      out, os, None)

    assert a(hq=30) == -2 and a(hq=512, qs=65536, os=65536) == -2 and a(bs=32) == -2
    assert a(d=64) == -2 and a(w=40000) == -2
    assert a(R=-1) == -1 and a(qs=100) == -1 and a(qsl=None) == -1 and a(c=None) == -1
    assert a(nb=0) == -1 and a(w=0) == -1 and a(scale=float("nan")) == -1
    assert a(c=FAKE + 8) == -3 and a(out=FAKE + 8) == -3 and a(qs=4100) == -3
    assert a(R=0) == 0 and a(rows=0) == 0


def test_binding():
    bf, u8 = torch.bfloat16, torch.uint8
    k = torch.zeros(2, 8, 128, dtype=bf)
    c = torch.zeros(4, 8, pkv.INT4_PAGE_BYTES, dtype=u8)
    sm = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.pkv_write_int4(k, k, c, sm)
    with pytest.raises(TypeError):
        pkv.pkv_write_int4(k.float(), k, c, sm)
    with pytest.raises(TypeError):
        pkv.pkv_attention_int4(None, c, sm, sm, sm, 1, 1.0, k)
