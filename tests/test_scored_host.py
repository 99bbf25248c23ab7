"""pkv_attention_scored: what the host refuses before touching a device."""
import pytest

FAKE = 0x10000  # a non-null, 16-byte aligned address; never dereferenced by these calls


@pytest.fixture(scope="module")
def lib():
    from paged_kv_attention_05_gb300 import build as b
    b.build()
    import paged_kv_attention_05_gb300 as pkv
    return pkv.load()


def call(lib, **kw):
    a = dict(q=FAKE, qs=4096, rows=4, hq=32, kc=FAKE, vc=FAKE, nb=10, bs=16, hkv=8, d=128,
             qsl=FAKE, sl=FAKE, bt=FAKE, w=4, R=2, scale=0.088, cap=0.0, window=0, slopes=None,
             prefix=None, out=FAKE, os=4096)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.pkv_attention_scored(*[a[x] for x in (
        "q", "qs", "rows", "hq", "kc", "vc", "nb", "bs", "hkv", "d", "qsl", "sl", "bt", "w", "R",
        "scale", "cap", "window", "slopes", "prefix", "out", "os")], None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("bad,code", [
    (dict(cap=-1.0), -1), (dict(cap=NAN), -1), (dict(cap=INF), -1), (dict(window=-1), -1),
    (dict(cap=1e-45), -1), (dict(cap=3e38), -1), (dict(scale=0.0), -1), (dict(scale=-0.1), -1),
    (dict(scale=INF), -1), (dict(scale=NAN), -1), (dict(hq=30), -2),
    (dict(hq=512, qs=65536, os=65536), -2), (dict(bs=32), -2), (dict(d=64), -2), (dict(R=-1), -1),
    (dict(rows=-1), -1), (dict(qs=100), -1), (dict(os=4088), -1), (dict(out=FAKE + 8), -3),
    (dict(q=FAKE + 2), -3), (dict(qs=4100), -3), (dict(qsl=None), -1), (dict(sl=None), -1),
    (dict(bt=None), -1), (dict(q=None), -1), (dict(out=None), -1), (dict(w=0), -1),
    (dict(w=40000), -2), (dict(hkv=0), -1), (dict(nb=0), -1),
])
def test_refused_on_the_host(lib, bad, code):
    assert call(lib, **bad) == code
    assert lib.pkv_last_error_string()


def test_an_empty_step_is_not_an_error(lib):
    assert call(lib, R=0) == 0
    assert call(lib, rows=0, cap=30.0, window=5) == 0


def test_binding_refuses_what_it_cannot_pass_on():
    torch = pytest.importorskip("torch")
    import paged_kv_attention_05_gb300 as pkv
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    kc = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):     # not on a device
        pkv.pkv_attention_scored(q, kc, kc, i, i, i, 1, 0.1, q)
    with pytest.raises(TypeError):
        pkv.pkv_attention_scored(q.float(), kc, kc, i, i, i, 1, 0.1, q)
