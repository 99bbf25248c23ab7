"""pkv_write_rope / pkv_write_rope_int8: what the host refuses before touching
a device, through the C ABI and through the Python binding."""
import pytest

FAKE = 0x10000  # a non-null, 16-byte aligned address; never dereferenced by these calls


@pytest.fixture(scope="module")
def lib():
    from paged_kv_attention_05_gb300 import build as b
    b.build()
    import paged_kv_attention_05_gb300 as pkv
    return pkv.load()


def call(lib, int8=False, **kw):
    a = dict(q=FAKE, qs=4096, hq=32, k=FAKE, ks=1024, v=FAKE, vs=1024, qw=None, kw=None, off=0.0,
             eps=1e-6, cs=FAKE, mp=100, rot=128, il=0, pos=FAKE, qo=FAKE, qos=4096, kc=FAKE,
             vc=FAKE, k_scale=0.1, v_scale=0.1, nb=10, bs=16, hkv=8, d=128, sm=FAKE, n=4)
    assert set(kw) <= set(a)
    a.update(kw)
    head = [a[x] for x in ("q", "qs", "hq", "k", "ks", "v", "vs", "qw", "kw", "off", "eps", "cs",
                           "mp", "rot", "il", "pos", "qo", "qos", "kc", "vc")]
    tail = [a[x] for x in ("nb", "bs", "hkv", "d", "sm", "n")] + [None]
    if int8:
        return lib.pkv_write_rope_int8(*head, a["k_scale"], a["v_scale"], *tail)
    return lib.pkv_write_rope(*head, *tail)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("bad,code", [
    (dict(bs=8), -2), (dict(d=64), -2), (dict(hkv=0), -1), (dict(hkv=40000), -2),
    (dict(hq=0), -1), (dict(hq=-1), -1), (dict(n=-1), -1), (dict(nb=0), -1),
    (dict(rot=0), -2), (dict(rot=8), -2), (dict(rot=24), -2), (dict(rot=136), -2),
    (dict(rot=256), -2), (dict(rot=-16), -2), (dict(mp=0), -1),
    (dict(qw=FAKE, eps=-1.0), -1), (dict(kw=FAKE, eps=float("nan")), -1),
    (dict(qw=FAKE, eps=float("inf")), -1), (dict(kw=FAKE, off=float("nan")), -1),
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(cs=None), -1),
    (dict(pos=None), -1), (dict(qo=None), -1), (dict(kc=None), -1), (dict(vc=None), -1),
    (dict(sm=None), -1), (dict(qs=4088), -1), (dict(qos=4088), -1), (dict(ks=1016), -1),
    (dict(vs=1016), -1), (dict(q=FAKE + 8), -3), (dict(qo=FAKE + 2), -3), (dict(cs=FAKE + 4), -3),
    (dict(qw=FAKE + 8), -3), (dict(kw=FAKE + 8), -3), (dict(qs=4100), -3), (dict(ks=1028), -3),
    (dict(vc=FAKE + 8), -3),
])
def test_refused_on_the_host(lib, int8, bad, code):
    assert call(lib, int8, **bad) == code
    assert lib.pkv_last_error_string()


def test_int8_scales_must_be_finite_and_positive(lib):
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert call(lib, True, k_scale=s) == -1
        assert call(lib, True, v_scale=s) == -1


def test_packed_structs_match_the_header():
    """The binding's struct formats against the C compiler's layout."""
    import os
    import subprocess
    import tempfile
    from paged_kv_attention_05_gb300 import _binding as b
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = r"""
#include <stddef.h>
#include <stdio.h>
#include "pkv.h"
int main(void) {
  printf("%zu %zu %zu %zu %zu %zu\n", sizeof(pkv_write_rope_args),
         offsetof(pkv_write_rope_args, num_heads), offsetof(pkv_write_rope_args, v_scale),
         sizeof(pkv_attention_scored_args), offsetof(pkv_attention_scored_args, num_heads),
         offsetof(pkv_attention_scored_args, softcap));
  return 0;
}
"""
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "t")
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(root, "include"), "-x", "c", "-",
                        "-o", exe], input=src, text=True, check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True,
                                              check=True).stdout.split()]
    assert got == [b._ROPE_ARGS.size, 19 * 8, b._ROPE_ARGS.size - 4,
                   b._SCORED_ARGS.size, 15 * 8, b._SCORED_ARGS.size - 4]


def test_packed_calls_check_like_the_others(lib):
    assert lib.pkv_write_rope_packed(None, 0) == -1
    assert lib.pkv_attention_scored_packed(None) == -1
    from paged_kv_attention_05_gb300 import _binding as b
    ok = dict(heads=(32, 8, 128, 16, 128, 0))
    pack = lambda heads, n=4, sc=0.1: b._ROPE_ARGS.pack(  # noqa: E731
        FAKE, 4096, FAKE, 1024, FAKE, 1024, 0, 0, FAKE, 100, FAKE, FAKE, 4096, FAKE, FAKE, 10,
        FAKE, n, 0, *heads, 0.0, 1e-6, sc, 0.1)
    assert lib.pkv_write_rope_packed(pack(n=0, **ok), 0) == 0
    assert lib.pkv_write_rope_packed(pack(n=-1, **ok), 0) == -1
    assert lib.pkv_write_rope_packed(pack((32, 8, 64, 16, 128, 0)), 0) == -2
    assert lib.pkv_write_rope_packed(pack((32, 8, 128, 16, 24, 0)), 1) == -2
    assert lib.pkv_write_rope_packed(pack(sc=0.0, n=0, **ok), 1) == -1
    assert lib.pkv_write_rope_packed(pack(sc=0.0, n=0, **ok), 0) == 0
    scored = lambda heads, scale=0.1, cap=0.0: b._SCORED_ARGS.pack(  # noqa: E731
        FAKE, 4096, 4, FAKE, FAKE, 10, FAKE, FAKE, FAKE, 4, 0, 0, FAKE, 4096, 0, *heads, scale,
        cap)
    assert lib.pkv_attention_scored_packed(scored((32, 8, 128, 16, 0, 0))) == 0
    assert lib.pkv_attention_scored_packed(scored((30, 8, 128, 16, 2, 0))) == -2
    assert lib.pkv_attention_scored_packed(scored((32, 8, 128, 16, 2, -1))) == -1
    assert lib.pkv_attention_scored_packed(scored((32, 8, 128, 16, 2, 0), cap=-1.0)) == -1


def test_no_tokens_is_not_an_error(lib):
    assert call(lib, n=0, q=None, k=None, v=None, sm=None) == 0
    assert call(lib, True, n=0) == 0


def test_binding_refuses_what_it_cannot_pass_on():
    torch = pytest.importorskip("torch")
    import paged_kv_attention_05_gb300 as pkv
    bf = dict(dtype=torch.bfloat16)
    q, k = torch.zeros(2, 8, 128, **bf), torch.zeros(2, 2, 128, **bf)
    kc = torch.zeros(4, 16, 2, 128, **bf)
    i = torch.zeros(2, dtype=torch.int64)
    cs = torch.zeros(10, 128)
    with pytest.raises(ValueError):     # not on a device
        pkv.pkv_write_rope(q, k, k, i, cs, kc, kc, i, q)
    with pytest.raises(TypeError):      # wrong type
        pkv.pkv_write_rope(q.float(), k, k, i, cs, kc, kc, i, q)
    with pytest.raises(TypeError):
        pkv.pkv_write_rope("q", k, k, i, cs, kc, kc, i, q)
