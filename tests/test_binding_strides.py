"""The binding and the strides of dimensions of size one, which address nothing:
views of one head or one row are taken whatever stride torch gives them, others
only with contiguous heads."""
import pytest

torch = pytest.importorskip("torch")

from paged_kv_attention_05_gb300 import _binding as b  # noqa: E402

D = 128


class Recorder:
    """Stands for the library: keeps the structs, enqueues nothing."""

    def __init__(self):
        self.rope = self.scored = None

    def pkv_write_rope_packed(self, args, int8):
        self.rope = b._ROPE_ARGS.unpack(args)
        return 0

    def pkv_attention_scored_packed(self, args):
        self.scored = b._SCORED_ARGS.unpack(args)
        return 0


@pytest.fixture
def lib(monkeypatch):
    r = Recorder()
    b._T()
    monkeypatch.setattr(b, "_lib", r)
    monkeypatch.setattr(b, "_get_device", lambda: -1)   # where a CPU tensor says that it is
    return r


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def one_head(n):
    """[n, 1, 128] as a model's transpose of [1, n, 128] gives it: stride(1) is n * 128."""
    t = bf(1, n, D).transpose(0, 1)
    assert t.stride() == (D, n * D, 1)
    return t


def one_row(heads):
    """[1, heads, 128] from [heads, 1, 128]: stride(0) is 128."""
    t = bf(heads, 1, D).transpose(0, 1)
    assert t.stride() == (D, D, 1)
    return t


def rope(q, k, v, q_out, n):
    i = torch.zeros(n, dtype=torch.int64)
    kc = bf(4, 16, k.shape[1], D)
    b.pkv_write_rope(q, k, v, i, torch.zeros(10, D), kc, kc.clone(), i, q_out, stream=0)


def scored(q, out, hkv):
    kc = bf(4, 16, hkv, D)
    i = torch.zeros(2, dtype=torch.int32)
    b.pkv_attention_scored(q, kc, kc.clone(), i, i, i.view(1, 2), 1, 0.1, out, stream=0)


def test_write_rope_takes_views_of_one_head(lib):
    rope(bf(5, 8, D), one_head(5), one_head(5), bf(5, 8, D), 5)
    assert lib.rope[1] == lib.rope[12] == 8 * D and lib.rope[3] == lib.rope[5] == D
    rope(one_head(5), one_head(5), bf(5, 1, D), one_head(5), 5)
    assert lib.rope[1] == lib.rope[12] == D


def test_write_rope_takes_views_of_one_row(lib):
    rope(one_row(8), one_row(2), one_row(2), one_row(8), 1)
    assert lib.rope[1] == lib.rope[12] == 8 * D and lib.rope[3] == lib.rope[5] == 2 * D


def test_scored_attention_takes_views_of_one_head_or_row(lib):
    scored(one_head(7), one_head(7), 1)
    assert lib.scored[1] == lib.scored[13] == D
    scored(one_row(8), one_row(8), 2)
    assert lib.scored[1] == lib.scored[13] == 8 * D
    scored(one_row(8), bf(3, 8, D), 2)     # (out may have more rows)
    assert lib.scored[1] == lib.scored[13] == 8 * D


def test_strides_that_count_are_still_refused(lib):
    good, two = bf(5, 2, D), bf(2, 5, D).transpose(0, 1)     # heads 5 rows apart
    for bad in ((two, good, good, good), (good, two, good, good), (good, good, two, good),
                (good, good, good, two)):
        with pytest.raises(ValueError):
            rope(*bad, 5)
    half = bf(5, 2, 2 * D)[..., ::2]
    with pytest.raises(ValueError):
        rope(half, good, good, good, 5)
    with pytest.raises(ValueError):
        rope(bf(5, 1, 2 * D)[..., ::2], good, good, bf(5, 1, D), 5)
    for q, out in ((two, good), (good, two), (half, good), (good, half)):
        with pytest.raises(ValueError):
            scored(q, out, 2)
    assert lib.rope is None and lib.scored is None


def test_rows_of_the_other_calls():
    assert b._rows3(bf(5, 4, D), "q") == 4 * D
    assert b._rows3(bf(5, 9 * D)[:, :4 * D].view(5, 4, D), "q") == 9 * D
    assert b._rows3(one_head(5), "k") == D
    assert b._rows3(one_row(8), "q") == 8 * D
    assert b._rows3(bf(8 * D, 1).t(), "out") == 8 * D
    for bad in (bf(2, 5, D).transpose(0, 1), bf(5, 2, 2 * D)[..., ::2], bf(5, 2 * D)[:, ::2],
                bf(2, 2, 2, D)):
        with pytest.raises(ValueError):
            b._rows3(bad, "q")
