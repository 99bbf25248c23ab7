"""Sizes that pkv_reserve_select refuses on the host (no GPU is touched)."""
import paged_kv_attention_05_gb300 as pkv


def test_more_rows_than_a_call_takes():
    """As pkv_select_pages refuses them; their room in bytes would not fit 64 bits."""
    from paged_kv_attention_05_gb300 import build
    build.build()
    lib = pkv.load()
    assert lib.pkv_reserve_select(1 << 31, 10, 8) == -2
    assert lib.pkv_reserve_select(1 << 40, 32768, 32767) == -2
    assert lib.pkv_reserve_select((1 << 63) - 1, 1, 1) == -2
