"""The room that pkv_select_pages' workspace takes, in a process of its own, read off the
device's free memory."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))

SCRIPT = r"""
import sys
sys.path[:0] = [%(root)r, %(here)r]
import torch
import paged_kv_attention_05_gb300 as pkv
import test_gpu_pages as P

pkv.pkv_num_sms()
torch.zeros(1, device="cuda")
free = lambda: torch.cuda.mem_get_info()[0]
PAGE = 2 << 20      # the device gives memory in such pieces
before = free()
# the most that rows share: the documented 340 MB, and no more
for rows, width, hkv in ((130, 32768, 8), (1 << 20, 32768, 8), (100000, 5, 32), (1, 32768, 512)):
    pkv.pkv_reserve_select(rows, width, hkv)
    took = before - free()
    assert took <= 340_000_000 + PAGE, (rows, width, hkv, took)
assert took >= 20 << 24
# what a row needs alone, where that is more
pkv.pkv_reserve_select(1, 32768, 600)
took = before - free()
need = 32768 * 600 * 20 + 65536 * 4
assert need <= took <= need + PAGE, took
reqs = [(50 * i %% 2500, 1) for i in range(130)]
q, bounds, reqs, bt, qsl, seq = P.a_case(16, 8, reqs, 3)
wide = torch.full((130, 32768), -1, dtype=torch.int32, device="cuda")
wide[:, :bt.shape[1]] = bt
P.check_select(q, bounds, reqs, wide, qsl, seq, 24, 1, 1)
assert pkv.pkv_get_error() == 0
print("as it should be")
"""


def test_room_of_the_selection():
    r = subprocess.run([sys.executable, "-c",
                        SCRIPT % {"root": os.path.dirname(HERE), "here": HERE}],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "as it should be" in r.stdout, r.stdout + r.stderr
