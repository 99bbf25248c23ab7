"""The first call of a process on a stream that does not wait for the legacy default
stream (as torch's side streams do not): workspaces and error words are zero before the
call's kernels run, in calls that make them, grow them, or follow a reservation at once.
In processes of their own: within the suite's the workspaces have long been made."""
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
import test_gpu_int4 as I

kind = sys.argv[1]
side = torch.cuda.Stream()
BITS = pkv.DEV_ERR_BITS

def select_case(width, rows, seed):
    reqs = [(50 * i %% 2500, 1) for i in range(rows)]
    q, bounds, reqs, bt, qsl, seq = P.a_case(16, 8, reqs, seed)
    wide = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    wide[:, :bt.shape[1]] = bt
    args = q, bounds, reqs, wide, qsl, seq
    want = P.select_ref(q, bounds, reqs, wide, 24, 1, 1)
    return args, want

def check_lists(got, want):
    n = want[0].shape[0] - 2
    assert torch.equal(got[1], want[1]) and torch.equal(got[0][:n], want[0][:n])

if kind.startswith("select"):
    # a clear of 26 MB, then one of 420
    cases = [select_case(2600, 20, 1), select_case(32768, 130, 3)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = []
        for args, _ in cases:
            if kind == "select after a reservation":
                pkv.pkv_reserve_select(args[0].shape[0], args[3].shape[1], 8)
            got += [P.run_select(*args, 24, 1, 1) for _ in range(3)]
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        check_lists(g, cases[i // 3][1])
elif kind.startswith("attention"):
    steps = [I.Step([(700, 1), (3000, 2), (0, 200)], 8, 2, 98),
             I.Step([(c, 1 + c %% 2) for c in range(900, 1150)], 8, 2, 99)]
    for s in steps:
        I.R.write(s.k, s.v, s.cache, s.slots)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        if kind == "attention after a reservation":
            pkv.pkv_reserve_workspace(300, 2000, 4096, 32, 2)
        for s in steps:
            s.attention()
            s.attention()
    torch.cuda.synchronize()
    for s in steps:
        s.check(kind)
else:
    # an error of the first call, and one of the call after a read of the word
    g = I.gen(1)
    cache, x = I.fill(2, 2, g), I.randn((3, 2, 128), g)
    slots = torch.tensor([-1, 32, 5], device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            pkv.pkv_write_int4(x, x, cache, slots)
            assert pkv.pkv_get_error() == BITS["SLOT_RANGE"]
torch.cuda.synchronize()
assert pkv.pkv_get_error() == 0
print("as it should be")
"""


@pytest.mark.parametrize("kind", ["select", "select after a reservation", "attention",
                                  "attention after a reservation", "errors"])
def test_first_calls_on_a_side_stream(kind):
    r = subprocess.run([sys.executable, "-c",
                        SCRIPT % {"root": os.path.dirname(HERE), "here": HERE}, kind],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "as it should be" in r.stdout, r.stdout + r.stderr
