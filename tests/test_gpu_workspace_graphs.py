"""The workspace that a captured graph holds, in processes of their own (within
the suite's process the workspace has long grown past what a test needs): growing it
keeps the old one where a graph was captured on it, and frees it where none was.
What was kept is read off the device's free memory, before any graph is replayed."""
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
from paged_kv_attention_05_gb300 import workloads as W
from gpu_util import DeviceStep

kind = sys.argv[1]
ds = DeviceStep(W.build(W.custom([700, 3000, 0], [1, 4, 200], 8, 2, seed=98)))
ds.write()
st, width = ds.step, ds.block_table.shape[1]

def scored():
    pkv.pkv_attention_scored(ds.q, ds.key_cache, ds.value_cache, ds.qsl, ds.seq_lens,
                             ds.block_table, 3, st.scale, ds.out, softcap=30.0)

def planned():
    pkv.pkv_plan(ds.q.shape[0], 8, 2, ds.qsl, ds.seq_lens, width, 3)
    for _ in range(2):
        pkv.pkv_attention_planned(ds.q, ds.key_cache, ds.value_cache, ds.block_table, st.scale,
                                  ds.out)

go = {"scored": scored, "plain": ds.attention, "planned": planned, "none": scored}[kind]
size = lambda r: pkv.pkv_workspace_size(r, 4096, 2048, 32, 8, pkv.pkv_num_sms())["bytes"]

def reserve(at_least):
    reqs = 8
    while size(reqs) < at_least:
        reqs *= 2
    pkv.pkv_reserve_workspace(reqs, 4096, 2048, 32, 8)
    return size(reqs) * 5 // 4      # (a workspace is made a quarter larger than asked for)

free = lambda: torch.cuda.mem_get_info()[0]
go()
first = reserve(1 << 28)
go()
torch.cuda.synchronize()
want = ds.out.clone()
n = int(st.query_start_loc[-1])
if kind != "none":
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
torch.cuda.synchronize()
before = free()
second = reserve(2 * first)
took = before - free()
slack = 16 << 20
assert second > first + 4 * slack
if kind == "none":
    assert abs(took - (second - first)) < slack, (took, first, second)
else:
    assert abs(took - second) < slack, (took, first, second)
    filler = torch.full((first,), 255, dtype=torch.uint8, device="cuda")
    for turn in range(3):
        ds.out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ds.out[:n], want[:n]), "replay %%d" %% turn
        ds.out.fill_(float("nan"))
        go()                        # on the larger one
        torch.cuda.synchronize()
        assert torch.equal(ds.out[:n], want[:n]), "call %%d" %% turn
    assert int(filler.min()) == 255
assert pkv.pkv_get_error() == 0
print("as it should be")
"""


@pytest.mark.parametrize("kind", ["scored", "plain", "planned", "none"])
def test_growing_the_workspace(kind):
    code = SCRIPT % {"root": os.path.dirname(HERE), "here": HERE}
    r = subprocess.run([sys.executable, "-c", code, kind], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "as it should be" in r.stdout, r.stdout + r.stderr
