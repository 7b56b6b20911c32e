"""paged_kv4_attention captured in a fresh process: one call of a head size, of any
form, is all that has to come before it."""
import os
import subprocess
import sys

import pytest

from conftest import REPO

pytestmark = pytest.mark.gpu

PROGRAM = r"""
import sys
import torch
from paged_attention_kv_gb300 import binding as pkv
d, first = int(sys.argv[1]), int(sys.argv[2])
gen = torch.Generator(device="cuda").manual_seed(1)
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
pool = pkv.alloc_kv4_cache(300, 2, d)
k, v = (torch.randn(300 * 16, 2, d, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
pkv.paged_kv4_write(k, v, torch.arange(300 * 16, dtype=torch.int32, device="cuda"), pool)
ws = pkv.alloc_kv4_workspace(pool)

def call(new):
    q = torch.randn(3 * new, 8, d, generator=gen, device="cuda").to(torch.bfloat16)
    table = torch.randperm(300, generator=gen, device="cuda").int().view(3, 100)
    return pkv.prepare_kv4_attention(q, pool, table, i32([new + 3, 900, 1600]), i32([0, new, 2 * new, 3 * new]), 0.1,
                                     max_query_len=new, workspace=ws)

calls = [call(n) for n in (1, 4, 12, 40, 200)]  # up to 8 rows of a head, 16, more, and chunks
calls[first]()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    for c in calls:
        c()
for c in calls:
    c.outputs.zero_()
g.replay()
torch.cuda.synchronize()
got = [c.outputs.clone() for c in calls]
assert all(torch.equal(c(), x) and x.any() for c, x in zip(calls, got))
print("same")
"""


@pytest.mark.parametrize("d,first", [(64, 0), (128, 0), (128, 4)])
def test_a_first_call_of_one_form_and_a_capture_of_all(d, first):
    res = subprocess.run([sys.executable, "-c", PROGRAM, str(d), str(first)], cwd=REPO, env=dict(os.environ, PYTHONPATH=REPO),
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout.strip() == "same", res.stderr[-2000:]
