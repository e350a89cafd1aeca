"""What the first calls of a process set up: each family of entry points its own kernels."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import json, sys
import torch
from torch.profiler import ProfilerActivity, profile
sys.path.insert(0, sys.argv[1])
import top_reduction_gb300 as lmh
z, u = torch.randn(4, 1024, device="cuda"), torch.rand(4, device="cuda")
x = torch.randn(2, 64, device="cuda").to(torch.bfloat16)
with profile(activities=[ProfilerActivity.CPU, ProfilerActivity.CUDA]):  # (its own start)
    z.sum().item()
def attributes(call):
    with profile(activities=[ProfilerActivity.CPU, ProfilerActivity.CUDA]) as prof:
        call()
        torch.cuda.synchronize()
    return sum(e.name == "cudaFuncSetAttribute" for e in prof.events())
t = lmh.Q4Table(torch.zeros(100, 32, dtype=torch.uint8, device="cuda"), torch.ones(100, 1, device="cuda"))
calls = [lambda: lmh.logprobs_from_logits(z), lambda: lmh.sample_from_logits(z, u), lambda: lmh.project_q4(x, t)]
print(json.dumps([attributes(c) for c in calls] + [attributes(c) for c in calls]))
"""


def test_a_call_sets_up_its_own_kernels_alone(lmh):
    """The first reduction does not wait for the draw's and the 4-bit projection's kernels to be loaded."""
    r = subprocess.run([sys.executable, "-c", SCRIPT, ROOT], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    reduction, draw, projection, *again = json.loads(r.stdout.splitlines()[-1])
    if reduction == 0:
        pytest.skip("the profiler does not see the runtime's calls here")
    assert draw > 0 and projection > 0
    assert again == [0, 0, 0]
