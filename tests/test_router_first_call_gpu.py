"""Expert counts around 48 KB of shared memory, each in a process whose first
router call it is (a larger call before it would have raised the limit)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CALL = """
import sys
import torch
import combine_send_counts_gb300 as ep
E = int(sys.argv[1])
w = torch.zeros((E, 8), dtype=torch.bfloat16, device="cuda")
w[[E - 1, 3], 0] = torch.tensor([2.0, 1.0], dtype=torch.bfloat16, device="cuda")
x = torch.ones((2, 8), dtype=torch.bfloat16, device="cuda")
idx, _ = ep.router_topk(x, w, 3)
assert idx.tolist() == [[E - 1, 3, 0]] * 2, idx
"""


@pytest.mark.parametrize("E", [6140, 6141, 6144, 6145])
def test_first_call(E):
    env = dict(os.environ, PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", CALL, str(E)], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
