"""Balance loss at the borders of what the call accepts."""
import os
import subprocess
import sys
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu

HERE = Path(__file__).resolve().parent

FIRST_CALL = """
import numpy as np, torch
import moe_expert_layer_topk_gb300 as m
import ops_ref
from test_gpu_balance import COEF, call, compare, inputs
for E, S in ({sizes}):
    T, k = 2000, 4
    l, idx, mask = inputs(T, E, k, seed=E)
    offsets = np.sort(np.random.RandomState(S).randint(0, T + 1, S + 1)).tolist()
    for grad in (False, True):
        o = call(l, idx, None, offsets, k, grad=grad)
        compare(o, ops_ref.balance(l.cpu().numpy(), idx.cpu().numpy(), None, offsets, k, *COEF))
assert m.moe_read_device_status(reset=True) == 0
print("fine")
"""


# 48 KB of dynamic shared memory, to the byte or one sequence either side of
# it: with the kernel's static variables more than a launch has unasked
@pytest.mark.parametrize("sizes", ["(128, 950), (236, 32)", "(128, 951), (192, 406)", "(192, 407),", "(236, 33),"])
def test_first_call_at_48_kb_of_shared_memory(sizes):
    """In a process of its own: an earlier, larger call would have asked for more."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.replace("{sizes}", sizes)], capture_output=True, text=True, timeout=300,
                       cwd=HERE.parent, env={**os.environ, "PYTHONPATH": f"{HERE.parent}:{HERE}"})
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]
