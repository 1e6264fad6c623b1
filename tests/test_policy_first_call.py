"""policy_loss as the first call of a process, with slices just below 48 KB (one GB300).

What a kernel was once allowed to take of shared memory it keeps, so a call of another size before
would hide that a launch asks for too little: each of the four forms of the gradient's kernel (two
types, rows of whole words or not) is called here for the first time.
"""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))

CODE = """
import sys
sys.path[:0] = [{root!r}, {here!r}]
import torch
import test_parity_policy as t
for R, V, dtype in {cases}:
    d = t.inputs(R, V, dtype, seed=V)
    got = t.call(d)
    t.check(d, got, t.oracle(d), 1.0, 0.05)
    assert t.vsd.device_status(got["ws"]) == 0
print("fine")
"""


# slices of 3041 to 3072 words: one CTA a row, two, or (a few rows) many
@pytest.mark.parametrize("cases", [
    "[(200, 24500, torch.bfloat16), (200, 24504, torch.bfloat16), (200, 12250, torch.float32), (200, 12260, torch.float32)]",
    "[(200, 49000, torch.bfloat16), (200, 49003, torch.bfloat16), (160, 24516, torch.float32), (160, 24517, torch.float32)]",
    "[(7, 122600, torch.bfloat16), (7, 122601, torch.bfloat16), (7, 61300, torch.float32), (7, 61301, torch.float32)]",
])
def test_first_call_of_a_process(spec, cases):
    code = CODE.format(root=os.path.dirname(HERE), here=HERE, cases=cases)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr[-2000:]
