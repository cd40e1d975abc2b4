"""hc_mixes_pre_backward at the Sinkhorn step counts around 48 KB of shared memory (GPU).

k_mix_backward keeps HC * 8 * (2 iters - 1) divisors beside a few hundred bytes of its own; what a
launch may use without asking is 48 KB for both together.  The calls run in a process of their own,
as one with more steps raises the limit for all that follow.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
CHILD = """
import sys
sys.path[:0] = [%r, %r]
import test_gpu_train as t
import sinkhorn_mixing_gb300 as hc
for copies, counts in ((4, (191, 192, 193)), (8, (95, 96, 97))):
    for iters in counts:
        for k8 in (True, False):
            c = t.pre_case(hc, 9, copies, 64, k8, seed=iters)
            t.check_pre(t.run_pre(hc, c, iters=iters), c, iters=iters)
assert hc.hc_device_error(clear=True) == 0
print("steps ok")
""" % (os.path.dirname(HERE), HERE)


def test_steps_around_the_shared_memory_limit():
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "steps ok" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
