"""A process whose daemon thread is inside the host module's calls when the interpreter ends:
Python ends such a thread by unwinding it, which must not abort the process.

The calls are ones that the library refuses, so that nothing but the module's own handling of
the lock is in question: torch's own calls (a loop of torch.empty on the device) abort there."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import threading
import torch
import block_scaled_precision_nvfp4_b200 as nv
a = torch.zeros(4, 24, dtype=torch.int8, device="cuda")     # K is no multiple of 16
s = torch.ones(4, device="cuda")
gemm = nv._host().fast_gemm
assert gemm(a, s, a, s) == nv.Status.INVALID_ARG
running = threading.Event()
def loop():
    for i in range(10000000):
        gemm(a, s, a, s)
        if i == 100:
            running.set()
threading.Thread(target=loop, daemon=True).start()
assert running.wait(60)
print("leaving", flush=True)
"""


def test_exit_with_a_daemon_thread_inside_a_call():
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
        assert "leaving" in r.stdout and r.returncode == 0, (r.returncode, r.stderr[-2000:])
