"""A process whose daemon thread is inside the host module's calls when the interpreter ends:
Python ends such a thread by unwinding it, which must not abort the process."""
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
x = torch.ones(16, 256, device="cuda", dtype=torch.bfloat16)
nv.int8_quantize_bf16(x)
assert nv._host().fast_quantize is not nv._no_fast_call
running = threading.Event()
def loop():
    for i in range(1000000):
        nv.int8_quantize_bf16(x)
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
