"""The first calls of the 8-bit projection in a process, from several threads at once
and with different widths."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import threading
import torch
from fibonacci_spaced_sparse_gb300 import api
FP8 = torch.float8_e4m3fn
widths = [512, 128, 384, 256]
data = []
for dm in widths:
    x, w = (torch.randint(0, 0x70, (n, dm), dtype=torch.uint8, device="cuda").view(FP8) for n in (4096, 768))
    data.append((x[None], torch.ones(1, 4096, device="cuda"), w, torch.ones(768, device="cuda")))
api._native()
torch.cuda.synchronize()
failed, start = [], threading.Barrier(len(widths))
def work(args):
    torch.cuda.set_device(0)
    side = torch.cuda.Stream()
    start.wait()
    try:
        for _ in range(3):
            api.sfa_qkv_rope_fp8(*args, rope_theta=0.0, stream=side)
    except Exception as e:
        failed.append(f"{args[0].shape[-1]}: {e}")
threads = [threading.Thread(target=work, args=(a,)) for a in data]
for t in threads:
    t.start()
for t in threads:
    t.join()
torch.cuda.synchronize()
print("failed:", failed)
raise SystemExit(1 if failed else 0)
"""


@pytest.mark.parametrize("turn", range(4))
def test_widths_of_several_threads_at_first_use(turn):
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=dict(os.environ, PYTHONPATH=ROOT), capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
