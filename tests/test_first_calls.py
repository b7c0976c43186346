"""Several threads whose first call of the library is a Linear, in a process of their own."""
import os
import subprocess
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu

PROGRAM = """
import threading
import torch
import fusion_add_rmsnorm_gb300 as gbf

N, K = 256, 512
x = torch.full((40, K), 0x38, dtype=torch.uint8, device="cuda")          # ones
w = torch.full((N, K), 0x38, dtype=torch.uint8, device="cuda")
xs, ws = torch.ones(40, K // 128, device="cuda"), torch.ones(N // 128, K // 128, device="cuda")
ys = [torch.zeros(40, N, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
bf = lambda t: t.view(torch.uint8).repeat_interleave(2, 1).view(torch.bfloat16).fill_(1.0)   # noqa: E731
xb, wb = bf(x), bf(w)
torch.cuda.synchronize()
start, wrong = threading.Barrier(8), []

def call(i):
    try:
        torch.cuda.set_device(0)
        start.wait()
        if i % 2:
            gbf.linear_fp8_block(x, xs, w, ws, None, ys[i], act=gbf.ACT_NONE)
        else:
            gbf.linear_bias_gelu(xb, wb, None, ys[i], act=gbf.ACT_NONE)
    except Exception as e:  # noqa: BLE001 - the main thread reports it
        wrong.append((i, repr(e)))

threads = [threading.Thread(target=call, args=(i,)) for i in range(8)]
for t in threads:
    t.start()
for t in threads:
    t.join()
torch.cuda.synchronize()
assert not wrong, wrong
assert all((y == K).all() for y in ys)
assert gbf.device_status()[0] == gbf.OK
print("ok")
"""


def test_first_calls_of_several_threads():
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0 and r.stdout.split() == ["ok"], r.stdout + r.stderr
