"""A process whose first block-scaled calls are captured into a graph: nothing is loaded, asked
for or raised on the way that a capture does not allow, and the graph gives what eager calls give."""
import os
import subprocess
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu

PROGRAM = """
import sys
import torch
import fusion_add_rmsnorm_gb300 as gbf

m, h, f = map(int, sys.argv[1:])
g = torch.Generator(device="cuda").manual_seed(m)
bf = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()                 # noqa: E731
codes = lambda r, d: (torch.zeros(r, d, dtype=torch.uint8, device="cuda"), torch.zeros(r, -(-d // 128), device="cuda"))  # noqa: E731
x, res, w, w_up = bf(m, h), bf(m, h), bf(h), bf(2 * f, h)
out, up = torch.zeros_like(x), torch.zeros(m, 2 * f, dtype=torch.bfloat16, device="cuda")
c1, c2 = codes(m, h), codes(m, f)
wq, ws = torch.zeros(2 * f, h, dtype=torch.uint8, device="cuda"), torch.zeros(-(-2 * f // 128), -(-h // 128), device="cuda")

def step():
    gbf.quantize_fp8_block(w_up, wq, ws, block_rows=128)
    gbf.add_rmsnorm_fp8_block(x, res, out, *c1, gbf.NORM_WEIGHT, weight=w)
    gbf.linear_fp8_block(*c1, wq, ws, None, up, act=gbf.ACT_NONE)
    gbf.gated_act_fp8_block(up, *c2, act=gbf.ACT_SILU)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
outs = (wq, ws, out, *c1, up, *c2)
graph.replay()
torch.cuda.synchronize()
first = [t.clone() for t in outs]
for t in outs:
    t.zero_()
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(first, outs)) and c2[0].any()
assert gbf.device_status()[0] == gbf.OK
print(*gbf.linear_fp8_block_plan(m, 2 * f, h))
"""


@pytest.mark.parametrize("m,h,f,rows", [(3, 400, 640, 16), (200, 1024, 512, None), (1000, 2048, 4096, 256)])
def test_first_calls_in_a_capture(m, h, f, rows):
    r = subprocess.run([sys.executable, "-c", PROGRAM, str(m), str(h), str(f)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert rows is None or int(r.stdout.split()[0]) == rows
