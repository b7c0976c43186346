"""The block-scaled calls where no GPU is to be seen: an error, and the process lives."""
import os
import subprocess
import sys

import pytest

from conftest import ROOT

PROGRAM = """
import ctypes, sys
import fusion_add_rmsnorm_gb300 as gbf
A = lambda i: ctypes.c_void_p((i + 1) << 40)
m = int(sys.argv[1])
lib = gbf.raw()
print(lib.gbfb_linear_fp8(A(0), A(1), A(2), A(3), None, A(4), m, 4096, 4096, 0, None),
      lib.gbfb_add_rmsnorm_fp8(A(0), A(1), A(2), None, 1, None, None, None, A(3), A(4), m, 4096, 1e-6, None),
      lib.gbfb_gated_act_fp8(A(0), A(1), A(2), m, 4096, 3, None), lib.gbfb_quantize_fp8(A(0), A(1), A(2), m, 4096, 1, None),
      lib.gbfb_quantize_fp8(A(0), A(1), A(2), m, 4096, 128, None))
"""


@pytest.mark.parametrize("m", [1, 32, 33, 1024, 8192])
def test_calls_without_a_device(m):
    r = subprocess.run([sys.executable, "-c", PROGRAM, str(m)], cwd=ROOT, capture_output=True, text=True, timeout=120,
                       env=dict(os.environ, CUDA_VISIBLE_DEVICES=""))
    assert r.returncode == 0, (r.returncode, r.stderr)
    assert r.stdout.split() == ["-4"] * 5                  # GBF_ELAUNCH
