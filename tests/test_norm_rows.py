"""How the norm's backward kernels share out rows, walked over on the host (no GPU needed)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = "/opt/rocm/bin/hipcc"


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
def test_every_row_and_gate_row_has_one_slot(tmp_path):
    exe = str(tmp_path / "norm_rows")
    r = subprocess.run([HIPCC, "--offload-host-only", "-O1", "-std=c++17", "-I",
                        os.path.join(ROOT, "block_scaled_fp4_06_amd", "csrc"),
                        os.path.join(ROOT, "tests", "native", "norm_rows_main.hip"), "-o", exe],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr
