"""The costs that attention's shares go by, checked on the host (no GPU needed): tests/flash_shares_check.cu
includes the kernels' header and adds the blocks' costs up one by one."""
import os
import shutil
import subprocess

import pytest

from int4_routed_expert_prerouter_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_costs_of_the_blocks_before_one_add_up(tmp_path):
    nvcc = build.nvcc()
    if shutil.which(nvcc) is None and not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path / "flash_shares_check")
    # device code only as PTX (no ptxas): the check runs the host functions
    subprocess.check_call([nvcc, "-gencode", "arch=compute_103a,code=compute_103a", "-std=c++17", "-O1",
                           "-I", os.path.join(ROOT, "include"),
                           "-I", os.path.join(ROOT, "int4_routed_expert_prerouter_gb300", "csrc"),
                           os.path.join(ROOT, "tests", "flash_shares_check.cu"), "-o", exe])
    out = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stdout[-4000:] + out.stderr[-2000:]
    assert "ALL OK" in out.stdout
