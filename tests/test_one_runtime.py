"""One HIP runtime in a process, whichever of the library and PyTorch a program calls first."""

import os
import subprocess
import sys

import pytest

import dbf_linear_fwd_amd as dbf

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HOST_CALL = "import dbf_linear_fwd_amd as dbf; dbf.dbf_mx_forward_plan(17, 4096, 4096, dbf.DBF_TYPE_E4M3)"
MAPS = "print(sorted({l.split()[-1] for l in open('/proc/self/maps') if 'libamdhip64' in l}))"


@pytest.mark.parametrize("program", [f"{HOST_CALL}; import torch; {MAPS}", f"import torch; {HOST_CALL}; {MAPS}"])
def test_one_hip_runtime(program):
    pytest.importorskip("torch")
    dbf.lib()
    out = subprocess.run([sys.executable, "-c", program], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr
    assert out.stdout.count("libamdhip64") == 1, out.stdout


@pytest.mark.gpu
def test_gpu_call_after_a_host_call(gpu):
    program = (f"{HOST_CALL}; import torch; g = dbf.group_rows(torch.tensor([2, 0, 1, 0], dtype=torch.int32, device='cuda'), 3); "
               "print(g.order.tolist(), g.offsets.tolist())")
    out = subprocess.run([sys.executable, "-c", program], cwd=ROOT, capture_output=True, text=True, timeout=100)
    assert out.returncode == 0, out.stderr
    assert out.stdout.split("\n")[0] == "[1, 3, 2, 0] [0, 2, 3, 4]"
