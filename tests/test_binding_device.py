"""How the binding finds the current device: torch's quick call where there is one,
its public one elsewhere; a first call brings CUDA up."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert done.returncode == 0, done.stdout + done.stderr
    return done.stdout.strip()


def test_without_torchs_quick_call():
    """A torch without it: its public call is taken (CUDA pretended, nothing is launched)."""
    assert run("""
import torch
import neighborhood_attention_video_gb300 as na
if hasattr(torch._C, "_cuda_getDevice"):
    del torch._C._cuda_getDevice
torch.cuda.is_available, torch.cuda.init, torch.cuda.current_device = lambda: True, lambda: None, lambda: 5
na._torch_module()
print(na._device())
""") == "5"


@pytest.mark.gpu
def test_first_call_of_a_process():
    """The status as the first use of CUDA, then an attention call."""
    assert run("""
import torch
import neighborhood_attention_video_gb300 as na
print(na.na3d_device_status())
q = torch.ones((1, 2, 3, 4, 1, 32), dtype=torch.bfloat16, device="cuda")
out = na.na3d_attention(q * 0, q, q, (1, 3, 3))
print(bool((out == 1).all()), na.na3d_device_status())
""").split() == ["0", "True", "0"]
