"""The training-step operators' Python binding on the CPU."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_imports_where_torch_has_no_raw_stream():
    """A torch built without CUDA does not have it; the module's CPU parts work there."""
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'): del torch._C._cuda_getCurrentRawStream\n"
            "from entropy_loss_gb300 import flp\n"
            "print(flp.SCHEDULES['auto'], flp._raw_stream.__name__)\n")
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert out.returncode == 0, out.stderr
    assert out.stdout.split()[1] == "_stream_of"
