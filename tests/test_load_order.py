"""The library and torch share one HIP runtime, whichever a program touches first."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
from bit_quantized_finetuning_quant_amd import qlora
assert qlora.linear_gated_workspace_bytes(4, 128, 256, 8) > 0  # a size helper, before anything on the GPU
import torch
with open("/proc/self/maps") as f:
    print(len({line.split()[-1] for line in f if "libamdhip64" in line}))
"""


def test_a_size_helper_before_torch_leaves_one_runtime():
    """With two of them, torch's first call on the GPU ends the process."""
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == "1"
