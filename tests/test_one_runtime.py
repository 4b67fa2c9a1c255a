"""CPU test: the library and PyTorch share one HIP runtime, whichever of them a program loads first."""

import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = """
import {first}
import rank_kv_block_amd as rk
rk.pred_rope_turns(64, 10000.0)
import torch
print(*sorted({{line.split()[-1] for line in open("/proc/self/maps") if "libamdhip64" in line}}))
"""


@pytest.mark.parametrize("first", ["rank_kv_block_amd", "torch"])
def test_one_hip_runtime(first):
    out = subprocess.run([sys.executable, "-c", CODE.format(first=first)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr
    assert len(out.stdout.split()) == 1, out.stdout
