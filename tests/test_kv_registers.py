"""Registers of eviction's selection, whose 1024 threads have 32 each: what does not fit goes to memory at every pass."""
from __future__ import annotations

import os
import re
import subprocess

from gemm_epilogue_02_gb300.build import ARCH, nvcc


def test_selection_keeps_its_registers(tmp_path):
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "kv_select_build.cu")
    run = subprocess.run([nvcc(), *ARCH, "-O3", "-std=c++17", "--expt-relaxed-constexpr", "-c", "-Xptxas", "-v", "-o",
                          str(tmp_path / "select.o"), src], check=True, capture_output=True, text=True)
    spills = re.findall(r"(\d+) bytes spill stores, (\d+) bytes spill loads", run.stdout + run.stderr)
    assert len(spills) == 3 and all(x == ("0", "0") for x in spills), spills
