"""The paged cache's kernels begin before the stream's previous kernel has ended
(programmatic dependent launches).  What that one and those before it have
written is visible only after a kernel's own griddepcontrol.wait, so no kernel
may touch global memory earlier, and all its threads have to pass the wait.
Read from the source, on a machine without a GPU."""
from __future__ import annotations

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gemm_epilogue_02_gb300", "csrc")
# What reads or writes through the kernels' parameter p (pointers are formed without brackets).
ACCESS = re.compile(r"\bp\.[\w.]+\s*\[|(?<=[=(,;{])\s*\*\s*p\.|__ldc[gs]|__stcg|atomic|cp_async|record_status|kv_row\(|kv_length\(|kv_sequence_of\(|"
                    r"\b(?:kept|list|w|to_w|mine|scores|stats)\[")


def kernels():
    """(name, body) of every kernel of the paged cache."""
    out = []
    for path in sorted(glob.glob(os.path.join(CSRC, "kv_*.cuh"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__[^;{]*?\b(kv_\w+_kernel)\s*\(", text):
            start = text.index("{", m.end())
            depth, at = 1, start + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[at], 0)
                at += 1
            out.append((m.group(1), text[start + 1:at - 1]))
    return out


def test_every_kernel_is_found():
    assert sorted(n for n, _ in kernels()) == ["kv_append_kernel", "kv_attend_kernel", "kv_gather_kernel", "kv_select_kernel",
                                               "kv_spread_kernel"]


@pytest.mark.parametrize("name,body", kernels(), ids=[n for n, _ in kernels()])
def test_no_access_before_the_wait(name, body):
    assert body.count("griddep_wait()") == 1, "one wait"
    before = body[:body.index("griddep_wait()")]
    assert before.count("{") == before.count("}") and before.rstrip().endswith((";", "}")), "reached by all threads"
    found = ACCESS.search(before)
    assert not found, found.group(0)
    assert "griddep_launch_dependents" not in before, "what may follow begins after the wait"
