"""Kernels around the cache's pages and of the head norms begin before the
stream's previous kernel has ended (programmatic dependent launches): none may
touch global memory, or let what follows begin, before its own
griddepcontrol.wait, and all its threads have to pass the wait.  Read from the
source, on a machine without a GPU."""
from __future__ import annotations

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gemm_epilogue_02_gb300", "csrc")
ACCESS = re.compile(r"\bp\.(?!turns|axis\b|side\b|dbg_y)[\w.]+\s*\[|__ldc[gs]|__stcs|atomic|cp_async|record_status|kv_length\(|fork_length\(|fork_child|take_pages|plan_moves|move_pages|cluster_sync|"
                    r"rope_read|rope_write|rope_stage_weights\(|\*p\.in_use|\blist\[|\bto\[")


def kernels():
    out = []
    for name in ("page_bounds.cuh", "page_pool.cuh", "rope.cuh"):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
        for m in re.finditer(r"__global__[^;{]*?\b(\w+_kernel)\s*\(", text):
            start = text.index("{", m.end())
            depth, at = 1, start + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[at], 0)
                at += 1
            out.append((m.group(1), text[start + 1:at - 1]))
    return out


def test_every_kernel_is_found():
    assert sorted(n for n, _ in kernels()) == [
        "page_bounds_kernel", "page_choose_kernel", "page_compact_few_kernel", "page_fork_few_kernel", "page_fork_kernel", "page_free_kernel", "page_move_kernel",
        "page_plan_kernel", "page_take_kernel", "rope_backward_kernel", "rope_kernel"]


@pytest.mark.parametrize("name,body", kernels(), ids=[n for n, _ in kernels()])
def test_no_access_before_the_wait(name, body):
    assert body.count("griddep_wait()") == 1, "one wait"
    before = body[:body.index("griddep_wait()")]
    assert before.count("{") == before.count("}") and (before.rstrip() or ";").endswith((";", "}")), "reached by all threads"
    assert not re.search(r"\breturn\s*;", before), "reached by all threads"
    found = ACCESS.search(before)
    assert not found, found.group(0)
    assert "griddep_launch_dependents" not in before, "what may follow begins after the wait"
