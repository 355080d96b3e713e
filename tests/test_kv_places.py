"""Where the paged cache's outputs go when the data of a call changes while it
runs, which no call may turn into an access outside its arrays: the functions
that decide it, as compiled for the host."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest

from gemm_epilogue_02_gb300.build import ARCH, nvcc


@pytest.fixture(scope="module")
def places(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("kv") / "libkvplaces.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "kv_host_places.cu")
    subprocess.run([nvcc(), *ARCH, "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", "-o", lib, src], check=True,
                   capture_output=True)
    p = ctypes.CDLL(lib)
    p.check_scored.argtypes, p.check_scored.restype = [ctypes.c_int] * 4 + [ctypes.c_longlong], ctypes.c_longlong
    return p


def test_kept_positions_stay_among_the_best(places):
    """Counts that do not belong together (a limit found in other weights than those that are placed by it) give no
    place outside 0 .. best - 1."""
    at = ctypes.c_int()
    odd = (-2 ** 31, -7, -1, 0, 1, 5, 63, 64, 100, 2 ** 31 - 1)
    for larger in (0, 1, 5, 63, 64, 1000, 2 ** 31 - 1):
        for ties in (0, 1, 64, 2 ** 31 - 1):
            for need in odd:
                for best in (0, 1, 6, 64, 2 ** 30):
                    ok = places.check_kept_place(larger, ties, need, best, ctypes.byref(at))
                    want = larger + min(ties, need)
                    assert ok == (0 <= want < best)
                    if ok:
                        assert at.value == want


def test_scores_stay_inside_what_the_page_lists_hold(places):
    """A step's positions past what the workspace has room for have no score, whatever tile they are said to be in."""
    for positions in (0, 1, 95, 96, 1000, 2 ** 30):
        for lo in (0, 1, positions // 2, max(0, positions - 1)):
            for tile in (0, 1, 10, 11184810, 11184826):
                for in_tile in (0, 16, 80):
                    first = lo + tile * 96 + in_tile
                    assert places.check_scored(lo, tile, 96, in_tile, positions) == max(0, positions - first)


def test_parts_are_joined_in_groups_that_fit(places):
    """The groups that attention's parts are joined in, for every number of parts that there can be: each part in one
    group, no more parts or groups than a block has room for, a counter and a slot of its own for every group."""
    limits = (ctypes.c_int * 3)()
    places.check_join_limits(limits)
    ctas, most, one_level = limits
    assert one_level <= most
    for parts in range(1, ctas + 1):
        fan, groups = most, 1
        if parts > one_level:
            fan = places.check_fan(parts)
            groups = -(-parts // fan)
        assert 1 <= fan <= most and 1 <= groups <= most and (groups - 1) * fan < parts <= groups * fan
        if groups == 1:
            assert parts <= most
            continue
        seen = []
        for group in range(groups):
            first = group * fan
            members = list(range(first, first + min(fan, parts - first)))
            assert members and all(m // fan == group for m in members)
            seen += members
        assert seen == list(range(parts))
        for first_run in (0, ctas - parts):
            heads = [places.check_slot(first_run + g * fan, first_run, 0, 1) for g in range(groups)]
            assert len(set(heads)) == groups and min(heads) >= 0 and max(heads) < 2 * ctas
