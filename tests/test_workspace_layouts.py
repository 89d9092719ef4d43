"""What gsi.h says of workspaces that calls share, held against the layouts
themselves, on the CPU (no kernel is launched: two layouts on one workspace that
is not cleared in between are never run)."""
import ctypes
import os
import re

import numpy as np
import pytest

from rank_gated_memory_amd import gsi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000  # aligned fake device address (never dereferenced)


def plan(sizes, at=FAKE, eps=0.05):
    """The host plan of one bf16 call for each (d, d_out, k, wave)."""
    n = len(sizes)
    arr = (gsi.GsiCallStruct * n)()
    for i, (d, d_out, k, wave) in enumerate(sizes):
        p = at + i * 0x10000000
        m = gsi.GsiMapStruct(d, d_out, k, 1, p, p + 0x8000000, p + 0xA000000)
        arr[i] = gsi.GsiCallStruct(m, p + 0xC000000, p + 0xD000000, eps, wave, 0, 0)
    host = np.zeros(int(gsi.lib().gsi_stack_plan_bytes(arr, n)), dtype=np.uint8)
    assert gsi.lib().gsi_stack_plan(arr, n, host.ctypes.data, host.size) == 0
    return host


def where(host):
    """(bytes of workspace, the status word's place among its counters)."""
    return int(gsi.lib().gsi_stack_workspace(host.ctypes.data)), int(gsi.lib().gsi_stack_status_offset(host.ctypes.data))


FIRST = [(4096, 12288, 256, 0), (4096, 16384, 256, 0)]   # a block's maps of its input
SECOND = [(4096, 4096, 256, 0), (16384, 4096, 512, 0)]   # and of attention's and the inner output


def test_counters_of_one_layout_lie_among_the_sums_of_another():
    """Why a workspace serves one layout: the two stacks of a decoder's block."""
    (bytes_a, at_a), (bytes_b, at_b) = where(plan(FIRST)), where(plan(SECOND))
    assert at_a < bytes_a <= at_b < bytes_b, "the first one's counters lie before the second one's: among its sums"


def test_layouts_go_by_sizes_and_waves_alone():
    """Stacks of the same sizes and waves may share one."""
    assert where(plan(FIRST)) == where(plan(FIRST, at=FAKE + (1 << 40), eps=0.2))
    waves = [(*FIRST[0][:3], 0), (*FIRST[1][:3], 1)]
    assert where(plan(FIRST)) != where(plan(waves))


@pytest.mark.parametrize("other", [dict(T=1), dict(T=256), dict(k=512)])
def test_linear_layouts_go_by_tokens_and_sizes(other):
    """(Of d alone two layouts may be the same: the header takes less for granted.)"""
    def bytes_of(T=64, d=4096, k=256):
        m = gsi.GsiMapStruct(d, 4096, k, 0, FAKE, FAKE, FAKE)
        return int(gsi.lib().gsi_linear_workspace(ctypes.byref(m), T))
    assert bytes_of() == bytes_of(T=64) != bytes_of(**other)


def test_the_header_says_so():
    text = re.sub(r"\s*\n \*\s*", " ", open(os.path.join(ROOT, "include", "gsi.h")).read())
    assert "A workspace serves one layout." in text
    assert "have a workspace each, or all of the buffer is zero-filled, in stream order, between" in text
    for word in ("gsi_stack(const void *plan_host", "gsi_linear(const gsi_map *map"):
        comment = text[:text.index(word)].rsplit("/*", 1)[1]
        assert "layout" in comment, word
