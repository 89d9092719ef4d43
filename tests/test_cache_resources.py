"""The paged cache's kernels as the compiler reports them at the build's own flags
(CPU only): none uses scratch memory, and each keeps the wavefronts that its grid
counts on.  gsi_cache_attend deals its work to as many workgroups of four
wavefronts as it takes the chip to hold at once: three a CU up to heads of 64,
two up to 128, one above."""
import os
import re

import pytest

from tests.test_kernel_resources import resource_usage

pytestmark = pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not installed")


@pytest.mark.parametrize("source,waves", [
    ("gsi_rotary.hip", {r"rotate_kernel": 8}),
    ("gsi_attend.hip", {r"attend_kernelI\w*Li[12]E": 3, r"attend_kernelI\w*Li[34]E": 2, r"attend_kernelI\w*Li[68]E": 1,
                        r"join_kernel": 4, r"mass_kernel": 4}),
    ("gsi_evict.hip", {r"select_kernel": 4, r"move_kernel": 8}),
])
def test_kernels_keep_their_occupancy_without_scratch(source, waves):
    usage = resource_usage(source)
    seen = set()
    for name, use in usage.items():
        hit = [p for p in waves if re.search(p, name)]
        assert len(hit) == 1, f"{name} in {source} is not listed once"
        seen.add(hit[0])
        assert use.get("Occupancy", 0) >= waves[hit[0]], f"{name}: {use}"
        assert use.get("ScratchSize", 1) == 0, f"{name} uses scratch memory: {use}"
    assert seen == set(waves)
