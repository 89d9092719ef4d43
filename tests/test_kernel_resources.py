"""Occupancy of the hot kernels as the compiler reports it for the build's own
flags (CPU only: hipcc cross-compiles for gfx950, nothing is launched).

The single-launch stack runs two workgroups of four wavefronts per CU (two
wavefronts per SIMD) and the batched output kernel one workgroup of eight;
both sit close to the 256 registers that allow it (as does the
instrumented build of the stack, whose timelines are only representative at
the product's grid).  A change that pushes a
kernel past them does not fail any numerical test, it halves the kernel's
resident wavefronts (the stack's grid follows the occupancy query), so it
is checked here."""
import os
import re
import subprocess

import pytest

from rank_gated_memory_amd import build

CSRC = os.path.join(build.PKG, "csrc")


def resource_usage(source, flags=build.FLAGS):
    """{kernel name: {field: value}} from clang's resource-usage remarks."""
    cmd = ["/opt/rocm/bin/hipcc", *[f for f in flags if f not in ("-shared", "-fPIC")],
           "--cuda-device-only", "-c", os.path.join(CSRC, source), "-o", os.devnull,
           "-Rpass-analysis=kernel-resource-usage"]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stderr[-2000:]
    kernels, name = {}, None
    for line in r.stderr.splitlines():
        m = re.search(r"remark:\s+Function Name: (\S+)", line)
        if m:
            name = m.group(1)
            kernels[name] = {}
            continue
        m = re.search(r"remark:\s+([A-Za-z ]+?)(?: \[[^\]]*\])?: (-?\d+)", line)
        if m and name:
            kernels[name][m.group(1).strip()] = int(m.group(2))
    return kernels


@pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not installed")
@pytest.mark.parametrize("source,pattern,waves,flags", [
    ("gsi_kernels.hip", r"stack_kernel", 2, build.FLAGS),
    # the instrumented build must run the same grid for its timeline to hold
    ("gsi_kernels.hip", r"stack_kernel", 2, build.TRACE_FLAGS),
    ("gsi_batched.hip", r"bout_kernel", 2, build.FLAGS),
], ids=["stack", "stack-traced", "bout"])
def test_hot_kernels_keep_their_occupancy(source, pattern, waves, flags):
    usage = resource_usage(source, flags)
    hits = {k: v for k, v in usage.items() if re.search(pattern, k)}
    assert hits, f"no {pattern} in the remarks of {source}"
    for k, v in hits.items():
        assert v.get("Occupancy", 0) >= waves, f"{k}: {v}"
        assert v.get("VGPRs Spill", 0) == 0, f"{k} spills registers: {v}"


@pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not installed")
def test_wide_maps_wait_for_their_stages(tmp_path):
    """The wide map kernels let the loads of the running step be under way when
    it ends (vmcnt counts them) and need every older one to have landed.  Were
    there fewer loads in a step than it allows, e.g. because the compiler had
    merged two, a stage could be read before it is there; no test of numbers
    would show that reliably, so the compiled steps are counted."""
    out = str(tmp_path / "wide.s")
    cmd = ["/opt/rocm/bin/hipcc", *[f for f in build.FLAGS if f not in ("-shared", "-fPIC")],
           "--cuda-device-only", "-S", os.path.join(CSRC, "gsi_maps_wide.hip"), "-o", out]
    assert subprocess.run(cmd, capture_output=True, timeout=900).returncode == 0
    loads, steps, allowed = 0, 0, None
    for line in open(out):
        op = line.split()[0] if line.split() else ""
        if re.match(r"(global|buffer|flat|scratch)_load", op):
            loads += 1
        elif op == "s_waitcnt" and "vmcnt" in line:
            allowed = int(re.search(r"vmcnt\((\d+)\)", line).group(1))
        elif op == "s_barrier":
            assert allowed is not None and allowed <= loads, f"{allowed} loads may be under way after {loads}"
            steps += allowed > 0
            loads, allowed = 0, None
        elif line.startswith((".LBB", "_Z")) or op.startswith(("s_cbranch", "s_branch")):
            loads, allowed = 0, None  # a step is straight-line code
    assert steps >= 4 * 4 + 4 * 6, steps  # four heights of bf16 tiles, two of each group size


@pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not installed")
@pytest.mark.parametrize("source,pattern,count,waves", [
    ("gsi_maps_stream.hip", r"stream_kernel", 8, 4),
    ("gsi_maps_wide.hip", r"wide_kernel", 4, 2),
    ("gsi_maps_wide.hip", r"small_kernel", 2, 4),
], ids=["stream", "wide", "small"])
def test_map_kernels_keep_their_occupancy(source, pattern, count, waves):
    """Two workgroups of eight wavefronts of the streaming kernels on a CU (or
    one of 16), one of the large tiles, four of the small ones; no spills."""
    hits = {k: v for k, v in resource_usage(source).items() if re.search(pattern, k)}
    assert len(hits) == count, sorted(hits)
    for k, v in hits.items():
        assert v.get("Occupancy", 0) >= waves, f"{k}: {v}"
        assert v.get("VGPRs Spill") == 0 and v.get("ScratchSize") == 0, f"{k} spills registers: {v}"
