"""The bench's decode step with a key-value cache at a budget, past the step from
which on all of the newest 512 entries are its own: every key head still moves one
entry at every step."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_step_of_the_cache_workload_moves_an_entry_per_head():
    r = subprocess.run([sys.executable, "bench.py", "--workload", "gptj6b-28L-cache", "--layers", "1", "--steps", "600",
                        "--warmup", "2"], cwd=ROOT, capture_output=True, text=True, timeout=110)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    line = json.loads(r.stdout.strip().splitlines()[-1])
    assert line["config"]["entries_moved"] == {"step": 16, "cache alone": 16}, line
    assert line["finite"] and line["status"] == 0
