"""Where attention over the paged cache reads, checked on the CPU: the kernel's
own functions for it (csrc/gsi_attend_at.h) in a host program, over every type,
size of a head, lane and piece."""
import os
import shutil
import subprocess

import pytest

from rank_gated_memory_amd import build

CSRC = os.path.join(build.PKG, "csrc")
COMPILER = shutil.which("g++") or "/opt/rocm/llvm/bin/clang++"

HEAD = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "@HEADER@"
using namespace gsi;
#define HOLD(what, ...)                                  \
  do {                                                   \
    if (!(what)) {                                       \
      std::printf("%s: ", #what);                        \
      std::printf(__VA_ARGS__);                          \
      std::printf("\n");                                 \
      std::exit(1);                                      \
    }                                                    \
  } while (0)
"""


def run(tmp_path, body, header="gsi_attend_at.h"):
    """The body of a main() over the functions of a header of the library."""
    source, program = tmp_path / "check.cpp", tmp_path / "check"
    source.write_text(HEAD.replace("@HEADER@", header) + "int main() {\n" + body + '\n  std::printf("held\\n");\n}\n')
    subprocess.run([COMPILER, "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-I", CSRC, str(source), "-o",
                    str(program)], check=True, timeout=120)
    r = subprocess.run([str(program)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.endswith("held\n"), r.stdout + r.stderr


@pytest.mark.parametrize("es", [2, 4])
def test_keys_are_read_within_their_entry(tmp_path, es):
    """Every piece lies in the key, and those that count are all of it, each once."""
    run(tmp_path, f"constexpr int es = {es};" + r"""
  for (int d = 8; d <= 256; d += 8) {
    const int ks = attend_ks(d);
    HOLD(32 * ks >= d, "d %d", d);
    std::vector<int> seen(d * es / 16);
    for (int c = 0; c < key_pieces(es, ks); ++c)
      for (int quad = 0; quad < 4; ++quad) {
        const int at = (int)piece_at(es, ks, d, c, quad);
        HOLD(at >= 0 && at % 16 == 0 && at + 16 <= d * es, "d %d, piece %d of quad %d: bytes %d to %d", d, c, quad, at, at + 16);
        if (!piece_inside(es, d, c, quad)) {
          HOLD(c >= key_guarded(es, ks), "d %d, piece %d of quad %d is not taken for zeros", d, c, quad);
          continue;
        }
        HOLD(at == 64 * c + 16 * quad, "d %d, piece %d of quad %d", d, c, quad);
        ++seen[at / 16];
      }
    for (int n : seen) HOLD(n == 1, "d %d: %d", d, n);
  }""")


@pytest.mark.parametrize("es", [2, 4])
def test_values_are_read_within_their_entry(tmp_path, es):
    """A lane's columns lie in the value, and the lanes' are all of it."""
    run(tmp_path, f"constexpr int es = {es};" + r"""
  for (int d = 8; d <= 256; d += 8) {
    const int ks = attend_ks(d), n = value_columns(ks);
    std::vector<int> seen(d);
    for (int l16 = 0; l16 < 16; ++l16) {
      const int at = first_column(ks, d, l16);
      HOLD(at >= 0 && at + n <= d && at * es % 4 == 0, "d %d, lane %d: columns %d to %d", d, l16, at, at + n);
      for (int j = 0; j < n; ++j) seen[at + j] = 1;
    }
    for (int e = 0; e < d; ++e) HOLD(seen[e], "d %d, column %d", d, e);
  }""")


@pytest.mark.parametrize("es", [2, 4])
def test_a_step_reads_each_slot_once(tmp_path, es):
    run(tmp_path, f"constexpr int es = {es};" + r"""
  std::vector<int> keys(attend_step(es)), values(attend_step(es));
  for (int l16 = 0; l16 < 16; ++l16)
    for (int u = 0; u < key_tiles(es); ++u) {
      HOLD(key_slot(es, l16) + 4 * u < 8, "lane %d", l16);
      ++keys.at(8 * key_block(es, l16) + key_slot(es, l16) + 4 * u);
    }
  for (int quad = 0; quad < 4; ++quad)
    for (int e = 0; e < value_slots(es); ++e) {
      HOLD(value_slot(es, quad) + e < 8, "quad %d", quad);
      ++values.at(8 * value_block(es, quad) + value_slot(es, quad) + e);
    }
  for (int t = 0; t < attend_step(es); ++t) HOLD(keys[t] == 1 && values[t] == 1, "slot %d", t);""")


def test_page_numbers_are_read_of_slots_in_use_alone(tmp_path):
    """Steps (of attention) and strips of 256 slots (of the mass) begin before a
    window and end behind a sequence: what they look up lies within."""
    run(tmp_path, r"""
  for (int n = 1; n < 700; n += n < 40 ? 1 : 37)
    for (int window = 0; window < n + 2; window += window < 40 ? 1 : 41) {
      const int first = window > 0 && n > window ? n - window : 0;
      for (const int unit : {attend_step(2), attend_step(4), 256})
        for (int t = first / unit * unit; t < n + 3 * unit; ++t) {
          const int at = slot_in_use(t, first, n);
          HOLD(first <= at && at < n, "slot %d for slot %d of %d to %d", at, t, first, n);
          HOLD(t < first || t >= n || at == t, "slot %d for slot %d of %d to %d", at, t, first, n);
        }
    }""")
