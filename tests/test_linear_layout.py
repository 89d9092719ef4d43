"""The regions of gsi_linear's workspace for more tokens than a launch takes, on the
CPU: the library's own arithmetic (csrc/gsi_layout.h) in a host program.  A call of
many tokens is several launches on one workspace, and a workspace serves call after
call without being cleared: no launch may write where another one counts."""
import pytest
import torch

from rank_gated_memory_amd import gsi, synth
from tests.test_cache_reads import run as run_program

BODY = r"""
  const int dims[][3] = {{64, 64, 8}, {4096, 4096, 256}, {8192, 1024, 256}, {8192, 8192, 1024}, {2048, 16384, 128}};
  const int tokens[] = {1, 5, 63, 64, 4095, 4096, 4097, 4096 + 63, 5000, 8192, 8193, 13000};
  for (const auto &m : dims)
    for (const int T : tokens) {
      const int d = m[0], d_out = m[1], k = m[2], es = 4;
      const LinearLayout layout = linear_layout(d, d_out, k, es, T);
      const WsLayout &w = layout.ws;
      for (int t0 = 0; t0 < T; t0 += kMaxCalls) {
        const int64_t n = std::min(T - t0, (int)kMaxCalls);
        const UnitShape &us = layout.of((int32_t)n), own = linear_shape(d, d_out, k, es, n);
        HOLD(us.a_units == own.a_units && us.groups == own.groups && us.fast_units == own.fast_units, "d %d, T %d", d, T);
        // counters, then gates, needs, prefixes and floats, then group counters, of this launch
        HOLD((uint64_t)(n + 1) * 4 <= w.gate_off, "d %d, k %d, T %d: %d counters", d, k, T, (int)n);
        HOLD(w.gate_off + (uint64_t)n * 16 <= w.need_off && w.need_off + (uint64_t)n * 4 <= w.pref_off, "T %d", T);
        HOLD(w.pref_off + (uint64_t)(n + 1) * 4 <= w.float_off, "T %d", T);
        const uint64_t floats = (uint64_t)n * (us.g_floats + us.part_floats) * 4;
        HOLD(w.float_off + floats <= w.gcnt_off, "d %d, k %d, T %d: floats of %d tokens", d, k, T, (int)n);
        HOLD(w.gcnt_off + (uint64_t)n * us.a_units * 4 <= w.total, "d %d, k %d, T %d", d, k, T);
      }
    }
"""


def test_launches_of_a_call_share_one_layout(tmp_path):
    run_program(tmp_path, BODY, header="gsi_layout.h")


@pytest.mark.gpu
@pytest.mark.parametrize("d,d_out,k", [(64, 64, 8), (8192, 64, 256)])
def test_many_tokens_again_and_again_on_one_workspace(d, d_out, k):
    """4096 tokens and five more in one call, three times on one workspace that is
    zero before the first: every time the bits of the two launches alone.  (8192
    columns by 256: the five tokens' projections are summed in two levels.)"""
    dev = torch.device("cuda:0")
    W = synth.gaussian_weight(d_out, d, (95, 0, 0, 0), dtype=torch.float32)
    v, u = synth.orthonormal_frame(d, k, 16, (95, 0, 0, 1))
    T = 4101
    mask = torch.zeros(T, dtype=torch.bool)
    mask[::11] = True
    X = synth.tokens(v, u, mask, (95, 0, 0))[0].to(torch.float32).to(dev)
    m = gsi.gsi_prepare(gsi.Map(W.to(dev), v.to(torch.float32).to(dev)))
    parts = [gsi.gsi_linear(m, X[:4096], 0.05), gsi.gsi_linear(m, X[4096:], 0.05)]
    want = [torch.cat(p) for p in zip(*parts)]
    ws = gsi.workspace(gsi.gsi_linear_workspace(m, T), dev)
    for _ in range(3):
        got = [torch.full_like(t, 7) for t in want]
        gsi.gsi_linear(m, X, 0.05, y=got[0], rho=got[1], slow=got[2], ws=ws)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert 0 < int(want[2].sum()) < T
