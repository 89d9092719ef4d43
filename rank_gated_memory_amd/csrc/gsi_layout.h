// Host arithmetic of the batch-1 path: the units of its launches and the regions of
// its workspace.  Nothing here is part of the public ABI.
#pragma once

#include <algorithm>

#include "gsi_internal.h"

namespace gsi {

struct WsLayout {
  uint64_t gate_off, need_off, pref_off, float_off, ctl_off, gcnt_off, total;
};

// The group counters of two-level partial sums follow the control words.
inline uint64_t gcnt_offset(uint64_t ctl_off, int64_t ctl) { return align_up(ctl_off + (uint64_t)ctl * 4, 256); }

// ctl: control words of the single-launch stack kernel (0 for gsi_linear);
// units_a: projection units (at most one group counter each)
inline WsLayout ws_layout(int64_t n, int64_t floats, int64_t ctl, int64_t units_a) {
  WsLayout w;
  w.gate_off = align_up((uint64_t)(n + 1) * 4, 256);
  w.need_off = align_up(w.gate_off + (uint64_t)n * 16, 256);
  w.pref_off = align_up(w.need_off + (uint64_t)n * 4, 256);
  w.float_off = align_up(w.pref_off + (uint64_t)(n + 1) * 4, 256);
  w.ctl_off = align_up(w.float_off + (uint64_t)floats * 4, 256);
  w.gcnt_off = gcnt_offset(w.ctl_off, ctl);
  w.total = align_up(w.gcnt_off + (uint64_t)units_a * 4, 256);
  return w;
}

// Bytes of V_k per projection unit of a stack plan: small enough that the
// gates of a step open progressively (output work overlaps projection in
// the single launch), large enough to amortise a unit's partial hand-off.
#ifndef GSI_PLAN_PROJ_UNIT_KB
#define GSI_PLAN_PROJ_UNIT_KB 384
#endif
inline int64_t plan_proj_target(int64_t total_v_bytes) {
  int64_t t = total_v_bytes / (256 * 4);
  if (t < 16 * 1024) t = 16 * 1024;
  if (t > GSI_PLAN_PROJ_UNIT_KB * 1024) t = GSI_PLAN_PROJ_UNIT_KB * 1024;
  return t;
}

// Unit shapes of every call of a (validated) plan, chosen wave by wave.
// A wave's projection units aim at (its V_k bytes) / 1024, clamped to
// [16 KiB, GSI_PLAN_PROJ_UNIT_KB], and at most kMaxPartials per call (the
// final sum of a call's partials is then one round of loads).  A wave whose fast
// outputs make fewer than kFineUnits ordinary units is latency-bound (the
// waves of a dependency-chained stack): it takes the smallest output units.
constexpr int64_t kFineUnits = 1024;
#ifndef GSI_PLAN_MAX_PARTIALS
#define GSI_PLAN_MAX_PARTIALS 64
#endif
constexpr int64_t kMaxPartials = GSI_PLAN_MAX_PARTIALS;
constexpr int64_t kTwoLevelUnitBytes = 64 * 1024;
constexpr int64_t kMaxPartials2 = 256;

// Unit shape of one call in a wave whose projection bytes total `wave_vbytes`
// and whose fast outputs make `wave_fast_units` ordinary units (the rule
// above).
inline UnitShape shape_in_wave(int32_t d, int32_t d_out, int32_t k, int es, int64_t wave_vbytes,
                               int64_t wave_fast_units) {
  const int64_t t = plan_proj_target(wave_vbytes);
  const bool fine = wave_fast_units < kFineUnits;
  const int64_t vi = (int64_t)d * k * es;
  int64_t ti = std::max<int64_t>(t, (vi + kMaxPartials - 1) / kMaxPartials);
  // Where the cap of kMaxPartials one-level partials would make the units
  // larger than the wave's target and than kTwoLevelUnitBytes (a wide V_k in
  // a latency-bound wave), up to kMaxPartials2 smaller units are summed in
  // two levels instead.
  if (ti > t && ti > kTwoLevelUnitBytes)
    ti = std::max<int64_t>({t, kTwoLevelUnitBytes, (vi + kMaxPartials2 - 1) / kMaxPartials2});
  return unit_shape(d, d_out, k, es, ti, fine);
}

// Unit shape of n tokens of one map: the n tokens are n calls of one wave, shaped as
// a stack plan would shape them (a few tokens are latency-bound and take the small
// units).
inline UnitShape linear_shape(int32_t d, int32_t d_out, int32_t k, int es, int64_t n) {
  const int64_t coarse = unit_shape(d, d_out, k, es, 1 << 20).fast_units;
  return shape_in_wave(d, d_out, k, es, (int64_t)d * k * es * n, coarse * n);
}

// T tokens go in launches of kMaxCalls and one of the rest, one after the other on
// one workspace: a region that has to be zero between launches must lie in the same
// place for all of them, or one would leave its sums in another's counters.  The
// regions are laid out once, each for the launch that needs most of it.
struct LinearLayout {
  UnitShape full, rest;  // of kMaxCalls tokens, and of the others
  WsLayout ws;
  const UnitShape &of(int32_t n) const { return n == kMaxCalls ? full : rest; }
};

inline LinearLayout linear_layout(int32_t d, int32_t d_out, int32_t k, int es, int32_t T) {
  LinearLayout r{};
  int64_t floats = 0, units = 0;
  const auto take = [&](int64_t n) {
    const UnitShape us = linear_shape(d, d_out, k, es, n);
    floats = std::max(floats, n * (us.g_floats + us.part_floats));
    units = std::max(units, n * us.a_units);
    return us;
  };
  if (T >= kMaxCalls) r.full = take(kMaxCalls);
  if (T % kMaxCalls) r.rest = take(T % kMaxCalls);
  r.ws = ws_layout(std::min(T, (int32_t)kMaxCalls), floats, 0, units);
  return r;
}

}  // namespace gsi
