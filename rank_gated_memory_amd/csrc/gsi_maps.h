// Plain linear maps (gsi_q4_linear, gsi_grouped_linear): what their kernels
// share.  Nothing here is part of the public ABI.
//
// Both entry points are one product, y[r] = W_e(r) x[src(r)], with the rows of
// y ordered by expert; gsi_q4_linear has one expert and every row.
//
// MFMA operand layouts as in gsi_batched.hip: for 16x16x32, lane l holds
// A[l % 16][8 (l / 16) + e], B[8 (l / 16) + e][l % 16] and accumulator i is
// C[4 (l / 16) + i][l % 16]; for 32x32x16, A[l % 32][8 (l / 32) + e],
// B[8 (l / 32) + e][l % 32] and accumulator i is
// C[8 (i / 4) + 4 (l / 32) + i % 4][l % 32]; for the fp32 16x16x4,
// A[l % 16][l / 16], B[l / 16][l % 16] and C as for 16x16x32.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/gsi.h"

namespace gsi {

struct MArgs {
  const uint8_t *W;
  const uint8_t *scales;
  const uint8_t *zeros;  // null: 8
  const uint8_t *x;
  uint8_t *y;
  const int32_t *offsets;  // null: one expert, rows [0, R)
  const int32_t *rows;     // null: row r reads x row r
  int64_t w_stride;        // bytes between maps
  int64_t ldx, ldy;        // elements
  int32_t d, d_out, n, R, T;
  int32_t groups;          // scale groups of a row
};

// A launch holds fewer than 2^32 threads.
constexpr int64_t kMostThreads = (1LL << 32) - 1;

enum Kind { kQ4Bf16, kQ4F32, kBf16, kF32 };

// Launchers; group is 0 for dense kinds.  launch_wide: dense bf16.
gsi_status launch_stream(const MArgs &a, Kind kind, int group, hipStream_t st);
gsi_status launch_wide(const MArgs &a, hipStream_t st);
gsi_status launch_small(const MArgs &a, Kind kind, hipStream_t st);       // dense
gsi_status launch_wide_q4(const MArgs &a, int group, hipStream_t st);  // bf16 x

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ bf16x8_t as_bf16x8(u32x4_t u) { return __builtin_bit_cast(bf16x8_t, u); }

// Rows [lo, hi) of expert e, clamped to the rows there are.
__device__ __forceinline__ void expert_rows(const MArgs &a, int e, int *lo, int *hi) {
  *lo = *hi = 0;
  if (a.offsets) {
    if (e < a.n) {
      *lo = min(max(a.offsets[e], 0), a.R);
      *hi = min(max(a.offsets[e + 1], *lo), a.R);
    }
  } else if (e == 0) {
    *hi = a.R;
  }
}

}  // namespace
}  // namespace gsi
