// The paged key-value cache (gsi_rotary, gsi_cache_append, gsi_cache_attend,
// gsi_cache_evict): what their kernels share.  Nothing here is part of the
// public ABI.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/gsi.h"

namespace gsi {

constexpr int64_t kMostLaunch = (1LL << 32) - 1;  // a launch holds fewer than 2^32 threads

// The pool and the tables of a call; strides in bytes.
struct Pool {
  uint8_t *K, *V;
  float *mass;
  int32_t *age;
  const int32_t *table;
  int64_t page_stride, head_stride, slot_stride, ld;
  int32_t pages, shift, heads, d, S, most;  // a page has 1 << shift slots
};

// Quotients n / by, exact where n * by stays below 2^32.
struct Div {
  uint32_t by, magic;
};

inline Div div_by(uint32_t by) { return {by, by > 1 ? (uint32_t)((1ull << 32) / by) + 1 : 0u}; }

struct Rows {  // T rows of heads; strides in bytes
  uint8_t *p;
  int64_t row, head;
  int32_t n;
};

struct RotateArgs {
  Rows q, qo, k, v;
  Pool c;
  const int32_t *seq, *slots;
  const double *freq;
  const void *positions;
  float amplitude;
  int32_t pos_bytes, T, d, turned, start;
};

struct AttendArgs {
  Pool c;
  Rows q, out;
  const int32_t *lengths;
  float *lse;
  uint8_t *ws;
  float scale;
  int32_t window, group;  // query heads of a key head
  bool accumulate;
};

struct EvictArgs {
  Pool c;
  const int32_t *to;  // null: in place
  int64_t to_ld;
  const int32_t *lengths;
  int32_t *lengths_out, *from;
  int32_t budget, recent;
};

gsi_status launch_rotate(const RotateArgs &a, int dtype, int layout, hipStream_t st);
bool attend_counts(const Pool &c);  // whether there are no more slots than are counted
size_t attend_workspace(const Pool &c, int dtype, int q_heads, bool accumulate);
gsi_status launch_attend(const AttendArgs &a, int dtype, hipStream_t st);
gsi_status launch_evict(const EvictArgs &a, int dtype, hipStream_t st);

namespace {

__device__ __forceinline__ uint32_t quotient(uint32_t n, Div d) { return d.magic ? __umulhi(n, d.magic) : n; }

__device__ __forceinline__ int clamped_length(const Pool &c, const int32_t *lengths, int s) {
  return min(max(lengths[s], 0), c.most << c.shift);
}

// The page of slot i of sequence s, or -1.
__device__ __forceinline__ int page_of(const Pool &c, int s, int i) {
  const int p = c.table[s * c.ld + (i >> c.shift)];
  return p >= 0 && p < c.pages ? p : -1;
}

// Bytes from K (V) to slot i's entry of head h on page p.
__device__ __forceinline__ int64_t entry_at(const Pool &c, int p, int h, int i) {
  return p * c.page_stride + h * c.head_stride + (i & ((1 << c.shift) - 1)) * c.slot_stride;
}

// Its place in mass and age.
__device__ __forceinline__ int64_t number_at(const Pool &c, int p, int h, int i) {
  return (((int64_t)p * c.heads + h) << c.shift) + (i & ((1 << c.shift) - 1));
}

// Sums over the lanes up to and with this one, in registers (a row's lanes by
// shifts, then the rows' last lanes to the rows behind).
template <int None, typename F>
__device__ __forceinline__ int joined_to(int v, const F &f) {  // of any f with f(None, x) = x
  v = f(v, __builtin_amdgcn_update_dpp(None, v, 0x111, 0xf, 0xf, false));  // row_shr 1
  v = f(v, __builtin_amdgcn_update_dpp(None, v, 0x112, 0xf, 0xf, false));
  v = f(v, __builtin_amdgcn_update_dpp(None, v, 0x114, 0xf, 0xf, false));
  v = f(v, __builtin_amdgcn_update_dpp(None, v, 0x118, 0xf, 0xf, false));
  v = f(v, __builtin_amdgcn_update_dpp(None, v, 0x142, 0xa, 0xf, false));  // row_bcast 15, rows 1 and 3
  v = f(v, __builtin_amdgcn_update_dpp(None, v, 0x143, 0xc, 0xf, false));  // row_bcast 31, rows 2 and 3
  return v;
}
__device__ __forceinline__ int sums_to(int v) {
  return joined_to<0>(v, [](int a, int b) { return a + b; });
}

}  // namespace
}  // namespace gsi
