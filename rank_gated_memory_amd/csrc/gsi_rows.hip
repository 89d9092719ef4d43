// Ordering the choices of a router by expert, and the weighted sum that
// undoes it (gsi_group_rows, gsi_group_combine).
#include <hip/hip_runtime.h>

#include "../../include/gsi.h"

namespace gsi {
namespace {

// gsi_group_rows: the stable order of n_flat expert numbers.
//
// The grouped row of a choice is (choices of smaller experts) + (earlier
// choices of the same expert).  One workgroup per expert, in one launch and
// without atomics: it counts the choices below and equal to its expert, which
// gives its first row, then walks the choices again and writes its own in
// order.  Each wavefront owns a contiguous span of the flat order, so the
// place of a choice is the span's start plus its rank among the span's
// ballots.  Workgroup n (one more than the experts) handles the dropped
// choices, the rows behind the last kept one and the last offset.
constexpr int kRowsThreads = 1024;
constexpr int kRowsWaves = kRowsThreads / 64;

template <typename I>
__global__ void __launch_bounds__(kRowsThreads)
group_rows_kernel(const I *ids, int n_flat, int top, int n, int32_t *offsets, int32_t *rows, int32_t *pos) {
  __shared__ int less_sh[kRowsWaves], mine_sh[kRowsWaves];
  const int e = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int span = ((n_flat + kRowsWaves - 1) / kRowsWaves + 63) / 64 * 64;
  const int lo = min((int64_t)n_flat, (int64_t)wave * span), hi = min((int64_t)n_flat, (int64_t)lo + span);
  // number of a choice: its expert, or n if it is dropped
  const auto number = [&](int f) {
    const I v = ids[f];
    return v >= 0 && v < (I)n ? (int)v : n;
  };
  int less = 0, mine = 0;
  for (int f = lo + lane; f < hi; f += 64) {
    const int v = number(f);
    less += v < e;
    mine += v == e;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    less += __shfl_xor(less, o, 64);
    mine += __shfl_xor(mine, o, 64);
  }
  if (lane == 0) {
    less_sh[wave] = less;
    mine_sh[wave] = mine;
  }
  __syncthreads();
  int first = 0, at = 0, total = 0;
  for (int w = 0; w < kRowsWaves; ++w) {
    first += less_sh[w];
    at += w < wave ? mine_sh[w] : 0;
    total += mine_sh[w];
  }
  if (threadIdx.x == 0) offsets[e] = first;  // e == n: the kept choices
  at += first;
  if (e == n) {
    for (int f = first + threadIdx.x; f < n_flat; f += kRowsThreads) rows[f] = -1;
    for (int f = lo + lane; f < hi; f += 64)
      if (number(f) == n) pos[f] = -1;
    return;
  }
  if (total == 0) return;
  for (int f0 = lo; f0 < hi; f0 += 64) {
    const int f = f0 + lane;
    const bool is = f < hi && number(f) == e;
    const uint64_t m = __ballot(is);
    if (is) {
      const int r = at + __popcll(m & ((1ull << lane) - 1));
      rows[r] = f / top;
      pos[f] = r;
    }
    at += __popcll(m);
  }
}

// gsi_group_combine: one pass over the rows, fp32 sums in the order of j.
template <typename E>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int n = 4;
  static __device__ void load(const float *p, float *v) {
    const float4 u = *reinterpret_cast<const float4 *>(p);
    v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
  }
  static __device__ void store(float *p, const float *v) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <>
struct Vec<__bf16> {
  static constexpr int n = 8;
  typedef __bf16 v8 __attribute__((ext_vector_type(8)));
  static __device__ void load(const __bf16 *p, float *v) {
    const v8 u = *reinterpret_cast<const v8 *>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)u[i];
  }
  static __device__ void store(__bf16 *p, const float *v) {
    v8 u;
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = (__bf16)v[i];
    *reinterpret_cast<v8 *>(p) = u;
  }
};

template <typename E>
__global__ void __launch_bounds__(256)
combine_kernel(const E *y, int64_t ldy, int R, const int32_t *pos, const float *weights, const E *base, int64_t ldb,
               E *out, int64_t ldo, int top, int d) {
  constexpr int V = Vec<E>::n;
  const int per = (d / V + 255) / 256;  // workgroups per token
  const int t = blockIdx.x / per;
  const int c = ((blockIdx.x % per) * 256 + threadIdx.x) * V;
  if (c >= d) return;
  float acc[V] = {}, v[V];
  if (base) Vec<E>::load(base + t * ldb + c, acc);
  for (int j = 0; j < top; ++j) {
    const int p = pos[(int64_t)t * top + j];
    if (p < 0 || p >= R) continue;
    const float w = weights ? weights[(int64_t)t * top + j] : 1.f;
    Vec<E>::load(y + p * ldy + c, v);
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] += w * v[i];
  }
  Vec<E>::store(out + t * ldo + c, acc);
}

inline bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace
}  // namespace gsi

using namespace gsi;

extern "C" {

gsi_status gsi_group_rows(const void *ids, int32_t ids_bytes, int32_t T, int32_t top, int32_t n,
                          int32_t *offsets, int32_t *rows, int32_t *pos, void *stream) {
  if (T < 0 || top < 1 || n < 1 || n > 1024 || (int64_t)T * top > (1 << 26)) return GSI_E_SHAPE;
  if (ids_bytes != 4 && ids_bytes != 8) return GSI_E_DTYPE;
  if (!offsets || (T > 0 && (!ids || !rows || !pos))) return GSI_E_NULL;
  if (!aligned(ids, ids_bytes) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(pos, 4)) return GSI_E_ALIGN;
  const int flat = T * top;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (ids_bytes == 4)
    group_rows_kernel<int32_t><<<n + 1, kRowsThreads, 0, st>>>(static_cast<const int32_t *>(ids), flat, top, n,
                                                               offsets, rows, pos);
  else
    group_rows_kernel<int64_t><<<n + 1, kRowsThreads, 0, st>>>(static_cast<const int64_t *>(ids), flat, top, n,
                                                               offsets, rows, pos);
  return hipGetLastError() == hipSuccess ? GSI_OK : GSI_E_HIP;
}

gsi_status gsi_group_combine(const void *y, int64_t ldy, int32_t R, const int32_t *pos,
                             const float *weights, const void *base, int64_t ldb, void *out,
                             int64_t ldo, int32_t T, int32_t top, int32_t d, int32_t dtype,
                             void *stream) {
  if (dtype != GSI_FP32 && dtype != GSI_BF16) return GSI_E_DTYPE;
  if (T < 0 || R < 0 || top < 1 || top > 64 || d < 8 || d % 8 || d > (1 << 20)) return GSI_E_SHAPE;
  const int vec = dtype == GSI_FP32 ? 4 : 8;
  constexpr int64_t far = INT64_MAX >> 33;  // fp32 rows this far apart: 2^31 of them stay within 64 bits
  if (ldo < d || (R > 0 && ldy < d) || (base && ldb < d) || ldo > far || ldy > far || ldb > far) return GSI_E_SHAPE;
  if (T == 0) return GSI_OK;
  if (!pos || !out || (R > 0 && !y)) return GSI_E_NULL;
  if (!aligned(y, 16) || !aligned(out, 16) || !aligned(base, 16) || !aligned(pos, 4) || !aligned(weights, 4) ||
      ldo % vec || (R > 0 && ldy % vec) || (base && ldb % vec))
    return GSI_E_ALIGN;
  const int64_t grid = (int64_t)T * ((d / vec + 255) / 256);
  if (grid > INT32_MAX) return GSI_E_SHAPE;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (dtype == GSI_FP32)
    combine_kernel<float><<<(unsigned)grid, 256, 0, st>>>(static_cast<const float *>(y), ldy, R, pos, weights,
                                                          static_cast<const float *>(base), ldb,
                                                          static_cast<float *>(out), ldo, top, d);
  else
    combine_kernel<__bf16><<<(unsigned)grid, 256, 0, st>>>(static_cast<const __bf16 *>(y), ldy, R, pos, weights,
                                                           static_cast<const __bf16 *>(base), ldb,
                                                           static_cast<__bf16 *>(out), ldo, top, d);
  return hipGetLastError() == hipSuccess ? GSI_OK : GSI_E_HIP;
}

}  // extern "C"
