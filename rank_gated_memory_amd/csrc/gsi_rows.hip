// Ordering the choices of a router by expert, and the weighted sum that
// undoes it (gsi_group_rows, gsi_group_combine).
#include <hip/hip_runtime.h>

#include <type_traits>

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

// Bound by the reads of all numbers by every workgroup, out of the L2s, twice:
// a lane reads four choices at once and has four such reads under way.
constexpr int kRowsAhead = 4;

template <typename I>
__global__ void __launch_bounds__(kRowsThreads)
group_rows_kernel(const I *ids, int n_flat, int top, int n, int32_t *offsets, int32_t *rows, int32_t *pos) {
  __shared__ int less_sh[kRowsWaves], mine_sh[kRowsWaves];
  const int e = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int span = ((n_flat + kRowsWaves - 1) / kRowsWaves + 255) / 256 * 256;
  const int lo = min((int64_t)n_flat, (int64_t)wave * span), hi = min((int64_t)n_flat, (int64_t)lo + span);
  struct Four {
    I v[4];
  };
  // calls use(f, v) with the choices v[0..3] = ids[f..f + 3] of the span, the
  // lanes in order; behind the span a number is -1, which no expert has
  const auto each = [&](const auto &use) {
    constexpr int kStep = 256 * kRowsAhead;
    int f0 = lo;
    for (; f0 + kStep <= hi; f0 += kStep) {
      Four v[kRowsAhead];
#pragma unroll
      for (int j = 0; j < kRowsAhead; ++j) __builtin_memcpy(&v[j], ids + f0 + 256 * j + 4 * lane, sizeof(Four));
#pragma unroll
      for (int j = 0; j < kRowsAhead; ++j) use(f0 + 256 * j + 4 * lane, v[j]);
    }
    for (; f0 < hi; f0 += 256) {
      Four v;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int f = f0 + 4 * lane + c;
        v.v[c] = ids[f < hi ? f : lo];
        if (f >= hi) v.v[c] = -1;
      }
      use(f0 + 4 * lane, v);
    }
  };
  typedef std::make_unsigned_t<I> U;  // a dropped number is at least n as such
  int less = 0, mine = 0;
  each([&](int, const Four &v) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      less += (U)v.v[c] < (U)e;
      mine += v.v[c] == (I)e;
    }
  });
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
  int first = 0, before = 0;
  for (int w = 0; w < kRowsWaves; ++w) {
    first += less_sh[w];
    before += w < wave ? mine_sh[w] : 0;
  }
  if (threadIdx.x == 0) offsets[e] = first;  // e == n: the kept choices
  if (e == n) {
    for (int f = first + threadIdx.x; f < n_flat; f += kRowsThreads) rows[f] = -1;
    each([&](int f, const Four &v) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (f + c < hi && (U)v.v[c] >= (U)n) pos[f + c] = -1;
    });
    return;
  }
  if (mine == 0) return;
  int at = first + before;
  each([&](int f, const Four &v) {
    bool is[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) is[c] = v.v[c] == (I)e;
    if (__ballot(is[0] || is[1] || is[2] || is[3]) == 0) return;
    // choices of earlier lanes, then this lane's own in order
    int r = at;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint64_t m = __ballot(is[c]);
      r += __popcll(m & ((1ull << lane) - 1));
      at += __popcll(m);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (is[c]) {
        rows[r] = (f + c) / top;
        pos[f + c] = r++;
      }
  });
}

// Many choices: three launches whose work grows with the choices alone.  The
// flat order is cut into blocks of kPlaceBlock choices (the last takes what is
// left); the block's counts per expert, and then its first rows per expert,
// lie in the block's own part of pos until the block overwrites them with its
// result, so no workspace is needed (a block has at least as many choices as
// there are experts).
// From this many choices on (16384 choices over 32 to 256 experts: 7.7 us in
// one launch, 11 in three; 32768 over 8: 10.6 and 10.5; 131072 over 256: 38
// and 15).
constexpr int kPlaceFrom = 32768;
constexpr int kPlaceBlock = 2048;
static_assert(kPlaceBlock >= 1024, "a block's part of pos holds a count for every expert");

__device__ __forceinline__ int place_end(int b, int n_flat) {
  return b == (int)gridDim.x - 1 ? n_flat : (b + 1) * kPlaceBlock;
}

template <typename I>
__global__ void __launch_bounds__(kRowsThreads) count_kernel(const I *ids, int n_flat, int n, int32_t *pos) {
  __shared__ int count[1024];
  for (int e = threadIdx.x; e < n; e += kRowsThreads) count[e] = 0;
  __syncthreads();
  const int lo = blockIdx.x * kPlaceBlock, hi = place_end(blockIdx.x, n_flat);
  for (int f = lo + threadIdx.x; f < hi; f += kRowsThreads) {
    const I v = ids[f];
    if (v >= 0 && v < (I)n) atomicAdd(&count[v], 1);  // a sum of integers: the order does not matter
  }
  __syncthreads();
  for (int e = threadIdx.x; e < n; e += kRowsThreads) pos[lo + e] = count[e];
}

// Every block's counts become the choices of the same expert in earlier
// blocks, the totals the experts' first rows.
__global__ void __launch_bounds__(kRowsThreads) scan_kernel(int blocks, int n, int32_t *offsets, int32_t *pos) {
  __shared__ int total[1024];
  const int e = threadIdx.x;
  int run = 0;
  if (e < n) {
    constexpr int kAhead = 16;
    for (int b0 = 0; b0 < blocks; b0 += kAhead) {
      int c[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) c[j] = b0 + j < blocks ? pos[(int64_t)(b0 + j) * kPlaceBlock + e] : 0;
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (b0 + j < blocks) pos[(int64_t)(b0 + j) * kPlaceBlock + e] = run;
        run += c[j];
      }
    }
  }
  total[e] = e < n ? run : 0;
  for (int o = 1; o < 1024; o <<= 1) {  // inclusive sums
    __syncthreads();
    const int before = e >= o ? total[e - o] : 0;
    __syncthreads();
    total[e] += before;
  }
  if (e < n) {
    offsets[e] = total[e] - run;
    if (e == n - 1) offsets[n] = total[e];
  }
}

template <typename I>
__global__ void __launch_bounds__(kRowsThreads)
place_kernel(const I *ids, int n_flat, int top, int n, const int32_t *offsets, int32_t *rows, int32_t *pos) {
  extern __shared__ int next[];  // [wavefront][expert]: the next row
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lo = blockIdx.x * kPlaceBlock, hi = place_end(blockIdx.x, n_flat);
  const int span = ((hi - lo + kRowsWaves - 1) / kRowsWaves + 63) / 64 * 64;
  const int f0 = min(lo + wave * span, hi), f1 = min(f0 + span, hi);
  for (int k = threadIdx.x; k < kRowsWaves * n; k += kRowsThreads) next[k] = 0;
  __syncthreads();
  int *const mine = next + wave * n;
  for (int f = f0 + lane; f < f1; f += 64) {
    const I v = ids[f];
    if (v >= 0 && v < (I)n) atomicAdd(&mine[v], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < n; e += kRowsThreads) {
    int run = offsets[e] + pos[lo + e];
    for (int w = 0; w < kRowsWaves; ++w) {
      const int c = next[w * n + e];
      next[w * n + e] = run;
      run += c;
    }
  }
  __syncthreads();
  for (int f = lo + threadIdx.x; f < hi; f += kRowsThreads)
    if (f >= offsets[n]) rows[f] = -1;
  for (int f = f0; f < f1; f += 64) {
    const bool in = f + lane < f1;
    const I v = in ? ids[f + lane] : (I)-1;
    const bool kept = v >= 0 && v < (I)n;
    const int e = kept ? (int)v : 0;
    // the lanes with this lane's expert, a bit of its number at a time
    uint64_t same = __ballot(kept);
    for (int bit = 1; bit < n; bit <<= 1) {
      const uint64_t m = __ballot(e & bit);
      same &= e & bit ? m : ~m;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    const int r = kept ? mine[e] + rank : -1;
    // every lane has read its row before the first of each expert moves it on
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (kept) {
      if (rank == 0) mine[e] = r + __popcll(same);
      rows[r] = (f + lane) / top;
    }
    if (in) pos[f + lane] = r;
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

template <typename I>
void launch_rows(const I *ids, int flat, int top, int n, int32_t *offsets, int32_t *rows, int32_t *pos,
                 hipStream_t st) {
  if (flat < kPlaceFrom) {
    group_rows_kernel<I><<<n + 1, kRowsThreads, 0, st>>>(ids, flat, top, n, offsets, rows, pos);
    return;
  }
  const int blocks = flat / kPlaceBlock;
  count_kernel<I><<<blocks, kRowsThreads, 0, st>>>(ids, flat, n, pos);
  scan_kernel<<<1, kRowsThreads, 0, st>>>(blocks, n, offsets, pos);
  place_kernel<I><<<blocks, kRowsThreads, (size_t)kRowsWaves * n * sizeof(int), st>>>(ids, flat, top, n, offsets, rows,
                                                                                  pos);
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

// Bound by HBM (8191 tokens of four rows of 4096 bf16 and a residual: 397 MB in
// 77 us, 5.1 TB/s, the rate of a copy).
// A token's positions and weights are the same for its whole workgroup; four
// rows are under way at a time.
template <typename E>
__global__ void __launch_bounds__(256)
combine_kernel(const E *y, int64_t ldy, int R, const int32_t *pos, const float *weights, const E *base, int64_t ldb,
               E *out, int64_t ldo, int top, int d, int per) {
  constexpr int V = Vec<E>::n, kAhead = 4;
  const int t = blockIdx.x / per;  // `per` workgroups of a token
  const int c = ((blockIdx.x - t * per) * 256 + threadIdx.x) * V;
  if (c >= d) return;
  float acc[V] = {};
  if (base) Vec<E>::load(base + t * ldb + c, acc);
  for (int j0 = 0; j0 < top; j0 += kAhead) {
    float w[kAhead], v[kAhead][V];
    bool has[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int64_t at = (int64_t)t * top + min(j0 + j, top - 1);
      const int p = pos[at];
      has[j] = j0 + j < top && p >= 0 && p < R;
      w[j] = weights ? weights[at] : 1.f;
      if (has[j]) Vec<E>::load(y + p * ldy + c, v[j]);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (!has[j]) continue;
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += w[j] * v[j][i];
    }
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
    launch_rows(static_cast<const int32_t *>(ids), flat, top, n, offsets, rows, pos, st);
  else
    launch_rows(static_cast<const int64_t *>(ids), flat, top, n, offsets, rows, pos, st);
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
  const int per = (d / vec + 255) / 256;
  const int64_t grid = (int64_t)T * per;
  if (grid * 256 > UINT32_MAX) return GSI_E_SHAPE;  // a launch holds fewer than 2^32 threads
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (dtype == GSI_FP32)
    combine_kernel<float><<<(unsigned)grid, 256, 0, st>>>(static_cast<const float *>(y), ldy, R, pos, weights,
                                                          static_cast<const float *>(base), ldb,
                                                          static_cast<float *>(out), ldo, top, d, per);
  else
    combine_kernel<__bf16><<<(unsigned)grid, 256, 0, st>>>(static_cast<const __bf16 *>(y), ldy, R, pos, weights,
                                                           static_cast<const __bf16 *>(base), ldb,
                                                           static_cast<__bf16 *>(out), ldo, top, d, per);
  return hipGetLastError() == hipSuccess ? GSI_OK : GSI_E_HIP;
}

}  // extern "C"
