// Attention of one new token of every sequence over the paged cache
// (gsi_cache_attend).
#include "gsi_cache.h"

namespace gsi {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

template <typename E>
__device__ __forceinline__ float score_of(const AttendArgs &a, const float *q, int page, int kh, int i) {
  const E *k = reinterpret_cast<const E *>(a.c.K + entry_at(a.c, page, kh, i));
  float v = 0.f;
  for (int e = 0; e < a.c.d; ++e) v += q[e] * (float)k[e];
  return v * a.scale;
}

// A workgroup per sequence and query head: 256 slots at a time, the running
// maximum and sum of the softmax, a thread per element of the output.
template <typename E>
__global__ void __launch_bounds__(kThreads) attend_kernel(AttendArgs a, float *lse) {
  __shared__ float q[256], p[kThreads], red[8];
  __shared__ int64_t at[kThreads];
  const int s = blockIdx.x / a.q.n, h = blockIdx.x % a.q.n, kh = h / a.group, tid = threadIdx.x, d = a.c.d;
  const int n = clamped_length(a.c, a.lengths, s), first = a.window > 0 ? max(0, n - a.window) : 0;
  const E *qp = reinterpret_cast<const E *>(a.q.p + s * a.q.row + h * a.q.head);
  if (tid < d) q[tid] = (float)qp[tid];
  float top = -INFINITY, sum = 0.f, acc = 0.f;
  for (int i0 = first; i0 < n; i0 += kThreads) {
    __syncthreads();
    const int i = i0 + tid, page = i < n ? page_of(a.c, s, i) : -1;
    const float score = page >= 0 ? score_of<E>(a, q, page, kh, i) : -INFINITY;
    at[tid] = page >= 0 ? entry_at(a.c, page, kh, i) : -1;
    const float m = wave_max(score);
    if (tid % 64 == 0) red[tid / 64] = m;
    __syncthreads();
    const float now = fmaxf(fmaxf(top, fmaxf(red[0], red[1])), fmaxf(red[2], red[3]));
    const float base = now == -INFINITY ? 0.f : now;
    p[tid] = at[tid] >= 0 ? expf(score - base) : 0.f;
    const float t = wave_sum(p[tid]), fade = expf(top - base);
    if (tid % 64 == 0) red[4 + tid / 64] = t;
    __syncthreads();
    sum = sum * fade + red[4] + red[5] + red[6] + red[7];
    acc *= fade;
    top = now;
    if (tid < d)
      for (int j = 0; j < kThreads; ++j)
        if (at[j] >= 0) acc += p[j] * (float)reinterpret_cast<const E *>(a.c.V + at[j])[tid];
  }
  E *out = reinterpret_cast<E *>(a.out.p + s * a.out.row + h * a.out.head);
  if (tid < d) out[tid] = (E)(sum == 0.f ? 0.f : acc / sum);
  const float l = sum == 0.f ? -INFINITY : top + logf(sum);
  if (tid == 0 && a.lse) a.lse[(int64_t)s * a.q.n + h] = l;
  if (tid == 0 && lse) lse[(int64_t)s * a.q.n + h] = l;
}

// A thread per sequence, key head and slot: the weights from the scores again.
template <typename E>
__global__ void __launch_bounds__(kThreads) mass_kernel(AttendArgs a, const float *lse, int strips) {
  const int strip = blockIdx.x % strips, sh = blockIdx.x / strips, s = sh / a.c.heads, kh = sh % a.c.heads;
  __shared__ float q[256];
  const int n = clamped_length(a.c, a.lengths, s), first = a.window > 0 ? max(0, n - a.window) : 0;
  const int i = strip * kThreads + threadIdx.x, page = i >= first && i < n ? page_of(a.c, s, i) : -1;
  float add = 0.f;
  for (int h = kh * a.group; h < (kh + 1) * a.group; ++h) {
    __syncthreads();
    if ((int)threadIdx.x < a.c.d)
      q[threadIdx.x] = (float)reinterpret_cast<const E *>(a.q.p + s * a.q.row + h * a.q.head)[threadIdx.x];
    __syncthreads();
    const float l = lse[(int64_t)s * a.q.n + h];
    if (page >= 0 && l != -INFINITY) add += expf(score_of<E>(a, q, page, kh, i) - l);
  }
  if (page >= 0) a.c.mass[number_at(a.c, page, kh, i)] += add;
}

template <typename E>
gsi_status launch_as(const AttendArgs &a, hipStream_t st) {
  float *lse = a.accumulate ? reinterpret_cast<float *>(a.ws) : nullptr;
  const int64_t rows = (int64_t)a.c.S * a.q.n;
  const int64_t strips = (((int64_t)a.c.most << a.c.shift) + kThreads - 1) / kThreads;
  const int64_t mass = (int64_t)a.c.S * a.c.heads * strips;
  if (rows * kThreads > kMostLaunch || (a.accumulate && mass * kThreads > kMostLaunch)) return GSI_E_SHAPE;
  attend_kernel<E><<<(unsigned)rows, kThreads, 0, st>>>(a, lse);
  if (a.accumulate && mass > 0) mass_kernel<E><<<(unsigned)mass, kThreads, 0, st>>>(a, lse, (int)strips);
  return hipGetLastError() == hipSuccess ? GSI_OK : GSI_E_HIP;
}

}  // namespace

size_t attend_workspace(const Pool &c, int, int q_heads, bool accumulate) {
  return accumulate ? (size_t)c.S * q_heads * 4 : 0;
}

gsi_status launch_attend(const AttendArgs &a, int dtype, hipStream_t st) {
  return dtype == GSI_FP32 ? launch_as<float>(a, st) : launch_as<__bf16>(a, st);
}

}  // namespace gsi
