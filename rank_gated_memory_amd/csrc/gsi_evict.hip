// Cutting the paged cache to a budget (gsi_cache_evict): which entries stay,
// and the moves that bring them below the budget.
#include "gsi_cache.h"

namespace gsi {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;

// Keys whose unsigned order is that of the scores.  NaN and an entry of no page
// are the least; the two zeros are alike.
__device__ __forceinline__ uint32_t mass_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return v != v ? 0u : u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint32_t age_key(int32_t v) { return (uint32_t)v ^ 0x80000000u; }

// Adds to the set `keep` (a bit per slot) the `count` slots below n outside it
// of the largest key, ties to the lowest slot; there are at least `count`.  The
// key of rank `count` is found eight bits at a time from the top.  words: LDS
// for a number per 64 slots.
template <typename Key>
__device__ void take_largest(int n, int count, uint64_t *keep, int *words, int *hist, const Key &key) {
  if (count <= 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = (n + 63) / 64;
  uint32_t prefix = 0;
  int need = count;
  const auto free_slot = [&](int i) { return i < n && !(keep[i >> 6] >> (i & 63) & 1); };
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      if (!free_slot(i)) continue;
      const uint32_t k = key(i);
      if (shift == 24 || k >> (shift + 8) == prefix) atomicAdd(&hist[k >> shift & 255], 1);  // integers: any order
    }
    __syncthreads();
    // from the top: the bin where the running count reaches `need`
    int above = 0, bin = 255;
    while (bin > 0 && above + hist[bin] < need) above += hist[bin--];
    need -= above;
    prefix = prefix << 8 | bin;
    __syncthreads();
  }
  // all keys above, and the first `need` slots of those that are it
  for (int w = wave; w < nw; w += kWaves) {
    const int i = w * 64 + lane;
    const uint64_t same = __ballot(free_slot(i) && key(i) == prefix);
    if (lane == 0) words[w] = __popcll(same);
  }
  __syncthreads();
  if (tid == 0)
    for (int w = 0, run = 0; w < nw; ++w) {
      const int c = words[w];
      words[w] = run;
      run += c;
    }
  __syncthreads();
  for (int w = wave; w < nw; w += kWaves) {
    const int i = w * 64 + lane;
    const bool is_free = free_slot(i);
    const uint32_t k = is_free ? key(i) : 0;
    const uint64_t same = __ballot(is_free && k == prefix);
    const int rank = words[w] + __popcll(same & ((1ull << lane) - 1));
    const uint64_t more = __ballot(is_free && (k > prefix || (k == prefix && rank < need)));
    if (lane == 0) keep[w] |= more;
  }
  __syncthreads();
}

// A workgroup per sequence and key head: `from`.
__global__ void __launch_bounds__(kThreads) select_kernel(EvictArgs a, int words) {
  extern __shared__ __attribute__((aligned(8))) uint8_t lds[];
  __shared__ int hist[256];
  uint64_t *const keep = reinterpret_cast<uint64_t *>(lds);
  int *const count = reinterpret_cast<int *>(keep + words);
  const int s = blockIdx.x / a.c.heads, h = blockIdx.x - s * a.c.heads, tid = threadIdx.x;
  const int n = clamped_length(a.c, a.lengths, s), budget = a.budget;
  int32_t *const from = a.from + ((int64_t)s * a.c.heads + h) * budget;
  if (h == 0 && tid == 0 && a.lengths_out) a.lengths_out[s] = min(n, budget);
  if (n <= budget) {
    for (int j = tid; j < budget; j += kThreads) from[j] = j < n ? j : -1;
    return;
  }
  const int nw = (n + 63) / 64;
  for (int w = tid; w < nw; w += kThreads) keep[w] = 0;
  __syncthreads();
  if (a.c.age) {
    take_largest(n, a.recent, keep, count, hist, [&](int i) {
      const int p = page_of(a.c, s, i);
      return p < 0 ? 0u : age_key(a.c.age[number_at(a.c, p, h, i)]);
    });
  } else {
    for (int w = tid; w < nw; w += kThreads) {
      const int lo = min(max(n - a.recent - w * 64, 0), 64), hi = min(n - w * 64, 64);  // bits [lo, hi)
      const uint64_t to_hi = hi == 64 ? ~0ull : (1ull << hi) - 1, to_lo = lo == 64 ? ~0ull : (1ull << lo) - 1;
      keep[w] = to_hi & ~to_lo;
    }
    __syncthreads();
  }
  take_largest(n, budget - a.recent, keep, count, hist, [&](int i) {
    const int p = page_of(a.c, s, i);
    return p < 0 ? 0u : mass_key(a.c.mass[number_at(a.c, p, h, i)]);
  });
  // kept slots before each word
  if (tid == 0)
    for (int w = 0, run = 0; w < nw; ++w) {
      count[w] = run;
      run += __popcll(keep[w]);
    }
  __syncthreads();
  const auto before = [&](int i) { return count[i >> 6] + __popcll(keep[i >> 6] & ((1ull << (i & 63)) - 1)); };
  const int low = before(budget);  // budget < n
  for (int j = tid; j < budget; j += kThreads) {
    if (keep[j >> 6] >> (j & 63) & 1) {
      from[j] = j;
      continue;
    }
    // the hole's rank among the holes is that of its filler among the kept slots behind
    const int rank = low + j - before(j);
    int lo = 0, hi = nw - 1;  // the last word with at most `rank` kept slots before it
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (count[mid] <= rank)
        lo = mid;
      else
        hi = mid - 1;
    }
    uint64_t bits = keep[lo];
    for (int k = rank - count[lo]; k > 0; --k) bits &= bits - 1;
    from[j] = lo * 64 + __ffsll((unsigned long long)bits) - 1;
  }
}

// 16 bytes of an entry's key and value per thread.
__global__ void __launch_bounds__(256) move_kernel(EvictArgs a, int strips, int pieces) {
  const int sh = blockIdx.x / strips, strip = blockIdx.x - sh * strips, s = sh / a.c.heads, h = sh - s * a.c.heads;
  const int64_t k = (int64_t)strip * 256 + threadIdx.x;
  const int j = (int)(k / pieces), piece = (int)(k - (int64_t)j * pieces);
  if (j >= a.budget) return;
  const int src = a.from[((int64_t)s * a.c.heads + h) * a.budget + j];
  if (src < 0 || (!a.to && src == j)) return;
  const int p = page_of(a.c, s, src);
  const int t = a.to ? a.to[s * a.to_ld + (j >> a.c.shift)] : a.c.table[s * a.c.ld + (j >> a.c.shift)];
  if (p < 0 || t < 0 || t >= a.c.pages) return;
  const int64_t at = entry_at(a.c, p, h, src) + 16 * piece, to = entry_at(a.c, t, h, j) + 16 * piece;
  *reinterpret_cast<uint4 *>(a.c.K + to) = *reinterpret_cast<const uint4 *>(a.c.K + at);
  *reinterpret_cast<uint4 *>(a.c.V + to) = *reinterpret_cast<const uint4 *>(a.c.V + at);
  if (piece == 0) {
    a.c.mass[number_at(a.c, t, h, j)] = a.c.mass[number_at(a.c, p, h, src)];
    if (a.c.age) a.c.age[number_at(a.c, t, h, j)] = a.c.age[number_at(a.c, p, h, src)];
  }
}

}  // namespace

gsi_status launch_evict(const EvictArgs &a, int dtype, hipStream_t st) {
  const int words = (a.c.most << a.c.shift) / 64 + 1;
  const int pieces = a.c.d * (dtype == GSI_FP32 ? 4 : 2) / 16;
  const int64_t rows = (int64_t)a.c.S * a.c.heads, strips = ((int64_t)a.budget * pieces + 255) / 256;
  if (rows * kThreads > kMostLaunch || rows * strips * 256 > kMostLaunch) return GSI_E_SHAPE;
  select_kernel<<<(unsigned)rows, kThreads, (size_t)words * 12, st>>>(a, words);
  if (hipGetLastError() != hipSuccess) return GSI_E_HIP;
  move_kernel<<<(unsigned)(rows * strips), 256, 0, st>>>(a, (int)strips, pieces);
  return hipGetLastError() == hipSuccess ? GSI_OK : GSI_E_HIP;
}

}  // namespace gsi
