// Cutting the paged cache to a budget (gsi_cache_evict): which entries stay,
// and the moves that bring them below the budget.
//
//   select_kernel : a workgroup per sequence and key head finds the entries that
//                   stay and writes, for every slot below the budget, where its
//                   entry comes from; few moves in place it makes itself.
//   move_kernel   : the moves.
//
// The newest entries and those of the largest mass are each found as all
// entries above a threshold, the key of the wanted rank, and the first ones at
// it.  The threshold comes eight bits at a time: entries that agree with it so
// far are counted by their next eight bits in LDS.  A lane holds the keys of four
// slots one after the other, which lie in one page, so that a load of 16 bytes
// reads them; up to 32768 slots stay in registers and are read once.  A call for
// a few thousand slots is bound by the latency of these reads and of the dozen
// barriers behind them, one for long sequences by the counting in LDS.
#include <utility>

#include "gsi_cache.h"

namespace gsi {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kFewMoves = 64;  // that select_kernel makes itself

// Keys whose unsigned order is that of the scores.  NaN and an entry of no page
// are the least; the two zeros are alike.
__device__ __forceinline__ uint32_t mass_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return v != v ? 0u : u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint32_t age_key(int32_t v) { return (uint32_t)v ^ 0x80000000u; }

struct Four {
  uint32_t v[4];
};

// LDS of a workgroup.
struct Shared {
  int hist[2][4][256];  // of the two selections' passes, zero at first
  uint32_t all[2][kWaves], any[2][kWaves];
  int part[kWaves];
  int2 moves[kFewMoves];
};

// counts[b] becomes the sum of the counts before it; returns after a barrier.
__device__ void sums_before(int *counts, int nb, Shared &sh) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = (nb + kThreads - 1) / kThreads, lo = min(tid * per, nb), hi = min(lo + per, nb);
  __syncthreads();
  int sum = 0;
  for (int b = lo; b < hi; ++b) sum += counts[b];
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(incl, o, 64);
    if (lane >= o) incl += u;
  }
  if (lane == 63) sh.part[wave] = incl;
  __syncthreads();
  int run = incl - sum;
  for (int w = 0; w < wave; ++w) run += sh.part[w];
  for (int b = lo; b < hi; ++b) {
    const int c = counts[b];
    counts[b] = run;
    run += c;
  }
  __syncthreads();
}

__device__ __forceinline__ uint64_t below(int lane) { return (1ull << lane) - 1; }

// The slots of a workgroup in blocks of 256: slot 256 b + 4 lane + e of a block,
// blocks dealt to the wavefronts in turn.  NB blocks at most of a wavefront, with
// their keys in registers; 0: any number, keys are read again each time.
constexpr int kBlock = 256;
template <int NB>
struct Slots {
  int n, lane, wave;
  uint64_t *keep;     // [block][e]: a bit per lane (for NB > 0 written at the end)
  uint32_t kept = 0;  // NB > 0: bit 4 k + e

  // f(k, b) for each of the wavefront's blocks; k is a constant, or the arrays
  // that it indexes would not stay in registers
  template <typename F>
  __device__ __forceinline__ void each(const F &f) const {
    if constexpr (NB > 0)
      unrolled(f, std::make_integer_sequence<int, NB>());
    else
      for (int b = wave; b * kBlock < n; b += kWaves) f(std::integral_constant<int, 0>{}, b);
  }
  template <typename F, int... K>
  __device__ __forceinline__ void unrolled(const F &f, std::integer_sequence<int, K...>) const {
    (((wave + kWaves * K) * kBlock < n ? f(std::integral_constant<int, K>{}, wave + kWaves * K) : void()), ...);
  }
  // bit e: slot e of this lane is there and not kept yet
  __device__ __forceinline__ uint32_t is_free(int k, int b) const {
    uint32_t mine;
    if constexpr (NB > 0) {
      mine = kept >> (4 * k);
    } else {
      mine = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) mine |= (uint32_t)(keep[4 * b + e] >> lane & 1) << e;
    }
    const int left = n - (b * kBlock + 4 * lane);
    return ~mine & (left >= 4 ? 15u : left <= 0 ? 0u : (1u << left) - 1);
  }
  __device__ __forceinline__ void take(int k, int b, uint32_t mine) {  // every lane of the wavefront
    if constexpr (NB > 0) {
      kept |= mine << (4 * k);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint64_t m = __ballot(mine >> e & 1);
        if (lane == 0) keep[4 * b + e] |= m;
      }
    }
  }
};

// Keeps the `count` free slots of the largest key, ties to the lowest slot;
// there are at least `count`.  keys(k, b): this lane's four keys; which: 0 or 1,
// the selection's LDS; counts: LDS for a number per block.
template <int NB, typename Keys>
__device__ __forceinline__ void take_largest(Slots<NB> &sl, int count, const Keys &keys, int which, int *counts,
                                             Shared &sh) {
  const int lane = sl.lane;
  // what all keys agree in, from the top, needs no counting
  uint32_t all = ~0u, any = 0;
  sl.each([&](auto k, int b) {
    const uint32_t is_free = sl.is_free(k, b);
    const Four key = keys(k, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      all &= is_free >> e & 1 ? key.v[e] : ~0u;
      any |= is_free >> e & 1 ? key.v[e] : 0u;
    }
  });
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    all &= __shfl_xor(all, o, 64);
    any |= __shfl_xor(any, o, 64);
  }
  if (lane == 0) sh.all[which][sl.wave] = all, sh.any[which][sl.wave] = any;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) all &= sh.all[which][w], any |= sh.any[which][w];
  const uint32_t differ = all ^ any;
  int shift = 32 - __clz(differ), need = count;  // bits from `shift` on are known: those of prefix
  uint64_t prefix = (uint64_t)all >> shift;
  bool tied = true;  // more slots at the threshold than are taken
  for (int pass = 0; shift > 0 && tied; ++pass) {
    const int low = max(shift - 8, 0);
    const uint32_t mask = (1u << (shift - low)) - 1;
    int *const hist = sh.hist[which][pass];
    sl.each([&](auto k, int b) {
      const uint32_t is_free = sl.is_free(k, b);
      const Four key = keys(k, b);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((is_free >> e & 1) && (uint64_t)key.v[e] >> shift == prefix)
          atomicAdd(&hist[key.v[e] >> low & mask], 1);  // integers: any order
    });
    __syncthreads();
    // from the top, four bins a lane: the bin where the running count reaches
    // `need`; every wavefront by itself
    const int4 h = *reinterpret_cast<const int4 *>(hist + 252 - 4 * lane);
    const int sum = h.x + h.y + h.z + h.w;
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(incl, o, 64);
      if (lane >= o) incl += u;
    }
    const int at = __ffsll((unsigned long long)__ballot(incl >= need)) - 1;
    int above = __builtin_amdgcn_readlane(incl - sum, at), bin = 255 - 4 * at;
    int c = __builtin_amdgcn_readlane(h.w, at);
    if (above + c < need) {
      above += c, --bin, c = __builtin_amdgcn_readlane(h.z, at);
      if (above + c < need) {
        above += c, --bin, c = __builtin_amdgcn_readlane(h.y, at);
        if (above + c < need) above += c, --bin, c = __builtin_amdgcn_readlane(h.x, at);
      }
    }
    need -= above;
    tied = c > need;
    prefix = prefix << (shift - low) | (uint32_t)bin;
    shift = low;
  }
  if (!tied) {
    sl.each([&](auto k, int b) {
      const Four key = keys(k, b);
      uint32_t mine = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) mine |= (uint32_t)((uint64_t)key.v[e] >> shift >= prefix) << e;
      sl.take(k, b, mine & sl.is_free(k, b));
    });
  } else {  // the first `need` slots with this very key
    const auto same_of = [&](const Four &key, uint32_t is_free) {
      uint32_t same = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) same |= (uint32_t)(key.v[e] == prefix) << e;
      return same & is_free;
    };
    sl.each([&](auto k, int b) {
      const uint32_t same = same_of(keys(k, b), sl.is_free(k, b));
      int c = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) c += __popcll(__ballot(same >> e & 1));
      if (lane == 0) counts[b] = c;
    });
    sums_before(counts, (sl.n + kBlock - 1) / kBlock, sh);
    sl.each([&](auto k, int b) {
      const uint32_t is_free = sl.is_free(k, b);
      const Four key = keys(k, b);
      const uint32_t same = same_of(key, is_free);
      int rank = counts[b];
#pragma unroll
      for (int e = 0; e < 4; ++e) rank += __popcll(__ballot(same >> e & 1) & below(lane));
      uint32_t mine = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (key.v[e] > prefix || ((same >> e & 1) && rank < need)) mine |= 1u << e;
        rank += same >> e & 1;
      }
      sl.take(k, b, mine & is_free);
    });
  }
  __syncthreads();
}

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void move_piece(const EvictArgs &a, int64_t from, int64_t to) {
  const u32x4_t k = *reinterpret_cast<const u32x4_t *>(a.c.K + from), v = *reinterpret_cast<const u32x4_t *>(a.c.V + from);
  *reinterpret_cast<u32x4_t *>(a.c.K + to) = k;
  *reinterpret_cast<u32x4_t *>(a.c.V + to) = v;
}

__device__ __forceinline__ void move_numbers(const EvictArgs &a, int64_t from, int64_t to) {
  a.c.mass[to] = a.c.mass[from];
  if (a.c.age) a.c.age[to] = a.c.age[from];
}

// blocks: for which there is LDS; pieces: of 16 bytes of a key.
template <int NB>
__global__ void __launch_bounds__(kThreads) select_kernel(EvictArgs a, int blocks, int pieces) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ __attribute__((aligned(16))) Shared sh;
  const int s = blockIdx.x / a.c.heads, h = blockIdx.x - s * a.c.heads, tid = threadIdx.x;
  const int n = clamped_length(a.c, a.lengths, s), budget = a.budget;
  int32_t *const from = a.from + ((int64_t)s * a.c.heads + h) * budget;
  if (h == 0 && tid == 0 && a.lengths_out) a.lengths_out[s] = min(n, budget);
  if (n <= budget) {
    for (int j = tid; j < budget; j += kThreads) from[j] = j < n ? j : -1;
    return;
  }
  const int nb = (n + kBlock - 1) / kBlock;
  int *const count = reinterpret_cast<int *>(lds + 32 * blocks);
  Slots<NB> sl{n, tid & 63, tid >> 6, reinterpret_cast<uint64_t *>(lds)};
  const bool by_age = a.c.age && a.recent > 0, by_mass = budget > a.recent;
  // This lane's four slots of a block: one page.  What lies behind the last slot
  // reads the last page's; an entry without a page reads page 0 and counts as
  // the least.
  const auto raw_page = [&](int b) {
    return a.c.table[s * a.c.ld + (min(b * kBlock + 4 * sl.lane, n - 1) >> a.c.shift)];
  };
  const auto is_page = [&](int p) { return (uint32_t)p < (uint32_t)a.c.pages; };
  const auto read = [&](const void *from_pool, int p, int b) {
    Four r;
    __builtin_memcpy(&r, static_cast<const uint32_t *>(from_pool) +
                             number_at(a.c, is_page(p) ? p : 0, h, b * kBlock + 4 * sl.lane), 16);
    return r;
  };
  const auto mass_keys = [&](int p, Four r) {
#pragma unroll
    for (int e = 0; e < 4; ++e) r.v[e] = is_page(p) ? mass_key(__uint_as_float(r.v[e])) : 0;
    return r;
  };
  const auto age_keys = [&](int p, Four r) {
#pragma unroll
    for (int e = 0; e < 4; ++e) r.v[e] = is_page(p) ? age_key((int32_t)r.v[e]) : 0;
    return r;
  };
  for (int k = tid; k < 2 * 4 * 256; k += kThreads) (&sh.hist[0][0][0])[k] = 0;
  // All reads of a selection at once, those of both where there are registers.
  constexpr bool kBoth = NB <= 1;
  int p[NB > 0 ? NB : 1];
  Four age[NB > 0 ? NB : 1], mass[NB > 0 ? NB : 1];
  const auto read_masses = [&] {
    sl.each([&](auto k, int b) { mass[k] = read(a.c.mass, p[k], b); });
  };
  if constexpr (NB > 0) {
    sl.each([&](auto k, int b) { p[k] = raw_page(b); });
    if (by_age) sl.each([&](auto k, int b) { age[k] = read(a.c.age, p[k], b); });
    if (kBoth && by_mass) read_masses();
    if (by_age) sl.each([&](auto k, int) { age[k] = age_keys(p[k], age[k]); });
  } else {
    for (int k = tid; k < 4 * nb; k += kThreads) sl.keep[k] = 0;
  }
  __syncthreads();
  if (by_age) {
    take_largest(sl, a.recent, [&](auto k, int b) {
      if constexpr (NB > 0) return age[k];
      const int page = raw_page(b);
      return age_keys(page, read(a.c.age, page, b));
    }, 0, count, sh);
  } else if (a.recent > 0) {
    sl.each([&](auto k, int b) {
      const int before = n - a.recent - (b * kBlock + 4 * sl.lane);  // slots of this lane before the newest
      sl.take(k, b, sl.is_free(k, b) & (before <= 0 ? 15u : before >= 4 ? 0u : 15u << before & 15u));
    });
    __syncthreads();
  }
  if (by_mass) {
    if constexpr (NB > 0) {
      if (!kBoth) read_masses();
      sl.each([&](auto k, int) { mass[k] = mass_keys(p[k], mass[k]); });
    }
    take_largest(sl, budget - a.recent, [&](auto k, int b) {
      if constexpr (NB > 0) return mass[k];
      const int page = raw_page(b);
      return mass_keys(page, read(a.c.mass, page, b));
    }, 1, count, sh);
  }
  // kept slots before each block
  sl.each([&](auto k, int b) {
    int c = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint64_t m;
      if constexpr (NB > 0) {
        m = __ballot(sl.kept >> (4 * k + e) & 1);
        if (sl.lane == 0) sl.keep[4 * b + e] = m;
      } else {
        m = sl.keep[4 * b + e];
      }
      c += __popcll(m);
    }
    if (sl.lane == 0) count[b] = c;
  });
  sums_before(count, nb, sh);
  const auto is_kept = [&](int i) { return sl.keep[4 * (i / kBlock) + (i & 3)] >> (i / 4 % 64) & 1; };
  // kept slots of a block's lanes before `lane`
  const auto lanes_before = [&](int b, int lane) {
    int c = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) c += __popcll(sl.keep[4 * b + e] & below(lane));
    return c;
  };
  const auto before = [&](int i) {
    int c = count[i / kBlock] + lanes_before(i / kBlock, i / 4 % 64);
    for (int e = 0; e < (i & 3); ++e) c += is_kept((i & ~3) + e);
    return c;
  };
  const int low = before(budget);  // budget < n
  const bool few = budget - low <= kFewMoves && !a.to;
  for (int j = tid; j < budget; j += kThreads) {
    if (is_kept(j)) {
      from[j] = j;
      continue;
    }
    // the hole's rank among the holes is that of its filler among the kept slots behind
    const int hole = j - before(j);
    int rank = low + hole, lo = budget / kBlock, hi = nb - 1;  // the last block with at most `rank` kept slots before it
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (count[mid] <= rank)
        lo = mid;
      else
        hi = mid - 1;
    }
    rank -= count[lo];
    int lane = 0;  // the last lane with at most `rank` before it
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
      if (lanes_before(lo, lane + o) <= rank) lane += o;
    rank -= lanes_before(lo, lane);
    int src = lo * kBlock + 4 * lane;
    for (; rank > 0 || !is_kept(src); ++src) rank -= (int)is_kept(src);
    from[j] = src;
    if (few) sh.moves[hole] = make_int2(src, j);
  }
  if (!few) return;
  __syncthreads();
  for (int k = sl.wave; k < budget - low; k += kWaves) {
    const int src = sh.moves[k].x, j = sh.moves[k].y, p = page_of(a.c, s, src), t = page_of(a.c, s, j);
    if (p < 0 || t < 0) continue;
    if (sl.lane < pieces) move_piece(a, entry_at(a.c, p, h, src) + 16 * sl.lane, entry_at(a.c, t, h, j) + 16 * sl.lane);
    if (sl.lane == 0) move_numbers(a, number_at(a.c, p, h, src), number_at(a.c, t, h, j));
  }
}

constexpr int kMoveRows = 4;  // of a thread

// 16 bytes of a key and of a value per thread and row; `side` rows at a time.
__global__ void __launch_bounds__(256) move_kernel(EvictArgs a, int strips, Div pieces) {
  const int sh = blockIdx.x / strips, strip = blockIdx.x - sh * strips, s = sh / a.c.heads, h = sh - s * a.c.heads;
  const int rows = 256 / pieces.by, row = quotient(threadIdx.x, pieces), piece = threadIdx.x - row * pieces.by;
  if (row >= rows) return;
  const int32_t *const from = a.from + ((int64_t)s * a.c.heads + h) * a.budget;
  int src[kMoveRows], p[kMoveRows] = {}, t[kMoveRows] = {};
#pragma unroll
  for (int k = 0; k < kMoveRows; ++k) {
    const int j = (strip * kMoveRows + k) * rows + row;
    src[k] = j < a.budget ? from[j] : -1;
    if (!a.to && src[k] == j) src[k] = -1;
  }
#pragma unroll
  for (int k = 0; k < kMoveRows; ++k) {
    const int j = (strip * kMoveRows + k) * rows + row;
    if (src[k] < 0) continue;
    p[k] = page_of(a.c, s, src[k]);
    t[k] = a.to ? a.to[s * a.to_ld + (j >> a.c.shift)] : a.c.table[s * a.c.ld + (j >> a.c.shift)];
    if (p[k] < 0 || t[k] < 0 || t[k] >= a.c.pages) src[k] = -1;
  }
  u32x4_t key[kMoveRows] = {}, value[kMoveRows] = {};
#pragma unroll
  for (int k = 0; k < kMoveRows; ++k) {
    if (src[k] < 0) continue;
    const int64_t at = entry_at(a.c, p[k], h, src[k]) + 16 * piece;
    key[k] = *reinterpret_cast<const u32x4_t *>(a.c.K + at);
    value[k] = *reinterpret_cast<const u32x4_t *>(a.c.V + at);
  }
#pragma unroll
  for (int k = 0; k < kMoveRows; ++k) {
    const int j = (strip * kMoveRows + k) * rows + row;
    if (src[k] < 0) continue;
    const int64_t to = entry_at(a.c, t[k], h, j) + 16 * piece;
    *reinterpret_cast<u32x4_t *>(a.c.K + to) = key[k];
    *reinterpret_cast<u32x4_t *>(a.c.V + to) = value[k];
    if (piece == 0) move_numbers(a, number_at(a.c, p[k], h, src[k]), number_at(a.c, t[k], h, j));
  }
}

}  // namespace

gsi_status launch_evict(const EvictArgs &a, int dtype, hipStream_t st) {
  const int slots = a.c.most << a.c.shift, blocks = slots / kBlock + 1;
  const int pieces = a.c.d * (dtype == GSI_FP32 ? 4 : 2) / 16, per = 256 / pieces * kMoveRows;
  const int64_t rows = (int64_t)a.c.S * a.c.heads, strips = (a.budget + per - 1) / per;
  if (rows * kThreads > kMostLaunch || rows * strips * 256 > kMostLaunch) return GSI_E_SHAPE;
  const size_t lds = (size_t)blocks * 36;
  if (slots <= kWaves * kBlock)
    select_kernel<1><<<(unsigned)rows, kThreads, lds, st>>>(a, blocks, pieces);
  else if (slots <= 8 * kWaves * kBlock)
    select_kernel<8><<<(unsigned)rows, kThreads, lds, st>>>(a, blocks, pieces);
  else
    select_kernel<0><<<(unsigned)rows, kThreads, lds, st>>>(a, blocks, pieces);
  if (hipGetLastError() != hipSuccess) return GSI_E_HIP;
  // In place no more move than there are slots behind the budget; select_kernel
  // has made few (and made again they change nothing: nothing is moved from
  // below the budget).
  if (!a.to && (a.budget >= slots || slots - a.budget <= kFewMoves || a.budget <= kFewMoves)) return GSI_OK;
  move_kernel<<<(unsigned)(rows * strips), 256, 0, st>>>(a, (int)strips, div_by(pieces));
  return hipGetLastError() == hipSuccess ? GSI_OK : GSI_E_HIP;
}

}  // namespace gsi
