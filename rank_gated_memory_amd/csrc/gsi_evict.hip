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
// barriers behind them (2049 slots, 128 workgroups: 12 us), one for long sequences by
// the counting in LDS of one CU each (30011 slots, 24 workgroups: 41 us).
#include <algorithm>
#include <utility>

#include "gsi_cache.h"

namespace gsi {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
// Moves that select_kernel makes itself.  16 sequences of 8 heads to 2048 of 2049
// (2112) entries: 13.2 (15.4) us, with move_kernel 21.9 (23.7).
constexpr int kFewMoves = 64;

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
  uint32_t all[kWaves], any[kWaves];
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
  const int incl = sums_to(sum);
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
// there are at least `count`.  keys(k, b): this lane's four keys; Common: they may
// agree in their upper bits, as ages do; hists: the selection's bins, zero; counts:
// LDS for a number per block.
template <bool Common, int NB, typename Keys>
__device__ __forceinline__ void take_largest(Slots<NB> &sl, int count, const Keys &keys, int (*hists)[256], int *counts,
                                             Shared &sh) {
  const int lane = sl.lane;
  int shift = 32, need = count;
  // keys from `base` on to base + span agree with the threshold so far
  uint32_t base = 0, span = ~0u;
  if constexpr (Common) {  // what all keys agree in, from the top, needs no counting
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
    all = joined_to<-1>(all, [](int x, int y) { return x & y; });
    any = joined_to<0>(any, [](int x, int y) { return x | y; });
    if (lane == 63) sh.all[sl.wave] = all, sh.any[sl.wave] = any;
    __syncthreads();
    all = sh.all[0], any = sh.any[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) all &= sh.all[w], any |= sh.any[w];
    shift = 32 - __clz(all ^ any);
    if (shift < 32) span = (1u << shift) - 1, base = all & ~span;
  }
  bool tied = true;  // more slots at the threshold than are taken
  for (int pass = 0; shift > 0 && tied; ++pass) {
    const int low = max(shift - 8, 0);
    int *const hist = hists[pass];
    sl.each([&](auto k, int b) {
      const uint32_t is_free = sl.is_free(k, b);
      const Four key = keys(k, b);
      // Neighbours often agree in these bits (ages are slots at first), and lanes
      // at one bin take their turns: a lane's run of one bin is counted at once,
      // and of the lanes' last runs those of the first lane's bin.
      uint32_t among = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) among |= (uint32_t)(key.v[e] - base <= span) << e;
      among &= is_free;
      if (__ballot(among != 0) == 0) return;  // few are left after a pass or two
      int bin = 0, c = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t off = key.v[e] - base;
        const bool in = among >> e & 1;
        if (in && c > 0 && (int)(off >> low) != bin) {
          atomicAdd(&hist[bin], c);  // integers: any order
          c = 0;
        }
        bin = in ? off >> low : bin;
        c += in;
      }
      const uint64_t last = __ballot(c > 0);
      if (last == 0) return;
      const int first = __ffsll((unsigned long long)last) - 1, common = __builtin_amdgcn_readlane(bin, first);
      const uint64_t same = last & __ballot(bin == common);
      const int sum = __popcll(same & __ballot(c & 1)) + 2 * __popcll(same & __ballot(c & 2)) +
                      4 * __popcll(same & __ballot(c & 4));
      if (lane == first)
        atomicAdd(&hist[common], sum);
      else if (c > 0 && bin != common)
        atomicAdd(&hist[bin], c);
    });
    __syncthreads();
    // from the top, four bins a lane: the bin where the running count reaches
    // `need`; every wavefront by itself
    const int4 h = *reinterpret_cast<const int4 *>(hist + 252 - 4 * lane);
    const int sum = h.x + h.y + h.z + h.w;
    const int incl = sums_to(sum);
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
    base += (uint32_t)bin << low;
    span = (1u << low) - 1;
    shift = low;
  }
  if (!tied) {
    sl.each([&](auto k, int b) {
      const Four key = keys(k, b);
      uint32_t mine = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) mine |= (uint32_t)(key.v[e] >= base) << e;
      sl.take(k, b, mine & sl.is_free(k, b));
    });
  } else {  // the first `need` slots with this very key
    const auto same_of = [&](const Four &key, uint32_t is_free) {
      uint32_t same = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) same |= (uint32_t)(key.v[e] == base) << e;
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
        if (key.v[e] > base || ((same >> e & 1) && rank < need)) mine |= 1u << e;
        rank += same >> e & 1;
      }
      sl.take(k, b, mine & is_free);
    });
  }
  __syncthreads();
}

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void move_piece(const EvictArgs &a, int64_t from, int64_t to) {
  const u32x4_t k = *reinterpret_cast<const u32x4_t *>(a.c.K + from);
  const u32x4_t v = *reinterpret_cast<const u32x4_t *>(a.c.V + from);
  *reinterpret_cast<u32x4_t *>(a.c.K + to) = k;
  *reinterpret_cast<u32x4_t *>(a.c.V + to) = v;
}

__device__ __forceinline__ void move_numbers(const EvictArgs &a, int64_t from, int64_t to) {
  a.c.mass[to] = a.c.mass[from];
  if (a.c.age) a.c.age[to] = a.c.age[from];
}

// blocks: for which there is LDS; holes: for which there is; pieces: of 16 bytes
// of a key.
template <int NB>
__global__ void __launch_bounds__(kThreads) select_kernel(EvictArgs a, int blocks, int holes, int pieces) {
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
  int p[NB > 0 ? NB : 1];
  Four age[NB > 0 ? NB : 1], mass[NB > 0 ? NB : 1];
  if constexpr (NB > 0) {  // all reads of both selections at once
    sl.each([&](auto k, int b) { p[k] = raw_page(b); });
    if (by_age) sl.each([&](auto k, int b) { age[k] = read(a.c.age, p[k], b); });
    if (by_mass) sl.each([&](auto k, int b) { mass[k] = read(a.c.mass, p[k], b); });
    if (by_age) sl.each([&](auto k, int) { age[k] = age_keys(p[k], age[k]); });
  } else {
    for (int k = tid; k < 4 * nb; k += kThreads) sl.keep[k] = 0;
  }
  __syncthreads();
  if (by_age) {
    take_largest<true>(sl, a.recent, [&](auto k, int b) {
      if constexpr (NB > 0) return age[k];
      const int page = raw_page(b);
      return age_keys(page, read(a.c.age, page, b));
    }, sh.hist[0], count, sh);
  } else if (a.recent > 0) {
    sl.each([&](auto k, int b) {
      const int before = n - a.recent - (b * kBlock + 4 * sl.lane);  // slots of this lane before the newest
      sl.take(k, b, sl.is_free(k, b) & (before <= 0 ? 15u : before >= 4 ? 0u : 15u << before & 15u));
    });
    __syncthreads();
  }
  if (by_mass) {
    if constexpr (NB > 0) sl.each([&](auto k, int) { mass[k] = mass_keys(p[k], mass[k]); });
    take_largest<false>(sl, budget - a.recent, [&](auto k, int b) {
      if constexpr (NB > 0) return mass[k];
      const int page = raw_page(b);
      return mass_keys(page, read(a.c.mass, page, b));
    }, sh.hist[1], count, sh);
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
  // of a lane's four slots, the kept ones and how many are kept before them
  const auto kept_of = [&](int b, int lane, uint32_t *kept) {
    int c = count[b];
    *kept = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint64_t w = sl.keep[4 * b + e];
      c += __popcll(w & below(lane));
      *kept |= (uint32_t)(w >> lane & 1) << e;
    }
    return c;
  };
  uint32_t kept;
  int low = kept_of(budget / kBlock, budget / 4 % 64, &kept);  // kept below the budget; budget < n
  low += __popc(kept & ((1u << (budget & 3)) - 1));
  const bool few = budget - low <= kFewMoves && !a.to;
  // The holes below the budget and the kept slots behind it, both in order, go
  // together: through a list of the holes in LDS, `holes` at a time.
  int *const list = count + blocks;
  for (int first = 0; first == 0 || first < budget - low; first += holes) {
    // loops that stay loops: code for every block waits longer for its fetch
#pragma unroll 1
    for (int b = sl.wave; b * kBlock < budget; b += kWaves) {
      const int i0 = b * kBlock + 4 * sl.lane;
      uint32_t mine;
      int hole = i0 - kept_of(b, sl.lane, &mine) - first;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (i0 + e >= budget) continue;
        if (mine >> e & 1) {
          if (first == 0) from[i0 + e] = i0 + e;
        } else {
          if (hole >= 0 && hole < holes) list[hole] = i0 + e;
          ++hole;
        }
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int b = budget / kBlock + sl.wave; b < nb; b += kWaves) {
      const int i0 = b * kBlock + 4 * sl.lane;
      uint32_t mine;
      int rank = kept_of(b, sl.lane, &mine) - low;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!(mine >> e & 1)) continue;
        const int hole = rank - first;
        if (i0 + e >= budget && hole >= 0 && hole < holes) {
          from[list[hole]] = i0 + e;
          if (few) sh.moves[rank] = make_int2(i0 + e, list[hole]);
        }
        ++rank;
      }
    }
    __syncthreads();
  }
  if (!few) return;
  for (int k = sl.wave; k < budget - low; k += kWaves) {
    const int src = sh.moves[k].x, j = sh.moves[k].y, p = page_of(a.c, s, src), t = page_of(a.c, s, j);
    if (p < 0 || t < 0) continue;
    if (sl.lane < pieces) move_piece(a, entry_at(a.c, p, h, src) + 16 * sl.lane, entry_at(a.c, t, h, j) + 16 * sl.lane);
    if (sl.lane == 0) move_numbers(a, number_at(a.c, p, h, src), number_at(a.c, t, h, j));
  }
}

constexpr int kMoveRows = 2;  // of a thread

// 16 bytes of a key and of a value per thread and row.  Reads and writes all that
// moves once: 98304000 bytes of 24 heads' entries into other pages in 23 us, 4.3
// TB/s (with 4 rows a thread 29 us).
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
  const int holes = std::max(1, std::min({a.budget, slots - a.budget, 8192}));
  const size_t lds = (size_t)blocks * 36 + (size_t)holes * 4;
  // As few blocks of keys in registers as hold the slots, us with 1, 2, 8 and 0 (in
  // memory) of a wavefront: 2049 to 2048 12.9, 13.5, 17.4, 17.6; 5003 to 777 (fp32)
  // -, 22.0, 25.9, 28.1; 30011 to 4000 -, -, 63.6, 79.6.  (From 8193 slots on keys in
  // LDS, short code and masses counted one by one: the same for few rows, but 2560
  // rows of 2049 slots 93 for 62 us, and equal masses, all at one address, 16 for 12.)
  if (slots <= kWaves * kBlock)
    select_kernel<1><<<(unsigned)rows, kThreads, lds, st>>>(a, blocks, holes, pieces);
  else if (slots <= 2 * kWaves * kBlock)
    select_kernel<2><<<(unsigned)rows, kThreads, lds, st>>>(a, blocks, holes, pieces);
  else if (slots <= 8 * kWaves * kBlock)
    select_kernel<8><<<(unsigned)rows, kThreads, lds, st>>>(a, blocks, holes, pieces);
  else
    select_kernel<0><<<(unsigned)rows, kThreads, lds, st>>>(a, blocks, holes, pieces);
  if (hipGetLastError() != hipSuccess) return GSI_E_HIP;
  // In place no more move than there are slots behind the budget; select_kernel
  // has made few (and made again they change nothing: nothing is moved from
  // below the budget).
  if (!a.to && (a.budget >= slots || slots - a.budget <= kFewMoves || a.budget <= kFewMoves)) return GSI_OK;
  move_kernel<<<(unsigned)(rows * strips), 256, 0, st>>>(a, (int)strips, div_by(pieces));
  return hipGetLastError() == hipSuccess ? GSI_OK : GSI_E_HIP;
}

}  // namespace gsi
