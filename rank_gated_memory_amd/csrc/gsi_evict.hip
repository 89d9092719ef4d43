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
// far are counted by their next eight bits in LDS.  Keys lie in registers (up to
// 4096 slots) or LDS (up to 32768), so an entry's mass and age are read once; a
// call for a few thousand slots is bound by the latency of these reads and of
// the dozen barriers behind them, one for long sequences by the counting.
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

// LDS of a workgroup.  words: as many 64-bit words as the slots need.
struct Shared {
  int hist[2][4][256];  // of the two selections' passes, zero at first
  uint32_t all[2][kWaves], any[2][kWaves];
  int part[kWaves];
  int2 moves[kFewMoves];
};

// words[w] becomes the sum of the words before it; returns after a barrier.
__device__ void sums_before(int *words, int nw, Shared &sh) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = (nw + kThreads - 1) / kThreads, lo = min(tid * per, nw), hi = min(lo + per, nw);
  __syncthreads();
  int sum = 0;
  for (int w = lo; w < hi; ++w) sum += words[w];
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
  for (int w = lo; w < hi; ++w) {
    const int c = words[w];
    words[w] = run;
    run += c;
  }
  __syncthreads();
}

// Where a selection's keys lie: four words of slots per wavefront in registers,
// LDS, or where they came from, read again each time.
enum Keys { kInRegisters, kInLds, kInMemory };
constexpr int kWords = 4;
constexpr int kMostInRegisters = kWords * kThreads, kMostInLds = 32 * 1024;

// The slots of a workgroup: slot 64 w + lane of word w, words dealt to the
// wavefronts in turn.
template <Keys K>
struct Slots {
  int n, lane, wave;
  uint64_t *keep;     // a bit per slot (from registers: written at the end)
  uint32_t kept = 0;  // in registers: bit r for this lane's slot of word r

  // f(r, w) for each of the wavefront's words; r is a constant, or the arrays
  // that it indexes would not stay in registers
  template <typename F>
  __device__ __forceinline__ void each(const F &f) const {
    if constexpr (K == kInRegisters) {
      unrolled(f, std::make_integer_sequence<int, kWords>());
    } else {
      for (int w = wave; w * 64 < n; w += kWaves) f(std::integral_constant<int, 0>{}, w);
    }
  }
  template <typename F, int... R>
  __device__ __forceinline__ void unrolled(const F &f, std::integer_sequence<int, R...>) const {
    ((wave * 64 + kWaves * 64 * R < n ? f(std::integral_constant<int, R>{}, wave + kWaves * R) : void()), ...);
  }
  __device__ __forceinline__ bool is_free(int r, int w) const {
    if (w * 64 + lane >= n) return false;
    if constexpr (K == kInRegisters) return !(kept >> r & 1);
    return !(keep[w] >> lane & 1);
  }
  // every lane of the wavefront
  __device__ __forceinline__ void take(int r, int w, bool mine) {
    if constexpr (K == kInRegisters) {
      kept |= (uint32_t)mine << r;
    } else {
      const uint64_t m = __ballot(mine);
      if (lane == 0) keep[w] |= m;
    }
  }
};

// Keeps the `count` free slots of the largest key, ties to the lowest slot;
// there are at least `count`.  which: 0 or 1, the selection's LDS.
template <Keys K, typename Key>
__device__ __forceinline__ void take_largest(Slots<K> &sl, int count, const Key &key, int which, int *words, Shared &sh) {
  if (count <= 0) return;
  const int lane = sl.lane;
  // what all keys agree in, from the top, needs no counting
  uint32_t all = ~0u, any = 0;
  sl.each([&](auto r, int w) {
    if (sl.is_free(r, w)) {
      const uint32_t k = key(r, w);
      all &= k;
      any |= k;
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
    sl.each([&](auto r, int w) {
      if (!sl.is_free(r, w)) return;
      const uint32_t k = key(r, w);
      if ((uint64_t)k >> shift == prefix) atomicAdd(&hist[k >> low & mask], 1);  // integers: any order
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
    sl.each([&](auto r, int w) { sl.take(r, w, sl.is_free(r, w) && (uint64_t)key(r, w) >> shift >= prefix); });
  } else {  // the first `need` slots with this very key
    sl.each([&](auto r, int w) {
      const int same = __popcll(__ballot(sl.is_free(r, w) && key(r, w) == prefix));
      if (lane == 0) words[w] = same;
    });
    sums_before(words, (sl.n + 63) / 64, sh);
    sl.each([&](auto r, int w) {
      const bool is_free = sl.is_free(r, w);
      const uint32_t k = is_free ? key(r, w) : 0;
      const int rank = words[w] + __popcll(__ballot(is_free && k == prefix) & ((1ull << lane) - 1));
      sl.take(r, w, is_free && (k > prefix || (k == prefix && rank < need)));
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

// words: 64-bit words of LDS for the slots; pieces: of 16 bytes of a key.
template <Keys K>
__global__ void __launch_bounds__(kThreads) select_kernel(EvictArgs a, int words, int pieces) {
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
  const int nw = (n + 63) / 64;
  int *const count = reinterpret_cast<int *>(lds + 8 * words);
  uint32_t *const keys = reinterpret_cast<uint32_t *>(lds + 12 * words);
  Slots<K> sl{n, tid & 63, tid >> 6, reinterpret_cast<uint64_t *>(lds)};
  const bool by_age = a.c.age && a.recent > 0;
  // An entry without a page reads page 0 and counts as the least.
  const auto raw_page = [&](int i) { return a.c.table[s * a.c.ld + (i >> a.c.shift)]; };
  const auto is_page = [&](int p) { return (uint32_t)p < (uint32_t)a.c.pages; };
  const auto read_age = [&](int p, int i) { return a.c.age[number_at(a.c, is_page(p) ? p : 0, h, i)]; };
  const auto read_mass = [&](int p, int i) { return a.c.mass[number_at(a.c, is_page(p) ? p : 0, h, i)]; };
  for (int k = tid; k < 2 * 4 * 256; k += kThreads) (&sh.hist[0][0][0])[k] = 0;
  uint32_t age[kWords] = {}, mass[kWords] = {};
  if constexpr (K == kInRegisters) {  // all reads at once: pages, then masses and ages
    int p[kWords];
    float m[kWords];
    int32_t t[kWords] = {};
    sl.each([&](auto r, int w) { p[r] = raw_page(min(w * 64 + sl.lane, n - 1)); });
    sl.each([&](auto r, int w) {
      const int i = min(w * 64 + sl.lane, n - 1);
      m[r] = read_mass(p[r], i);
      if (by_age) t[r] = read_age(p[r], i);
    });
    sl.each([&](auto r, int) {
      mass[r] = is_page(p[r]) ? mass_key(m[r]) : 0;
      age[r] = is_page(p[r]) ? age_key(t[r]) : 0;
    });
  } else {
    for (int w = tid; w < nw; w += kThreads) sl.keep[w] = 0;
  }
  // into LDS, eight reads of a thread at once
  const auto stage = [&](const auto &read, const auto &key_of) {
    constexpr int kAhead = 8;
    for (int i0 = tid; i0 < n; i0 += kAhead * kThreads) {
      int p[kAhead];
      decltype(read(0, 0)) v[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) p[j] = raw_page(min(i0 + j * kThreads, n - 1));
#pragma unroll
      for (int j = 0; j < kAhead; ++j) v[j] = read(p[j], min(i0 + j * kThreads, n - 1));
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i0 + j * kThreads < n) keys[i0 + j * kThreads] = is_page(p[j]) ? key_of(v[j]) : 0;
    }
    __syncthreads();
  };
  const auto select = [&](int which, int wanted, const uint32_t *own, const auto &read, const auto &key_of) {
    if (wanted <= 0) return;
    if constexpr (K == kInLds) stage(read, key_of);
    take_largest(sl, wanted, [&](auto r, int w) {
      if constexpr (K == kInRegisters) return own[r];
      const int i = w * 64 + sl.lane;
      if constexpr (K == kInLds) return keys[i];
      const int p = raw_page(i);
      return is_page(p) ? key_of(read(p, i)) : 0;
    }, which, count, sh);
  };
  __syncthreads();
  if (by_age) {
    select(0, a.recent, age, read_age, age_key);
  } else if (a.recent > 0) {
    sl.each([&](auto r, int w) {
      const int i = w * 64 + sl.lane;
      sl.take(r, w, i < n && i >= n - a.recent);
    });
    __syncthreads();
  }
  select(1, budget - a.recent, mass, read_mass, mass_key);
  // kept slots before each word
  sl.each([&](auto r, int w) {
    uint64_t m;
    if constexpr (K == kInRegisters) {
      m = __ballot(sl.kept >> r & 1);
      if (sl.lane == 0) sl.keep[w] = m;
    } else {
      m = sl.keep[w];
    }
    if (sl.lane == 0) count[w] = __popcll(m);
  });
  sums_before(count, nw, sh);
  const auto before = [&](int i) { return count[i >> 6] + __popcll(sl.keep[i >> 6] & ((1ull << (i & 63)) - 1)); };
  const int low = before(budget);  // budget < n
  const bool few = budget - low <= kFewMoves && !a.to;
  for (int j = tid; j < budget; j += kThreads) {
    if (sl.keep[j >> 6] >> (j & 63) & 1) {
      from[j] = j;
      continue;
    }
    // the hole's rank among the holes is that of its filler among the kept slots behind
    const int hole = j - before(j), rank = low + hole;
    int lo = budget >> 6, hi = nw - 1;  // the last word with at most `rank` kept slots before it
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (count[mid] <= rank)
        lo = mid;
      else
        hi = mid - 1;
    }
    uint64_t bits = sl.keep[lo];
    for (int k = rank - count[lo]; k > 0; --k) bits &= bits - 1;
    const int src = lo * 64 + __ffsll((unsigned long long)bits) - 1;
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
  const int slots = a.c.most << a.c.shift, words = slots / 64 + 1;
  const int pieces = a.c.d * (dtype == GSI_FP32 ? 4 : 2) / 16, per = 256 / pieces * kMoveRows;
  const int64_t rows = (int64_t)a.c.S * a.c.heads, strips = (a.budget + per - 1) / per;
  if (rows * kThreads > kMostLaunch || rows * strips * 256 > kMostLaunch) return GSI_E_SHAPE;
  const auto lds = ((size_t)words * 12 + 15) / 16 * 16;
  if (slots <= kMostInRegisters)
    select_kernel<kInRegisters><<<(unsigned)rows, kThreads, lds, st>>>(a, words, pieces);
  else if (slots <= kMostInLds)
    select_kernel<kInLds><<<(unsigned)rows, kThreads, lds + (size_t)slots * 4, st>>>(a, words, pieces);
  else
    select_kernel<kInMemory><<<(unsigned)rows, kThreads, lds, st>>>(a, words, pieces);
  if (hipGetLastError() != hipSuccess) return GSI_E_HIP;
  // In place no more move than there are slots behind the budget; select_kernel
  // has made few (and made again they change nothing: nothing is moved from
  // below the budget).
  if (!a.to && (a.budget >= slots || slots - a.budget <= kFewMoves || a.budget <= kFewMoves)) return GSI_OK;
  move_kernel<<<(unsigned)(rows * strips), 256, 0, st>>>(a, (int)strips, div_by(pieces));
  return hipGetLastError() == hipSuccess ? GSI_OK : GSI_E_HIP;
}

}  // namespace gsi
