// Attention of one new token of every sequence over the paged cache on gfx950
// MFMA (gsi_cache_attend).
//
//   attend_kernel : the slots of a sequence and key head (a row) are counted in
//                   units, four steps of 32 slots (bf16; 16 in fp32), one for each
//                   wavefront of a workgroup.  All rows' units, one after the
//                   other, are dealt to as many workgroups as the chip holds at
//                   once in shares of equal cost, from the lengths as they are:
//                   no workgroup is idle however the lengths differ.  A workgroup
//                   takes up to 16 query heads of its rows (a tile); where a key
//                   head has more, a share has a workgroup for each tile.  A
//                   step's keys and values are read once, straight into the
//                   registers that the matrix instructions take them from.  One
//                   pass with the running maximum and sum of the softmax;
//                   wavefronts are joined through LDS.
//   join_kernel   : rows that a share's end cuts, from the workspace.
//   mass_kernel   : the weights added to the mass, from the scores that
//                   attend_kernel has left in the workspace.
//
// The products.  S^T = K Q^T has slots as rows and query heads as columns, so
// accumulator i of a lane belongs to head l % 16, and the rows of K's tiles are
// dealt so that a lane gets the scores of consecutive slots (bf16: 8 (l / 16) +
// 0..7 over two tiles; fp32: 4 (l / 16) + 0..3).  That is just what the lane has
// to hold of P as the operand A of O = P V: no weight changes its lane.  The
// operand B wants, in a lane, the same slots' values of one column; a lane
// therefore loads for these slots a run of consecutive columns, each column's
// values of two slots are packed with one byte permute (bf16; in fp32 they are
// the operand as they are), and instruction j gives column j of every lane's
// run.  No value goes through LDS and no layout of the pool other than rows is
// needed.  With fewer than 16 query heads the other rows of the tile are idle:
// at 16 B a clock and CU from HBM the matrix cores are at 5 % (bf16) or 30 %
// (fp32) of their rate even then.  The workgroups of a share's tiles run on one
// XCD at one time, so that one of them reads from HBM and all from its L2: 64
// sequences of 2000 slots, 8 key heads for 256, 524 MB, 121 us (16 query heads for
// each key head: 103; with the tiles one after the other 190).  Two tiles in one
// workgroup's registers: 64 sequences of 2000 slots, one key head for 32, 39 us, in
// two workgroups 28 then and 25 now.
//
// Bound by HBM where the lengths fill the chip: two sequences of 131071 slots, 8
// heads of 128, 537 MB in 95 us, 5.7 TB/s; 64 of 1 to 4096 slots, 40 heads of 128,
// 700 MB in 143 us with the scores kept, 4.9.  One sequence of 1777 slots of 16
// heads of 256, 29 MB, takes 12 us and 4 for the join: a launch's latency, a
// length's, a page number's, and the keys' and values' own.
//
// Weights are two bf16 numbers, p = hi + lo to 2^-16, multiplied in two
// instructions, so that in bf16 too only the result's own rounding shows.  hi is p
// cut off, and lo what is left, at least 2^-126: where p is not 0 both are above
// it, and a value that is infinite gives the same infinity with both (hi rounded,
// lo may be 0 or below it, and their sum NaN).
#include <algorithm>
#include <type_traits>

#include "gsi_attend_at.h"
#include "gsi_cache.h"

namespace gsi {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// How a launch splits its work, and its workspace.  A workgroup leaves at most
// two rows unfinished: 2 b for one that an earlier workgroup has begun, 2 b + 1
// for one that it begins.
struct Plan {
  int tiles;   // of a key head
  int kept;    // query heads of a tile at most
  int shares;  // workgroups of a tile
  int scores_row;
  float *stats;    // [tiles][2 shares][kept]: maximum (times log2 e) and sum
  float *partial;  // [tiles][2 shares][kept][d], values' sums over that sum
  float *level;    // [S * heads]: log2 of the sum of all weights, infinity for none
  float *scores;   // [S * heads][scores_row], times log2 e
};

template <typename E>
constexpr int kStep = attend_step(sizeof(E));

// The slots [first, n) of a sequence in steps [lo, lo + steps), and in units.
struct Span {
  int n, first, lo, steps, units;
};

template <typename E>
__device__ __forceinline__ Span span_of(const AttendArgs &a, int n) {
  Span r;
  r.n = n;
  r.first = a.window > 0 ? max(0, n - a.window) : 0;
  r.lo = r.first / kStep<E>;
  r.steps = (n + kStep<E> - 1) / kStep<E> - r.lo;
  r.units = max(1, (r.steps + kWaves - 1) / kWaves);  // no slots: a unit that writes zeros
  return r;
}

// A sequence, its length, and the things of those before it.
struct Sequence {
  int s, n, before;
};

// The sequences one after the other, count(n) things each for n slots: all
// things, and where a thing or a sequence is.  By every wavefront; the lengths
// of the first 64 sequences are read once.
template <typename Count>
struct Counted {
  const AttendArgs &a;
  const Count &count;
  int length, first, first_to, sum;

  __device__ __forceinline__ Counted(const AttendArgs &args, const Count &c) : a(args), count(c) {
    const int lane = threadIdx.x & 63, S = a.c.S;
    length = clamped_length(a.c, a.lengths, min(lane, S - 1));
    first = lane < S ? count(length) : 0;
    first_to = sums_to(first);
    int more = 0;
    for (int s = lane + 64; s < S; s += 64) more += count(clamped_length(a.c, a.lengths, s));
    sum = __builtin_amdgcn_readlane(first_to, 63);
    if (S > 64) sum += __builtin_amdgcn_readlane(sums_to(more), 63);
  }
  // the first sequence that `is` holds for, of its number and the things up to and with it
  template <typename Is>
  __device__ __forceinline__ Sequence search(const Is &is) const {
    const int lane = threadIdx.x & 63, S = a.c.S;
    int run = 0;
    for (int s0 = 0; s0 < S; s0 += 64) {
      const int n = s0 == 0 ? length : clamped_length(a.c, a.lengths, min(s0 + lane, S - 1));
      const int mine = s0 == 0 ? first : s0 + lane < S ? count(n) : 0;
      const int incl = s0 == 0 ? first_to : sums_to(mine);
      const uint64_t over = __ballot(is(s0 + lane, run + incl));
      if (over) {
        const int l = __ffsll((unsigned long long)over) - 1;
        return {s0 + l, __builtin_amdgcn_readlane(n, l), run + __builtin_amdgcn_readlane(incl - mine, l)};
      }
      run += __builtin_amdgcn_readlane(incl, 63);
    }
    return {S - 1, 0, run};
  }
  __device__ __forceinline__ Sequence of_thing(int v) const {
    return search([&](int, int to) { return to > v; });
  }
  __device__ __forceinline__ Sequence number(int s) const {
    return search([&](int i, int) { return i == s; });
  }
};

// A quotient of wave-uniform numbers below 2^62, in 32 bits where they are; where
// not, bit by bit: the compiler's own steps for 64 bits are long, and code that is
// jumped over is waited for too.
__device__ __forceinline__ int64_t over(int64_t n, int64_t by) {
  if (__builtin_expect((uint64_t)(n | by) >> 32 == 0, 1))
    // a division's steps are vector instructions: back to scalar registers
    return (int64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)n / (uint32_t)by));
  int64_t q = 0, rest = 0;
#pragma unroll 1
  for (int k = 61; k >= 0; --k) {
    rest = rest * 2 + (n >> k & 1);
    const bool in = rest >= by;
    rest -= in ? by : 0;
    q = q * 2 + in;
  }
  return q;
}

// Where a unit is: a row of a sequence, its length, and the row's units before it.
struct Place {
  int s, kh, n, skip;
  int64_t at;  // the cost before it
};

// The shares of all rows' units.  A unit costs two and a row one, what its first
// loads and its join take (64 ragged sequences of 40 heads, 6 rows of a share in
// the mean: 158 us by units alone, where the shares of many short rows end last,
// 143 so); share b begins with the first unit at or behind b / of of the cost.
// Units are at most three apart: a share is not empty where it has as much; where
// that is not so, units alone are the cost.
template <typename Count>
struct Shares {
  const AttendArgs &a;
  const Counted<Count> &counted;
  int of, unit;  // shares, and a unit's cost
  int64_t all;

  __device__ __forceinline__ Shares(const AttendArgs &args, const Plan &p, const Counted<Count> &c)
      : a(args), counted(c), unit(2) {
    all = (int64_t)cost(c.sum, a.c.S) * a.c.heads;
    if (all < 3 * (int64_t)p.shares) {
      unit = 1;
      all = (int64_t)c.sum * a.c.heads;
    }
    of = (int)min((int64_t)p.shares, all);
  }
  // of a key head's units in so many rows
  __device__ __forceinline__ int cost(int units, int rows) const { return unit * units + (unit - 1) * rows; }
  __device__ __forceinline__ int64_t start_of(const Sequence &q, int kh, int units) const {
    return (int64_t)cost(q.before, q.s) * a.c.heads + (int64_t)cost(units, 1) * kh;
  }
  __device__ __forceinline__ int owner(int64_t at) const { return (int)over((at + 1) * of - 1, all); }
  __device__ __forceinline__ int64_t part(int b) const { return over(b * all, of); }
  __device__ __forceinline__ Place begin(int b) const {
    const int64_t at = part(b);
    const int v = (int)over(at, a.c.heads);
    const Sequence q = counted.search([&](int s, int to) { return cost(to, s + 1) > v; });
    const int units = counted.count(q.n), row = cost(units, 1);
    const int64_t in = at - (int64_t)cost(q.before, q.s) * a.c.heads;
    Place r{q.s, (int)over(in, row), q.n, 0, at};
    const int off = (int)(in - (int64_t)r.kh * row);
    r.skip = (off + unit - 1) >> (unit - 1);
    if (r.skip < units) {
      r.at += unit * r.skip - off;
    } else {  // the next row
      r.at += row - off;
      r.skip = 0;
      if (++r.kh == a.c.heads) {
        r.kh = 0;
        r.n = clamped_length(a.c, a.lengths, ++r.s);
      }
    }
    return r;
  }
};

// The largest (the sum) of a value over the four lanes l % 16 + 16 k.
__device__ __forceinline__ float quads_max(float v) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float quads_sum(float v) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ float exp2_of(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ __forceinline__ float log2_of(float v) { return __builtin_amdgcn_logf(v); }

// Weights are 2^8 at most (see below), and values times their sum over many slots
// may pass the largest number where the result does not.  Values are therefore added
// up with weights times this, which over so many slots sum to less than 1.  (In turn
// products below 2^-126 lose their digits: values of 2^-87 at 2^30 slots.)
__device__ __forceinline__ float down_of(int slots) {
  return __uint_as_float((uint32_t)(127 - 41 + __clz(slots)) << 23);  // 2^-9 / slots, rounded down
}

// Where -inf is the maximum so far nothing has a weight: any finite number does
// for it in the exponent.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }

__device__ __forceinline__ void finish_row(const AttendArgs &a, const Plan &p, int64_t row, float top, float total) {
  const float level = top + log2_of(total);
  if (a.lse) a.lse[row] = total == 0.f ? -INFINITY : level * 0.69314718055994531f;
  if (p.level) p.level[row] = total == 0.f ? INFINITY : level;
}

// KS: the head's size in units of 32, rounded up.
template <typename E, int KS>
__global__ void __launch_bounds__(kThreads, KS <= 2 ? 3 : KS <= 4 ? 2 : 1) attend_kernel(AttendArgs a, Plan p) {
  constexpr bool f32 = sizeof(E) == 4;
  constexpr int es = sizeof(E), step = kStep<E>;
  constexpr int KT = key_tiles(es);        // tiles of keys of a step
  constexpr int CH = key_pieces(es, KS);   // 16-byte pieces of a key that a lane holds
  constexpr int VT = value_slots(es);      // slots whose scores and values a lane holds
  constexpr int NC = value_columns(KS);    // columns of a value that a lane holds
  constexpr int VD = NC * es / 4;          // dwords
  // whether the next segment's first loads go out before the present one is done:
  // for fp32 heads above 96 there are no registers for it
  constexpr bool kAhead = !f32 || KS <= 3;
  constexpr int GC = key_guarded(es, KS);  // pieces from here on may lie behind the key
  // rows of 16-byte pieces, four rows apart on other banks
  __shared__ __attribute__((aligned(16))) float red[kWaves][16][32 * KS + 4];
  __shared__ float red_m[kWaves][16], red_l[kWaves][16];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int quad = lane >> 4, l16 = lane & 15, d = a.c.d;
  // eight shares' first tiles, their second ones ..: workgroups go to the XCDs in turn
  const int eight = blockIdx.x / 8, tile = p.tiles == 1 ? 0 : eight % p.tiles;
  const int share = eight / p.tiles * 8 + blockIdx.x % 8;
  const auto units_of = [&](int n) { return span_of<E>(a, n).units; };
  const Counted counted(a, units_of);
  const Shares sh(a, p, counted);
  if (share >= sh.of) return;

  // A row's part in this share: its units from `skip` on, `mine` of them, and of
  // this wavefront the steps st, st + kWaves, .. below end.
  struct Segment {
    int s, kh, skip, mine, st, end;
    Span sp;
  };
  int64_t left;  // cost of the share behind the present segment
  const auto place = [&](Segment &g) {
    g.mine = (int)min((int64_t)(g.sp.units - g.skip), (left + sh.unit - 1) >> (sh.unit - 1));
    g.st = g.sp.lo + g.skip * kWaves + wave;
    g.end = g.sp.lo + min(g.sp.steps, (g.skip + g.mine) * kWaves);
    left -= sh.unit * g.mine + (g.skip + g.mine == g.sp.units ? sh.unit - 1 : 0);
  };
  Segment seg;
  {
    const Place at = sh.begin(share);
    seg.s = at.s, seg.kh = at.kh, seg.skip = at.skip;
    seg.sp = span_of<E>(a, __builtin_amdgcn_readfirstlane(at.n));
    left = sh.part(share + 1) - at.at;
    place(seg);
  }

  // A lane's keys (and its values) of a step lie in one block of 8 slots, so in one
  // page.  Its first column, and its offsets from the start of the block: the last
  // run of columns ends with the value.  (One page for a whole step, in scalar
  // registers, where pages hold whole steps: 3 % slower to 2 % faster.)
  const int col0 = first_column(KS, d, l16);
  const int kblock = key_block(es, l16), vblock = value_block(es, quad);
  const uint32_t ss = (uint32_t)a.c.slot_stride, pages = a.c.pages;
  const uint32_t ko = key_slot(es, l16) * ss, vo = value_slot(es, quad) * ss + col0 * es;
  const float scale2 = a.scale * 1.4426950408889634f;

  // The page numbers of this lane's keys and values, as the table has them: they
  // are checked where they are used, a step later, so that nothing waits for
  // them here.  Slots before the first and behind the last read those ones' and are
  // masked.
  struct Where {
    uint32_t k, v;
  };
  const auto pages_of = [&](const Segment &g, int st) {
    const int32_t *const table = a.c.table + g.s * a.c.ld;
    const auto page = [&](int t) { return (uint32_t)table[slot_in_use(t, g.sp.first, g.sp.n) >> a.c.shift]; };
    return Where{page(st * step + 8 * kblock), page(st * step + 8 * vblock)};
  };
  const auto start_of = [&](const Segment &g, uint32_t page, int t) {
    return entry_at(a.c, page < pages ? page : 0, g.kh, t);
  };
  u32x4_t q[CH];  // this lane's query head as the operand B of S^T
  u32x4_t k[KT][CH];
  uint32_t v[VT][VD];
  const auto load_q = [&](const Segment &g) {
    const int live = a.group - tile * 16;
    const uint8_t *const at = a.q.p + g.s * a.q.row + (g.kh * a.group + tile * 16 + l16) * a.q.head;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      q[c] = u32x4_t{0, 0, 0, 0};
      if (l16 < live && piece_inside(es, d, c, quad)) q[c] = *reinterpret_cast<const u32x4_t *>(at + 64 * c + 16 * quad);
    }
  };
  // The addresses are formed one after the other: all at once they would take as
  // many registers as what they load.
  const auto here = [](const uint8_t *at) {
    asm volatile("" : "+v"(at));
    return at;
  };
  const auto load_k = [&](const Segment &g, const Where &w, int st) {
    const uint8_t *at = here(a.c.K + start_of(g, w.k, st * step + 8 * kblock));
#pragma unroll
    for (int u = 0; u < KT; ++u) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        k[u][c] = *reinterpret_cast<const u32x4_t *>(at + (ko + piece_at(es, KS, d, c, quad)));
      }
      if (u + 1 < KT) at = here(at + 4 * (uint64_t)ss);
    }
  };
  const auto load_v = [&](const Segment &g, const Where &w, int st) {
    const uint8_t *at = here(a.c.V + start_of(g, w.v, st * step + 8 * vblock));
    struct Run {
      uint32_t w[VD];
    };
#pragma unroll
    for (int e = 0; e < VT; ++e) {
      __builtin_memcpy(v[e], at + vo, sizeof(Run));
      at = here(at + ss);
    }
  };

  Where now{}, next{};
  if (seg.st < seg.end) {
    now = pages_of(seg, seg.st);
    next = pages_of(seg, seg.st + kWaves);
  }
  load_q(seg);
  if (seg.st < seg.end) {
    load_k(seg, now, seg.st);
    load_v(seg, now, seg.st);
  }
  for (;;) {
    // The next segment, whose first loads go out as this one's last are used: while
    // the wavefronts are joined nothing has to be waited for.
    const bool last = left <= 0;
    Segment then = seg;
    Where then_now{}, then_next{};
    if (!last) {  // then this segment ends its row
      if (++then.kh == a.c.heads) {
        then.kh = 0;
        then.sp = span_of<E>(a, __builtin_amdgcn_readfirstlane(clamped_length(a.c, a.lengths, ++then.s)));
      }
      then.skip = 0;
      place(then);
      if (then.st < then.end) {
        then_now = pages_of(then, then.st);
        then_next = pages_of(then, then.st + kWaves);
      }
    }
    const bool ahead = !last && then.st < then.end;
    const bool whole = seg.mine == seg.sp.units;
    const int s = seg.s, live = min(16, a.group - tile * 16);  // query heads of this tile
    const int head0 = seg.kh * a.group + tile * 16;
    const Span &sp = seg.sp;

    f32x4_t acc[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) acc[j] = f32x4_t{0, 0, 0, 0};
    float m = -INFINITY, sum = 0.f;  // of head l16; the sum over this lane's slots
    const float down = down_of(seg.mine * step);
    if (kAhead && seg.st >= seg.end && !last) {  // no step of this wavefront
      load_q(then);
      if (ahead) {
        load_k(then, then_now, then.st);
        load_v(then, then_now, then.st);
      }
    }
    for (int st = seg.st; st < seg.end; st += kWaves) {
      f32x4_t sc[KT];
#pragma unroll
      for (int u = 0; u < KT; ++u) {
        sc[u] = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          if (c >= GC && !piece_inside(es, d, c, quad)) k[u][c] = u32x4_t{0, 0, 0, 0};
          if constexpr (f32) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              sc[u] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k[u][c][i]), __uint_as_float(q[c][i]), sc[u],
                                                           0, 0, 0);
          } else {
            sc[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, k[u][c]),
                                                            __builtin_bit_cast(bf16x8_t, q[c]), sc[u], 0, 0, 0);
          }
        }
      }
      // the next step's keys into the registers that have just been read
      const bool more = st + kWaves < seg.end;
      const Where after = pages_of(seg, st + 2 * kWaves);
      if (more) {
        load_k(seg, next, st + kWaves);
      } else if (kAhead && !last) {
        load_q(then);
        if (ahead) load_k(then, then_now, then.st);
      }
      float w[VT];
#pragma unroll
      for (int i = 0; i < VT; ++i) w[i] = sc[i / 4][i % 4] * scale2;
      const int t0 = st * step;
      // the ends of the sequence and pages that are none: no score, no value
      uint32_t in[VT];
#pragma unroll
      for (int i = 0; i < VT; ++i) {
        const int t = t0 + VT * quad + i;
        in[i] = t >= sp.first && t < sp.n && now.v < pages ? ~0u : 0u;
        w[i] = in[i] ? w[i] : -INFINITY;
      }
      if (p.scores && l16 < live) {
        float *const to = p.scores + ((int64_t)s * a.q.n + head0 + l16) * p.scores_row + t0 + VT * quad;
#pragma unroll
        for (int i = 0; i < VT; i += 4)
          *reinterpret_cast<f32x4_t *>(to + i) = f32x4_t{w[i], w[i + 1], w[i + 2], w[i + 3]};
      }
      // The maximum moves only when a score is 2^8 times it in weight: sums and
      // weights then stay within 2^8 of what they would be, far from any limit,
      // and most steps leave the sums so far as they are.
      float top = w[0];
#pragma unroll
      for (int i = 1; i < VT; ++i) top = fmaxf(top, w[i]);
      if (__any(top > m + 8.f)) {
        const float to = fmaxf(m, quads_max(top)), fade = exp2_of(m - base_of(to));
        m = to;
        sum *= fade;
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __shfl(fade, 4 * quad + i, 64);
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[j][i] *= f[i];
      }
      const float base = base_of(m);
#pragma unroll
      for (int i = 0; i < VT; ++i) {
        w[i] = exp2_of(w[i] - base);
        sum += w[i];
        w[i] *= down;
      }
      if constexpr (f32) {
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int e = 0; e < VT; ++e)
            acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(w[e], __uint_as_float(v[e][j] & in[e]), acc[j], 0, 0, 0);
      } else {
        bf16x8_t hi, lo;
        uint32_t both[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) both[t] = (in[2 * t] & 0xffffu) | (in[2 * t + 1] & 0xffff0000u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float cut = __uint_as_float(__float_as_uint(w[i]) & 0xffff0000u);
          hi[i] = (__bf16)cut;
          lo[i] = (__bf16)__builtin_amdgcn_fmed3f(w[i] - cut, 0x1p-126f, w[i]);
        }
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          u32x4_t o;
#pragma unroll
          for (int t = 0; t < 4; ++t)
            o[t] = __builtin_amdgcn_perm(v[2 * t + 1][j / 2], v[2 * t][j / 2], j & 1 ? 0x07060302u : 0x05040100u) &
                   both[t];
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, __builtin_bit_cast(bf16x8_t, o), acc[j], 0, 0, 0);
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, __builtin_bit_cast(bf16x8_t, o), acc[j], 0, 0, 0);
        }
      }
      if (more)
        load_v(seg, next, st + kWaves);
      else if (kAhead && ahead)
        load_v(then, then_now, then.st);
      now = next;
      next = after;
    }

    // The four wavefronts' sums at their common maximum.  Every wavefront has every
    // head's, in lane l16; a thread then adds four columns of a head.
    sum = quads_sum(sum);
    if (lane < 16) red_m[wave][lane] = m, red_l[wave][lane] = sum;
    __syncthreads();
    float ms[kWaves], ls[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) ms[w] = red_m[w][l16], ls[w] = red_l[w][l16];
    const float top = fmaxf(fmaxf(ms[0], ms[1]), fmaxf(ms[2], ms[3])), base = base_of(top);
    float total = 0.f, f[4];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) total += ls[w] * exp2_of(ms[w] - base);
    const uint64_t none = __ballot(total == 0.f);  // heads without a weight
    // this wavefront's sums are divided before they are added to the others'
    const float share_of = exp2_of(m - base) / (total * down);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __shfl(share_of, 4 * quad + i, 64);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (4 * quad + i >= live) continue;
#pragma unroll
      for (int j = 0; j < NC; j += 2)
        *reinterpret_cast<f32x2_t *>(&red[wave][4 * quad + i][col0 + j]) =
            f32x2_t{acc[j][i] * f[i], acc[j + 1][i] * f[i]};
    }
    __syncthreads();
    const int64_t slot = (2 * ((int64_t)tile * p.shares + share) + (seg.skip == 0)) * p.kept;
    if (wave == 0 && lane < live) {
      if (whole)
        finish_row(a, p, (int64_t)s * a.q.n + head0 + lane, top, total);
      else
        *reinterpret_cast<f32x2_t *>(p.stats + 2 * (slot + lane)) = f32x2_t{top, total};
    }
    constexpr int W = KS == 3 ? 32 : KS == 6 ? 64 : 8 * KS;  // threads of a head
    const int c = 4 * (threadIdx.x % W);
    for (int h0 = 0; h0 < live; h0 += kThreads / W) {
      const int h = h0 + threadIdx.x / W;
      if (h >= live || c >= d) continue;
      f32x4_t o = *reinterpret_cast<const f32x4_t *>(&red[0][h][c]);
#pragma unroll
      for (int w = 1; w < kWaves; ++w) o += *reinterpret_cast<const f32x4_t *>(&red[w][h][c]);
      if (none >> h & 1) o = f32x4_t{0, 0, 0, 0};
      if (whole) {
        typedef E out_t __attribute__((ext_vector_type(4)));
        out_t r;
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = (E)o[e];
        *reinterpret_cast<out_t *>(a.out.p + s * a.out.row + (head0 + h) * a.out.head + c * es) = r;
      } else {
        *reinterpret_cast<f32x4_t *>(p.partial + (slot + h) * d + c) = o;
      }
    }
    if (last) return;
    seg = then;
    now = then_now, next = then_next;
    if (!kAhead) {
      load_q(seg);
      if (ahead) {
        load_k(seg, now, seg.st);
        load_v(seg, now, seg.st);
      }
    }
    __syncthreads();  // the sums have been read
  }
}

// A maximum and the sum of weights at it.
struct Stat {
  float m, l;
};

// Query heads that a workgroup of join_kernel takes: four columns a thread.
inline __host__ __device__ int heads_at_once(int d) { return max(1, 4 * kThreads / d); }

// Joins the rows that are cut.  By `cuts`, `sets` workgroups for each tile and share's
// end join the row that this end cuts, if no earlier one cuts it, heads_at_once()
// query heads each; otherwise a workgroup takes a query head of a sequence.
// All latency: the lengths, and then all pieces' statistics and sums at once.
// (A first round for the statistics and second ones for eight pieces at a time
// took 5 us more for 65 pieces; 1024 threads, which take all pieces in one round,
// lose 3 us to their sums in LDS, and in many workgroups 10 us to their start.)
template <typename E>
__global__ void __launch_bounds__(kThreads) join_kernel(AttendArgs a, Plan p, bool cuts, int sets) {
  __shared__ __attribute__((aligned(16))) float red[kThreads * 4];
  __shared__ float red_m[kThreads], red_l[kThreads];
  const int tid = threadIdx.x, d = a.c.d;
  const auto units_of = [&](int n) { return span_of<E>(a, n).units; };
  const Counted counted(a, units_of);
  const Shares sh(a, p, counted);
  int64_t start;
  int s, first, units, kh, tile, in_tile, live;
  if (cuts) {
    const int set = blockIdx.x % sets, most = heads_at_once(d), share = blockIdx.x / sets % (p.shares - 1) + 1;
    tile = blockIdx.x / sets / (p.shares - 1);
    if (share >= sh.of) return;
    const Place cut = sh.begin(share);
    if (cut.skip == 0) return;
    s = cut.s, kh = cut.kh;
    units = units_of(cut.n);
    start = cut.at - sh.unit * cut.skip;
    first = sh.owner(start);
    if (share != first + 1) return;
    in_tile = set * most;
    live = min(min(16, a.group - tile * 16) - in_tile, most);
    if (live <= 0) return;
  } else {
    s = blockIdx.x / a.q.n;
    const int h = blockIdx.x - s * a.q.n;
    kh = h / a.group, tile = (h - kh * a.group) / 16, in_tile = (h - kh * a.group) % 16, live = 1;
    const Sequence at = counted.number(s);
    units = units_of(at.n);
    start = sh.start_of(at, kh, units);
    first = sh.owner(start);
  }
  const int pieces = sh.owner(start + (int64_t)sh.unit * (units - 1)) - first + 1;
  if (pieces <= 1) return;
  const int head0 = kh * a.group + tile * 16 + in_tile;
  // `sides` threads share four columns of a head, each takes every sides-th piece
  const float down = down_of(units * kWaves * kStep<E>);
  const int items = live * d / 4, sides = kThreads / items, side = tid / items, item = tid - side * items;
  const int h = 4 * item / d, c = 4 * item - h * d;
  if (side < sides) {
    constexpr int kAhead = 12;
    f32x4_t o = {0, 0, 0, 0};
    Stat all{-INFINITY, 0.f};
    for (int at0 = 0; at0 < pieces; at0 += kAhead * sides) {
      const int i0 = at0 + side;
      f32x4_t u[kAhead] = {};
      Stat t[kAhead] = {};
      float top = all.m;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (at0 + k * sides >= pieces) continue;  // of every side
        const int i = min(i0 + k * sides, pieces - 1);
        const int64_t at = (2 * ((int64_t)tile * p.shares + first + i) + (i == 0)) * p.kept + in_tile + h;
        u[k] = *reinterpret_cast<const f32x4_t *>(p.partial + at * d + c);
        t[k] = *reinterpret_cast<const Stat *>(p.stats + 2 * at);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (i0 + k * sides < pieces) top = fmaxf(top, t[k].m);
      const float base = base_of(top), fade = exp2_of(all.m - base);
      all = {top, all.l * fade};
      o *= fade;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (i0 + k * sides >= pieces) continue;
        const float f = t[k].l * exp2_of(t[k].m - base);
        all.l += f;
        o += u[k] * (f * down);
      }
    }
    *reinterpret_cast<f32x4_t *>(red + 4 * tid) = o;
    red_m[tid] = all.m, red_l[tid] = all.l;
  }
  __syncthreads();
  if (side != 0) return;
  float top = red_m[item], total = 0.f;
  for (int w = 1; w < sides; ++w) top = fmaxf(top, red_m[w * items + item]);
  f32x4_t v = {0, 0, 0, 0};
  for (int w = 0; w < sides; ++w) {
    const float f = exp2_of(red_m[w * items + item] - base_of(top));
    total += red_l[w * items + item] * f;
    v += *reinterpret_cast<const f32x4_t *>(red + 4 * (w * items + item)) * f;
  }
  if (c == 0) finish_row(a, p, (int64_t)s * a.q.n + head0 + h, top, total);
  E *const out = reinterpret_cast<E *>(a.out.p + s * a.out.row + (head0 + h) * a.out.head) + c;
#pragma unroll
  for (int k = 0; k < 4; ++k) out[k] = (E)(total == 0.f ? 0.f : v[k] / (total * down));
}

constexpr int kMassSlots = 256;  // of a strip
constexpr int kMassGrid = 2048;

// The strips of kMassSlots slots of all sequences and key heads, four slots a
// lane, which lie in one page.  `sharers` wavefronts (1 or 4) divide a strip's
// query heads.  Bound by latency: lengths, pages, then masses and scores.  64
// ragged sequences of 40 heads: 9.7 us, 24 of 2 key heads of 32 query heads 4.1 us.
// (A strip for a whole workgroup, one slot a thread: 14.5 and 4.0 us.)
__global__ void __launch_bounds__(kThreads) mass_kernel(AttendArgs a, Plan p, int sharers) {
  __shared__ __attribute__((aligned(16))) float sums[kWaves][kMassSlots];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int own = wave & (sharers - 1), at_once = kWaves / sharers;
  const auto first_of = [&](int n) { return a.window > 0 ? max(0, n - a.window) : 0; };
  const auto strips = [&](int n) { return (n + kMassSlots - 1) / kMassSlots - first_of(n) / kMassSlots; };
  const Counted counted(a, strips);
  const int64_t all = (int64_t)counted.sum * a.c.heads;
  for (int64_t at0 = (int64_t)blockIdx.x * at_once; at0 < all; at0 += (int64_t)gridDim.x * at_once) {
    const int64_t at = at0 + wave / sharers;
    const bool has = at < all;
    const Sequence seq = counted.of_thing((int)over(has ? at : 0, a.c.heads));
    const int s = seq.s, n = seq.n, first = first_of(n);
    const int in = (int)((has ? at : 0) - (int64_t)seq.before * a.c.heads), of = strips(n);
    const int kh = (int)over(in, of), strip = in - kh * of;
    const int i = (first / kMassSlots + strip) * kMassSlots + 4 * lane;
    const int64_t row0 = (int64_t)s * a.q.n + kh * a.group;
    const int page = page_of(a.c, s, slot_in_use(i, first, n));
    float *const number = a.c.mass + number_at(a.c, max(page, 0), kh, i);
    f32x4_t mass = {0, 0, 0, 0}, add = {0, 0, 0, 0};
    if (own == 0) __builtin_memcpy(&mass, number, 16);
    const float *const score = p.scores + row0 * p.scores_row + min(i, p.scores_row - 4);
    for (int h0 = own; h0 < a.group; h0 += 8 * sharers) {
      f32x4_t u[8];
      float level[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int h = min(h0 + j * sharers, a.group - 1);
        level[j] = p.level[row0 + h];
        u[j] = *reinterpret_cast<const f32x4_t *>(score + (int64_t)h * p.scores_row);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) add[e] += h0 + j * sharers < a.group ? exp2_of(u[j][e] - level[j]) : 0.f;
    }
    if (sharers > 1) {
      *reinterpret_cast<f32x4_t *>(&sums[wave][4 * lane]) = add;
      __syncthreads();
      if (own == 0)
        for (int w = 1; w < sharers; ++w) add += *reinterpret_cast<const f32x4_t *>(&sums[wave + w][4 * lane]);
      __syncthreads();
    }
    if (own != 0 || !has || page < 0) continue;
    mass += add;  // rounded once
    if (i >= first && i + 4 <= n) {
      __builtin_memcpy(number, &mass, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e >= first && i + e < n) number[e] = mass[e];
    }
  }
}

// Workgroups that the chip holds at once, by the registers of the kernel.  With 1, 2,
// 3 and 4 for each CU, us: 64 ragged sequences of 40 heads of 128 201, 163, 181, 165; of
// 8 heads of 64 34, 28, 27, 31; 16 of 4000 slots of 8 heads of 64 35, 30, 31, 34, of 256
// 101, 105, 113.
inline int shares_for(int d) { return 256 * (d <= 64 ? 3 : d <= 128 ? 2 : 1); }

template <typename E>
Plan plan_of(const Pool &c, int q_heads, bool accumulate, uint8_t *ws, size_t *bytes) {
  Plan p{};
  const int64_t slots = (int64_t)c.most << c.shift;
  const int64_t units = std::max<int64_t>(1, (slots + kWaves * kStep<E> - 1) / (kWaves * kStep<E>));
  p.tiles = (q_heads / c.heads + 15) / 16;
  p.kept = std::min(q_heads / c.heads, 16);
  // of each tile as many on every XCD, or some would wait for a place
  const int shares = std::max(8, shares_for(c.d) / p.tiles / 8 * 8);
  p.shares = (int)std::min<int64_t>(shares, c.S * units * c.heads);
  p.scores_row = (int)((slots + 31) / 32 * 32);
  size_t at = 0;
  const auto take = [&](size_t floats) {
    float *const r = ws ? reinterpret_cast<float *>(ws + at) : nullptr;
    at += (floats * 4 + 15) / 16 * 16;
    return r;
  };
  if (units > 1) {
    p.stats = take((size_t)p.tiles * p.shares * 2 * p.kept * 2);
    p.partial = take((size_t)p.tiles * p.shares * 2 * p.kept * c.d);
  }
  if (accumulate) {
    p.level = take((size_t)c.S * q_heads);
    p.scores = take((size_t)c.S * q_heads * p.scores_row);
  }
  if (bytes) *bytes = at;
  return p;
}

template <typename E>
gsi_status launch_as(const AttendArgs &a, hipStream_t st) {
  const Plan p = plan_of<E>(a.c, a.q.n, a.accumulate, a.ws, nullptr);
  const unsigned grid = (p.shares + 7) / 8 * 8 * p.tiles;
  const auto go = [&](auto ks) {
    attend_kernel<E, decltype(ks)::value><<<grid, kThreads, 0, st>>>(a, p);
  };
  const int ks = attend_ks(a.c.d);
  if (ks == 1)
    go(std::integral_constant<int, 1>{});
  else if (ks == 2)
    go(std::integral_constant<int, 2>{});
  else if (ks == 3)
    go(std::integral_constant<int, 3>{});
  else if (ks == 4)
    go(std::integral_constant<int, 4>{});
  else if (ks == 6)
    go(std::integral_constant<int, 6>{});
  else
    go(std::integral_constant<int, 8>{});
  if (hipGetLastError() != hipSuccess) return GSI_E_HIP;
  if (p.stats && p.shares > 1) {
    const int most = heads_at_once(a.c.d), sets = (p.kept + most - 1) / most;
    const int64_t by_cuts = (int64_t)(p.shares - 1) * p.tiles * sets, by_heads = (int64_t)a.c.S * a.q.n;
    // A query head for each workgroup has more threads for many pieces, as long as
    // they run at once.  By heads and by cuts, us: 2000 slots of 2 key heads for 64, 4
    // sequences (256 heads) 12.3 and 13.9, 24 (1536) 17.8 and 16.9, 64 (4096) 29.1 and
    // 22.4; 1 to 8000 slots, 16 (1024) 22.5 and 27.4, 32 (2048) 25.7 both; 2000 slots of 8
    // key heads for 32, 24 (768) 20.1 and 20.2, 64 (2048) 28.1 and 24.7.
    const bool cuts = by_heads > 1536 && by_cuts < by_heads;
    join_kernel<E><<<(unsigned)(cuts ? by_cuts : by_heads), kThreads, 0, st>>>(a, p, cuts, sets);
    if (hipGetLastError() != hipSuccess) return GSI_E_HIP;
  }
  if (a.accumulate && a.c.most > 0) {
    const int64_t strips = (((int64_t)a.c.most << a.c.shift) + kMassSlots - 1) / kMassSlots * a.c.S * a.c.heads;
    // A wavefront alone where its heads' scores are one round of loads: with four
    // for a strip 64 sequences of 2000 slots, 8 key heads for 64, take 1.3 us more;
    // 24 sequences of 2 key heads of 32 take 2.3 us less.
    const int sharers = a.group > 8 ? 4 : 1, at_once = kWaves / sharers;
    const int64_t grid = std::min<int64_t>((strips + at_once - 1) / at_once, kMassGrid);
    mass_kernel<<<(unsigned)grid, kThreads, 0, st>>>(a, p, sharers);
    if (hipGetLastError() != hipSuccess) return GSI_E_HIP;
  }
  return GSI_OK;
}

}  // namespace

// Units of 64 slots or more, one of a sequence at least, cost two, and a row one: that
// of a key head is counted in 32 bits.
bool attend_counts(const Pool &c) { return (((int64_t)c.most << c.shift) / 32 + 3) * c.S <= INT32_MAX; }

size_t attend_workspace(const Pool &c, int dtype, int q_heads, bool accumulate) {
  size_t bytes = 0;
  if (dtype == GSI_FP32)
    plan_of<float>(c, q_heads, accumulate, nullptr, &bytes);
  else
    plan_of<__bf16>(c, q_heads, accumulate, nullptr, &bytes);
  return bytes;
}

gsi_status launch_attend(const AttendArgs &a, int dtype, hipStream_t st) {
  return dtype == GSI_FP32 ? launch_as<float>(a, st) : launch_as<__bf16>(a, st);
}

}  // namespace gsi
