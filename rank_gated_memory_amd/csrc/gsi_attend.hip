// Attention of one new token of every sequence over the paged cache on gfx950
// MFMA (gsi_cache_attend).
//
//   attend_kernel : the slots of a sequence and key head are cut into pieces, a
//                   workgroup each; its four wavefronts take the piece's steps
//                   of 32 slots (bf16; 16 in fp32) in turn.  A step's keys and
//                   values are read once, straight into the registers that the
//                   matrix instructions take them from, for up to 16 query
//                   heads of the key head.  One pass with the running maximum
//                   and sum of the softmax; the wavefronts are joined through
//                   LDS, pieces through the workspace.
//   join_kernel   : the pieces of a row, and the weights added to the mass from
//                   the scores that attend_kernel has left in the workspace.
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
// (fp32) of their rate even then.
//
// Weights are rounded to bf16 twice, p = hi + lo to 2^-17, and multiplied in two
// instructions, so that in bf16 too only the result's own rounding shows.
#include <algorithm>
#include <type_traits>

#include "gsi_cache.h"

namespace gsi {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMostPieces = 256;

// How a launch splits its work, and its workspace.
struct Plan {
  int pieces;   // of a row at most
  int least;    // steps of a piece at least
  int tiles;    // of 16 query heads of a key head
  int row;      // scores of a row
  float *stats;    // [S * heads][pieces]: maximum (times log2 e) and sum
  float *partial;  // [S * heads][pieces][d], sums at that maximum
  float *scores;   // [S * heads][row], times log2 e
};

template <typename E>
constexpr int kStep = sizeof(E) == 2 ? 32 : 16;

// The steps of a sequence and its pieces.
struct Span {
  int n, first, lo, steps, per, pieces;  // slots [first, n); steps [lo, lo + steps), `per` a piece
};

template <typename E>
__device__ __forceinline__ Span span_of(const AttendArgs &a, const Plan &p, int s) {
  Span r;
  r.n = clamped_length(a.c, a.lengths, s);
  r.first = a.window > 0 ? max(0, r.n - a.window) : 0;
  r.lo = r.first / kStep<E>;
  r.steps = (r.n + kStep<E> - 1) / kStep<E> - r.lo;
  r.per = max(p.least, (r.steps + p.pieces - 1) / p.pieces);
  r.pieces = (r.steps + r.per - 1) / r.per;
  return r;
}

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

// Where -inf is the maximum so far nothing has a weight: any finite number does
// for it in the exponent.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }

// KS: the head's size in units of 32, rounded up.  Uniform: a page holds whole
// steps, so that a step has one page; otherwise each 8 slots have one.
template <typename E, int KS, bool Uniform>
__global__ void __launch_bounds__(kThreads, KS <= 4 ? 2 : 1) attend_kernel(AttendArgs a, Plan p) {
  constexpr bool f32 = sizeof(E) == 4;
  constexpr int es = sizeof(E), step = kStep<E>;
  constexpr int KT = f32 ? 1 : 2;          // tiles of keys of a step
  constexpr int CH = f32 ? 2 * KS : KS;    // 16-byte pieces of a key that a lane holds
  constexpr int CE = f32 ? 16 : 32;        // elements of a key in piece c of the four lanes
  constexpr int VT = f32 ? 4 : 8;          // slots whose scores and values a lane holds
  constexpr int NC = 2 * KS;               // columns of a value that a lane holds
  constexpr int VD = NC * es / 4;          // dwords
  constexpr int GC = CH - (f32 ? 2 : 1) * (KS > 4 ? 2 : 1);  // pieces from here on may lie behind the key
  __shared__ float red[kWaves][16][32 * KS];
  __shared__ float red_m[kWaves][16], red_l[kWaves][16];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int quad = lane >> 4, l16 = lane & 15, d = a.c.d;
  int b = blockIdx.x;
  const int piece = b % p.pieces;
  b /= p.pieces;
  const int tile = b % p.tiles;
  b /= p.tiles;
  const int kh = b % a.c.heads, s = b / a.c.heads;
  const Span sp = span_of<E>(a, p, s);
  const int live = min(16, a.group - tile * 16);  // query heads of this tile
  const int head0 = kh * a.group + tile * 16;
  if (piece >= sp.pieces && !(piece == 0 && sp.pieces == 0)) return;

  // this lane's query head as the operand B of S^T
  u32x4_t q[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e = c * CE + 16 / es * quad;
    q[c] = u32x4_t{0, 0, 0, 0};
    if (l16 < live && e < d)
      q[c] = *reinterpret_cast<const u32x4_t *>(a.q.p + s * a.q.row + (head0 + l16) * a.q.head + e * es);
  }

  // this lane's first column, and its offsets from the start of a step (of a
  // block of 8 slots): the last run of columns ends with the value
  const int col0 = min(l16 * NC, d - NC);
  const int ktoken = f32 ? (Uniform ? l16 : l16 & 7) : (Uniform ? 8 * (l16 >> 2) : 0) + (l16 & 3);
  const int vtoken = f32 ? (Uniform ? 4 * quad : 4 * (quad & 1)) : (Uniform ? 8 * quad : 0);
  const int kblock = f32 ? l16 >> 3 : l16 >> 2, vblock = f32 ? quad >> 1 : quad;
  const uint32_t ss = (uint32_t)a.c.slot_stride;
  const uint32_t ko = ktoken * ss + 16 * quad, vo = vtoken * ss + col0 * es;
  const int32_t *const table = a.c.table + s * a.c.ld;

  struct Where {
    int k, v;  // pages of this lane's keys and values, -1 for none
  };
  const auto pages_of = [&](int st) {
    const auto page = [&](int t) {
      if (t >= sp.n) return -1;
      const int g = table[t >> a.c.shift];
      return (uint32_t)g < (uint32_t)a.c.pages ? g : -1;
    };
    Where w;
    if constexpr (Uniform) {
      w.k = w.v = __builtin_amdgcn_readfirstlane(page(st * step));
    } else {
      w.k = page(st * step + 8 * kblock);
      w.v = page(st * step + 8 * vblock);
    }
    return w;
  };
  u32x4_t k[KT][CH];
  uint32_t v[VT][VD];
  const auto load_k = [&](const Where &w, int st) {
    const uint8_t *const at = a.c.K + entry_at(a.c, max(w.k, 0), kh, st * step + (Uniform ? 0 : 8 * kblock));
#pragma unroll
    for (int u = 0; u < KT; ++u)
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const uint32_t in = c < GC || c * CE + 16 / es * quad < d ? c * 64 : 0;
        k[u][c] = *reinterpret_cast<const u32x4_t *>(at + 4 * u * (uint64_t)ss + (ko + in));
      }
  };
  const auto load_v = [&](const Where &w, int st) {
    const uint8_t *const at = a.c.V + entry_at(a.c, max(w.v, 0), kh, st * step + (Uniform ? 0 : 8 * vblock));
    struct Run {
      uint32_t w[VD];
    };
#pragma unroll
    for (int e = 0; e < VT; ++e) __builtin_memcpy(v[e], at + e * (uint64_t)ss + vo, sizeof(Run));
  };

  const float scale2 = a.scale * 1.4426950408889634f;
  f32x4_t acc[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) acc[j] = f32x4_t{0, 0, 0, 0};
  float m = -INFINITY, sum = 0.f;  // of head l16; the sum over this lane's slots
  const int end = sp.lo + min(sp.steps, (piece + 1) * sp.per);
  int st = sp.lo + piece * sp.per + wave;
  Where now = pages_of(st < end ? st : 0), next = now;
  if (st < end) {
    load_k(now, st);
    load_v(now, st);
    if (st + kWaves < end) next = pages_of(st + kWaves);
  }
  for (; st < end; st += kWaves) {
    f32x4_t sc[KT];
#pragma unroll
    for (int u = 0; u < KT; ++u) {
      sc[u] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (c >= GC && c * CE + 16 / es * quad >= d) k[u][c] = u32x4_t{0, 0, 0, 0};
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
    const bool more = st + kWaves < end;
    Where after = next;
    if (more) {
      load_k(next, st + kWaves);
      if (st + 2 * kWaves < end) after = pages_of(st + 2 * kWaves);
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
      in[i] = t >= sp.first && t < sp.n && now.v >= 0 ? ~0u : 0u;
      w[i] = in[i] ? w[i] : -INFINITY;
    }
    if (p.scores && l16 < live) {
      float *const to = p.scores + ((int64_t)s * a.q.n + head0 + l16) * p.row + t0 + VT * quad;
#pragma unroll
      for (int i = 0; i < VT; i += 4) *reinterpret_cast<f32x4_t *>(to + i) = f32x4_t{w[i], w[i + 1], w[i + 2], w[i + 3]};
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
        hi[i] = (__bf16)w[i];
        lo[i] = (__bf16)(w[i] - (float)hi[i]);
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
    if (more) load_v(next, st + kWaves);
    now = next;
    next = after;
  }

  // the four wavefronts' sums at their common maximum
  sum = quads_sum(sum);
  if (lane < 16) red_m[wave][lane] = m, red_l[wave][lane] = sum;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int h = 4 * quad + i;
    float top = red_m[0][h];
    for (int w = 1; w < kWaves; ++w) top = fmaxf(top, red_m[w][h]);
    const float f = exp2_of(red_m[wave][h] - base_of(top));
    if (h < live)
#pragma unroll
      for (int j = 0; j < NC; ++j) red[wave][h][col0 + j] = acc[j][i] * f;
  }
  __syncthreads();
  const bool whole = sp.pieces <= 1;
  for (int h = wave; h < live; h += kWaves) {
    float top = red_m[0][h], total = 0.f;
    for (int w = 1; w < kWaves; ++w) top = fmaxf(top, red_m[w][h]);
    for (int w = 0; w < kWaves; ++w) total += red_l[w][h] * exp2_of(red_m[w][h] - base_of(top));
    const int64_t row = (int64_t)s * a.q.n + head0 + h, at = row * p.pieces + piece;
    if (lane == 0) {
      if (p.stats) p.stats[2 * at] = top, p.stats[2 * at + 1] = total;
      if (whole && a.lse) a.lse[row] = total == 0.f ? -INFINITY : (top + log2_of(total)) * 0.69314718055994531f;
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    for (int c = lane; c < d; c += 64) {
      float o = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) o += red[w][h][c];
      if (whole)
        reinterpret_cast<E *>(a.out.p + s * a.out.row + (head0 + h) * a.out.head)[c] = (E)(total == 0.f ? 0.f : o * inv);
      else
        p.partial[at * d + c] = o;
    }
  }
}

// log2 of the sum of a row's weights, from its pieces' statistics; by a wavefront.
__device__ __forceinline__ float joined(const float *stats, int pieces, float *top_out) {
  const int lane = threadIdx.x & 63;
  float top = -INFINITY, total = 0.f;
  for (int i = lane; i < pieces; i += 64) top = fmaxf(top, stats[2 * i]);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
  for (int i = lane; i < pieces; i += 64) total += stats[2 * i + 1] * exp2_of(stats[2 * i] - base_of(top));
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o, 64);
  *top_out = top;
  return total;
}

constexpr int kMassSlots = 1024;  // of a workgroup

// Workgroups below `rows` join a row each, those behind add the weights of
// kMassSlots slots of a sequence and key head.
template <typename E>
__global__ void __launch_bounds__(kThreads) join_kernel(AttendArgs a, Plan p, int rows, int strips) {
  __shared__ float red[kWaves][256];
  __shared__ float level[4096];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, d = a.c.d;
  if ((int)blockIdx.x < rows) {
    const int row = blockIdx.x, s = row / a.q.n, h = row - s * a.q.n;
    const Span sp = span_of<E>(a, p, s);
    if (sp.pieces <= 1) return;
    const float *const stats = p.stats + (int64_t)row * p.pieces * 2;
    float top;
    const float total = joined(stats, sp.pieces, &top), base = base_of(top);
    float o[4] = {};
    if (4 * lane < d) {
      for (int i = wave; i < sp.pieces; i += kWaves) {
        const float f = exp2_of(stats[2 * i] - base);
        const f32x4_t u = *reinterpret_cast<const f32x4_t *>(p.partial + ((int64_t)row * p.pieces + i) * d + 4 * lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] += u[j] * f;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) red[wave][4 * lane + j] = o[j];
    }
    __syncthreads();
    if ((int)threadIdx.x < d) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += red[w][threadIdx.x];
      reinterpret_cast<E *>(a.out.p + s * a.out.row + h * a.out.head)[threadIdx.x] = (E)(total == 0.f ? 0.f : v / total);
    }
    if (threadIdx.x == 0 && a.lse)
      a.lse[row] = total == 0.f ? -INFINITY : (top + log2_of(total)) * 0.69314718055994531f;
    return;
  }
  const int b = blockIdx.x - rows, strip = b % strips, kh = b / strips % a.c.heads, s = b / strips / a.c.heads;
  const Span sp = span_of<E>(a, p, s);
  const int lo = max(sp.first, strip * kMassSlots), hi = min(sp.n, (strip + 1) * kMassSlots);
  if (lo >= hi) return;
  const int64_t row0 = (int64_t)s * a.q.n + kh * a.group;
  for (int h = wave; h < a.group; h += kWaves) {
    float top;
    const float total = joined(p.stats + (row0 + h) * p.pieces * 2, sp.pieces, &top);
    if (lane == 0) level[h] = total == 0.f ? INFINITY : top + log2_of(total);
  }
  __syncthreads();
  for (int i = lo + threadIdx.x; i < hi; i += kThreads) {
    const int page = page_of(a.c, s, i);
    if (page < 0) continue;
    float add = 0.f;
    for (int h = 0; h < a.group; ++h) add += exp2_of(p.scores[(row0 + h) * p.row + i] - level[h]);
    a.c.mass[number_at(a.c, page, kh, i)] += add;
  }
}

template <typename E>
Plan plan_of(const Pool &c, int q_heads, bool accumulate, uint8_t *ws, size_t *bytes) {
  Plan p{};
  const int64_t slots = (int64_t)c.most << c.shift, steps = (slots + kStep<E> - 1) / kStep<E>;
  p.tiles = (q_heads / c.heads + 15) / 16;
  const int64_t rows = std::max<int64_t>(1, (int64_t)c.S * c.heads * p.tiles);
  // Pieces enough that the chip has four rounds of workgroups, two to a CU, of
  // at least 128 slots; where rows alone do, of 1024 slots, so that no long
  // sequence is left at the end.
  int64_t want = 1024 / rows, least = kWaves;
  const int64_t longest = 1024 / kStep<E>;
  want = std::max<int64_t>(want, (steps + longest - 1) / longest);
  if (rows >= 1024) least = longest;
  want = std::min<int64_t>({want, kMostPieces, (steps + least - 1) / least});
  p.pieces = (int)std::max<int64_t>(1, want);
  p.least = (int)least;
  p.row = (int)((slots + 31) / 32 * 32);
  const size_t all = (size_t)c.S * q_heads;
  size_t at = 0;
  const auto take = [&](size_t floats) {
    float *const r = ws ? reinterpret_cast<float *>(ws + at) : nullptr;
    at += (floats * 4 + 15) / 16 * 16;
    return r;
  };
  if (p.pieces > 1 || accumulate) p.stats = take(all * p.pieces * 2);
  if (p.pieces > 1) p.partial = take(all * p.pieces * c.d);
  if (accumulate) p.scores = take(all * p.row);
  if (bytes) *bytes = at;
  return p;
}

template <typename E>
gsi_status launch_as(const AttendArgs &a, hipStream_t st) {
  const Plan p = plan_of<E>(a.c, a.q.n, a.accumulate, a.ws, nullptr);
  const int64_t grid = (int64_t)a.c.S * a.c.heads * p.tiles * p.pieces;
  const int64_t rows = p.pieces > 1 ? (int64_t)a.c.S * a.q.n : 0;
  const int64_t strips = ((int64_t)a.c.most << a.c.shift) / kMassSlots + 1;
  const int64_t second = rows + (a.accumulate ? (int64_t)a.c.S * a.c.heads * strips : 0);
  if (grid * kThreads > kMostLaunch || second * kThreads > kMostLaunch) return GSI_E_SHAPE;
  const bool uniform = 1 << a.c.shift >= kStep<E>;
  const auto go = [&](auto ks) {
    constexpr int KS = decltype(ks)::value;
    if (uniform)
      attend_kernel<E, KS, true><<<(unsigned)grid, kThreads, 0, st>>>(a, p);
    else
      attend_kernel<E, KS, false><<<(unsigned)grid, kThreads, 0, st>>>(a, p);
  };
  const int ks = (a.c.d + 31) / 32;
  if (ks == 1)
    go(std::integral_constant<int, 1>{});
  else if (ks == 2)
    go(std::integral_constant<int, 2>{});
  else if (ks == 3)
    go(std::integral_constant<int, 3>{});
  else if (ks == 4)
    go(std::integral_constant<int, 4>{});
  else if (ks <= 6)
    go(std::integral_constant<int, 6>{});
  else
    go(std::integral_constant<int, 8>{});
  if (hipGetLastError() != hipSuccess) return GSI_E_HIP;
  if (second == 0) return GSI_OK;
  join_kernel<E><<<(unsigned)second, kThreads, 0, st>>>(a, p, (int)rows, (int)strips);
  return hipGetLastError() == hipSuccess ? GSI_OK : GSI_E_HIP;
}

}  // namespace

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
