// Plain linear maps on gfx950 MFMA: weights in 4 bits and weights of many
// experts (gsi_q4_linear, gsi_grouped_linear).
//
// Both entry points are one product, y[r] = W_e(r) x[src(r)], with the rows
// of y ordered by expert; gsi_q4_linear has one expert and every row.
//
//   stream_kernel : every output row block of 16 (times RB) weight rows
//                   reads its weights once per chunk of 16 * TB tokens.
//
// 4-bit weights.  With w = s (q - z) a group's share of y is
//   s (sum q x - z sum x) = s (sum (16 + q) x - (16 + z) sum x).
// 16 + q is the bf16 0x4180 | q << 3, so two codes decode with one shift and
// one and-or, exactly, and the matrix core multiplies them with bf16 x
// exactly; sum x of the group comes from the same instruction with ones for
// weights.  fp32 x is split into three bf16 parts (8 + 8 + 8 bits, exact),
// each its own product.  Only the group's fp32 sums are rounded.
//
// MFMA operand layouts as in gsi_batched.hip: for 16x16x32, lane l holds
// A[l % 16][8 (l / 16) + e], B[8 (l / 16) + e][l % 16] and accumulator i is
// C[4 (l / 16) + i][l % 16]; for the fp32 16x16x4, A[l % 16][l / 16] and
// B[l / 16][l % 16].  A holds tokens and B weight rows, so that a lane's
// accumulators all belong to one weight row and take one scale.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "../../include/gsi.h"

namespace gsi {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

struct MArgs {
  const uint8_t *W;
  const uint8_t *scales;
  const uint8_t *zeros;  // null: 8
  const uint8_t *x;
  uint8_t *y;
  const int32_t *offsets;  // null: one expert, rows [0, R)
  const int32_t *rows;     // null: row r reads x row r
  int64_t w_stride;        // bytes between maps
  int64_t ldx, ldy;        // elements
  int32_t d, d_out, n, R, T;
  int32_t groups;          // scale groups of a row
};

enum Kind { kQ4Bf16, kQ4F32, kBf16, kF32 };

__device__ __forceinline__ bf16x8_t as_bf16x8(u32x4_t u) { return __builtin_bit_cast(bf16x8_t, u); }

// The chunk of rows that slot `s` of a launch computes: experts in order,
// each in chunks of `chunk` rows.  Every wavefront looks it up by itself.
struct Chunk {
  int e, row, count;  // count 0: the slot is behind the last chunk
};

__device__ __forceinline__ Chunk find_chunk(const MArgs &a, int s, int chunk) {
  if (!a.offsets) {
    const int row = s * chunk;
    return {0, row, min(chunk, a.R - row)};
  }
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int e0 = 0; e0 < a.n; e0 += 64) {
    const int e = e0 + lane;
    int lo = 0, hi = 0;
    if (e < a.n) {
      lo = min(max(a.offsets[e], 0), a.R);
      hi = min(max(a.offsets[e + 1], lo), a.R);
    }
    const int mine = (hi - lo + chunk - 1) / chunk;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(incl, o, 64);
      if (lane >= o) incl += u;
    }
    const uint64_t over = __ballot(before + incl > s);
    if (over) {
      const int l = __ffsll((unsigned long long)over) - 1;
      const int k = s - before - (__shfl(incl, l, 64) - __shfl(mine, l, 64));
      const int row = __shfl(lo, l, 64) + k * chunk;
      return {e0 + l, row, min(chunk, __shfl(hi, l, 64) - row)};
    }
    before += __shfl(incl, 63, 64);
  }
  return {0, 0, 0};
}

// Columns of one step: one 16-byte load of each of 64 lanes, 64 bytes of
// each of 16 weight rows.
template <Kind K>
constexpr int step_columns() {
  return K == kQ4Bf16 || K == kQ4F32 ? 128 : K == kBf16 ? 32 : 16;
}

// Eight codes as bf16 16 + q, in the order of the nibbles 0 4 1 5 2 6 3 7.
__device__ __forceinline__ bf16x8_t decode(uint32_t c) {
  u32x4_t o;
  o[0] = ((c << 3) & 0x00780078u) | 0x41804180u;
  o[1] = ((c >> 1) & 0x00780078u) | 0x41804180u;
  o[2] = ((c >> 5) & 0x00780078u) | 0x41804180u;
  o[3] = ((c >> 9) & 0x00780078u) | 0x41804180u;
  return as_bf16x8(o);
}

// Eight values (four dwords of bf16 pairs) in that order.
__device__ __forceinline__ u32x4_t pair_order(u32x4_t v) {
  u32x4_t o;
  o[0] = __builtin_amdgcn_perm(v[2], v[0], 0x05040100u);
  o[1] = __builtin_amdgcn_perm(v[2], v[0], 0x07060302u);
  o[2] = __builtin_amdgcn_perm(v[3], v[1], 0x05040100u);
  o[3] = __builtin_amdgcn_perm(v[3], v[1], 0x07060302u);
  return o;
}

// fp32 as three bf16 parts, by truncation: 24 significant bits are 8 + 8 + 8,
// so their sum is the value.  Parts of Inf and NaN are not finite.
__device__ __forceinline__ void split3(float v, uint32_t (&p)[3]) {
  const uint32_t h = __float_as_uint(v) & 0xffff0000u;
  const float r = v - __uint_as_float(h);
  const uint32_t m = __float_as_uint(r) & 0xffff0000u;
  const float s = r - __uint_as_float(m);
  p[0] = h;
  p[1] = m;
  p[2] = __float_as_uint(s);
}

__device__ __forceinline__ uint32_t high_pair(uint32_t a, uint32_t b) {  // bf16 of a (low) and b (high)
  return __builtin_amdgcn_perm(b, a, 0x07060302u);
}

// x of one step and one token block in operand order.
template <Kind K>
struct XFrag;
template <>
struct XFrag<kBf16> {
  bf16x8_t v;
};
template <>
struct XFrag<kF32> {
  f32x4_t v;
};
template <>
struct XFrag<kQ4Bf16> {
  bf16x8_t v[1][4];
};
template <>
struct XFrag<kQ4F32> {
  bf16x8_t v[3][4];
};

// G: scale group (4-bit).  Product i of a step covers, for G = 128, columns
// 32 quad + 8 i + e of the step; for smaller groups columns 32 i + 8 quad + e,
// so that no product mixes groups.
template <Kind K, int G>
__device__ __forceinline__ void load_x(XFrag<K> &f, const uint8_t *x, int col, int d, int quad) {
  if constexpr (K == kBf16) {
    const int c = col + 8 * quad;
    u32x4_t u = {0, 0, 0, 0};
    if (c < d) u = *reinterpret_cast<const u32x4_t *>(x + 2 * (int64_t)c);
    f.v = as_bf16x8(u);
  } else if constexpr (K == kF32) {
    const int c = col + 4 * quad;
    f32x4_t u = {0, 0, 0, 0};
    if (c < d) u = *reinterpret_cast<const f32x4_t *>(x + 4 * (int64_t)c);
    f.v = u;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = col + (G == 128 ? 32 * quad + 8 * i : 32 * i + 8 * quad);
      if constexpr (K == kQ4Bf16) {
        u32x4_t u = {0, 0, 0, 0};
        if (c < d) u = *reinterpret_cast<const u32x4_t *>(x + 2 * (int64_t)c);
        f.v[0][i] = as_bf16x8(pair_order(u));
      } else {
        f32x4_t u[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
        if (c < d) {
          u[0] = *reinterpret_cast<const f32x4_t *>(x + 4 * (int64_t)c);
          u[1] = *reinterpret_cast<const f32x4_t *>(x + 4 * (int64_t)c + 16);
        }
        u32x4_t o[3];
#pragma unroll
        for (int p = 0; p < 4; ++p) {  // pair p: values p and p + 4
          uint32_t lo[3], hi[3];
          split3(u[0][p], lo);
          split3(u[1][p], hi);
#pragma unroll
          for (int k = 0; k < 3; ++k) o[k][p] = high_pair(lo[k], hi[k]);
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) f.v[k][i] = as_bf16x8(o[k]);
      }
    }
  }
}

// One wavefront's share of 16 weight rows times RB against 16 tokens times
// TB; the NW wavefronts of a workgroup take the steps of a row in turn and
// their sums are joined through LDS in a fixed order.
template <Kind K, int G, int TB, int RB, int NW>
__global__ void __launch_bounds__(NW * 64) stream_kernel(MArgs a) {
  constexpr int C = step_columns<K>();
  constexpr bool q4 = K == kQ4Bf16 || K == kQ4F32;
  constexpr bool out32 = K == kQ4F32 || K == kF32;
  constexpr int XP = K == kQ4F32 ? 3 : 1;
  constexpr int es = out32 ? 4 : 2;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, quad = lane >> 4;
  const int blocks = (a.d_out + 16 * RB - 1) / (16 * RB);
  const Chunk ch = find_chunk(a, blockIdx.x / blocks, 16 * TB);
  if (ch.count <= 0) return;
  const int i0 = blockIdx.x % blocks * (16 * RB);

  const uint8_t *xp[TB];
#pragma unroll
  for (int t = 0; t < TB; ++t) {
    const int r = ch.row + min(16 * t + l16, ch.count - 1);
    const int src = a.rows ? a.rows[r] : r;
    // rows behind the chunk and sources outside x read some valid row; what
    // they give is not stored
    xp[t] = a.x + (int64_t)(src < 0 || src >= a.T ? 0 : src) * a.ldx * es;
  }
  const uint8_t *wp[RB];
  int64_t sp[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    const int i = min(i0 + 16 * b + l16, a.d_out - 1);
    if constexpr (q4) {
      wp[b] = a.W + ch.e * a.w_stride + (int64_t)i * (a.d / 2);
      sp[b] = ((int64_t)ch.e * a.d_out + i) * a.groups;
    } else {
      wp[b] = a.W + ch.e * a.w_stride + (int64_t)i * a.d * es;
      sp[b] = 0;
    }
  }

  f32x4_t acc[RB][TB] = {};
  const u32x4_t one_bits = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
  const bf16x8_t ones = as_bf16x8(one_bits);
  const f32x4_t zero4 = {0, 0, 0, 0};
  for (int col = wave * C; col < a.d; col += NW * C) {
    u32x4_t w[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      w[b] = u32x4_t{0, 0, 0, 0};
      const int byte = col / C * 64 + 16 * quad;
      const int row_bytes = q4 ? a.d / 2 : a.d * es;
      if (byte < row_bytes) w[b] = *reinterpret_cast<const u32x4_t *>(wp[b] + byte);
    }
    XFrag<K> x[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) load_x<K, G>(x[t], xp[t], col, a.d, quad);

    if constexpr (K == kBf16) {
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int t = 0; t < TB; ++t)
          acc[b][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[t].v, as_bf16x8(w[b]), acc[b][t], 0, 0, 0);
    } else if constexpr (K == kF32) {
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int t = 0; t < TB; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[b][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[t].v[i], __uint_as_float(w[b][i]), acc[b][t], 0, 0, 0);
    } else {
      constexpr int NG = 128 / G, PG = 4 / NG;  // groups of a step, products of a group
      f32x4_t sx[TB][NG];
#pragma unroll
      for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          sx[t][g] = zero4;
#pragma unroll
          for (int i = 0; i < PG; ++i)
#pragma unroll
            for (int p = 0; p < XP; ++p)
              sx[t][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[t].v[p][g * PG + i], ones, sx[t][g], 0, 0, 0);
        }
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        u32x4_t c = w[b];
        if constexpr (G < 128) {  // dword j of quad i <- dword i of quad j
          uint32_t c0 = c[0], c1 = c[1], c2 = c[2], c3 = c[3];
          auto u = __builtin_amdgcn_permlane32_swap(c0, c2, false, false);
          c0 = u[0], c2 = u[1];
          u = __builtin_amdgcn_permlane32_swap(c1, c3, false, false);
          c1 = u[0], c3 = u[1];
          u = __builtin_amdgcn_permlane16_swap(c0, c1, false, false);
          c[0] = u[0], c[1] = u[1];
          u = __builtin_amdgcn_permlane16_swap(c2, c3, false, false);
          c[2] = u[0], c[3] = u[1];
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const int64_t at = sp[b] + min(col / G + g, a.groups - 1);
          const float s = out32 ? reinterpret_cast<const float *>(a.scales)[at]
                                : __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(a.scales)[at] << 16);
          const float z = 16.f + (float)(a.zeros ? a.zeros[at] & 15 : 8);
#pragma unroll
          for (int t = 0; t < TB; ++t) {
            f32x4_t q = zero4;
#pragma unroll
            for (int i = 0; i < PG; ++i)
#pragma unroll
              for (int p = 0; p < XP; ++p)
                q = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[t].v[p][g * PG + i], decode(c[g * PG + i]), q, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[b][t][i] += s * (q[i] - z * sx[t][g][i]);
          }
        }
      }
    }
  }

  __shared__ float red[NW][RB * TB * 256];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[wave][(b * TB + t) * 256 + (4 * quad + i) * 16 + l16] = acc[b][t][i];
  __syncthreads();
  for (int k = threadIdx.x; k < RB * TB * 256; k += NW * 64) {
    const int b = k / (TB * 256), token = k / 16 % (16 * TB), i = i0 + 16 * b + k % 16;
    if (token >= ch.count || i >= a.d_out) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += red[w][k];
    const int r = ch.row + token;
    if (a.rows) {
      const int src = a.rows[r];
      if (src < 0 || src >= a.T) v = 0.f;
    }
    if constexpr (out32)
      reinterpret_cast<float *>(a.y)[r * a.ldy + i] = v;
    else
      reinterpret_cast<__bf16 *>(a.y)[r * a.ldy + i] = (__bf16)v;
  }
}

// ---- many rows per expert ----

typedef float f32x16_t __attribute__((ext_vector_type(16)));

// The tiles of a launch.  Each expert's rows are cut into full row tiles of
// BM and one shorter rest; every full tile comes before any rest, so that the
// last round of the workgroups is made of short ones.  The full tiles are
// dealt to the 8 XCDs (workgroup b runs on XCD b % 8) in contiguous shares, so
// that workgroups that share an L2 work on neighbouring tiles: groups of
// kSlotGroup row tiles, in each all column tiles, in each the row tiles.  The
// rests, of all heights, are dealt one by one.
constexpr int kXcds = 8;
constexpr int kSlotGroup = 4;

struct Tile {
  int e, row, count, col;  // count 0: behind the last
};

__device__ __forceinline__ void expert_rows(const MArgs &a, int e, int *lo, int *hi) {
  *lo = *hi = 0;
  if (a.offsets) {
    if (e < a.n) {
      *lo = min(max(a.offsets[e], 0), a.R);
      *hi = min(max(a.offsets[e + 1], *lo), a.R);
    }
  } else if (e == 0) {
    *hi = a.R;
  }
}

struct Tiles {
  int full, rest;  // row tiles
};

template <int BM>
__device__ __forceinline__ Tiles count_tiles(const MArgs &a) {
  int full = 0, rest = 0;
  for (int e0 = 0; e0 < a.n; e0 += 64) {
    int lo, hi;
    expert_rows(a, e0 + (threadIdx.x & 63), &lo, &hi);
    full += (hi - lo) / BM;
    rest += (hi - lo) % BM != 0;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    full += __shfl_xor(full, o, 64);
    rest += __shfl_xor(rest, o, 64);
  }
  return {__builtin_amdgcn_readfirstlane(full), __builtin_amdgcn_readfirstlane(rest)};
}

// Tile number `at` of XCD `xcd`.
template <int BM>
__device__ __forceinline__ Tile find_tile(const MArgs &a, const Tiles &n, int col_tiles, int xcd, int64_t at) {
  const int lane = threadIdx.x & 63;
  const int64_t full_tiles = (int64_t)n.full * col_tiles, rest_tiles = (int64_t)n.rest * col_tiles;
  const int64_t share = (full_tiles + kXcds - 1) / kXcds;
  const int64_t first = xcd * share, mine = max((int64_t)0, min(share, full_tiles - first));
  const bool is_full = at < mine;
  int slot, col;
  if (is_full) {
    const int64_t t = first + at;
    const int g = (int)(t / (kSlotGroup * col_tiles)), in = (int)(t - (int64_t)g * kSlotGroup * col_tiles);
    const int wide = min(kSlotGroup, n.full - g * kSlotGroup);
    slot = g * kSlotGroup + in % wide;
    col = in / wide;
  } else {
    const int64_t t = (at - mine) * kXcds + xcd;
    if (t >= rest_tiles) return {0, 0, 0, 0};
    slot = (int)(t / col_tiles);
    col = (int)(t - (int64_t)slot * col_tiles);
  }
  int before = 0;
  for (int e0 = 0; e0 < a.n; e0 += 64) {
    int lo, hi;
    expert_rows(a, e0 + lane, &lo, &hi);
    const int has = is_full ? (hi - lo) / BM : ((hi - lo) % BM != 0);
    int incl = has;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(incl, o, 64);
      if (lane >= o) incl += u;
    }
    const uint64_t over = __ballot(before + incl > slot);
    if (over) {
      const int l = __ffsll((unsigned long long)over) - 1;
      const int k = slot - before - (__builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(has, l));
      const int row = __builtin_amdgcn_readlane(lo, l), rows = __builtin_amdgcn_readlane(hi, l) - row;
      const int skip = is_full ? k * BM : rows / BM * BM;
      return {e0 + l, row + skip, min(BM, rows - skip), col};
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return {0, 0, 0, 0};
}

// A tile row is BK columns in 16-byte pieces; piece c of row r lies at
// position c ^ swizzle(r), so that the 16 rows that a read touches at once lie
// in different banks.
template <int BK>
__device__ __forceinline__ int swizzle(int r) {
  return BK == 64 ? r & 7 : (r >> 2) & 3;
}
template <int BK>
__device__ __forceinline__ int tile_at(int r, int c) {
  return r * (BK * 2) + ((c ^ swizzle<BK>(r)) << 4);
}

__device__ const u32x4_t kZeros = {0, 0, 0, 0};

// 64 lanes' 16 bytes each, from anywhere, to 1 KiB of LDS in lane order.
__device__ __forceinline__ void to_lds(const void *src, void *dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                   (__attribute__((address_space(3))) void *)dst, 16, 0, 0);
}

// Every wavefront's own loads to LDS but the last N have landed, then all wavefronts'.
template <int N>
__device__ __forceinline__ void landed() {
  static_assert(N < 64, "vmcnt");
  // the builtin, so that the compiler's own count knows of the wait
  __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4 << 14) | (7 << 4));  // vmcnt(N) lgkmcnt(0)
  asm volatile("s_barrier" ::: "memory");
}

// bf16 tiles of 256 tokens x 256 weight rows on 8 wavefronts, 2 x 4 of them,
// each 32 TM tokens x 64 weight rows.  The columns go by in stages of 32; four
// stages lie in LDS, filled by direct loads in a stream that runs on from one
// tile into the next.
constexpr int kWideBM = 256, kWideBN = 256, kWideBK = 32;
constexpr int kWideStage = (kWideBM + kWideBN) * kWideBK * 2;
constexpr int kWideLoads = kWideStage / 1024 / 8;  // loads of a wavefront per stage, half x, half W

// Where a wavefront's loads of a stage come from.
struct WideSource {
  const uint8_t *x[kWideLoads / 2], *w[kWideLoads / 2];
  int left;  // columns from this lane's next piece to the row's end
};

__device__ __forceinline__ WideSource wide_source(const MArgs &a, const Tile &tl, int wave, int lane) {
  constexpr int L = kWideLoads / 2, RK = 16;  // rows of a KiB
  // first column of this lane's piece: the same in all its rows, which lie
  // whole KiB apart
  const int sub = lane >> 2, piece = ((lane & 3) ^ swizzle<kWideBK>(sub)) * 8;
  WideSource f;
  f.left = tl.count > 0 ? a.d - piece : 0;
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int m = (wave * L + i) * RK + sub;
    f.x[i] = f.w[i] = nullptr;
    if (tl.count > 0) {
      const int r = tl.row + min(m, tl.count - 1);
      const int src = a.rows ? a.rows[r] : r;
      f.x[i] = a.x + ((int64_t)(src < 0 || src >= a.T ? 0 : src) * a.ldx + piece) * 2;
      f.w[i] = a.W + tl.e * a.w_stride + ((int64_t)min(tl.col * kWideBN + m, a.d_out - 1) * a.d + piece) * 2;
    }
  }
  return f;
}

// Brings the next 32 columns.  A piece behind d is read from zeros, for x and
// for W (their product must be zero), and so is a whole stage behind the last.
__device__ __forceinline__ void wide_fetch(WideSource &f, uint8_t *st, int wave) {
  constexpr int L = kWideLoads / 2;
  const uint64_t zeros = reinterpret_cast<uint64_t>(&kZeros);
  const uint64_t in = (int64_t)(-f.left) >> 63;  // all ones while left > 0
  f.left -= kWideBK;
#pragma unroll
  for (int i = 0; i < L; ++i) {
    to_lds(reinterpret_cast<const void *>((reinterpret_cast<uint64_t>(f.x[i]) & in) | (zeros & ~in)),
           st + (wave * L + i) * 1024);
    f.x[i] += 2 * kWideBK;
  }
#pragma unroll
  for (int i = 0; i < L; ++i) {
    to_lds(reinterpret_cast<const void *>((reinterpret_cast<uint64_t>(f.w[i]) & in) | (zeros & ~in)),
           st + kWideBM * kWideBK * 2 + (wave * L + i) * 1024);
    f.w[i] += 2 * kWideBK;
  }
}

// One tile of at most 64 TM tokens.  Its first two stages have landed and the
// third is on its way when it begins; it leaves those of the next tile (`nf`) so.
template <int TM>
__device__ __forceinline__ void wide_tile(const MArgs &a, const Tile &tl, WideSource &f, const WideSource &nf,
                                          uint8_t *lds0, uint8_t *lds1, uint8_t *lds2, uint8_t *lds3) {
  constexpr int TN = 2, kBlock = 32 * kWideBK * 2;  // 32 x 32 blocks of weight rows; bytes of 32 rows
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3, l32 = lane & 31, half = lane >> 5;
  // which of this lane's tokens have a source; 0 for those behind the tile
  uint32_t valid = 0;
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int m = (wm * TM + j) * 32 + l32;
    if (m < tl.count) {
      const int src = a.rows ? a.rows[tl.row + m] : tl.row + m;
      valid |= (src >= 0 && src < a.T ? 1u : 0u) << j;
    }
  }

  f32x16_t acc[TN][TM] = {};
  int xat[2], wat[2];  // the swizzle of a row depends on its place in a block only
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    xat[s] = wm * TM * kBlock + tile_at<kWideBK>(l32, 2 * s + half);
    wat[s] = kWideBM * kWideBK * 2 + wn * TN * kBlock + tile_at<kWideBK>(l32, 2 * s + half);
  }
  bf16x8_t wf[2][TN], xf[2][TM];
  const auto read = [&](const uint8_t *st, int s) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
      wf[s][j] = as_bf16x8(*reinterpret_cast<const u32x4_t *>(st + wat[s] + j * kBlock));
#pragma unroll
    for (int j = 0; j < TM; ++j)
      xf[s][j] = as_bf16x8(*reinterpret_cast<const u32x4_t *>(st + xat[s] + j * kBlock));
  };
  const auto multiply = [&](int s) {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
      for (int i = 0; i < TN; ++i)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wf[s][i], xf[s][j], acc[i][j], 0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
  };
  // One step multiplies the stage `cur`, whose first 16 columns are in
  // registers, and leaves those of `next` there.  Loads to LDS are issued
  // between two products, where every read of LDS has come back: the compiler
  // waits for all of them after such a load.  When a step ends only its own
  // loads may be under way, so a stage has two steps to arrive; it is filled
  // after the barrier behind its last reads.
  const auto step = [&](const uint8_t *cur, const uint8_t *next, uint8_t *fill) {
    read(cur, 1);
    multiply(0);
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    wide_fetch(f, fill, wave);
    read(next, 0);
    multiply(1);
    landed<kWideLoads>();
  };
  read(lds0, 0);
  for (int k = 128; k < a.d; k += 128) {
    step(lds0, lds1, lds3);
    step(lds1, lds2, lds0);
    step(lds2, lds3, lds1);
    step(lds3, lds0, lds2);
  }
  // the last 128 columns (zeros behind d)
  step(lds0, lds1, lds3);
  f = nf;
  step(lds1, lds2, lds0);
  step(lds2, lds3, lds1);
  step(lds3, lds0, lds2);

  // Of each 16 weight rows of a token the lower lanes take eight and the
  // upper ones the others, 16 bytes each.
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int m = (wm * TM + j) * 32 + l32;
    uint8_t *const yp = a.y + 2 * ((int64_t)(tl.row + m) * a.ldy);
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int q = 0; q < 4; q += 2) {
        uint32_t v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
          const bf16x2_t p = {(__bf16)acc[i][j][4 * q + 2 * r], (__bf16)acc[i][j][4 * q + 2 * r + 1]};
          v[r] = valid >> j & 1 ? __builtin_bit_cast(uint32_t, p) : 0u;
        }
        const auto s0 = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
        const auto s1 = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
        const int o = tl.col * kWideBN + (wn * TN + i) * 32 + 8 * q + 8 * half;
        if (m < tl.count && o < a.d_out)
          *reinterpret_cast<u32x4_t *>(yp + 2 * o) = u32x4_t{s0[0], s1[0], s0[1], s1[1]};
      }
  }
}

// A workgroup for every CU, each walking its XCD's tiles; an expert's rest
// takes the smallest of four heights that holds it.
__global__ void __launch_bounds__(512) wide_kernel(MArgs a) {
  // stages as separate objects, so that the compiler sees that filling one
  // does not touch the others
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[kWideStage];
  __shared__ __attribute__((aligned(1024))) uint8_t lds1[kWideStage];
  __shared__ __attribute__((aligned(1024))) uint8_t lds2[kWideStage];
  __shared__ __attribute__((aligned(1024))) uint8_t lds3[kWideStage];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col_tiles = (a.d_out + kWideBN - 1) / kWideBN;
  const Tiles n = count_tiles<kWideBM>(a);
  const int xcd = blockIdx.x % kXcds, stride = gridDim.x / kXcds;
  int64_t at = blockIdx.x / kXcds;
  Tile tl = find_tile<kWideBM>(a, n, col_tiles, xcd, at);
  if (tl.count <= 0) return;
  WideSource f = wide_source(a, tl, wave, lane);
  wide_fetch(f, lds0, wave);
  wide_fetch(f, lds1, wave);
  wide_fetch(f, lds2, wave);
  landed<kWideLoads>();
  for (;;) {
    at += stride;
    const Tile next = find_tile<kWideBM>(a, n, col_tiles, xcd, at);
    const WideSource nf = wide_source(a, next, wave, lane);
    if (tl.count > 192)
      wide_tile<4>(a, tl, f, nf, lds0, lds1, lds2, lds3);
    else if (tl.count > 128)
      wide_tile<3>(a, tl, f, nf, lds0, lds1, lds2, lds3);
    else if (tl.count > 64)
      wide_tile<2>(a, tl, f, nf, lds0, lds1, lds2, lds3);
    else
      wide_tile<1>(a, tl, f, nf, lds0, lds1, lds2, lds3);
    if (next.count <= 0) break;
    tl = next;
  }
  // no load may reach the LDS after the workgroup has left it
  landed<0>();
}

gsi_status launch_wide(const MArgs &a, hipStream_t st) {
  constexpr int kCus = 256;
  wide_kernel<<<kCus, 512, 0, st>>>(a);
  return hipGetLastError() == hipSuccess ? GSI_OK : GSI_E_HIP;
}

template <Kind K, int G>
gsi_status launch(const MArgs &a, hipStream_t st) {
  constexpr int TB = 1, RB = 1, NW = 8;
  const int64_t blocks = (a.d_out + 16 * RB - 1) / (16 * RB);
  const int64_t slots = (a.R + 16 * TB - 1) / (16 * TB) + (a.offsets ? (a.n < a.R ? a.n : a.R) : 0);
  if (blocks * slots > INT32_MAX) return GSI_E_SHAPE;
  stream_kernel<K, G, TB, RB, NW><<<(unsigned)(blocks * slots), NW * 64, 0, st>>>(a);
  return hipGetLastError() == hipSuccess ? GSI_OK : GSI_E_HIP;
}

inline bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

gsi_status check_weights(const gsi_weights *w) {
  if (!w) return GSI_E_NULL;
  if (w->dtype != GSI_FP32 && w->dtype != GSI_BF16) return GSI_E_DTYPE;
  if (w->bits != 0 && w->bits != 4) return GSI_E_DTYPE;
  if (w->n < 1 || w->n > 4096 || w->d_out < 8 || w->d_out % 8 || w->d_out > (1 << 24)) return GSI_E_SHAPE;
  if (w->d < 8 || w->d % (w->bits ? 32 : 8) || w->d > (1 << 20)) return GSI_E_SHAPE;
  const int es = w->dtype == GSI_FP32 ? 4 : 2;
  if (w->bits) {
    if ((w->group != 32 && w->group != 64 && w->group != 128) || w->stride != 0) return GSI_E_SHAPE;
  } else if (w->group != 0 || (w->n > 1 && w->stride < (int64_t)w->d_out * w->d) || w->stride > (INT64_MAX >> 16)) {
    return GSI_E_SHAPE;
  }
  if (!w->W || (w->bits && !w->scales)) return GSI_E_NULL;
  if (!aligned(w->W, 16) || (w->bits && !aligned(w->scales, es)) || (!w->bits && w->n > 1 && w->stride * es % 16))
    return GSI_E_ALIGN;
  return GSI_OK;
}

gsi_status run_maps(const gsi_weights *w, const void *x, int64_t ldx, int32_t T, const int32_t *offsets,
                    const int32_t *rows, void *y, int64_t ldy, int32_t R, void *stream) {
  const int es = w->dtype == GSI_FP32 ? 4 : 2;
  if (ldx < w->d || ldy < w->d_out || ldx > INT64_MAX / 4 / T || ldy > INT64_MAX / 4 / R) return GSI_E_SHAPE;
  if (!x || !y) return GSI_E_NULL;
  if (!aligned(x, 16) || !aligned(y, 16) || ldx * es % 16 || ldy * es % 16 || !aligned(offsets, 4) || !aligned(rows, 4))
    return GSI_E_ALIGN;
  MArgs a{};
  a.W = static_cast<const uint8_t *>(w->W);
  a.scales = static_cast<const uint8_t *>(w->scales);
  a.zeros = w->zeros;
  a.x = static_cast<const uint8_t *>(x);
  a.y = static_cast<uint8_t *>(y);
  a.offsets = offsets;
  a.rows = rows;
  a.w_stride = w->bits ? (int64_t)w->d_out * (w->d / 2) : w->stride * es;
  a.ldx = ldx;
  a.ldy = ldy;
  a.d = w->d;
  a.d_out = w->d_out;
  a.n = w->n;
  a.R = R;
  a.T = T;
  a.groups = w->bits ? (w->d + w->group - 1) / w->group : 0;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const int per = R / (w->n < R ? w->n : R);
  if (w->bits == 0 && w->dtype == GSI_BF16 && per >= 64) return launch_wide(a, st);
  if (w->bits == 0) return w->dtype == GSI_FP32 ? launch<kF32, 0>(a, st) : launch<kBf16, 0>(a, st);
  if (w->dtype == GSI_FP32)
    return w->group == 128 ? launch<kQ4F32, 128>(a, st)
                           : (w->group == 64 ? launch<kQ4F32, 64>(a, st) : launch<kQ4F32, 32>(a, st));
  return w->group == 128 ? launch<kQ4Bf16, 128>(a, st)
                         : (w->group == 64 ? launch<kQ4Bf16, 64>(a, st) : launch<kQ4Bf16, 32>(a, st));
}

}  // namespace
}  // namespace gsi

using namespace gsi;

extern "C" {

gsi_status gsi_q4_linear(const gsi_weights *w, const void *x, int64_t ldx, void *y, int64_t ldy,
                         int32_t T, void *stream) {
  const gsi_status s = check_weights(w);
  if (s != GSI_OK) return s;
  if (w->bits != 4) return GSI_E_DTYPE;
  if (w->n != 1 || T < 0) return GSI_E_SHAPE;
  if (T == 0) return GSI_OK;
  return run_maps(w, x, ldx, T, nullptr, nullptr, y, ldy, T, stream);
}

gsi_status gsi_grouped_linear(const gsi_weights *w, const void *x, int64_t ldx, int32_t T,
                              const int32_t *offsets, const int32_t *rows, void *y, int64_t ldy,
                              int32_t R, void *stream) {
  const gsi_status s = check_weights(w);
  if (s != GSI_OK) return s;
  if (R < 0 || T < 0 || (R > 0 && T == 0)) return GSI_E_SHAPE;
  if (R == 0) return GSI_OK;
  if (!offsets) return GSI_E_NULL;
  return run_maps(w, x, ldx, T, offsets, rows, y, ldy, R, stream);
}

}  // extern "C"
