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
