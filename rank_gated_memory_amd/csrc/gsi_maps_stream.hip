// Plain linear maps with few rows per expert on gfx950 MFMA.
//
//   stream_kernel : the weights of an expert are read once for a chunk of up
//                   to 16 rows.  At one token a weight is used once, so the
//                   chunk's x is staged in LDS and the wavefronts do nothing
//                   but stream weights into registers, a batch of loads ahead
//                   of the products: many bytes at a few rows are bound by
//                   HBM, few bytes by launch and latency, and from some ten
//                   rows on the products, with the codes decoded again for
//                   every 16 rows, count for more than the bytes.  A wavefront
//                   owns 16 weight rows; where there are fewer such blocks
//                   than the chip has wavefronts, several split the columns of
//                   a block and are joined through LDS in a fixed order.
//                   Further chunks of an expert read its weights again, out of
//                   the L2s.  (Chunks of 32 and 64 rows, with two blocks of
//                   weight rows per wavefront, were slower at every number of
//                   rows when they were tried: 28 and 69 us against 22 and 23
//                   for 24 and 40 tokens of a 4-bit 4096 x 4096 map, which
//                   take 10.5 and 13 now.) Times on weights called again and
//                   again, and in brackets on weights from HBM: 128 bf16
//                   experts' maps 1024 -> 2048, a row each, 538 MB: 97 us (97:
//                   5.5 TB/s).  8 experts' bf16 maps 2048 -> 2816 for one
//                   token, 92 MB: 18.4 us (21.1: 4.4 TB/s).  24 tokens' 192
//                   rows over 128 experts in 4 bits, 4096 -> 1536, 110 to 142
//                   MB: 30 to 54 us (33 to 58), by how uneven the experts are.
//                   A 4-bit 4096 x 4096 map for one token, 8.8 MB: 6.0 us
//                   (6.3), most of it launch and latency; 5 tokens 4096 ->
//                   50400, 113 MB: 30 us (33), where reading the weights in
//                   this pattern alone took 23.  With more tokens the staging
//                   of x shows: 13 fp32 tokens 5120 -> 13824, 47 MB: 28 us
//                   (29.5).
//
// 4-bit weights.  With w = s (q - z) a group's share of y is
//   s (sum q x - z sum x) = s (sum (16 + q) x - (16 + z) sum x).
// 16 + q is the bf16 0x4180 | q << 3, so two codes decode with one shift and
// one and-or, exactly, and the matrix core multiplies them with bf16 x
// exactly; sum x of the group comes from the same instruction with ones for
// weights.  The two sums cancel, so a group's fp32 error is one of sum (32 + q
// + z) |x|: with x of one sign and groups of 128 up to 11 times that of a
// plain fp32 product (1.0e-6 of sum |w x| at most, 2.2e-7 there).  fp32 x is
// split into three bf16 parts (8 + 8 + 8 bits, exact), each its own product.
// Only the group's fp32 sums are rounded.
//
// The matrix operand A holds tokens and B weight rows, so that a lane's
// accumulators all belong to one weight row and take one scale.  Row m of A
// is token 4 (m % 4) + m / 4 of the chunk: up to four tokens then need only
// the first accumulator of every lane.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "gsi_maps.h"

namespace gsi {
namespace {

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
    int lo, hi;
    expert_rows(a, e, &lo, &hi);
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

// The constants of decode(), in registers: with literals (v & mask) | bits
// takes two instructions instead of one.
struct DecodeBits {
  uint32_t mask = 0x00780078u, one = 0x41804180u, low = 0x0f0f0f0fu, sixteen = 0x10101010u;
  __device__ __forceinline__ DecodeBits() {
    asm("" : "+s"(mask), "+v"(one));
    asm("" : "+s"(low), "+v"(sixteen));
  }
};

// Eight codes as bf16 16 + q, in the order of the nibbles 0 4 1 5 2 6 3 7.
__device__ __forceinline__ bf16x8_t decode(uint32_t c, const DecodeBits &k) {
  u32x4_t o;
  o[0] = ((c << 3) & k.mask) | k.one;
  o[1] = ((c >> 1) & k.mask) | k.one;
  o[2] = ((c >> 5) & k.mask) | k.one;
  o[3] = ((c >> 9) & k.mask) | k.one;
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

// Eight fp32 values as bf16 part p of each, in the order of pair_order.
__device__ __forceinline__ void split_octet(const f32x4_t (&u)[2], bf16x8_t (&out)[3]) {
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
  for (int k = 0; k < 3; ++k) out[k] = as_bf16x8(o[k]);
}

// A step is 64 bytes of each weight row: one 16-byte load of each of 64 lanes.
template <Kind K>
constexpr int kStepColumns = K == kQ4Bf16 || K == kQ4F32 ? 128 : K == kBf16 ? 32 : 16;

constexpr int kStreamWaves = 16;  // at most, of a workgroup that has the CU for itself; 8 of one that shares it
constexpr int kStreamLds = 64 * 1024;        // x of a chunk; two workgroups of a CU hold theirs
constexpr int kStreamLdsAlone = 144 * 1024;  // of a workgroup that has the CU for itself

// How a launch splits its work.
struct StreamShape {
  int split;         // wavefronts that share the columns of a block of weight rows
  int strips;        // workgroups per chunk
  int room;          // bytes of LDS for x
  int waves;         // of a workgroup
};

template <Kind K, int G, int U>
struct Stream {
  static constexpr bool q4 = K == kQ4Bf16 || K == kQ4F32;
  static constexpr bool f32 = K == kQ4F32 || K == kF32;
  static constexpr int es = f32 ? 4 : 2;
  static constexpr int C = kStepColumns<K>;
  static constexpr int XP = K == kQ4F32 ? 3 : 1;       // parts of x
  static constexpr int xes = K == kF32 ? 4 : 2;        // bytes of a part
  static constexpr int NG = q4 ? 128 / G : 1;          // scale groups of a step
  static constexpr int BG = U * NG;                    // of a batch
  static constexpr int SW = f32 ? BG : (BG + 1) / 2;   // their scales and zeros in dwords
  static constexpr int ZW = (BG + 3) / 4;

  // U steps of weights with their scales
  struct Batch {
    u32x4_t w[U];
    uint32_t s[SW], z[ZW];
  };

  const MArgs &a;
  DecodeBits bits;
  int quad, l16, row_bytes;
  // the block's first row, and this lane's offsets from there: 32 bits, for at
  // most 16 rows
  const uint8_t *wp, *sp, *zp;
  uint32_t wo, so, zo;

  __device__ __forceinline__ Stream(const MArgs &args, int lane) : a(args) {
    quad = lane >> 4, l16 = lane & 15;
    row_bytes = q4 ? a.d / 2 : a.d * es;
  }

  // The block of weight rows from i0 < d_out on; rows behind the last read
  // the last, and what they give is not stored.
  __device__ __forceinline__ void rows_from(int e, int i0) {
    const int64_t row = (int64_t)e * a.d_out + i0;
    const uint32_t i = min(l16, a.d_out - 1 - i0);
    wp = a.W + e * a.w_stride + (int64_t)i0 * row_bytes;
    wo = i * row_bytes + 16 * quad;
    if constexpr (q4) {
      sp = a.scales + row * a.groups * es;
      so = i * a.groups * es;
      // without zeros their loads read 16 bytes of the scales, which there are
      // at least, and the value is dropped
      zp = a.zeros ? a.zeros + row * a.groups : a.scales;
      zo = a.zeros ? i * a.groups : 0;
    }
  }

  template <typename T, int M, int N>
  __device__ __forceinline__ static void copy_run(uint32_t (&o)[N], const uint8_t *p) {
    struct Run {
      T v[M];
    };
    __builtin_memcpy(o, p, sizeof(Run));
  }

  // The U whole steps from `step` on.
  __device__ __forceinline__ void load(Batch &o, int step) const {
#pragma unroll
    for (int u = 0; u < U; ++u) o.w[u] = *reinterpret_cast<const u32x4_t *>(wp + (wo + (uint32_t)step * 64) + u * 64);
    if constexpr (q4) {
      using T = std::conditional_t<f32, uint32_t, uint16_t>;
      copy_run<T, BG>(o.s, sp + (so + (uint32_t)(step * NG * es)));
      copy_run<uint8_t, BG>(o.z, zp + (zo + (uint32_t)(a.zeros ? step * NG : 0)));
    }
  }

  // Step `step` alone as step 0 of a batch; it may end behind the row.
  __device__ __forceinline__ void load_last(Batch &o, int step) const {
    o.w[0] = u32x4_t{0, 0, 0, 0};
    if (step * 64 + 16 * quad < row_bytes) o.w[0] = *reinterpret_cast<const u32x4_t *>(wp + (wo + (uint32_t)step * 64));
    if constexpr (q4) {
#pragma unroll
      for (int g = 0; g < SW; ++g) o.s[g] = 0;
      o.z[0] = 0;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int at = min(step * NG + g, a.groups - 1);  // behind the last group x is zero
        if constexpr (f32)
          o.s[g] = *reinterpret_cast<const uint32_t *>(sp + (so + 4u * at));
        else
          o.s[g / 2] |= (uint32_t) * reinterpret_cast<const uint16_t *>(sp + (so + 2u * at)) << (16 * (g & 1));
        o.z[0] |= (uint32_t)zp[zo + (a.zeros ? at : 0)] << (8 * g);
      }
    }
  }

  __device__ __forceinline__ static int x_stride(int columns) { return columns * xes + 16; }

  // x of the chunk's columns [c0, c0 + columns) into LDS: a plane of tokens for
  // each part, zeros behind d and for rows without a source, octets in the
  // order of decode() where the weights are codes.  Only the chunk's own rows
  // are written; those behind them are never read.
  __device__ __forceinline__ void stage(uint8_t *lds, const Chunk &ch, int c0, int columns, int threads) const {
    constexpr int V = K == kF32 ? 4 : 8;  // columns of a 16-byte piece
    const int pieces = columns / V, stride = x_stride(columns);
    for (int k = threadIdx.x; k < ch.count * pieces; k += threads) {
      const int m = k / pieces, p = k - m * pieces, c = c0 + p * V;
      const int src = a.rows ? a.rows[ch.row + m] : ch.row + m;
      const bool in = c < a.d && src >= 0 && src < a.T;
      const uint8_t *at = a.x + ((int64_t)(in ? src : 0) * a.ldx + c) * es;
      uint8_t *const to = lds + m * stride + p * 16;
      if constexpr (K == kQ4F32) {
        f32x4_t u[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
        if (in) {
          u[0] = *reinterpret_cast<const f32x4_t *>(at);
          u[1] = *reinterpret_cast<const f32x4_t *>(at + 16);
        }
        bf16x8_t o[3];
        split_octet(u, o);
#pragma unroll
        for (int q = 0; q < 3; ++q) *reinterpret_cast<bf16x8_t *>(to + q * (ch.count * stride)) = o[q];
      } else {
        u32x4_t u = {0, 0, 0, 0};
        if (in) u = *reinterpret_cast<const u32x4_t *>(at);
        *reinterpret_cast<u32x4_t *>(to) = q4 ? pair_order(u) : u;
      }
    }
  }

  // Where this lane's token lies in LDS; a lane without a token reads the first.
  struct Token {
    const uint8_t *x;
    int plane;
  };
  __device__ __forceinline__ Token token(const uint8_t *lds, const Chunk &ch, int columns) const {
    const int stride = x_stride(columns), m = 4 * (l16 & 3) + (l16 >> 2);
    return {lds + (m < ch.count ? m : 0) * stride + quad * (q4 && G == 128 ? 64 : 16), ch.count * stride};
  }

  // The products of a batch's first N steps into acc, x from `at` bytes on;
  // accumulators from NI on stay zero.
  template <int NI, int N>
  __device__ __forceinline__ void multiply(f32x4_t &acc, const Batch &o, const Token &tk, int at) const {
    uint32_t z16[ZW];  // 16 + zero, a byte each
    if constexpr (q4) {
#pragma unroll
      for (int k = 0; k < ZW; ++k) z16[k] = a.zeros ? (o.z[k] & bits.low) | bits.sixteen : 0x18181818u;
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
      // step by step: hoisting the reads of x over all steps costs wavefronts
      __builtin_amdgcn_sched_barrier(0);
      const int xo = at + u * C * xes;
      if constexpr (!q4) {
        const u32x4_t x = *reinterpret_cast<const u32x4_t *>(tk.x + xo);
        if constexpr (K == kBf16) {
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(x), as_bf16x8(o.w[u]), acc, 0, 0, 0);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x[i]), __uint_as_float(o.w[u][i]), acc, 0, 0, 0);
        }
      } else {
        // Product i of a step covers, for G = 128, columns 32 quad + 8 i + e;
        // for smaller groups columns 32 i + 8 quad + e, so that no product
        // mixes groups.
        constexpr int PG = 4 / NG;  // products of a group
        const f32x4_t zero4 = {0, 0, 0, 0};
        const u32x4_t ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
        u32x4_t c = o.w[u];
        if constexpr (G < 128) {  // dword j of quad i <- dword i of quad j
          const auto p = __builtin_amdgcn_permlane32_swap(c[0], c[2], false, false);
          const auto q = __builtin_amdgcn_permlane32_swap(c[1], c[3], false, false);
          const auto r = __builtin_amdgcn_permlane16_swap(p[0], q[0], false, false);
          const auto s = __builtin_amdgcn_permlane16_swap(p[1], q[1], false, false);
          c = u32x4_t{r[0], r[1], s[0], s[1]};
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const int k = u * NG + g;
          const float s = f32 ? __uint_as_float(o.s[k])
                              : __uint_as_float(k & 1 ? o.s[k / 2] & 0xffff0000u : o.s[k / 2] << 16);
          const float z = (float)(z16[k / 4] >> (8 * (k & 3)) & 255);
          f32x4_t q = zero4, sx = zero4;
#pragma unroll
          for (int i = 0; i < PG; ++i) {
            const bf16x8_t w = decode(c[g * PG + i], bits);
#pragma unroll
            for (int p = 0; p < XP; ++p) {
              const bf16x8_t x = as_bf16x8(*reinterpret_cast<const u32x4_t *>(tk.x + p * tk.plane + xo +
                                                                              (g * PG + i) * (G == 128 ? 16 : 64)));
              sx = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, as_bf16x8(ones), sx, 0, 0, 0);
              q = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w, q, 0, 0, 0);
            }
          }
#pragma unroll
          for (int i = 0; i < NI; ++i) acc[i] += s * (q[i] - z * sx[i]);
          // here, not after the next batch's loads, where the compiler would
          // carry q and sx of every group to
          asm volatile("" : "+v"(acc));
        }
      }
    }
  }
};

// Columns of `tokens` rows of x that fit into `room` bytes: all `padded` ones of
// a row, or whole batches.
template <typename S, int U>
__host__ __device__ constexpr int columns_in(int room, int tokens, int padded) {
  const int fit = (room / (tokens * S::XP) - 16) / S::xes;
  return fit >= padded ? padded : fit / (S::C * U) * (S::C * U);
}

template <Kind K, int G, int U>
__global__ void __launch_bounds__(kStreamWaves * 64, 4) stream_kernel(MArgs a, StreamShape sh) {
  using S = Stream<K, G, U>;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ float red[kStreamWaves][256];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Chunk ch = find_chunk(a, blockIdx.x / sh.strips, 16);
  if (ch.count <= 0) return;
  S s(a, lane);
  // a workgroup's wavefronts: sh.waves / sh.split blocks of weight rows, the
  // columns of each in `split` shares of whole batches
  const int side = wave / sh.split, share = wave % sh.split, sides = sh.waves / sh.split;
  const int blocks = (a.d_out + 15) / 16, groups = (blocks + sides - 1) / sides;
  // accumulators of a lane that hold tokens
  const int live = S::q4 ? (ch.count + 3) / 4 : 4;
  // columns of x in LDS at a time, whole steps, and the parts of d
  const int padded = (a.d + S::C - 1) / S::C * S::C;
  const int columns = __builtin_amdgcn_readfirstlane(columns_in<S, U>(sh.room, ch.count, padded));
  const int parts = (a.d + columns - 1) / columns;
  const auto tk = s.token(lds, ch, columns);
  // a part's columns: whole batches, dealt to the split in even shares; what
  // is left of the row goes to the last share, step by step
  const auto share_of = [&](int part, int *step0, int *first, int *end, int *rest, int *last) {
    const int c0 = part * columns, width = min(columns, a.d - c0), batches = width / (S::C * U);
    *step0 = c0 / S::C;
    *first = *step0 + batches * share / sh.split * U;
    *end = *step0 + batches * (share + 1) / sh.split * U;
    *rest = *step0 + batches * U;
    *last = share == sh.split - 1 ? *step0 + (width + S::C - 1) / S::C : 0;
  };
  // Of every part and of every block the first batch is on its way before the
  // wavefront is done with the last one.
  typename S::Batch o[2];
  const auto first_batch = [&](int g, int part) {
    int step0, first, end, rest, last;
    share_of(part, &step0, &first, &end, &rest, &last);
    s.rows_from(ch.e, min((g * sides + side) * 16, a.d_out - 1));
    if (first < end) s.load(o[0], first);
  };
  int g = blockIdx.x % sh.strips;
  if (g < groups) first_batch(g, 0);
  for (; g < groups; g += sh.strips) {
    f32x4_t acc = {};
    for (int part = 0; part < parts; ++part) {
      int step0, first, end, rest, last;
      share_of(part, &step0, &first, &end, &rest, &last);
      if (parts > 1 || g < sh.strips) {
        if (part > 0 || g >= sh.strips) __syncthreads();
        s.stage(lds, ch, part * columns, columns, sh.waves * 64);
        __syncthreads();
      }
      const auto run = [&](auto ni) {
        constexpr int NI = decltype(ni)::value;
        for (int step = first; step < end; step += 2 * U) {
          if (step + U < end) s.load(o[1], step + U);
          s.template multiply<NI, U>(acc, o[0], tk, (step - step0) * S::C * S::xes);
          if (step + 2 * U < end) s.load(o[0], step + 2 * U);
          if (step + U < end) s.template multiply<NI, U>(acc, o[1], tk, (step + U - step0) * S::C * S::xes);
        }
        for (int step = rest; step < last; ++step) {
          s.load_last(o[0], step);
          s.template multiply<NI, 1>(acc, o[0], tk, (step - step0) * S::C * S::xes);
        }
      };
      if (live == 1)
        run(std::integral_constant<int, 1>{});
      else if (live == 2)
        run(std::integral_constant<int, 2>{});
      else
        run(std::integral_constant<int, 4>{});
      if (part + 1 < parts)
        first_batch(g, part + 1);
      else if (g + sh.strips < groups)
        first_batch(g + sh.strips, 0);
    }
    // one output: token k / 16 and weight row k % 16 of block `b`
    const auto put = [&](int b, int k, float v) {
      // here: the compiler would carry the addresses of every output through all
      // blocks, in registers that the bf16 form of groups of 32 does not have (it
      // spilled two; 5 tokens 4096 -> 50400, weights from HBM: 40.8 -> 39.9 us);
      // the other forms keep them (bf16 without groups is 3 % faster so)
      if constexpr (S::q4 && G == 32) asm volatile("" : "+v"(k));
      const int i = (g * sides + b) * 16 + k % 16, r = ch.row + k / 16;
      if (k / 16 >= ch.count || i >= a.d_out) return;
      if (a.rows) {
        const int src = a.rows[r];
        if (src < 0 || src >= a.T) v = 0.f;
      }
      if constexpr (S::f32)
        reinterpret_cast<float *>(a.y)[r * a.ldy + i] = v;
      else
        reinterpret_cast<__bf16 *>(a.y)[r * a.ldy + i] = (__bf16)v;
    };
    if (sh.split > 1) {
      if (g >= sh.strips) __syncthreads();  // the sums of the last block have been read
#pragma unroll
      for (int i = 0; i < 4; ++i) red[wave][(4 * i + s.quad) * 16 + s.l16] = acc[i];
      __syncthreads();
      for (int k = threadIdx.x; k < sides * 256; k += sh.waves * 64) {
        float v = 0.f;
        for (int w = 0; w < sh.split; ++w) v += red[k / 256 * sh.split + w][k % 256];
        put(k / 256, k % 256, v);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) put(side, (4 * i + s.quad) * 16 + s.l16, acc[i]);
    }
  }
}

template <Kind K, int G, int U>
gsi_status launch_as(const MArgs &a, hipStream_t st) {
  using S = Stream<K, G, U>;
  static_assert(16 * S::XP * (S::C * U * S::xes + 16) <= kStreamLds, "one batch of columns fits");
  const int experts = a.n < a.R ? a.n : a.R;
  const int64_t chunks = ((int64_t)a.R + 15) / 16 + (a.offsets ? experts : 0);  // a.R + 15 may pass 2^31
  // The cheapest shape, in half batches that a wavefront goes through in a row
  // until the last chunk is done: joining a split block costs about one, and
  // x that does not fit, one part after the other, two for each part.  Then a
  // workgroup may also have the CU for itself, with fewer and longer parts (16
  // tokens through a 4-bit 16384 -> 4096 map: 63 us in parts of 1536 columns,
  // two workgroups on a CU, and 38 us in parts of 4096, one on a CU; 300 tokens
  // over 32 experts 4096 -> 1024: 61 and 70 us), of 8 wavefronts or of 16 (64
  // tokens 4096 -> 16384: 34 and 31 us; 48 tokens 16384 -> 4096: 53 and 41; 16
  // tokens 4096 -> 4096, whose blocks 16 leave on half of the CUs: 10.2 and
  // 10.4; the first map above, where 16 wavefronts would take 32 us, is one
  // that this cost gets wrong).
  const int64_t busy = a.offsets ? std::max<int64_t>(experts, a.R / 16) : chunks;  // chunks with rows, about
  // Experts with more rows than others: more and smaller workgroups than run at
  // once even that out (100 tokens, six of 128 experts each, bf16 1024 -> 2048:
  // 63 us with one round of workgroups, 48 with two, 45 with four or eight; 24
  // tokens, eight of 128 experts in 4 bits, 4096 -> 1536: 71, 45, 30 and 30).
  const int64_t uneven = a.offsets && a.R > a.n ? 4 : 1;
  const int tokens = a.R < 16 ? a.R : 16;
  const int unit = S::C * U, padded = (a.d + S::C - 1) / S::C * S::C, blocks = (a.d_out + 15) / 16;
  StreamShape sh{};
  double best = INFINITY;
  for (int mode = 0; mode < 3; ++mode) {  // two workgroups on a CU, one of 8 wavefronts, one of 16
    const bool alone = mode > 0;
    const int columns = columns_in<S, U>(alone ? kStreamLdsAlone : kStreamLds, tokens, padded);
    const int parts = (a.d + columns - 1) / columns;
    const int batches = (columns + unit - 1) / unit;
    const int waves = mode == 2 ? kStreamWaves : kStreamWaves / 2;
    const int64_t at_once = alone ? 256 : 512, want = (uneven * at_once + busy - 1) / busy;
    for (int split = 1; split <= waves && (split == 1 || split <= batches); split *= 2) {
      const int sides = waves / split, groups = (blocks + sides - 1) / sides;
      // x that fits is staged once for all of a workgroup's blocks
      const int strips = parts > 1 ? groups : (int)std::min<int64_t>(groups, want);
      const int64_t part = 2 * ((batches + split - 1) / split) + (parts > 1 ? 2 : 0);
      const int64_t turn = (groups + strips - 1) / strips * (parts * part + (split > 1 ? 1 : 0));
      // workgroups that share a CU overlap: their last round need not be full
      const double load = (double)strips * busy / at_once;
      const double cost = turn * (alone ? std::ceil(load) : std::max(1.0, load));
      if (cost < best) best = cost, sh = {split, strips, tokens * S::XP * (columns * S::xes + 16), waves};
    }
    if (parts == 1 && !alone) break;
  }
  if (chunks * sh.strips * sh.waves * 64 > kMostThreads) return GSI_E_SHAPE;
  stream_kernel<K, G, U><<<(unsigned)(chunks * sh.strips), sh.waves * 64, sh.room, st>>>(a, sh);
  return hipGetLastError() == hipSuccess ? GSI_OK : GSI_E_HIP;
}

template <Kind K>
gsi_status launch_codes(const MArgs &a, int group, hipStream_t st) {
  constexpr int U = K == kQ4F32 ? 2 : 4;  // three parts of x leave room for fewer columns in LDS
  return group == 128 ? launch_as<K, 128, U>(a, st)
                      : (group == 64 ? launch_as<K, 64, U>(a, st) : launch_as<K, 32, U>(a, st));
}

}  // namespace

gsi_status launch_stream(const MArgs &a, Kind kind, int group, hipStream_t st) {
  switch (kind) {
    case kQ4Bf16: return launch_codes<kQ4Bf16>(a, group, st);
    case kQ4F32: return launch_codes<kQ4F32>(a, group, st);
    case kBf16: return launch_as<kBf16, 128, 4>(a, st);
    default: return launch_as<kF32, 128, 4>(a, st);
  }
}

}  // namespace gsi
