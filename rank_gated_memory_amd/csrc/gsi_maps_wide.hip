// Plain linear maps with many rows per expert on gfx950 MFMA, in tiles that
// use every byte of W for many rows:
//
//   wide_kernel    : bf16, 256 x 256 tiles
//   q4_wide_kernel : 4-bit weights and bf16 x, 256 x 128 tiles
//   small_kernel   : 64 x 64 tiles, fp32 and few bf16 rows
//
// All stage their operands through LDS by direct loads, several stages ahead.
#include "gsi_maps.h"

namespace gsi {
namespace {

typedef float f32x16_t __attribute__((ext_vector_type(16)));

// The tiles of a launch.  Each expert's rows are cut into full row tiles of
// BM and one shorter rest, of one of four heights.  The full tiles are dealt
// to the 8 XCDs (workgroup b runs on XCD b % 8) in contiguous shares, so that
// workgroups that share an L2 work on neighbouring tiles: groups of kSlotGroup
// row tiles, in each all column tiles, in each the row tiles.  The rests are
// dealt one by one.  An XCD's list holds its full tiles and then its rests, the
// high ones first, so that workgroups that take them in order end together.
constexpr int kXcds = 8;
constexpr int kSlotGroup = 4;
constexpr int kHeights = 4;

struct Tile {
  int e, row, count, col;  // count 0: behind the last
};

// Row tiles of each kind: kind 0 is full, kind k a rest of at most
// (kHeights + 1 - k) quarters of BM.
struct Tiles {
  int of[kHeights + 1];
};

template <int BM>
__device__ __forceinline__ int rest_kind(int rows) {  // 0 without a rest
  const int rest = rows % BM;
  return rest ? kHeights + 1 - (rest + BM / kHeights - 1) / (BM / kHeights) : 0;
}

template <int BM>
__device__ __forceinline__ Tiles count_tiles(const MArgs &a) {
  Tiles n = {};
  for (int e0 = 0; e0 < a.n; e0 += 64) {
    int lo, hi;
    expert_rows(a, e0 + (threadIdx.x & 63), &lo, &hi);
    n.of[0] += (hi - lo) / BM;
    const int kind = rest_kind<BM>(hi - lo);
#pragma unroll
    for (int k = 1; k <= kHeights; ++k) n.of[k] += __popcll(__ballot(kind == k));
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) n.of[0] += __shfl_xor(n.of[0], o, 64);
#pragma unroll
  for (int k = 0; k <= kHeights; ++k) n.of[k] = __builtin_amdgcn_readfirstlane(n.of[k]);
  return n;
}

// The tiles of XCD `xcd`: full ones, and all.
__device__ __forceinline__ int64_t full_share(const Tiles &n, int col_tiles, int xcd, int64_t *first) {
  const int64_t tiles = (int64_t)n.of[0] * col_tiles, share = (tiles + kXcds - 1) / kXcds;
  *first = xcd * share;
  return max((int64_t)0, min(share, tiles - *first));
}

__device__ __forceinline__ int64_t all_share(const Tiles &n, int col_tiles, int xcd) {
  int64_t first, rests = 0;
#pragma unroll
  for (int k = 1; k <= kHeights; ++k) rests += n.of[k];
  return full_share(n, col_tiles, xcd, &first) + (rests * col_tiles - xcd + kXcds - 1) / kXcds;
}

// Tile number `at` of XCD `xcd`.
template <int BM>
__device__ __forceinline__ Tile find_tile(const MArgs &a, const Tiles &n, int col_tiles, int xcd, int64_t at) {
  const int lane = threadIdx.x & 63;
  if (at >= all_share(n, col_tiles, xcd)) return {0, 0, 0, 0};
  int64_t first;
  const int64_t mine = full_share(n, col_tiles, xcd, &first);
  int kind = 0, slot, col;
  if (at < mine) {
    const int64_t t = first + at;
    const int g = (int)(t / (kSlotGroup * col_tiles)), in = (int)(t - (int64_t)g * kSlotGroup * col_tiles);
    const int wide = min(kSlotGroup, n.of[0] - g * kSlotGroup);
    slot = g * kSlotGroup + in % wide;
    col = in / wide;
  } else {
    const int64_t t = (at - mine) * kXcds + xcd;
    slot = (int)(t / col_tiles);
    col = (int)(t - (int64_t)slot * col_tiles);
    for (kind = 1; kind < kHeights && slot >= n.of[kind]; ++kind) slot -= n.of[kind];
  }
  int before = 0;
  for (int e0 = 0; e0 < a.n; e0 += 64) {
    int lo, hi;
    expert_rows(a, e0 + lane, &lo, &hi);
    const int has = kind == 0 ? (hi - lo) / BM : rest_kind<BM>(hi - lo) == kind;
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
      const int skip = kind == 0 ? k * BM : rows / BM * BM;
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

// Every wavefront's own loads but the last N have landed, then all wavefronts'.
// Loads return in order, so N may count any load issued since those that are
// waited for; it must not be more than there are (a test counts them in the
// compiled code).
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
// tile into the next.  Bound by the matrix cores and the clock they leave (one
// 8192^3 product: 1140 to 1180 TFLOP/s, MFMA busy 61 % of the cycles at 1.76 GHz).
// 4096 tokens, four of 32 ragged experts each, 2048 -> 4096: 275 GFLOP in 325
// to 350 us; with as many rows for every expert 305 (before the order of the
// tiles was tuned: two stages of 64 columns 3 % slower than four of 32, loads
// through registers 11 %).
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

// A workgroup for every CU.  The workgroups of an XCD take its list in turn,
// every second turn from the other end, which gives each about the same; XCDs
// with odd numbers walk their turns backwards, so that low rests, which are
// bound by the weights from HBM, run beside full tiles of other XCDs, which are
// not (the ragged prompt above: 375 us with the list taken in order, 350 so;
// every second workgroup backwards instead of every second XCD parts
// neighbours that share an L2: 302 -> 365 us with even experts).
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
  const int xcd = blockIdx.x % kXcds, me = blockIdx.x / kXcds, all = gridDim.x / kXcds;
  const int64_t tiles = all_share(n, col_tiles, xcd), turns = (tiles + all - 1) / all;
  const auto tile_of = [&](int64_t k) -> Tile {  // of this workgroup's turn k
    if (k >= turns) return {0, 0, 0, 0};
    const int64_t r = xcd & 1 ? turns - 1 - k : k;
    return find_tile<kWideBM>(a, n, col_tiles, xcd, r * all + (r & 1 ? all - 1 - me : me));
  };
  int64_t k = 0;
  Tile tl = tile_of(0);
  if (tl.count <= 0) tl = tile_of(k = 1);  // the last turn is not for all
  if (tl.count <= 0) return;
  WideSource f = wide_source(a, tl, wave, lane);
  wide_fetch(f, lds0, wave);
  wide_fetch(f, lds1, wave);
  wide_fetch(f, lds2, wave);
  landed<kWideLoads>();
  for (;;) {
    const Tile next = tile_of(++k);
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

// 4-bit weights: tiles of 256 tokens x 128 weight rows on 8 wavefronts, 4 x 2
// of them, each 32 TM tokens x 64 weight rows.  x arrives in LDS as above; the
// codes go through registers, 64 bytes of each weight row at a time, and are
// decoded once for all 256 tokens, to q - z, which bf16 holds exactly.  Every
// group has a sum of its own in the matrix core's accumulators and is added
// to the fp32 total with the group's scale, so nothing is rounded but fp32
// sums.  Here A holds tokens and B weight rows: a lane's accumulators belong
// to one weight row of each block and take one scale.  Bound by issue: the
// decoding and the scaling of the group sums run beside the products (2047
// tokens 4096 -> 16384, groups of 128: 275 GFLOP in 324 us, 850 TFLOP/s, MFMA
// busy 35 %; 764 us in the streaming kernel).
constexpr int kQ4BN = 128;
constexpr int kQ4X = kWideBM * kWideBK * 2, kQ4W = kQ4BN * kWideBK * 2;  // bytes of a stage

// A stage's x and W, objects of their own: the compiler lets a store to LDS
// wait for every load to LDS that may go to the same object.
struct Q4Stage {
  uint8_t *x, *w;
};

template <int G, int TM>
__device__ __forceinline__ void q4_tile(const MArgs &a, const Tile &tl, const Q4Stage &lds0, const Q4Stage &lds1,
                                        const Q4Stage &lds2, const Q4Stage &lds3) {
  constexpr int TN = 2, kBlock = 32 * kWideBK * 2, NG = 128 / G;  // groups of 128 columns
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, l32 = lane & 31, half = lane >> 5;
  const int i0 = tl.col * kQ4BN;

  // x: two loads to LDS of a wavefront per stage
  const int sub = lane >> 2, piece = ((lane & 3) ^ swizzle<kWideBK>(sub)) * 8;
  const uint8_t *xp[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = tl.row + min((wave * 2 + i) * 16 + sub, tl.count - 1);
    const int src = a.rows ? a.rows[r] : r;
    xp[i] = a.x + ((int64_t)(src < 0 || src >= a.T ? 0 : src) * a.ldx + piece) * 2;
  }
  int left = a.d - piece;
  const uint64_t zero_page = reinterpret_cast<uint64_t>(&kZeros);
  const auto fetch = [&](const Q4Stage &st) {
    const uint64_t in = (int64_t)(-left) >> 63;  // all ones while left > 0
    left -= kWideBK;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      to_lds(reinterpret_cast<const void *>((reinterpret_cast<uint64_t>(xp[i]) & in) | (zero_page & ~in)),
             st.x + (wave * 2 + i) * 1024);
      xp[i] += 2 * kWideBK;
    }
  };

  // Codes: this thread's 16 bytes of weight row tid / 4, columns 32 (tid % 4)
  // on of each 128, and the zeros of their groups.  Behind d it reads the
  // row's first bytes and the last group's zero: x is zero there.
  const int wr = tid >> 2, part = tid & 3, row_bytes = a.d / 2;
  const int64_t row = (int64_t)tl.e * a.d_out + min(i0 + wr, a.d_out - 1);
  const uint8_t *const cp = a.W + tl.e * a.w_stride + (int64_t)min(i0 + wr, a.d_out - 1) * row_bytes;
  // without zeros as many bytes of the scales are read and dropped: a step's
  // wait counts its loads
  const uint8_t *const zp = (a.zeros ? a.zeros : a.scales) + row * a.groups;
  struct Codes {
    u32x4_t c;
    uint32_t z[NG];
  };
  const auto load_codes = [&](Codes &o, int n) {
    const int at = n * 64 + 16 * part;
    o.c = *reinterpret_cast<const u32x4_t *>(cp + (at < row_bytes ? at : 0));
#pragma unroll
    for (int g = 0; g < NG; ++g) o.z[g] = zp[min(n * NG + g, a.groups - 1)];
  };
  // Stage s of 128 columns: its 32 codes of the row lie with lane s of the
  // row's four lanes, dword p for lane p.
  uint32_t mine[4];  // all ones for this lane's dword
#pragma unroll
  for (int p = 0; p < 4; ++p) mine[p] = part == p ? ~0u : 0u;
  const auto decode_to = [&](const Q4Stage &st, const Codes &o, auto sc) {
    constexpr int s = decltype(sc)::value, kPerm = s * 0x55;  // every lane of four reads lane s
    uint32_t c = 0;
#pragma unroll
    for (int p = 0; p < 4; ++p) c |= __builtin_amdgcn_mov_dpp(o.c[p], kPerm, 0xf, 0xf, true) & mine[p];
    const float z = a.zeros ? (float)(o.z[s * 32 / G] & 15) : 8.f;
    const uint32_t even = c & 0x0f0f0f0fu, odd = c >> 4 & 0x0f0f0f0fu;
    u32x4_t w;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float lo = (float)(even >> (8 * k) & 255) - z, hi = (float)(odd >> (8 * k) & 255) - z;
      w[k] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
    }
    *reinterpret_cast<u32x4_t *>(st.w + tile_at<kWideBK>(wr, part)) = w;
  };

  // scales of this lane's weight rows
  const uint16_t *sp[TN];
#pragma unroll
  for (int i = 0; i < TN; ++i)
    sp[i] = reinterpret_cast<const uint16_t *>(a.scales) +
            ((int64_t)tl.e * a.d_out + min(i0 + wn * 64 + i * 32 + l32, a.d_out - 1)) * a.groups;
  const auto load_scales = [&](uint32_t (&o)[NG][TN], int n) {
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int i = 0; i < TN; ++i) o[g][i] = sp[i][min(n * NG + g, a.groups - 1)];
  };

  f32x16_t total[TN][TM] = {}, sum[TN][TM];
  int xat[2], wat[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    xat[s] = wm * TM * kBlock + tile_at<kWideBK>(l32, 2 * s + half);
    wat[s] = wn * TN * kBlock + tile_at<kWideBK>(l32, 2 * s + half);
  }
  bf16x8_t wf[2][TN], xf[2][TM];
  const auto read = [&](const Q4Stage &st, int s) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
      wf[s][j] = as_bf16x8(*reinterpret_cast<const u32x4_t *>(st.w + wat[s] + j * kBlock));
#pragma unroll
    for (int j = 0; j < TM; ++j)
      xf[s][j] = as_bf16x8(*reinterpret_cast<const u32x4_t *>(st.x + xat[s] + j * kBlock));
  };
  const auto multiply = [&](int s, auto first) {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
    const f32x16_t none = {};
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
      for (int i = 0; i < TN; ++i)
        sum[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xf[s][j], wf[s][i], decltype(first)::value ? none : sum[i][j],
                                                            0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
  };
  uint32_t sc[NG][TN];
  // Step s of 128 columns, as in wide_tile; N loads of its own may be under
  // way when it ends.
  const auto step = [&](auto sc_, const Q4Stage &cur, const Q4Stage &next, const Q4Stage &fill, const Codes &o,
                        auto n) {
    constexpr int s = decltype(sc_)::value, per = G / 32;
    read(cur, 1);
    multiply(0, std::integral_constant<bool, s % per == 0>{});
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    fetch(fill);
    decode_to(fill, o, std::integral_constant<int, (s + 3) % 4>{});
    read(next, 0);
    multiply(1, std::false_type{});
    if constexpr ((s + 1) % per == 0) {
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        const float f = __uint_as_float(sc[s / per][i] << 16);
#pragma unroll
        for (int j = 0; j < TM; ++j) {
#pragma unroll
          for (int e = 0; e < 16; ++e) total[i][j][e] += f * sum[i][j][e];
          asm volatile("" : "+v"(total[i][j]));  // here: the compiler would carry the sums on
        }
      }
    }
    landed<decltype(n)::value>();
  };

  constexpr int kOwn = 2, kMore = 1 + NG + NG * TN;  // loads of a step; of codes, zeros and scales
  const int rounds = (a.d + 127) / 128;
  Codes c0, c1, c2;
  load_codes(c0, 0);
  load_codes(c1, 1);
  load_scales(sc, 0);
  fetch(lds0);
  fetch(lds1);
  fetch(lds2);
  decode_to(lds0, c0, std::integral_constant<int, 0>{});
  decode_to(lds1, c0, std::integral_constant<int, 1>{});
  decode_to(lds2, c0, std::integral_constant<int, 2>{});
  landed<0>();
  read(lds0, 0);
  for (int n = 0; n < rounds; ++n) {
    uint32_t sn[NG][TN];
    load_codes(c2, n + 2);
    load_scales(sn, n + 1);
    step(std::integral_constant<int, 0>{}, lds0, lds1, lds3, c0, std::integral_constant<int, kOwn + kMore>{});
    step(std::integral_constant<int, 1>{}, lds1, lds2, lds0, c1, std::integral_constant<int, kOwn>{});
    step(std::integral_constant<int, 2>{}, lds2, lds3, lds1, c1, std::integral_constant<int, kOwn>{});
    step(std::integral_constant<int, 3>{}, lds3, lds0, lds2, c1, std::integral_constant<int, kOwn>{});
    c0 = c1;
    c1 = c2;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int i = 0; i < TN; ++i) sc[g][i] = sn[g][i];
  }
  landed<0>();

#pragma unroll
  for (int j = 0; j < TM; ++j)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int m = (wm * TM + j) * 32 + 8 * (e / 4) + 4 * half + e % 4;
      if (m >= tl.count) continue;
      const int r = tl.row + m;
      const int src = a.rows ? a.rows[r] : r;
      const bool has = src >= 0 && src < a.T;
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        const int o = i0 + wn * 64 + i * 32 + l32;
        if (o < a.d_out) reinterpret_cast<__bf16 *>(a.y)[r * a.ldy + o] = has ? (__bf16)total[i][j][e] : (__bf16)0.f;
      }
    }
}

template <int G>
__global__ void __launch_bounds__(512) q4_wide_kernel(MArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t x0[kQ4X], x1[kQ4X], x2[kQ4X], x3[kQ4X];
  __shared__ __attribute__((aligned(1024))) uint8_t w0[kQ4W], w1[kQ4W], w2[kQ4W], w3[kQ4W];
  const Tiles n = count_tiles<kWideBM>(a);
  const Tile tl = find_tile<kWideBM>(a, n, (a.d_out + kQ4BN - 1) / kQ4BN, blockIdx.x % kXcds, blockIdx.x / kXcds);
  if (tl.count <= 0) return;
  if (tl.count > 128)
    q4_tile<G, 2>(a, tl, {x0, w0}, {x1, w1}, {x2, w2}, {x3, w3});
  else
    q4_tile<G, 1>(a, tl, {x0, w0}, {x1, w1}, {x2, w2}, {x3, w3});
}

// Small tiles: 64 tokens x 64 weight rows on four wavefronts, 2 x 2 of them,
// each 32 x 32, for fp32 (whose products are slow enough to be bound by them
// at any tile) and for bf16 with too few large tiles for the chip.  Several
// workgroups share a CU.  A stage is 64 bytes of each row; the 16 bytes that a
// lane reads of a row are one operand of 8 columns in bf16 and four of one
// column in fp32, lanes 32 to 63 taking the other columns.  A tile of at most
// 32 tokens has each pair of wavefronts take half of every stage, and their
// sums joined (200 tokens, four of 8 experts each, fp32 2048 -> 2048: 99 us with
// the second half of the tokens idle, 89 so; tiles of 32 tokens throughout: 96).
// fp32 is bound by its products where there are rows enough (333 tokens, three
// of 8 ragged experts each, 1000 -> 1208: 2.4 GFLOP in 38 us, 63 TFLOP/s of the
// 135 that a large product reaches; MFMA busy 33 %; 96 us in the streaming
// kernel).
constexpr int kSmallB = 64;
constexpr int kSmallStage = 2 * kSmallB * 64;

template <bool F32>
__global__ void __launch_bounds__(256) small_kernel(MArgs a) {
  constexpr int es = F32 ? 4 : 2, C = 64 / es;  // columns of a stage
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[kSmallStage];
  __shared__ __attribute__((aligned(1024))) uint8_t lds1[kSmallStage];
  __shared__ __attribute__((aligned(1024))) uint8_t lds2[kSmallStage];
  __shared__ __attribute__((aligned(1024))) uint8_t lds3[kSmallStage];
  const Tiles n = count_tiles<kSmallB>(a);
  const Tile tl =
      find_tile<kSmallB>(a, n, (a.d_out + kSmallB - 1) / kSmallB, blockIdx.x % kXcds, blockIdx.x / kXcds);
  if (tl.count <= 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1, l32 = lane & 31, half = lane >> 5;
  const int i0 = tl.col * kSmallB;

  // a KiB of x and a KiB of W of each stage
  const int sub = lane >> 2, piece = ((lane & 3) ^ swizzle<32>(sub)) * 16, m0 = wave * 16 + sub;
  const uint8_t *xp, *wp;
  {
    const int r = tl.row + min(m0, tl.count - 1);
    const int src = a.rows ? a.rows[r] : r;
    xp = a.x + (int64_t)(src < 0 || src >= a.T ? 0 : src) * a.ldx * es + piece;
    wp = a.W + tl.e * a.w_stride + (int64_t)min(i0 + m0, a.d_out - 1) * a.d * es + piece;
  }
  int left = a.d * es - piece;  // bytes from this lane's next piece to the row's end
  const uint64_t zeros = reinterpret_cast<uint64_t>(&kZeros);
  const auto fetch = [&](uint8_t *st) {
    const uint64_t in = (int64_t)(-left) >> 63;
    left -= 64;
    to_lds(reinterpret_cast<const void *>((reinterpret_cast<uint64_t>(xp) & in) | (zeros & ~in)), st + wave * 1024);
    to_lds(reinterpret_cast<const void *>((reinterpret_cast<uint64_t>(wp) & in) | (zeros & ~in)),
           st + kSmallB * 64 + wave * 1024);
    xp += 64;
    wp += 64;
  };

  f32x16_t acc = {};
  // where the operands of half a stage lie; in a low tile both halves of the
  // wavefronts have the same tokens and each its own half of every stage
  const bool low = tl.count <= 32;
  int xat[2], wat[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    xat[s] = (low ? 0 : wm * 2048) + tile_at<32>(l32, 2 * s + half);
    wat[s] = kSmallB * 64 + wn * 2048 + tile_at<32>(l32, 2 * s + half);
  }
  u32x4_t wf[2], xf[2];
  const auto read = [&](const uint8_t *st, int s) {
    wf[s] = *reinterpret_cast<const u32x4_t *>(st + wat[s]);
    xf[s] = *reinterpret_cast<const u32x4_t *>(st + xat[s]);
  };
  const auto multiply = [&](int s) {
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(wf[s][i]), __uint_as_float(xf[s][i]), acc, 0, 0, 0);
    } else {
      acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(wf[s]), as_bf16x8(xf[s]), acc, 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  const auto step = [&](const uint8_t *cur, const uint8_t *next, uint8_t *fill) {  // as in wide_tile
    read(cur, 1);
    multiply(0);
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    fetch(fill);
    read(next, 0);
    multiply(1);
    landed<2>();
  };
  // of a low tile: registers p hold this stage, the others take the next
  const int mine = xat[wm], mine_w = wat[wm];
  const auto read_low = [&](const uint8_t *st, int p) {
    wf[p] = *reinterpret_cast<const u32x4_t *>(st + mine_w);
    xf[p] = *reinterpret_cast<const u32x4_t *>(st + mine);
  };
  const auto step_low = [&](int p, const uint8_t *next, uint8_t *fill) {
    fetch(fill);
    read_low(next, 1 - p);
    multiply(p);
    landed<2>();
  };
  fetch(lds0);
  fetch(lds1);
  fetch(lds2);
  landed<2>();
  if (low) {
    read_low(lds0, 0);
    for (int k = 0; k < a.d; k += 4 * C) {
      step_low(0, lds1, lds3);
      step_low(1, lds2, lds0);
      step_low(0, lds3, lds1);
      step_low(1, lds0, lds2);
    }
  } else {
    read(lds0, 0);
    for (int k = 0; k < a.d; k += 4 * C) {
      step(lds0, lds1, lds3);
      step(lds1, lds2, lds0);
      step(lds2, lds3, lds1);
      step(lds3, lds0, lds2);
    }
  }
  landed<0>();

  if (low) {  // the sums of the second halves, in the room of a stage
    static_assert(2 * 16 * 64 * 4 <= kSmallStage);
    float *const other = reinterpret_cast<float *>(lds0) + wn * (16 * 64) + lane;
    if (wm) {
#pragma unroll
      for (int i = 0; i < 16; ++i) other[i * 64] = acc[i];
    }
    landed<0>();
    if (wm) return;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] += other[i * 64];
  }
  const int m = wm * 32 + l32;
  if (m >= tl.count) return;
  const int r = tl.row + m, src = a.rows ? a.rows[r] : r;
  const bool has = src >= 0 && src < a.T;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int o = i0 + wn * 32 + 8 * q + 4 * half;
    if (o >= a.d_out) continue;
    f32x4_t v = {acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
    if (!has) v = f32x4_t{0, 0, 0, 0};
    uint8_t *const yp = a.y + (r * a.ldy + o) * es;
    if constexpr (F32) {
      *reinterpret_cast<f32x4_t *>(yp) = v;
    } else {
      typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
      *reinterpret_cast<bf16x4_t *>(yp) = bf16x4_t{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
    }
  }
}

}  // namespace

gsi_status launch_wide(const MArgs &a, hipStream_t st) {
  constexpr int kCus = 256;
  wide_kernel<<<kCus, 512, 0, st>>>(a);
  return hipGetLastError() == hipSuccess ? GSI_OK : GSI_E_HIP;
}

gsi_status launch_wide_q4(const MArgs &a, int group, hipStream_t st) {
  // full tiles and rests: at most R / 256 of the ones and one rest per expert
  // with rows, each list rounded up to whole shares
  const int64_t slots = a.R / kWideBM + (a.n < a.R ? a.n : a.R);
  const int64_t grid = (slots * ((a.d_out + kQ4BN - 1) / kQ4BN) + 2 * kXcds) / kXcds * kXcds;
  if (grid * 512 > kMostThreads) return GSI_E_SHAPE;
  if (group == 128)
    q4_wide_kernel<128><<<(unsigned)grid, 512, 0, st>>>(a);
  else if (group == 64)
    q4_wide_kernel<64><<<(unsigned)grid, 512, 0, st>>>(a);
  else
    q4_wide_kernel<32><<<(unsigned)grid, 512, 0, st>>>(a);
  return hipGetLastError() == hipSuccess ? GSI_OK : GSI_E_HIP;
}

gsi_status launch_small(const MArgs &a, Kind kind, hipStream_t st) {
  const int64_t slots = a.R / kSmallB + (a.n < a.R ? a.n : a.R);
  const int64_t grid = (slots * ((a.d_out + kSmallB - 1) / kSmallB) + 2 * kXcds) / kXcds * kXcds;
  if (grid * 256 > kMostThreads) return GSI_E_SHAPE;
  if (kind == kF32)
    small_kernel<true><<<(unsigned)grid, 256, 0, st>>>(a);
  else
    small_kernel<false><<<(unsigned)grid, 256, 0, st>>>(a);
  return hipGetLastError() == hipSuccess ? GSI_OK : GSI_E_HIP;
}

}  // namespace gsi
