// Rotary positions and appending to the paged cache (gsi_rotary,
// gsi_cache_append): one kernel that turns rows of heads and writes them to
// rows or to the pages.
#include "gsi_cache.h"

namespace gsi {
namespace {

constexpr int kThreads = 256;
constexpr int kMostPairs = 128;
constexpr int kMostTokens = 8;  // of a workgroup

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

// A workgroup's items one after the other: the units of its tokens' query heads,
// of their key heads and of their value heads.  Queries go token by token, as
// their rows lie; keys and values head by head, each for all tokens, so that
// entries that lie side by side in a page are written together (4939 tokens of
// 16 heads of 256 into pages of 32: 59 and 54 us).
struct Split {
  Div turn_units, copy_units;   // of a head that is turned, and of one that is copied
  Div q_heads;
  int tokens;                   // of a workgroup
  int strips;                   // workgroups that share them
  int q_items, k_items, items;  // of a token: queries' end, keys' end, values' end
};

// What a workgroup's tokens share: amplitude times cos and sin of their angles,
// and where their entries lie.
struct Tokens {
  float2 turn[kMostTokens][kMostPairs];
  int64_t entry[kMostTokens];   // bytes from K (V) to head 0's entry
  int64_t number[kMostTokens];  // of head 0 in mass and age
  bool has[kMostTokens];
};

__device__ __forceinline__ int64_t position_of(const RotateArgs &a, int t) {
  return a.pos_bytes == 8 ? static_cast<const int64_t *>(a.positions)[t]
                          : (int64_t) static_cast<const int32_t *>(a.positions)[t];
}

__device__ __forceinline__ void prepare(const RotateArgs &a, Tokens &k, int t0, int tokens, bool first) {
  const int pairs = a.turned / 2, tid = threadIdx.x;
  if (a.slots && tid < tokens) {
    const int row = t0 + tid, s = a.seq ? a.seq[row] : row, slot = a.slots[row];
    int page = -1;
    if (s >= 0 && s < a.c.S && slot >= 0 && slot < a.c.most << a.c.shift) page = page_of(a.c, s, slot);
    k.has[tid] = page >= 0;
    k.entry[tid] = entry_at(a.c, max(page, 0), 0, slot);
    k.number[tid] = number_at(a.c, max(page, 0), 0, slot);
  }
  for (int i = tid; i < tokens * pairs; i += kThreads) {
    const int t = i / pairs, pair = i - t * pairs;
    // In turns, and of these the part of one turn: p * f has the rounding of
    // f alone, so an angle at position p is off by p f 2^-52 at most, and the
    // fp32 sine and cosine see a number in [-1, 1].
    const double p = (double)position_of(a, t0 + t), f = a.freq[pair] * 0.15915494309189533577;
    const float r = (float)(2.0 * fma(p, f, -rint(p * f)));
    float s, c;
    sincospif(r, &s, &c);
    k.turn[t][pair] = make_float2(a.amplitude * c, a.amplitude * s);
  }
  __syncthreads();
  if (!a.slots || !first) return;
  for (int i = tid; i < tokens * a.c.heads; i += kThreads) {
    const int t = i / a.c.heads, h = i - t * a.c.heads, row = t0 + t;
    if (!k.has[t]) continue;
    const int64_t at = k.number[t] + ((int64_t)h << a.c.shift);
    if (a.c.mass) a.c.mass[at] = 0.f;
    if (a.c.age)
      a.c.age[at] = a.positions ? (int32_t)min(max(position_of(a, row), (int64_t)INT32_MIN), (int64_t)INT32_MAX)
                                : a.slots[row];
  }
}

// An item's token, head and unit; to is null where there is nothing to do.
struct Item {
  const uint8_t *from;
  uint8_t *to;
  int t, unit;
  bool turns;
};

__device__ __forceinline__ Item item_of(const RotateArgs &a, const Split &sp, const Tokens &k, int t0, int tokens,
                                        int item) {
  Item r;
  const bool query = item < tokens * sp.q_items, key = item < tokens * sp.k_items;
  const Div du = key ? sp.turn_units : sp.copy_units;
  const int at = item - tokens * (query ? 0 : key ? sp.q_items : sp.k_items), line = quotient(at, du);
  const int along = tokens == 1 ? line : tokens == kMostTokens ? line / kMostTokens : line / tokens;
  const int before = quotient(line, sp.q_heads);
  const int h = query ? line - before * sp.q_heads.by : along;
  const Rows &src = query ? a.q : key ? a.k : a.v;
  r.unit = at - line * du.by;
  r.t = query ? before : line - along * tokens;
  r.turns = key;
  r.from = src.p + (t0 + r.t) * src.row + h * src.head;
  if (query)
    r.to = a.qo.p + (t0 + r.t) * a.qo.row + h * a.qo.head;
  else
    r.to = k.has[r.t] ? (key ? a.c.K : a.c.V) + k.entry[r.t] + h * a.c.head_stride : nullptr;
  return r;
}

// Bound by HBM for many tokens (8191 of 40 heads of 128: 168 MB in 30 us, 5.6
// TB/s; 4939 of 16 heads of 256 with their keys and values into the pages: 243
// MB), by latency for few: the position, the sine and cosine, the head.  The
// angles are formed once for all heads of a token.
template <typename E, bool Halves>
__global__ void __launch_bounds__(kThreads, 8) rotate_kernel(RotateArgs a, Split sp) {
  __shared__ Tokens k;
  constexpr int es = sizeof(E), V = 16 / es;
  constexpr int kAhead = Halves ? 2 : 4;  // items of a thread under way, of two pieces and of one
  typedef E vec __attribute__((ext_vector_type(V)));
  const int group = blockIdx.x / sp.strips, strip = blockIdx.x - group * sp.strips;
  const int t0 = group * sp.tokens, tokens = min(sp.tokens, a.T - t0), pairs = a.turned / 2;
  prepare(a, k, t0, tokens, strip == 0);
  const int all = tokens * sp.items, step = sp.strips * kThreads;
  for (int i0 = strip * kThreads + threadIdx.x; i0 < all; i0 += kAhead * step) {
    uint8_t *to[kAhead];
    u32x4_t x0[kAhead], x1[kAhead];
    int at[kAhead], turn[kAhead];  // of the (first) piece, and its first pair or -1
    const float2 *w[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j * step;
      to[j] = nullptr;
      x0[j] = x1[j] = u32x4_t{0, 0, 0, 0};
      at[j] = 0;
      turn[j] = -1;
      w[j] = k.turn[0];
      if (i >= all) continue;
      const Item it = item_of(a, sp, k, t0, tokens, i);
      w[j] = k.turn[it.t];
      to[j] = it.to;
      at[j] = it.unit * 16;
      if (it.turns) {
        if constexpr (Halves) {  // two pieces, or a piece of those that stay
          const int half = pairs / V;
          if (it.unit < half) {
            at[j] = (a.start + it.unit * V) * es;
            turn[j] = it.unit * V;
          } else {
            const int e = (it.unit - half) * V;
            at[j] = (e < a.start ? e : e + a.turned) * es;
          }
        } else {
          const int e = it.unit * V - a.start;
          if (e >= 0 && e < a.turned) turn[j] = e / 2;
        }
        if (turn[j] < 0 && it.from == it.to) to[j] = nullptr;  // in place
      }
      if (!to[j]) continue;
      x0[j] = *reinterpret_cast<const u32x4_t *>(it.from + at[j]);
      if (Halves && turn[j] >= 0) x1[j] = *reinterpret_cast<const u32x4_t *>(it.from + at[j] + pairs * es);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (!to[j]) continue;
      if (turn[j] >= 0) {
        const float2 *const u = w[j] + turn[j];
        const vec a0 = __builtin_bit_cast(vec, x0[j]), a1 = __builtin_bit_cast(vec, x1[j]);
        vec y0, y1;
        if constexpr (Halves) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            y0[e] = (E)((float)a0[e] * u[e].x - (float)a1[e] * u[e].y);
            y1[e] = (E)((float)a1[e] * u[e].x + (float)a0[e] * u[e].y);
          }
          *reinterpret_cast<vec *>(to[j] + at[j] + pairs * es) = y1;
        } else {
#pragma unroll
          for (int e = 0; e < V; e += 2) {
            y0[e] = (E)((float)a0[e] * u[e / 2].x - (float)a0[e + 1] * u[e / 2].y);
            y0[e + 1] = (E)((float)a0[e + 1] * u[e / 2].x + (float)a0[e] * u[e / 2].y);
          }
        }
        x0[j] = __builtin_bit_cast(u32x4_t, y0);
      }
      *reinterpret_cast<u32x4_t *>(to[j] + at[j]) = x0[j];
    }
  }
}

// The same where pieces of 16 bytes do not end where the turned part does: a
// unit is a pair, or an element of those that stay.
template <typename E, bool Halves>
__global__ void __launch_bounds__(kThreads) rotate_elements_kernel(RotateArgs a, Split sp) {
  __shared__ Tokens k;
  const int group = blockIdx.x / sp.strips, strip = blockIdx.x - group * sp.strips;
  const int t0 = group * sp.tokens, tokens = min(sp.tokens, a.T - t0), pairs = a.turned / 2;
  prepare(a, k, t0, tokens, strip == 0);
  const int all = tokens * sp.items, step = sp.strips * kThreads;
  for (int i = strip * kThreads + threadIdx.x; i < all; i += step) {
    const Item it = item_of(a, sp, k, t0, tokens, i);
    if (!it.to) continue;
    const E *const from = reinterpret_cast<const E *>(it.from);
    E *const to = reinterpret_cast<E *>(it.to);
    if (!it.turns) {
      reinterpret_cast<u32x4_t *>(to)[it.unit] = reinterpret_cast<const u32x4_t *>(from)[it.unit];
    } else if (it.unit < pairs) {
      const int i0 = a.start + (Halves ? it.unit : 2 * it.unit), i1 = i0 + (Halves ? pairs : 1);
      const float2 u = k.turn[it.t][it.unit];
      const float x0 = (float)from[i0], x1 = (float)from[i1];
      to[i0] = (E)(x0 * u.x - x1 * u.y);
      to[i1] = (E)(x1 * u.x + x0 * u.y);
    } else if (from != to) {
      const int e = it.unit - pairs, at = e < a.start ? e : e + a.turned;
      to[at] = from[at];
    }
  }
}

template <typename E, bool Halves>
gsi_status launch_as(const RotateArgs &a, bool whole, hipStream_t st) {
  constexpr int V = 16 / sizeof(E);
  const int pairs = a.turned / 2, copies = a.d / V;
  const int turn_units = !whole ? a.d - pairs : Halves ? copies - pairs / V : copies;
  Split sp{};
  sp.turn_units = div_by(turn_units);
  sp.copy_units = div_by(copies);
  sp.q_heads = div_by(a.q.n > 0 ? a.q.n : 1);
  sp.q_items = a.q.n * turn_units;
  sp.k_items = sp.q_items + a.k.n * turn_units;
  sp.items = sp.k_items + a.v.n * copies;
  // Tokens share a workgroup where there are enough of them to fill the chip.
  sp.tokens = a.T >= 2048 ? kMostTokens : 1;
  const int64_t groups = ((int64_t)a.T + sp.tokens - 1) / sp.tokens;
  const int64_t per = ((int64_t)sp.tokens * sp.items + kThreads - 1) / kThreads;
  const int64_t most = 2048 / groups > 1 ? 2048 / groups : 1;
  sp.strips = (int)(per < most ? per : most);
  if (groups * sp.strips * kThreads > kMostLaunch) return GSI_E_SHAPE;
  const unsigned grid = (unsigned)(groups * sp.strips);
  if (whole)
    rotate_kernel<E, Halves><<<grid, kThreads, 0, st>>>(a, sp);
  else
    rotate_elements_kernel<E, Halves><<<grid, kThreads, 0, st>>>(a, sp);
  return hipGetLastError() == hipSuccess ? GSI_OK : GSI_E_HIP;
}

template <typename E>
gsi_status launch_of(const RotateArgs &a, int layout, hipStream_t st) {
  constexpr int V = 16 / sizeof(E);
  const bool halves = layout == GSI_ROTARY_HALVES;
  const bool whole = a.start % V == 0 && (halves ? a.turned / 2 : a.turned) % V == 0;
  return halves ? launch_as<E, true>(a, whole, st) : launch_as<E, false>(a, whole, st);
}

}  // namespace

gsi_status launch_rotate(const RotateArgs &a, int dtype, int layout, hipStream_t st) {
  return dtype == GSI_FP32 ? launch_of<float>(a, layout, st) : launch_of<__bf16>(a, layout, st);
}

}  // namespace gsi
