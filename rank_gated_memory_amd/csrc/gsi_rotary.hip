// Rotary positions and appending to the paged cache (gsi_rotary,
// gsi_cache_append): one kernel that turns rows of heads and writes them to
// rows or to the pages.
#include <type_traits>

#include "gsi_cache.h"

namespace gsi {
namespace {

constexpr int kThreads = 256;
constexpr int kMostPairs = 128;

// A 16-byte piece of a head in fp32, and single elements.
template <typename E, int V>
struct Piece {
  typedef E vec __attribute__((ext_vector_type(V)));
  static __device__ __forceinline__ void load(const uint8_t *p, float (&v)[V]) {
    const vec u = *reinterpret_cast<const vec *>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = (float)u[i];
  }
  static __device__ __forceinline__ void store(uint8_t *p, const float (&v)[V]) {
    vec u;
#pragma unroll
    for (int i = 0; i < V; ++i) u[i] = (E)v[i];
    *reinterpret_cast<vec *>(p) = u;
  }
  static __device__ __forceinline__ void copy(uint8_t *to, const uint8_t *from) {
    *reinterpret_cast<vec *>(to) = *reinterpret_cast<const vec *>(from);
  }
};
template <typename E>
struct Piece<E, 1> {
  static __device__ __forceinline__ void copy(uint8_t *to, const uint8_t *from) {
    *reinterpret_cast<E *>(to) = *reinterpret_cast<const E *>(from);
  }
};

struct Split {
  Div turn_units, copy_units, heads_q, heads_k;
  int tokens;   // of a workgroup
  int strips;   // workgroups that share them
  int q_items, k_items, items;  // of a token: queries end, keys end, values end
};

// V: elements of a 16-byte piece, or 1 where pieces do not end where the turned
// part does.
template <typename E, int V, bool Halves>
__global__ void __launch_bounds__(kThreads) rotate_kernel(RotateArgs a, Split sp) {
  __shared__ float2 turn[4][kMostPairs];  // amplitude times cos and sin of a token's angles
  constexpr int es = sizeof(E);
  const int group = blockIdx.x / sp.strips, strip = blockIdx.x - group * sp.strips;
  const int t0 = group * sp.tokens, tokens = min(sp.tokens, a.T - t0), pairs = a.turned / 2;
  const auto position = [&](int t) {
    return a.pos_bytes == 8 ? static_cast<const int64_t *>(a.positions)[t]
                            : (int64_t) static_cast<const int32_t *>(a.positions)[t];
  };
  for (int k = threadIdx.x; k < tokens * pairs; k += kThreads) {
    const int t = k / pairs, i = k - t * pairs;
    // In turns, and of these the part of one turn: p * f has the rounding of
    // f alone, so an angle at position p is off by p f 2^-52 at most, and the
    // fp32 sine and cosine see a number in [-1/2, 1/2].
    const double p = (double)position(t0 + t), f = a.freq[i] * 0.15915494309189533577;
    const float r = (float)(2.0 * fma(p, f, -rint(p * f)));
    float s, c;
    sincospif(r, &s, &c);
    turn[t][i] = make_float2(a.amplitude * c, a.amplitude * s);
  }
  __syncthreads();
  for (int k = strip * kThreads + threadIdx.x; k < tokens * sp.items; k += sp.strips * kThreads) {
    const int t = k / sp.items, item = k - t * sp.items, row = t0 + t;
    // the head and the unit, where they come from and go to
    const uint8_t *from;
    uint8_t *to;
    int unit;
    bool turns = true;
    if (item < sp.q_items) {
      const int h = quotient(item, sp.turn_units);
      unit = item - h * sp.turn_units.by;
      from = a.q.p + row * a.q.row + h * a.q.head;
      to = a.qo.p + row * a.qo.row + h * a.qo.head;
    } else {
      const bool key = item < sp.k_items;
      const Div du = key ? sp.turn_units : sp.copy_units;
      const int at = item - (key ? sp.q_items : sp.k_items), h = quotient(at, du);
      unit = at - h * du.by;
      turns = key;
      const int s = a.seq ? a.seq[row] : row, slot = a.slots[row];
      if (s < 0 || s >= a.c.S || slot < 0 || slot >= a.c.most << a.c.shift) continue;
      const int page = page_of(a.c, s, slot);
      if (page < 0) continue;
      const Rows &src = key ? a.k : a.v;
      from = src.p + row * src.row + h * src.head;
      to = (key ? a.c.K : a.c.V) + entry_at(a.c, page, h, slot);
      if (key && unit == 0) {
        const int64_t n = number_at(a.c, page, h, slot);
        if (a.c.mass) a.c.mass[n] = 0.f;
        if (a.c.age)
          a.c.age[n] = a.positions ? (int32_t)min(max(position(row), (int64_t)INT32_MIN), (int64_t)INT32_MAX) : slot;
      }
    }
    if (!turns) {
      Piece<E, 16 / es>::copy(to + unit * 16, from + unit * 16);
      continue;
    }
    const float2 *const w = turn[t];
    if constexpr (V == 1) {  // a pair, or an element of those that stay
      if (unit < pairs) {
        const int i0 = a.start + (Halves ? unit : 2 * unit), i1 = i0 + (Halves ? pairs : 1);
        const float x0 = (float)reinterpret_cast<const E *>(from)[i0], x1 = (float)reinterpret_cast<const E *>(from)[i1];
        reinterpret_cast<E *>(to)[i0] = (E)(x0 * w[unit].x - x1 * w[unit].y);
        reinterpret_cast<E *>(to)[i1] = (E)(x1 * w[unit].x + x0 * w[unit].y);
      } else {
        const int i = unit - pairs, e = i < a.start ? i : i + a.turned;
        if (from != to) Piece<E, 1>::copy(to + e * es, from + e * es);
      }
    } else if constexpr (Halves) {  // two pieces, or a piece of those that stay
      const int half = pairs / V;
      if (unit < half) {
        const int i0 = a.start + unit * V;
        float x0[V], x1[V], y0[V], y1[V];
        Piece<E, V>::load(from + i0 * es, x0);
        Piece<E, V>::load(from + (i0 + pairs) * es, x1);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float2 u = w[unit * V + i];
          y0[i] = x0[i] * u.x - x1[i] * u.y;
          y1[i] = x1[i] * u.x + x0[i] * u.y;
        }
        Piece<E, V>::store(to + i0 * es, y0);
        Piece<E, V>::store(to + (i0 + pairs) * es, y1);
      } else if (from != to) {
        const int i = unit - half, e = i * V < a.start ? i * V : i * V + a.turned;
        Piece<E, V>::copy(to + e * es, from + e * es);
      }
    } else {
      const int e = unit * V, i = e - a.start;
      if (i >= 0 && i < a.turned) {
        float x[V], y[V];
        Piece<E, V>::load(from + e * es, x);
#pragma unroll
        for (int j = 0; j < V; j += 2) {
          const float2 u = w[(i + j) / 2];
          y[j] = x[j] * u.x - x[j + 1] * u.y;
          y[j + 1] = x[j + 1] * u.x + x[j] * u.y;
        }
        Piece<E, V>::store(to + e * es, y);
      } else if (from != to) {
        Piece<E, V>::copy(to + e * es, from + e * es);
      }
    }
  }
}

template <typename E, int V, bool Halves>
gsi_status launch_as(const RotateArgs &a, hipStream_t st) {
  const int pairs = a.turned / 2, copies = a.d * (int)sizeof(E) / 16;
  const int turn_units = V == 1 ? a.d - pairs : (Halves ? a.d / V - pairs / V : a.d / V);
  Split sp{};
  sp.turn_units = div_by(turn_units);
  sp.copy_units = div_by(copies);
  sp.q_items = a.q.n * turn_units;
  sp.k_items = sp.q_items + a.k.n * turn_units;
  sp.items = sp.k_items + a.v.n * copies;
  sp.tokens = a.T >= 2048 ? 4 : 1;
  const int64_t groups = ((int64_t)a.T + sp.tokens - 1) / sp.tokens;
  const int64_t per = ((int64_t)sp.tokens * sp.items + kThreads - 1) / kThreads;
  const int64_t most = 2048 / groups > 1 ? 2048 / groups : 1;
  sp.strips = (int)(per < most ? per : most);
  if (groups * sp.strips * kThreads > kMostLaunch) return GSI_E_SHAPE;
  rotate_kernel<E, V, Halves><<<(unsigned)(groups * sp.strips), kThreads, 0, st>>>(a, sp);
  return hipGetLastError() == hipSuccess ? GSI_OK : GSI_E_HIP;
}

template <typename E>
gsi_status launch_of(const RotateArgs &a, int layout, hipStream_t st) {
  constexpr int V = 16 / sizeof(E);
  const bool halves = layout == GSI_ROTARY_HALVES;
  const bool whole = a.start % V == 0 && (halves ? a.turned / 2 : a.turned) % V == 0;
  if (whole) return halves ? launch_as<E, V, true>(a, st) : launch_as<E, V, false>(a, st);
  return halves ? launch_as<E, 1, true>(a, st) : launch_as<E, 1, false>(a, st);
}

}  // namespace

gsi_status launch_rotate(const RotateArgs &a, int dtype, int layout, hipStream_t st) {
  return dtype == GSI_FP32 ? launch_of<float>(a, layout, st) : launch_of<__bf16>(a, layout, st);
}

}  // namespace gsi
