// Rotary positions and appending to the paged cache (gsi_rotary,
// gsi_cache_append): one kernel that turns rows of heads and writes them to
// rows or to the pages.
#include "gsi_cache.h"

namespace gsi {
namespace {

constexpr int kThreads = 256;
constexpr int kMostPairs = 128;
constexpr int kMostTokens = 4;  // of a workgroup

typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

// A workgroup's items one after the other: the units of its tokens' query heads,
// of their key heads and of their value heads.  Queries go token by token, as
// their rows lie; keys and values head by head, each for all tokens, as entries
// lie side by side in a page.
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
  float2 turn[kMostTokens][kMostPairs + 8];  // a run's last pairs may lie behind
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

// Fewer elements than 8 bytes hold, in pieces of 4 and 2 bytes.
template <typename E>
__device__ __forceinline__ uint64_t load_few(const uint8_t *at, int count) {
  uint64_t v = 0;
  uint32_t four = 0;
  if constexpr (sizeof(E) == 4) {
    if (count > 0) __builtin_memcpy(&four, at, 4);
    v = four;
  } else {
    uint16_t two = 0;
    if (count & 2) __builtin_memcpy(&four, at, 4);
    if (count & 1) __builtin_memcpy(&two, at + 2 * (count & 2), 2);
    v = (uint64_t)two << 16 * (count & 2) | four;
  }
  return v;
}
template <typename E>
__device__ __forceinline__ void store_few(uint8_t *at, uint64_t v, int count) {
  const uint32_t four = (uint32_t)v;
  if constexpr (sizeof(E) == 4) {
    if (count > 0) __builtin_memcpy(at, &four, 4);
  } else {
    const uint16_t two = (uint16_t)(v >> 16 * (count & 2));
    if (count & 2) __builtin_memcpy(at, &four, 4);
    if (count & 1) __builtin_memcpy(at + 2 * (count & 2), &two, 2);
  }
}

// A run of `count` elements, 16 bytes of them where they are all there.
template <bool Whole, typename vec, typename E, int V>
__device__ __forceinline__ vec load_run(const uint8_t *at, int count) {
  vec v = {};
  if (Whole || count == V) {
    __builtin_memcpy(&v, Whole ? __builtin_assume_aligned(at, 16) : at, 16);
  } else if (count > 0) {
    const bool half = count >= V / 2;
    uint64_t two[2] = {0, 0};
    if (half) __builtin_memcpy(two, at, 8);
    const uint64_t rest = load_few<E>(at + (half ? 8 : 0), count % (V / 2));
    two[half ? 1 : 0] = rest;
    __builtin_memcpy(&v, two, 16);
  }
  return v;
}
template <bool Whole, typename vec, typename E, int V>
__device__ __forceinline__ void store_run(uint8_t *at, const vec &v, int count) {
  if (Whole || count == V) {
    __builtin_memcpy(Whole ? __builtin_assume_aligned(at, 16) : at, &v, 16);
  } else if (count > 0) {
    const bool half = count >= V / 2;
    uint64_t two[2];
    __builtin_memcpy(two, &v, 16);
    if (half) __builtin_memcpy(at, two, 8);
    store_few<E>(at + (half ? 8 : 0), half ? two[1] : two[0], count % (V / 2));
  }
}

// Bound by HBM for many tokens (8191 of 40 heads of 128: 168 MB in 29 us, 5.8
// TB/s; 4939 of 16 heads of 256 with their keys and values into the pages: 243
// MB in 54 us, 4.5 TB/s), by latency for few (one token of 16 heads of 256 3 us):
// the position, the sine and cosine, the head.  The angles are formed once for all
// heads of a token.  Whole: runs of 16 bytes end where the turned part does;
// otherwise the turned part, what lies before it and what lies behind are cut into
// runs each by itself, at any address.  Their last run then ends where the part
// does and repeats what the run before it has; in place, where that would turn
// elements twice, it is the shorter rest (8191 tokens of 40 heads of 128 in halves,
// bf16: all turned 27 us, 100 elements of each 29, in place 35).
template <typename E, bool Halves, bool Whole>
__global__ void __launch_bounds__(kThreads, 8) rotate_kernel(RotateArgs a, Split sp) {
  __shared__ Tokens k;
  constexpr int es = sizeof(E), V = 16 / es;
  // items of a thread under way: 64 bytes read, and half for runs of any length,
  // as much as eight wavefronts' registers hold
  constexpr int kAhead = Halves ? (Whole ? 2 : 1) : (Whole ? 4 : 2);
  typedef E vec __attribute__((ext_vector_type(V)));
  const int group = blockIdx.x / sp.strips, strip = blockIdx.x - group * sp.strips;
  const int t0 = group * sp.tokens, tokens = min(sp.tokens, a.T - t0), pairs = a.turned / 2;
  const int run = Halves ? pairs : a.turned, runs = (run + V - 1) / V, left = (a.start + V - 1) / V;
  prepare(a, k, t0, tokens, strip == 0);
  const int all = tokens * sp.items, step = sp.strips * kThreads;
  for (int i0 = strip * kThreads + threadIdx.x; i0 < all; i0 += kAhead * step) {
    uint8_t *to[kAhead];
    vec x0[kAhead], x1[kAhead];
    int count[kAhead], turn[kAhead];  // of the (first) run, and its first pair or -1
    const float2 *w[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j * step;
      to[j] = nullptr;
      x0[j] = x1[j] = vec{};
      count[j] = V;
      turn[j] = -1;
      w[j] = k.turn[0];
      if (i >= all) continue;
      const Item it = item_of(a, sp, k, t0, tokens, i);
      w[j] = k.turn[it.t];
      int e = it.unit * V;
      if (it.turns) {
        // the part that the run is of, and where that begins
        const bool turns = it.unit < runs, before = it.unit < runs + left;
        const int part = turns ? run : before ? a.start : a.d - a.start - a.turned;
        const int first = turns ? a.start : before ? 0 : a.start + a.turned;
        e -= V * (turns ? 0 : before ? runs : runs + left);
        if (!Whole) {
          if (it.from != it.to && part >= V)
            e = min(e, part - V);  // again what the run before has: the same values
          else
            count[j] = min(V, part - e);
        }
        if (turns) turn[j] = Halves ? e : e / 2;
        e += first;
      }
      if (!it.to || (it.turns && turn[j] < 0 && it.from == it.to)) continue;  // no entry; in place
      const uint8_t *const from = it.from + e * es;
      to[j] = it.to + e * es;
      x0[j] = load_run<Whole, vec, E, V>(from, count[j]);
      if (Halves && turn[j] >= 0) x1[j] = load_run<Whole, vec, E, V>(from + pairs * es, count[j]);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (!to[j]) continue;
      if (turn[j] >= 0) {
        const float2 *const u = w[j] + turn[j];
        vec y0, y1;
        if constexpr (Halves) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            y0[e] = (E)((float)x0[j][e] * u[e].x - (float)x1[j][e] * u[e].y);
            y1[e] = (E)((float)x1[j][e] * u[e].x + (float)x0[j][e] * u[e].y);
          }
          store_run<Whole, vec, E, V>(to[j] + pairs * es, y1, count[j]);
        } else {
#pragma unroll
          for (int e = 0; e < V; e += 2) {
            y0[e] = (E)((float)x0[j][e] * u[e / 2].x - (float)x0[j][e + 1] * u[e / 2].y);
            y0[e + 1] = (E)((float)x0[j][e + 1] * u[e / 2].x + (float)x0[j][e] * u[e / 2].y);
          }
        }
        x0[j] = y0;
      }
      store_run<Whole, vec, E, V>(to[j], x0[j], count[j]);
    }
  }
}

template <typename E, bool Halves>
gsi_status launch_as(const RotateArgs &a, bool whole, hipStream_t st) {
  constexpr int V = 16 / sizeof(E);
  const int pairs = a.turned / 2, copies = a.d / V;
  const int run = Halves ? pairs : a.turned, behind = a.d - a.start - a.turned;
  const int turn_units = (run + V - 1) / V + (a.start + V - 1) / V + (behind + V - 1) / V;
  Split sp{};
  sp.turn_units = div_by(turn_units);
  sp.copy_units = div_by(copies);
  sp.q_heads = div_by(a.q.n > 0 ? a.q.n : 1);
  sp.q_items = a.q.n * turn_units;
  sp.k_items = sp.q_items + a.k.n * turn_units;
  sp.items = sp.k_items + a.v.n * copies;
  // Tokens share a workgroup, and with it the wait for positions and pages, where
  // there are enough to fill the chip and one has little to move.  One token and
  // four, us, bf16 in halves: 8191 of 8 heads of 64 9.2 and 5.7, of 16 heads of 128 13.4
  // and 12.6, of 24 17.3 and 18.0, of 40 29.3 and 32.4; into pages, 3 prompts up to
  // 16000 of 8 query and 8 key heads of 64 32.5 and 23.0, of 16 and 16 of 256 169 and
  // 187; 1000 of 8 heads of 128 4.0 and 3.9, of 16 heads of 256 6.0 and 6.5.
  const int bytes = (a.q.n + a.k.n + a.v.n) * a.d * (int)sizeof(E);
  sp.tokens = a.T >= 2048 && bytes < 6144 ? kMostTokens : 1;
  const int64_t groups = ((int64_t)a.T + sp.tokens - 1) / sp.tokens;
  const int64_t per = ((int64_t)sp.tokens * sp.items + kThreads - 1) / kThreads;
  const int64_t most = 2048 / groups > 1 ? 2048 / groups : 1;
  sp.strips = (int)(per < most ? per : most);
  if (groups * sp.strips * kThreads > kMostLaunch) return GSI_E_SHAPE;
  const unsigned grid = (unsigned)(groups * sp.strips);
  if (whole)
    rotate_kernel<E, Halves, true><<<grid, kThreads, 0, st>>>(a, sp);
  else
    rotate_kernel<E, Halves, false><<<grid, kThreads, 0, st>>>(a, sp);
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
