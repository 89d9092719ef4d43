// Entry points of the plain linear maps: argument checks and the choice of kernel.
#include "gsi_maps.h"

namespace gsi {
namespace {

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

// Which kernel: the rows per expert and the tiles there are decide, both known
// from the call's sizes alone (the offsets are on the device).
gsi_status choose(const MArgs &a, const gsi_weights &w, hipStream_t st) {
  const bool f32 = w.dtype == GSI_FP32;
  const int64_t experts = a.n < a.R ? a.n : a.R, per = a.R / experts;
  if (w.bits == 4) {
    // Large tiles once they beat streaming the weights for every 16 rows: as
    // many tiles as CUs, or fewer, take as long as about 9000 blocks of 16 x 16
    // there (4096 -> 16384: 64 tokens 61 us in tiles, 31 us streamed; 160 tokens
    // 77 and 79; 512 tokens 83 and 173; 4096 -> 4096: 512 tokens 74 and 50, 576
    // tokens 75 and 77; 9120 -> 4608: 384 tokens 173 and 120, 640 tokens 171 and
    // 177; 32 experts 2048 -> 2048: 1200 rows 68 and 48, 1600 rows 68 and 63,
    // 2400 rows 69 and 86; weights called again and again).  Next to the limit
    // the streaming kernel is up to a fifth faster on the tiles' side: 128 tokens
    // 4096 -> 16384 61 and 51 us, 512 tokens 9120 -> 4608 172 and 153.
    const int64_t tiles = (a.R / 256 + experts) * ((a.d_out + 127) / 128);
    const int64_t blocks = (a.R / 16 + experts) * ((a.d_out + 15) / 16);
    if (!f32 && blocks >= 9000 && blocks / 9000. >= tiles / 256.) return launch_wide_q4(a, w.group, st);
    return launch_stream(a, f32 ? kQ4F32 : kQ4Bf16, w.group, st);
  }
  // Streaming for few rows per expert, and as long as its blocks of 16 x 16 do
  // not go round the chip twice: one small tile per CU or less is all latency.
  // Streamed and in small tiles, on weights called again and again and in
  // brackets from HBM:
  //   16 bf16 experts 2048 -> 2048   8 rows each: 25 (29) and 23 (35) us
  //                                 16 rows:      26 (30) and 24 (35)
  //   64 bf16 experts 2048 -> 2816   8 rows each: 154 (153) and 165 (164)
  //                                 16 rows:      161 (160) and 165 (165),
  //                                               156 (159) in large tiles
  //   16 fp32 experts 2048 -> 2048  12 rows each: 50 (64) and 51 (63)
  //   bf16, 8 experts 4096 -> 256, 40 rows, 448 blocks: 16 (16) and 18 (45)
  //         4 experts 4096 -> 1024, 24 rows, 640 blocks: 15 (16) and 28 (44)
  //                                 40 rows, 896 blocks: 31 (32) and 30 (46)
  //         8 experts 1024 -> 512, 33 rows, 768 blocks: 12 (12) and 8 (14)
  //   fp32, 4 experts 4096 -> 1024, 40 rows, 896 blocks: 57 (60) and 74 (96)
  // So the two are alike around the limits on repeated weights; on weights from
  // HBM streaming would serve up to 16 rows of bf16 and some more blocks.
  const int64_t blocks = (a.R / 16 + experts) * ((a.d_out + 15) / 16);
  if (per <= (f32 ? 12 : 8) || blocks <= 800) return launch_stream(a, f32 ? kF32 : kBf16, 0, st);
  // Large tiles where there is at least one for every CU, or half as many full
  // ones, as far as the rows and experts tell (large and small tiles: 64 experts
  // 2048 -> 4096, 32 rows each: 197 and 248 us; 16 experts 2048 -> 1024, 100
  // rows: 34 and 26 us; 8 experts 2048 -> 2048, 300 rows: 53 and 55 us, 512
  // rows: 54 and 76; 256 rows each, counted as twice the tiles there are: 53 and
  // 43; 2 experts 4096 -> 4096, 256 rows: 93 and 35).
  const int64_t tiles = (a.R / 256 + experts) * ((a.d_out + 255) / 256);
  if (!f32 && (tiles >= 256 || (tiles >= 128 && per >= 128))) return launch_wide(a, st);
  return launch_small(a, f32 ? kF32 : kBf16, st);
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
  return choose(a, *w, st);
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
