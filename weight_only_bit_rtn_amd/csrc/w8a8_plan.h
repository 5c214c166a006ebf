// w8a8_plan.h -- which kernel and tiles take a product or a gradient in 8-bit
// integers: host arithmetic on sizes and the device's number of CUs, without HIP,
// so that a program without a GPU can ask too.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace lowbit {

// Tiles of a product: `whole` of them, as many as fill the CUs some times over,
// are computed by one workgroup each, and each of the `rest` by `splits`
// workgroups that share its steps and leave their sums in the workspace for a
// second kernel to join.
struct TilePlan {
  int tiles_m, tiles_n, whole, rest, splits;
  int blocks() const { return whole + rest * splits; }
};
// The plan that should finish first, and when.  A CU takes alone_us for a step
// of a tile that it has to itself, and shared_us for each tile's where it has
// several workgroups; a join costs about 7 us, and the partial sums (tile_bytes
// for each share) are written and read again at about 8 TB/s (they stay in the
// caches).
inline TilePlan plan_tiles(int64_t tm, int64_t tn, int cus, int steps, double alone_us,
                           double shared_us, double tile_bytes, double* us) {
  const int64_t tiles = tm * tn, rest = tiles % cus, whole = tiles - rest;
  const int64_t rounds = (tiles + cus - 1) / cus;
  TilePlan best{(int)tm, (int)tn, (int)tiles, 0, 1};
  *us = rounds * steps * (rounds > 1 ? shared_us : alone_us);
  for (int z = 2; rest > 0 && z <= 16 && z <= steps / 4; z++) {
    const int64_t more = (rest * z + cus - 1) / cus;
    const double work = (double)(whole / cus) * steps + (double)(more * ((steps + z - 1) / z));
    const double t = work * (whole / cus + more > 1 ? shared_us : alone_us) + 7.0 +
                     (double)rest * z * tile_bytes * 2 / 8e6;
    if (t < *us) {
      best.whole = (int)whole;
      best.rest = (int)rest;
      best.splits = z;
      *us = t;
    }
  }
  return best;
}

// ---------------------------------------------------------------------------
// products: few_kernel, the rings of skinny_kernel, or tiles
// ---------------------------------------------------------------------------
// few_kernel's tokens have their codes in LDS; up to kFusedMost values it makes
// them itself.
constexpr int kFewMostCodes = 128 * 1024;
constexpr int kFusedMost = 16384;
constexpr int kFewChunk = 1024;  // bytes of a row per load

// Bytes of one token's codes in LDS: whole chunks, zeros behind the last.
constexpr int few_pitch(int K) {
  return (K + kFewChunk - 1) / kFewChunk * kFewChunk;
}

// Up to here whole rows read this way beat the rings of w8a8_skinny.hip, in us a
// call on weights rotated over 1 GiB: linear 2x11008x4096 12.1 / 16.3, 2x28672x8192
// 42.6 / 44.5; gated 4x4096x4096 12.1 / 16.4, though 4x28672x8192 84.0 / 83.1.  With
// kernels for more tokens, on weights in the last-level cache: linear 4x28672x8192
// 43.2 / 41.2, 8x12288x12288 33.6 / 28.3, gated 8x28672x8192 95.9 / 89.3.
inline bool few_takes(int64_t T, int64_t K, bool gated) {
  return T <= (gated ? 4 : 2) && T * few_pitch((int)K) <= kFewMostCodes;
}

// skinny_kernel takes up to 16 tokens in any case.
constexpr int kSkinnyMostT = 64;

// The rings' time, fitted to kernels on weights in the last-level cache: the tokens
// are read again with each tile of 16 weight rows.  In us a call, against 64 x 128
// tiles of w8a8_gemm.hip, on weights rotated over 1 GiB (in brackets: in the cache):
// 64x28672x8192 84 / 57 (64 / 41), gated 64x28672x8192 115 / 98, 64x12288x12288
// 60 / 46 (43 / 33), but 24x12288x12288 41.8 / 40.9 (30.9 / 31.4) and, where those
// would have to share few tiles out, 64x4096x4096 16.1 / 19.4, 45x4096x11008 from
// codes 17.4 / 17.0 (13.6 / 16.8).
inline double skinny_us(int64_t T, int64_t N, int64_t K, bool gated) {
  const double bytes = (double)N * K * (gated ? 2 : 1);
  const double tokens = (double)((T + 15) / 16) / (gated ? 2 : 1);
  return 1.5 + bytes * (0.165 + 0.03 * tokens) * 1e-6;
}

// Tile shapes: tokens, weight rows, bytes of k per step, and what a step of one
// tile takes of a CU's time when there is one tile for each CU at most, and when
// there are more (us; fitted to calls, so part of what lies around the steps is in
// it: 192 x 192 takes 0.88 us a step and 13-16 us around them).  The larger the tile
// the less is loaded per output; the smaller ones are for sizes that would leave CUs
// idle or pad much, and for those that wait for the weights.  Steps of 128 bytes
// read whole cache lines and halve the barriers; the last three have no LDS for three
// buffers of them, and two are slower (gated 4096x28672x8192 by a tenth).
// With a shape and without it, us a call on weights rotated over 1 GiB: 64 x 128 on
// 64x49152x12288 143 / 155, gated 64x11008x4096 30.0 / 32.3; 128 x 128 on
// 128x28672x8192 64 / 72, 1000x4096x4096 33.5 / 42; 256 x 128 on 250x28672x8192
// 82 / 105, 2000x4096x4096 50.5 / 53; 192 x 192 on gated 333x11008x4096 47 / 58; 256 x
// 384 on 4096x12288x12288 531 / 577, gated 4096x28672x8192 1822 / 1856.
struct ProductShape {
  int mt, nt, step;
  double alone_us, shared_us;
};
constexpr ProductShape kProductShapes[] = {
    {64, 128, 128, 0.55, 0.70},  {128, 128, 128, 0.63, 0.80}, {256, 128, 128, 1.15, 1.32},
    {192, 192, 128, 1.35, 1.50}, {256, 192, 64, 0.90, 0.90},  {256, 256, 64, 1.03, 1.03},
    {256, 384, 64, 1.42, 1.42}};

// The kernel and shape that should finish first.
struct GemmPlan {
  TilePlan tiles;
  int shape;  // -1: the rings of w8a8_skinny.hip
  size_t part_bytes() const {
    if (shape < 0) return 0;
    const ProductShape& t = kProductShapes[shape];
    return (size_t)tiles.rest * tiles.splits * t.mt * t.nt * 4;
  }
};
inline GemmPlan gemm_plan(int64_t T, int64_t N, int64_t K, bool gated, int cus) {
  const int64_t rows = gated ? 2 * N : N;
  GemmPlan best{{}, -1};
  if (T <= 16) return best;
  double least = T <= kSkinnyMostT ? skinny_us(T, N, K, gated) : 1e30;
  for (int i = 0; i < (int)(sizeof(kProductShapes) / sizeof(kProductShapes[0])); i++) {
    const ProductShape& t = kProductShapes[i];
    double us;
    const int steps = (int)((K + t.step - 1) / t.step);
    const TilePlan plan = plan_tiles((T + t.mt - 1) / t.mt, (rows + t.nt - 1) / t.nt, cus, steps,
                                     t.alone_us, t.shared_us, (double)t.mt * t.nt * 4, &us);
    us += 2;  // the ring's first filling, and the outputs
    if (us < least) {
      best = {plan, i};
      least = us;
    }
  }
  return best;
}

// ---------------------------------------------------------------------------
// gradients
// ---------------------------------------------------------------------------
constexpr int kStepN = 64;  // weight rows per pipeline step

// Tile shapes: tokens, columns of dx, and what a step of 64 weight rows of one
// tile takes of a CU's time when the CU has no other workgroup, and when it has
// (us; fitted so that the shapes come out in the order of whole calls.  Steps alone
// take 1.12 of 128 x 256, 1.39 of 256 x 192, 1.53 of 256 x 256, and with those
// 2000x4096x4096 took 83 for 80 us and gated 128x28672x8192 168 for 152, though
// gated 300x11008x4096 93 for 95).  64 x 256 reads the tokens' factors half as often
// as 64 x 128 and pays where the weights are large (with and without it, on weights
// rotated over 1 GiB: gated 64x28672x8192 117 / 138 us, 61x11008x4096 39 / 42); for 16
// or 32 tokens, whose factors are fewer, 256 columns gave nothing (gated
// 16x28672x8192 117 / 122, linear 10x12288x12288 40.5 / 37.5).
struct GradShape {
  int mt, kt;
  double alone_us, shared_us;
};
// 128 x 256 beside 128 x 128: 2000x4096x4096 80 / 83, gated 128x28672x8192 152 / 168,
// 300x11008x4096 95 / 101, but 1000x1024x1024 24.9 / 22.1, where it is not taken.
constexpr GradShape kGradShapes[] = {
    {16, 128, 0.40, 0.32},  {32, 128, 0.40, 0.32},  {64, 128, 0.50, 0.40},  {64, 256, 0.64, 0.64},
    {128, 128, 0.74, 0.55}, {128, 256, 1.06, 1.06}, {256, 192, 1.20, 1.20}, {256, 256, 1.60, 1.60}};

// The shape that should finish first, of those that hold T tokens without waste.
struct GradPlan {
  TilePlan tiles;
  int shape;
  size_t part_bytes() const {
    return (size_t)tiles.rest * tiles.splits * kGradShapes[shape].mt * kGradShapes[shape].kt * 4;
  }
};
inline GradPlan grad_plan(int64_t T, int64_t K, int steps, int cus) {
  const int from = T <= 16 ? 0 : T <= 32 ? 1 : T <= 64 ? 2 : 4;
  const int to = T <= 32 ? from : T <= 64 ? 3 : 7;
  GradPlan best{};
  double least = 0;
  for (int i = from; i <= to; i++) {
    const GradShape& t = kGradShapes[i];
    double us;
    const TilePlan plan = plan_tiles((T + t.mt - 1) / t.mt, (K + t.kt - 1) / t.kt, cus, steps,
                                     t.alone_us, t.shared_us, (double)t.mt * t.kt * 4, &us);
    if (least == 0 || us < least) {
      best = {plan, i};
      least = us;
    }
  }
  return best;
}

}  // namespace lowbit
