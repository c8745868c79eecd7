// How the gated linear unit is computed: which kernel takes a forward, which tiles a product has and how many workgroups share
// a sum, each by estimated time. No HIP in here: sizes and the number of compute units in, a choice out.
#pragma once

#include <stdint.h>

namespace rwkv7 {
namespace glu {

constexpr int kBK = 64;       // of k in a step of the tiles
constexpr int kCols32 = 64;   // columns of a tile of the float32 instructions, of each weight
constexpr int kStep32 = 32;   // of k
constexpr int kMostTM32 = 5;  // two workgroups on a compute unit: 128 registers a thread, 60 KB of LDS

struct Sizes {
  int64_t M, D, F;
  bool f32;
};

// Products of bfloat16 pieces that a product of the operands' type takes.
inline int pairs(bool f32) { return f32 ? 6 : 1; }
inline int64_t steps_of(int64_t K, int segments) { return (K + kBK - 1) / kBK * segments; }

// ---- tiles

// Shapes of a workgroup's tile, and what a step of 64 k and a tile's beginning and end take where as many workgroups as
// fit share a compute unit, in us: from products of 4096 to 8192 rows and columns, whose tiles fill the compute units
// evenly. 256 x 256: 1,340 TFLOP/s; 128 x 256: 1,080; two of 128 x 128 (64 x 256 in the forward): 1,050.
enum Shape { kLarge, kHalf, kSmall, kShapes };
struct ShapeInfo {
  int bm, bn;
  int per_cu;
  float step_us, ends_us;
};
// bn of the forward: columns of both weights
constexpr ShapeInfo kForwardShapes[kShapes] = {{256, 128, 1, 1.55f, 5.f}, {128, 128, 1, 0.96f, 4.f}, {64, 128, 2, 1.f, 4.f}};
constexpr ShapeInfo kGradShapes[kShapes] = {{256, 256, 1, 1.55f, 5.f}, {128, 256, 1, 0.96f, 4.f}, {128, 128, 2, 1.f, 4.f}};

// A product: its sizes, how many of them, and the steps of its sum.
struct Product {
  int64_t M, N, count, steps;
  int64_t tiles(const ShapeInfo& f) const { return (M + f.bm - 1) / f.bm * ((N + f.bn - 1) / f.bn) * count; }
  // written by each part and read again, at 5 TB/s, with the join's launch
  float join_us(int splits) const { return splits > 1 ? 4.f + (splits * 8.f + 4.f) * count * M * N * 2e-7f : 0.f; }
};
struct Plan {
  Shape shape;
  int splits[2];
  float us;
};

// When the last of two kinds of workgroups is done, of which `slots` run at a time, the longer kind before the other:
// n[i] of them of us[i] each.
inline float finish(int64_t (&n)[2], float (&us)[2], int64_t slots) {
  if (us[1] > us[0]) {
    const int64_t k = n[0];
    n[0] = n[1], n[1] = k;
    const float t = us[0];
    us[0] = us[1], us[1] = t;
  }
  // slots that are free early and late behind the first kind
  const int64_t late = n[0] % slots;
  float t[2] = {n[0] / slots * us[0], (n[0] / slots + 1) * us[0]};
  const int64_t count[2] = {slots - late, late};
  float end = late ? t[1] : t[0];
  int64_t left = n[1];
  if (left > 8 * slots) {  // whole rounds, which both kinds of slots take alike
    const int64_t rounds = left / slots - 4;
    left -= rounds * slots;
    t[0] += rounds * us[1], t[1] += rounds * us[1];
  }
  while (left > 0) {
    const int i = count[1] == 0 || t[0] <= t[1] ? 0 : 1;
    left -= count[i];
    t[i] += us[1];
    end = end > t[i] ? end : t[i];
  }
  return end;
}

// The shape and the numbers of parts of the sums with the least estimated time. Parts fill the compute units where
// there are few tiles, and level the last round of workgroups; a second kernel adds them.
inline Plan plan(const ShapeInfo (&shapes)[kShapes], const Product (&job)[2], int cus) {
  constexpr int kSplits[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32};
  Plan best{kLarge, {1, 1}, 0.f};
  bool any = false;
  for (int s = 0; s < kShapes; ++s) {
    const ShapeInfo& f = shapes[s];
    const int64_t slots = (int64_t)cus * f.per_cu, tiles[2] = {job[0].tiles(f), job[1].tiles(f)};
    for (int a : kSplits) {
      if (a > 1 && (tiles[0] * a > 4 * slots || job[0].steps < 4 * a)) break;
      for (int b : kSplits) {
        if (b > 1 && (tiles[1] * b > 4 * slots || job[1].steps < 4 * b)) break;
        int64_t n[2] = {tiles[0] * a, tiles[1] * b};
        float us[2] = {(job[0].steps + a - 1) / a * f.step_us + f.ends_us, (job[1].steps + b - 1) / b * f.step_us + f.ends_us};
        const float joins = job[0].join_us(a) + job[1].join_us(b);
        if (any && (n[0] * us[0] + n[1] * us[1]) / slots + joins >= best.us) continue;  // at least that
        const float t = finish(n, us, slots) + joins;
        if (!any || t < best.us) any = true, best = Plan{(Shape)s, {a, b}, t};
      }
    }
  }
  return best;
}

// ---- few rows

// Rows of whole 4 bytes, which a lane loads at least, may go by the kernel that reads the weights once for 32 of them.
inline bool fits_few(const Sizes& c) { return c.f32 || (c.D % 2 == 0 && c.F % 2 == 0); }
// 64 columns a workgroup; float32 32 where such workgroups fit side by side, one a compute unit: 1 x 2048 x 5504 17 us and 20, 1 x
// 2048 x 8192 (256 workgroups) 22 and 24, 32 rows there 26 and 38; 1 x 2048 x 10944 (342) 32 and 29, 32 rows there 47 and 39. In
// bfloat16 they would have half lines of a row (1 x 2048 x 5504 21 us and 12.6).
inline int few_columns(const Sizes& c, int cus) { return c.f32 && (c.F + 31) / 32 <= cus ? 32 : 64; }

// Up to 32 rows. A workgroup's k come one after the other, or the weights' bytes count (7.2 TB/s), which tiles have to read
// too. Tiles of so few rows take their steps, or the bytes, and for each part of the sums that the join adds half a us.
// The constants lie between what weights from the last-level cache take and what those from memory do, so that no call measured
// of either kind is more than 11% slower than by few rows.
constexpr float kFewStart = 5.f, kFewTilesStart = 6.f, kFewTilesPart = 0.55f;
inline float weights_us(const Sizes& c) { return 2.f * c.D * c.F * (c.f32 ? 4 : 2) / 7.2e6f; }
inline float few_us(const Sizes& c, int cus) {
  const bool one = c.M <= 16;  // tile of 16 rows
  const float k = c.f32 ? (one ? 0.0065f : 0.0095f) * (few_columns(c, cus) / 32) : one ? 0.0045f : 0.0046f;
  const float walk = kFewStart + c.D * k, read = 3.f + weights_us(c);
  return walk > read ? walk : read;
}
// The least that a plan of tiles may be estimated to take: with n steps in p parts 0.55 p + n / p us at least 1.48 sqrt(n).
// Most calls of few rows end there, as the plan takes the host up to 0.9 us.
inline bool few_at_once(const Sizes& c, int cus) {
  const float few = few_us(c, cus);
  if (c.f32) return few <= 23.f + weights_us(c) * 1.5f;  // pieces are 1.5 times as many bytes, written and read
  const float n = (float)steps_of(c.D, 1), more = few - kFewTilesStart;
  return more <= weights_us(c) || more * more <= 4.f * kFewTilesPart * n;
}
// Both ways in us, bfloat16 in a graph, weights from the cache: 1 x 2048 x 5504 11.3 and 18.6, 32 x 2048 x 2048 14.9 and 15.5, 8 x
// 4096 x 2048 19.8 and 21.7, 32 x 4096 x 2048 26 and 23, 32 x 4096 x 4096 27 and 29, 1 x 8192 x 512 33 and 26, 32 x 8192 x 4096 48
// and 38, 32 x 8192 x 8192 55 and 62, 1 x 16384 x 256 62 and 29, 32 x 16384 x 512 89 and 32; from memory: 1 x 2048 x 5504 17 and 21,
// 32 x 2048 x 2048 23 and 18, 16 x 4096 x 2048 38 and 23, 32 x 4096 x 4096 44 and 32, 32 x 8192 x 8192 87 and 74, 32 x 16384 x 512
// 156 and 34.
inline bool few_rows(const Sizes& c, const Plan& how, int cus) {
  const int p = how.splits[0];
  const float steps = (float)((steps_of(c.D, 1) + p - 1) / p), bytes = weights_us(c);
  return few_us(c, cus) <= kFewTilesStart + (p > 1 ? kFewTilesPart * p : 0.f) + (steps > bytes ? steps : bytes);
}

// More rows do too where the workgroups of 32 rows each fit side by side and each takes less time (its k one after the
// other) than tiles are estimated to: 64 rows of D=2048 F=5504 19 us and 25 by tiles, 256 of D=768 F=2048 10 and 20; 96 of
// D=2048 F=5504, more workgroups than compute units, 35 and 25, 64 of D=16384 F=1024 88 and 38; float32 128 of D=768
// F=2048 13 and 14.
inline bool few_rows_each(const Sizes& c, float tiles_us, int cus) {
  if (!fits_few(c)) return false;
  const int64_t groups = (c.M + 31) / 32 * ((c.F + few_columns(c, cus) - 1) / few_columns(c, cus));
  const float us = 6.f + c.D * (c.f32 ? 0.0003f * few_columns(c, cus) : 0.0051f);
  return groups <= cus && us < tiles_us;
}

// ---- a forward

// The float32 instructions' tile with the least estimated time: of its steps, by rows, on the compute unit with the most
// tiles (1 to 64 rows of tiles, of sizes 40 x 64 x 96 to 4096 x 4096 x 4096: within 10%). It is taken where that is less
// than the estimate for pieces: 515 x 770 x 2049 43 us and 55, 700 x 768 x 2048 41 and 54, 7 x 770 x 2049 13 and 42;
// 2048 x 768 x 2048 102 and 81, 4096 x 4096 x 4096 1,950 and 1,255.
struct F32Plan {
  int tm = 0;
  float us = 1e30f;
};
inline F32Plan plan_f32(const Sizes& c, int cus) {
  constexpr float kStepUs[kMostTM32] = {0.29f, 0.49f, 0.725f, 0.96f, 1.21f}, kWaitUs = 0.1f, kEndsUs = 7.f;
  F32Plan best;
  for (int tm = 1; tm <= kMostTM32; ++tm) {
    const int64_t tiles = (c.M + 16 * tm - 1) / (16 * tm) * ((c.F + kCols32 - 1) / kCols32);
    if (tiles > (int64_t(1) << 22)) continue;  // a grid's threads are counted in 32 bits
    const float us = kEndsUs + (c.D + kStep32 - 1) / kStep32 * ((tiles + cus - 1) / cus * kStepUs[tm - 1] + kWaitUs);
    if (us < best.us) best.tm = tm, best.us = us;
  }
  return best;
}

enum Way { kFew, kInstructions, kTiles };
struct ForwardPlan {
  Way way;
  int tm;      // kInstructions: rows of a tile, in 16
  Plan tiles;  // kTiles
};
inline ForwardPlan plan_forward(const Sizes& c, int cus) {
  ForwardPlan o{kFew, 0, Plan{}};
  const bool one = c.M <= 32 && fits_few(c);  // a workgroup has all rows
  if (one && few_at_once(c, cus)) return o;
  const Product job[2] = {{c.M, c.F, 1, steps_of(c.D, pairs(c.f32))}, {0, 0, 0, 0}};
  o.tiles = plan(kForwardShapes, job, cus);
  if (c.f32) {
    // the pieces come first: 4 bytes read and 6 written an element
    const float pieces = 8.f + (2.f * c.D * c.F + (float)c.M * c.D) * 10 / 6e6f;
    const F32Plan f32 = plan_f32(c, cus);
    const float us = o.tiles.us + pieces;
    // Pieces of few rows take some 15 us more than estimated. Few rows and pieces: 32 x 8192 x 512 83 us and 59, 32 x
    // 16384 x 256 161 and 76, 1 x 16384 x 256 76 and 73, 32 x 4096 x 256 38 and 48, 32 x 8192 x 1024 83 and 82.
    if (one ? few_us(c, cus) <= us + 15.f : few_rows_each(c, f32.us < us ? f32.us : us, cus)) return o;
    o.way = f32.us < us ? kInstructions : kTiles;
    o.tm = f32.tm;
  } else {
    // products this small take some 10 us more than estimated
    if (one ? few_rows(c, o.tiles, cus) : few_rows_each(c, o.tiles.us + 10.f, cus)) return o;
    o.way = kTiles;
  }
  return o;
}

}  // namespace glu
}  // namespace rwkv7
