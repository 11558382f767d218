// The block-scaled product's choice of kernel (fp8.hip), by sizes and strides
// alone.  Host code without HIP, so that it can be looked at without a GPU.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "reshard.h"

namespace rs {

enum class MatmulShape { kStream16x64, kStream16x16, kStream32x32, kFar64x256, k256x256, k128x256, k64x256, k64x128, k64x64 };

inline MatmulShape matmul_shape(const rs_fp8_matmul& mm, bool gathered) {
  const int64_t kblocks = (mm.k + 127) / 128;
  const int64_t rows = mm.m / (mm.n_groups ? mm.n_groups : 1);  // a group's, on average
  if (mm.a_rows == 0 || kblocks == 0 || rows <= (mm.n_groups ? 4 : 32)) {
    // Few rows (or nothing to add up): b streams through registers.  Measured
    // (us, this choice against the nearest other): 32 experts of 4096 x 7168,
    // two rows each, 133 with 16 x 64 per workgroup, 136 with 32 x 64; 32 of 2816
    // x 621, two rows each, 14.7 with 16 x 64, 16.2 with tiles of 64 x 128; but
    // five rows each over 64 experts of 2048 x 1024 24 with tiles, 27 with 16 x
    // 64, and sixteen of 4096 x 7168 167 with tiles, 183 with 32 x 64.  One
    // product 7168 x 4096: one row 9.0 with 16 x 16, 10.5 with 16 x 32; 20 rows
    // 11.6 with 32 x 32, 13.2 with tiles of 64 x 64; but 33 rows 13.3 with tiles,
    // 17 with 32 x 64.
    if (mm.n_groups && rows <= 4) return MatmulShape::kStream16x64;
    return !mm.n_groups && rows <= 16 ? MatmulShape::kStream16x16 : MatmulShape::kStream32x32;
  }
  // Operands too far apart for load offsets of 32 bits, which count from a
  // tile's first row or, of gathered rows, from a: one shape with 64-bit ones,
  // which has the registers for them.  Measured (us): 8192 rows gathered from 4.3
  // GB over 32 experts of 7168 x 2048 278, streamed 921 (from 4.1 GB, 32 bits:
  // 211); 16,384 x 4096 x 7168 772, streamed 3,566 (32 bits: 388).  (A stride of
  // a single row may hold anything.)
  const int64_t kFar = int64_t(1) << 32;
  const int64_t a_reach = mm.a_rows > 1 ? gathered ? mm.a_rows : 256 : 0;
  const bool one_b_scale = mm.n <= 1 || (mm.b_block_rows != 1 && mm.n <= 128 && (mm.b_split == 0 || mm.b_split == mm.n));
  if (a_reach * mm.a_stride >= kFar || a_reach * mm.a_scale_stride * 4 >= kFar || (mm.n > 1 ? 256 * mm.b_stride : 0) >= kFar ||
      (one_b_scale ? 0 : (mm.n + 256) * mm.b_scale_stride * 4) >= kFar)
    return MatmulShape::kFar64x256;
  // The tile shape with the least expected time: rounds of workgroups over
  // the chip, each of a fixed time and a time per step, fitted to measured
  // times (us): with every compute unit busy, or with one workgroup a unit
  // where there is less than a round, or with groups, whose matrices come from
  // memory one after the other and not from L2.  Groups are taken to end half
  // a tile early.  Measured (us, tiles of 256 x 256, 128 x 256, 64 x 256,
  // 64 x 128, 64 x 64; * = chosen): 4096 x 4096 x 4096 64* 78 104 103 197;
  // 1024 x 8192 x 4096 52 39* 51 53 100; 2048 x 2048 x 2048 28 21 16.5* 16.7 32;
  // 256 x 7168 x 4096 48 34 25 19* 27; 100 x 1000 x 4096 45 33 24 18 11.6*;
  // 32 groups, 8192 x 4096 x 4096 235* 272 320 335 679; 4096 x 4096 x 7168 323
  // 272* 332 378 655; 1536 x 4096 x 7168 244 215 209* 215 330.
  struct Tile {
    MatmulShape shape;
    int bm, bn, slots, blocks;  // rows, columns, workgroups a round, k blocks a step
    float fixed, alone, busy, grouped;
  };
  static constexpr Tile kTiles[] = {{MatmulShape::k256x256, 256, 256, 256, 1, 8.0f, 1.17f, 1.65f, 1.65f},
                                    {MatmulShape::k128x256, 128, 256, 256, 1, 4.4f, 0.90f, 1.10f, 1.10f},
                                    {MatmulShape::k64x256, 64, 256, 256, 1, 3.4f, 0.67f, 0.74f, 0.86f},
                                    {MatmulShape::k64x128, 64, 128, 512, 1, 2.8f, 0.43f, 0.70f, 0.88f},
                                    {MatmulShape::k64x64, 64, 64, 256, 4, 3.0f, 0.95f, 1.20f, 4.00f}};
  MatmulShape best = kTiles[0].shape;
  float least = 0.0f;
  for (const Tile& t : kTiles) {
    int64_t tiles = (mm.m + t.bm - 1) / t.bm;
    if (mm.n_groups) tiles = std::max(int64_t(mm.n_groups), mm.m / t.bm + mm.n_groups / 2);
    tiles *= (mm.n + t.bn - 1) / t.bn;
    const int64_t steps = (kblocks + t.blocks - 1) / t.blocks, rounds = (tiles + t.slots - 1) / t.slots;
    const bool few = tiles <= 256;  // one workgroup a unit
    const float step = !mm.n_groups ? (few ? t.alone : t.busy) : few && t.slots > 256 ? t.grouped / 2 : t.grouped;
    const float cost = float(rounds) * (t.fixed + float(steps) * step);
    if (least == 0.0f || cost < least) best = t.shape, least = cost;
  }
  return best;
}

}  // namespace rs
