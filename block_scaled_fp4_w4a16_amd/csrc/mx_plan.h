// Which kernel, tiles and K parts an MXFP4 product runs with: rules on its sizes and the device's compute units. Host code
// with no other dependency, so that a program without a GPU can ask too.
#pragma once
#include <stdint.h>

namespace mx {

// Stages of 256 positions.
inline int stages_of(int64_t K) { return (int)((K + 255) / 256); }

// How a product is run.
struct Plan {
  int tile;    // 0: rows_kernel, else gemm_kernel with tiles of 64, 128 or 256
  int parts;   // K parts
  int per;     // stages per part (even)
  int64_t ldp; // floats per row of a plane
  int64_t first_n;  // > 0: columns [0, first_n) in tiles of 256, the others as a product of their own
  double us;   // what it is taken to cost
};

// What a tile costs, in microseconds as measured on 256 compute units with 16-bit outputs and operands that come again (those
// of a few MB from the caches): a launch with its first loads and last stores, each further round's stores, and a stage of
// 256 positions with one workgroup on a unit (256: with every unit busy; a few workgroups of 256 run a stage in 1.2) and
// with two (64 and 128: two fit; their stages run at 16 and 28 outputs per nanosecond, those of 256 at 37).
struct TileCost {
  int tile;
  double launch, round, one, two;
};
constexpr TileCost TILE_COSTS[] = {{64, 3.2, 0.6, 0.27, 0.5}, {128, 4.4, 1.6, 0.67, 1.15}, {256, 9.0, 4.0, 1.75, 0}};

inline double tiles_us(const TileCost& c, int64_t work, int stages, int cus) {
  const int64_t slots = (c.two > 0 ? 2 : 1) * (int64_t)cus, full = work / slots, rest = work - full * slots;
  double last = rest > cus ? c.two : c.one;
  if (c.two == 0) last = 1.2 + (c.one - 1.2) * rest / cus;
  return c.launch + (full + (rest > 0) - 1) * c.round + stages * (full * (c.two > 0 ? c.two : c.one) + (rest > 0 ? last : 0));
}

// The cheapest of the tiles and K parts by those figures. Parts (only where one round of tiles leaves units idle) cost a
// second kernel and their planes' way to memory and back: 2.5 us and 1.2 bytes per picosecond. For example 333 x 2560,
// K = 9728: tiles of 64 take 13.1 us, of 128 28.9 us; 64 x 2560, K = 9728: 12.8 us, in 4 parts 9.3 us.
// Where the last round of tiles of 256 would be a small one (split), the columns that fill whole rounds are one product and
// the others a second in tiles that fill the device.
inline Plan plan_of(int64_t M, int64_t N, int64_t K, int cus, bool split = true) {
  Plan p{};
  p.ldp = (N + 3) / 4 * 4;
  const int stages = stages_of(K);
  p.parts = 1;
  p.per = (stages + 1) & ~1;
  p.us = 1e30;
  // up to 16 rows: rows_kernel, by its chunk pairs and tiles of 16 (4096 x 4096 at M = 1 and 16: 2.8 and 3.2 us, tiles of 64
  // 7.2; 28672 x 8192: 26.4 and 31.9 us against 25.9 and 27.0). The figure takes the work as spread over the device; few
  // columns with a long K take longer (1 x 16 x 2^20: 216 us, where 17 rows in K parts take 70; 16 x 128 x 65536: 16.8, 12.7)
  if (M <= 16) p.us = 1.8 + (double)((N + 15) / 16) * stages * (0.00034 + 0.00001 * M);
  const double least = 3.5 + N * K * (17 / 32.) / 5e6;  // the weights' bytes at 5 TB/s
  for (const TileCost& c : TILE_COSTS) {
    const int64_t tiles = ((M + c.tile - 1) / c.tile) * ((N + c.tile - 1) / c.tile);
    for (int want = 1; want <= 16; want *= 2) {
      const int per = ((stages + want - 1) / want + 1) & ~1, parts = (stages + per - 1) / per;
      if (want > 1 && (c.tile == 256 || parts != want || tiles * parts > cus)) break;
      double us = tiles_us(c, tiles * parts, per, cus);
      if (us < least) us = least;
      if (parts > 1) us += 2.5 + parts * M * p.ldp * 4 / 1.2e6;
      if (us < p.us) p.us = us, p.tile = c.tile, p.parts = parts, p.per = per;
    }
  }
  if (split) {
    const TileCost& c = TILE_COSTS[2];
    const int64_t down = (M + 255) / 256, across = (N + 255) / 256, fit = down * across / cus * cus / down;
    if (fit > 0 && fit < across) {
      const Plan rest = plan_of(M, N - fit * 256, K, cus, false);
      const double us = tiles_us(c, down * fit, (stages + 1) & ~1, cus) + rest.us;
      if (rest.parts == 1 && us < 0.95 * p.us)
        p.us = us, p.tile = 256, p.parts = 1, p.per = (stages + 1) & ~1, p.first_n = fit * 256;
    }
  }
  return p;
}

inline int64_t plane_bytes(const Plan& p, int64_t M) { return p.parts > 1 ? p.parts * M * p.ldp * 4 : 0; }

// Whether dense activations are quantised inside the product, else into the workspace before it. Each workgroup of 16
// weight rows then quantises all of them again, which pays while rows and rounds are few. With weights that come again, 4096 x
// 4096 at M = 1, 4 and 8 takes 4.2, 4.6 and 5.3 us against 4.8, 4.9 and 5.1 in two kernels, 9728 x 2560 at M = 1 and 4 5.9 and
// 6.7 against 6.4 and 6.8, 14336 x 4096 at M = 1 12.3 against 9.5.
inline bool fused(int64_t M, int64_t N, int64_t K) {
  return M <= 16 && (N + 15) / 16 * stages_of(K) * (M + 3) <= 32768;
}

}  // namespace mx
