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
// `costs`: what an epilogue makes of the tiles' figures. Where K is in parts the second kernel has it, which is taken to cost what it
// does in tiles of 64, so that it has no say in how many parts there are (20 x 635, K = 8192 with a bias: in 8 parts 8.5 us, in 16
// 10.0, whole 10.9). `room`: bytes that the planes may take.
inline Plan plan_of(int64_t M, int64_t N, int64_t K, int cus, bool split = true, const TileCost* costs = TILE_COSTS,
                    int64_t room = INT64_MAX) {
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
  for (int i = 0; i < 3; ++i) {
    const int64_t tile = costs[i].tile, tiles = ((M + tile - 1) / tile) * ((N + tile - 1) / tile);
    for (int want = 1; want <= 16; want *= 2) {
      const int per = ((stages + want - 1) / want + 1) & ~1, parts = (stages + per - 1) / per;
      if (want > 1 && (tile == 256 || parts != want || tiles * parts > cus || parts * M * p.ldp * 4 > room)) break;
      double us = tiles_us(parts > 1 ? TILE_COSTS[i] : costs[i], tiles * parts, per, cus);
      if (us < least) us = least;
      if (parts > 1) us += 2.5 + parts * M * p.ldp * 4 / 1.2e6 + (costs[0].launch - TILE_COSTS[0].launch);
      if (us < p.us) p.us = us, p.tile = (int)tile, p.parts = parts, p.per = per;
    }
  }
  if (split) {
    const TileCost& c = costs[2];
    const int64_t down = (M + 255) / 256, across = (N + 255) / 256, fit = down * across / cus * cus / down;
    if (fit > 0 && fit < across) {
      // the second product has no planes; a product without an epilogue whose second one would want them stays one
      const Plan rest = plan_of(M, N - fit * 256, K, cus, false, costs, costs == TILE_COSTS ? room : 0);
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

// The figures of tiles with an epilogue: what it adds to each round, as measured at 8192 x 14336 x 4096 and 8192 x 9728 x 2560 with
// 16-bit outputs. The matrix core idles through it in tiles of 256, one of which fits a unit; tiles of 128 cover each other's. So
// gelu onto a residual at 8192 x 9728 x 2560 takes 211 us in tiles of 256 and 173 in tiles of 128, a bias alone 127 and 126; at
// 14336 x 4096 369 and 372, 251 and 285.
struct EpilogueCosts {
  TileCost of[3];
};
inline EpilogueCosts epilogue_costs(bool erf, bool other_activation, bool residual, bool z) {
  EpilogueCosts e{{TILE_COSTS[0], TILE_COSTS[1], TILE_COSTS[2]}};
  const double more[3] = {0.3 + (erf ? 0.8 : other_activation ? 0.3 : 0) + (residual ? 1 : 0) + (z ? 2 : 0),
                          0.2 + (erf ? 2.5 : other_activation ? 0.8 : 0) + (residual ? 3.5 : 0) + (z ? 9 : 0),
                          3.7 + (erf ? 8 : other_activation ? 2.4 : 0) + (residual ? 9.7 : 0) + (z ? 13 : 0)};
  for (int i = 0; i < 3; ++i) e.of[i].launch += more[i], e.of[i].round += more[i];
  return e;
}

// Tiles of rows in groups: 64, 64 x 128 (WIDE; few rows of many groups, bound by the weights' bytes), 128 and 256 square. All but
// those of 64 are taken as streams, so that a round costs its stages and its way out; those of 64, which have more stages on
// their way, are for what leaves units idle (200 rows in 8 groups, 1024 columns, K = 2560: 6.6 us, in 64 x 128 8.7).
constexpr int WIDE = 96;
inline int tile_rows(int tile) { return tile == WIDE ? 64 : tile; }
inline int tile_columns(int tile) { return tile == WIDE ? 128 : tile; }
constexpr TileCost GROUPED_COSTS[] = {{64, 5, 4, 0.27, 0.5}, {WIDE, 6.3, 2.3, 0.6, 0.95}, {128, 7, 4.4, 0.75, 1.1}, {256, 15, 11, 1.75, 0}};
constexpr TileCost GRADIENT_COSTS[] = {{128, 7.5, 3.5, 0.8, 1.25}, {256, 11, 7, 1.75, 0}};

// The tiles of a product of T rows in E groups, whose sizes only the device knows, with N columns and depth K: the cheapest
// by those figures for groups of equal size, each of which ends inside a tile. 0: rows_grouped_kernel, for up to 16 rows.
// Measured in tiles of 64 x 128, 128 and 256, in us: 512 rows in 64 groups, 2560 columns, K = 1024: 18, 20, 33; 4000 in 32, 2560,
// 2560: 38, 33, 51; 8192 in 16, 4096, 2560: 80, 66, 75; 4096 in 8, 14336, 4096: 216, 176, 186; 16384 in 8: 828, 639, 568. Where the
// weights' bytes set the time of more than one, their own figures decide: 2000 in 64, 1024, 2560: 17.9, 19.5, 28.1, in tiles of 64 20.2.
inline int grouped_tile(int64_t T, int64_t N, int64_t K, int64_t E, int cus) {
  if (T <= 16) return 0;
  const double some = E < T ? E : T, each = T / some, least = 3.5 + some * N * K * (17 / 32.) / 5e6;
  int tile = 0;
  double best = 1e30;
  for (const TileCost& c : GROUPED_COSTS) {
    const double down = each / tile_rows(c.tile) + 0.5, rows = some * (down > 1 ? down : 1);
    double us = tiles_us(c, (int64_t)(rows * ((N + tile_columns(c.tile) - 1) / tile_columns(c.tile))), (stages_of(K) + 1) & ~1, cus);
    if (us < least) us = least + 0.01 * us;
    if (us < best) best = us, tile = c.tile;
  }
  return tile;
}

// The tiles of E products of M x N outputs that contract T rows between them. With the gradient's quantisation, in tiles of 128 and
// 256: 8192 rows, 16 of 4096 x 2560: 154 and 150 us; 16384, 2 of 4096 x 4096: 197 and 169; 200 rows, 8 of 1024 x 2560 in FP32: 29 and 42.
inline int gradient_tile(int64_t T, int64_t M, int64_t N, int64_t E, int cus) {
  int tile = 0;
  double best = 1e30;
  for (const TileCost& c : GRADIENT_COSTS) {
    const int64_t tiles = E * ((M + c.tile - 1) / c.tile) * ((N + c.tile - 1) / c.tile);
    const double us = tiles_us(c, tiles, (stages_of((T + E - 1) / E) + 1) & ~1, cus);
    if (us < best) best = us, tile = c.tile;
  }
  return tile;
}

}  // namespace mx
