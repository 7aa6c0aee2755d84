// Rows in groups (one per expert) whose bounds lie in device memory: reading them, and finding a tile's group.
#pragma once
#include "mx.h"

namespace mx {

constexpr int MAX_GROUPS = 512;
constexpr int UNIT = 256;  // positions that every group's part of an operand along the rows is padded to: a stage of the tiles

// Group e's rows are [start[e], start[e + 1]). `offsets` null: `each` rows per group.
struct Groups {
  const void* offsets;
  int E, wide;  // wide: 64-bit offsets
  int each;
};

// Tables in LDS: start[E + 1], and in the quantisation units[E + 1] with the units in front of each group. The products' tiles have the
// number of all units behind start and find a tile's group from start each time, so that two of them fit a compute unit however
// many groups there are: 40000 rows in 384 groups of 1024 x 1024 take 57 us, with both tables, one workgroup to a unit, 84.
constexpr int group_table_bytes(int E) { return ((E + 2) * 4 + 15) & ~15; }

// Bound e of the groups, in [0, T]: whatever the memory holds, no row past T belongs to a group.
__device__ __forceinline__ int bound_at(const Groups& g, int e, int T) {
  int64_t v;
  if (!g.offsets) v = (int64_t)e * g.each;
  else v = g.wide ? static_cast<const int64_t*>(g.offsets)[e] : static_cast<const int32_t*>(g.offsets)[e];
  return (int)(v < 0 ? 0 : v > T ? T : v);
}

// Inclusive scans over the wave's lanes, of values that are not negative: within rows of 16, then rows 1 and 3 take the last of
// the row before, rows 2 and 3 the last of the first half. A few cycles a step, where exchanges through LDS take a hundred.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ int from_lane(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, ROWS == 0xf);
}
constexpr int DPP_ROW_SHR = 0x110, DPP_WAVE_SHR1 = 0x138, DPP_ROW_BCAST15 = 0x142, DPP_ROW_BCAST31 = 0x143;
template <class F>
__device__ __forceinline__ int scan(int v, F op) {
  v = op(v, from_lane<DPP_ROW_SHR + 1>(v));
  v = op(v, from_lane<DPP_ROW_SHR + 2>(v));
  v = op(v, from_lane<DPP_ROW_SHR + 4>(v));
  v = op(v, from_lane<DPP_ROW_SHR + 8>(v));
  v = op(v, from_lane<DPP_ROW_BCAST15, 0xa>(v));
  return op(v, from_lane<DPP_ROW_BCAST31, 0xc>(v));
}
__device__ __forceinline__ int scan_max(int v) {
  return scan(v, [](int a, int b) { return max(a, b); });
}
__device__ __forceinline__ int scan_sum(int v) {
  return scan(v, [](int a, int b) { return a + b; });
}

// Fills the tables (one wave; the caller's barrier makes them visible), `units` where it is given, and returns the number of units.
// Bounds that decrease count as the largest in front of them, so that groups never overlap and their rows are T at most.
template <int UNIT_ROWS>
__device__ __forceinline__ int read_groups(const Groups& g, int T, int* start, int* units, int lane) {
  int most = 0, sum = 0;
  for (int base = 0; base <= g.E; base += 64) {
    const int e = base + lane;
    const int v = max(scan_max(e <= g.E ? bound_at(g, e, T) : 0), most);
    // the units of group e - 1, which ends here; the first lane's began in the 64 bounds before
    int before = from_lane<DPP_WAVE_SHR1>(v);
    if (lane == 0) before = base ? most : v;
    const int n = scan_sum((v - before + UNIT_ROWS - 1) / UNIT_ROWS) + sum;
    if (e <= g.E) {
      start[e] = v;
      if (units) units[e] = n;
    }
    most = __builtin_amdgcn_readlane(v, 63);
    sum = __builtin_amdgcn_readlane(n, 63);
  }
  return sum;
}

// The group that unit u lies in: as many groups end at or before it.
__device__ __forceinline__ int group_of(const int* units, int E, int u, int lane) {
  int e = 0;
  for (int base = 0; base < E; base += 64) {
    const bool past = base + lane < E && units[min(base + lane + 1, E)] <= u;
    e += __builtin_popcountll(__builtin_amdgcn_ballot_w64(past));
  }
  return e;
}

// The same by the rows' bounds alone, and the units in front of the group.
struct Found {
  int e, before;
};
template <int UNIT_ROWS>
__device__ __forceinline__ Found find_group(const int* start, int E, int u, int lane) {
  Found f{0, 0};
  for (int base = 0; base < E; base += 64) {
    const int rows = start[min(base + lane + 1, E)] - start[min(base + lane, E)];
    const int n = f.before + scan_sum((rows + UNIT_ROWS - 1) / UNIT_ROWS);
    const int past = __builtin_popcountll(__builtin_amdgcn_ballot_w64(base + lane < E && n <= u));
    f.e += past;
    if (past > 0) f.before = __builtin_amdgcn_readlane(n, past - 1);
    if (past < 64) break;
  }
  return f;
}
// The units in front of group e.
template <int UNIT_ROWS>
__device__ __forceinline__ int units_before(const int* start, int e, int lane) {
  int sum = 0;
  for (int base = 0; base < e; base += 64) {
    const int rows = start[min(base + lane + 1, e)] - start[min(base + lane, e)];
    sum += __builtin_amdgcn_readlane(scan_sum((rows + UNIT_ROWS - 1) / UNIT_ROWS), 63);
  }
  return sum;
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Row r of those that belong to no group (in front of the first and behind the last), of `rest` in all.
__device__ __forceinline__ int row_outside(int r, int first, int end) { return r < first ? r : end + r - first; }

// ------------------------------------------------------------------------------------------------ host side

static inline int check_groups(const fp4_groups* g) {
  if (!g || !g->offsets) return FP4_ERR_ARG;
  if (g->bits != 32 && g->bits != 64) return FP4_ERR_ARG;
  if (g->count < 1) return FP4_ERR_SHAPE;
  if (g->count > MAX_GROUPS) return FP4_ERR_UNSUPPORTED;
  return fp4_aligned(g->offsets, (uintptr_t)g->bits / 8) ? FP4_OK : FP4_ERR_ALIGN;
}

static inline Groups groups_of(const fp4_groups& g) { return {g.offsets, (int)g.count, g.bits == 64, 0}; }

// The most tiles of `rows` rows that T rows in E groups can make.
static inline int64_t most_tiles(int64_t T, int64_t E, int64_t rows) {
  const int64_t some = E < T ? E : T;
  return (T - some) / rows + some;
}

int launch_rows_grouped(int x_type, int out_type, int T, int N, int K, const Groups& groups, const void* x, int64_t ldx, const fp4_mx* a,
                        const fp4_mx& b, int64_t step_q, int64_t step_s, const fp4_epilogue* epi, void* y, int64_t ldy, int fill,
                        hipStream_t st);

}  // namespace mx
