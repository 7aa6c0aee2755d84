// Tiles of MXFP4 products with an epilogue, of products whose rows are in groups with operands of their own, and of products
// that contract each group's rows: the stages of mx_tile.h, fed by other jobs and followed by another way out.
//
// The sums leave through LDS as FP32 (y's rounding comes behind the residual), 16 rows of a wave's columns at a time: a lane then
// holds 8 neighbouring columns of a row (4 of FP32), so that residual, z and y move in whole lines, and bias and activation
// are taken in between. The residual's values are asked for two parts before they are added.
#pragma once
#include "mx_epilogue.h"
#include "mx_groups.h"
#include "mx_tile.h"

namespace mx {

enum Mode {
  DENSE,   // y = f(A B^T + bias) + residual
  ROWS,    // the same, A's rows and y's in groups, each with rows of B and a bias of its own
  DEPTH,   // y_e = A_e B_e^T over the positions of group e
};

struct Args {
  fp4_mx a, b;
  void* y;
  int64_t ldy;
  int M, N, K;            // DEPTH: K rows in groups
  int tiles_m, tiles_n;   // ROWS: tiles_m is not known
  int fill;               // ROWS: rows of no group become the residual, or zero
  fp4_epilogue epi;
  Groups groups;
  int64_t step_q, step_s;  // ROWS: bytes from one group's B to the next
};

// A tile: first row and column, the row behind the last that counts, its group, its stages, the blocks of its depth, and
// where its depth begins, in blocks.
struct Piece {
  int m0, n0, end, e, s1, nb, from;
};

// As place() of mx_gemm.hip's kernel, within one group's tiles.
__device__ __forceinline__ void walk(int t, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int BAND = 4;
  const int per = BAND * tiles_n, band = t / per, in = t - band * per;
  const int h = min(BAND, tiles_m - band * BAND);
  tn = in / h;
  tm = band * BAND + in - tn * h;
}

// Sums S of a wave, 16 rows and the columns of a half, to its LDS.
template <int S, class G, int SPLIT>
__device__ __forceinline__ void stage_sums(const f32x4 (&acc)[G::TM][G::TN], uint8_t* in) {
  constexpr int TJ = G::TN / SPLIT;
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    f32x4 v = acc[S / SPLIT][S % SPLIT * TJ + j];
    asm volatile("; part %1" : "+a"(v) : "n"(S));  // nothing to do, but different in each part (stage_any)
    *reinterpret_cast<f32x4*>(in + j * 64) = v;
  }
}
// The same for s in [FROM, TO): registers have no index, so a branch finds them. Branches alike would be made one again, with
// the sums in memory.
template <int FROM, int TO, class G, int SPLIT>
__device__ __forceinline__ void stage_any(int s, const f32x4 (&acc)[G::TM][G::TN], uint8_t* in) {
  if constexpr (TO - FROM == 1) {
    stage_sums<FROM, G, SPLIT>(acc, in);
  } else {
    constexpr int MID = (FROM + TO) / 2;
    if (s < MID) stage_any<FROM, MID, G, SPLIT>(s, acc, in);
    else stage_any<MID, TO, G, SPLIT>(s, acc, in);
  }
}

// This wave's sums, rows row0 + 16 i .., columns col0 + 16 j .., to y; rows from `end` on and columns from N on are not there.
// One loop body serves every 16 rows: written out, 256 sums' way through it would be 130 KB of code.
template <int OUT, class G>
__device__ __forceinline__ void store_epilogue(const f32x4 (&acc)[G::TM][G::TN], const fp4_epilogue& epi, int64_t bias_at, void* y,
                                               int64_t ldy, int row0, int end, int col0, int N, int lane, uint8_t* stage) {
  constexpr int SPLIT = G::TN == 8 ? 2 : 1, COLS = 16 * G::TN / SPLIT, STRIDE = COLS * 4 + 16, ALL = G::TM * SPLIT;
  constexpr int W = OUT == FP4_TYPE_F32 ? 4 : 8;                   // columns of a lane
  constexpr int PER = COLS / W, ROWS = 64 / PER, STEPS = 16 / ROWS;  // lanes per row, rows per step
  const int n = lane & 15, g = lane >> 4;
  uint8_t* const in = stage + n * STRIDE + 16 * g;
  const uint8_t* const out = stage + lane / PER * STRIDE + lane % PER * (4 * W);
  const int row_of = row0 + lane / PER, col_of = col0 + lane % PER * W;
  const int all = min(ALL, (end - row0 + 15) / 16 * SPLIT);
  if (all <= 0 || col0 >= N) return;

  float bias[SPLIT][W];
#pragma unroll
  for (int h = 0; h < SPLIT; ++h) {
#pragma unroll
    for (int i = 0; i < W; ++i) bias[h][i] = 0;
    const int c = col_of + h * COLS;
    if (epi.bias && c < N) values_of(epi.bias_type, load_raw<W>(epi.bias_type, epi.bias, bias_at + c, N - c), bias[h]);
  }
  // part s: row tile s / SPLIT, columns' half s % SPLIT
  Raw<W> ahead[2][STEPS] = {};
  const auto ask = [&](int s, Raw<W>(&r)[STEPS]) {
    const int row = row_of + 16 * (s / SPLIT), col = col_of + s % SPLIT * COLS;
#pragma unroll
    for (int k = 0; k < STEPS; ++k)
      if (row + k * ROWS < end && col < N)
        r[k] = load_raw<W>(epi.residual_type, epi.residual, (int64_t)(row + k * ROWS) * epi.ldr + col, N - col);
  };
  if (epi.residual) {
    ask(0, ahead[0]);
    if (all > 1) ask(1, ahead[1]);
  }
#pragma unroll 1
  for (int s = 0; s < all; ++s) {
    stage_any<0, ALL, G, SPLIT>(s, acc, in);
    asm volatile("" ::: "memory");  // one wave's LDS accesses stay in order: no barrier
    float add[STEPS][W];
    if (epi.residual) {
#pragma unroll
      for (int k = 0; k < STEPS; ++k) {
        values_of(epi.residual_type, ahead[0][k], add[k]);
        ahead[0][k] = ahead[1][k];
      }
      if (s + 2 < all) ask(s + 2, ahead[1]);
    }
    const int row = row_of + 16 * (s / SPLIT), col = col_of + s % SPLIT * COLS, left = N - col;
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
      float f[W];
      __builtin_memcpy(f, out + k * ROWS * STRIDE, 4 * W);
      const bool there = row + k * ROWS < end && col < N;
#pragma unroll
      for (int i = 0; i < W; ++i) f[i] += SPLIT == 2 && s % SPLIT ? bias[SPLIT - 1][i] : bias[0][i];
      if (epi.z && there) store_values<FP4_TYPE_F32>(epi.z, (int64_t)(row + k * ROWS) * epi.ldz + col, f, left);
      activate(epi.activation, f);
      if (epi.residual)
#pragma unroll
        for (int i = 0; i < W; ++i) f[i] += add[k][i];
      if (there) store_values<OUT>(y, (int64_t)(row + k * ROWS) * ldy + col, f, left);
    }
    asm volatile("" ::: "memory");
  }
}

// Rows of no group: the residual, or zero.
template <int OUT>
__device__ __forceinline__ void fill_row(const fp4_epilogue& epi, void* y, int64_t ldy, int64_t row, int N, int thread, int threads) {
  for (int c = thread; c < N; c += threads) {
    float f[1] = {0};
    if (epi.residual) values_of(epi.residual_type, load_raw<1>(epi.residual_type, epi.residual, row * epi.ldr + c, 1), f);
    store_values<OUT>(y, row * ldy + c, f, 1);
  }
}

// Whether a workgroup takes several tiles: tiles of which one fits a compute unit. (The others overlap by sharing a unit.)
template <class G>
constexpr bool STREAMED = G::NBUF == 2 && G::LDS > 80 * 1024;

template <class G, int OUT, Mode MODE>
__global__ void __launch_bounds__(G::THREADS, G::LDS > 80 * 1024 ? G::WAVES / 4 : G::WAVES / 2) product_kernel(Args p) {
  constexpr int BM = G::BM, BN = G::BN, NBUF = G::NBUF;
  extern __shared__ uint8_t lds[];
  Wave<G> w;
  w.lds = lds;
  w.lane = threadIdx.x & 63;
  w.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = w.lane & 15, g = w.lane >> 4;
  const int N = p.N;
  w.src.ldqa = (int)p.a.ldq, w.src.ldqb = (int)p.b.ldq, w.src.ldsa = (int)p.a.lds, w.src.ldsb = (int)p.b.lds;

  int* const start = reinterpret_cast<int*>(lds + G::LDS);
  int* const units = start + p.groups.E + 1;
  int total = p.tiles_m * p.tiles_n;
  if constexpr (MODE != DENSE) {
    if (w.wave == 0) read_groups<MODE == ROWS ? BM : UNIT>(p.groups, MODE == ROWS ? p.M : p.K, start, units, w.lane);
    __syncthreads();
    if constexpr (MODE == DEPTH) total *= p.groups.E;
    if constexpr (MODE == ROWS) {
      total = uniform(units[p.groups.E]) * p.tiles_n;
      if (p.fill) {
        const int first = uniform(start[0]), last = uniform(start[p.groups.E]);
        for (int r = blockIdx.x; r < first + p.M - last; r += gridDim.x)
          fill_row<OUT>(p.epi, p.y, p.ldy, row_outside(r, first, last), N, threadIdx.x, G::THREADS);
      }
      if ((int)blockIdx.x >= total) return;
    }
  }

  const auto set_depth = [&](int nb) {  // this lane's valid blocks of the last group of four chunks
    w.last_group = max((nb + GM_STAGE_BLOCKS - 1) / GM_STAGE_BLOCKS - 1, 0) >> 1;
    w.tail = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (16 * w.last_group + 4 * c + g < nb) w.tail |= 0xffu << (8 * c);
  };

  // this wave's first rows in LDS (multiples of 16)
  const int arow = w.wave / G::WN * (BM / G::WM), brow = BM + w.wave % G::WN * (BN / G::WN);
  const uint32_t at = n * GM_ROW_BYTES + ((g ^ swizzle(n)) << 4);
  w.frag_a = arow * GM_ROW_BYTES + at, w.frag_b = brow * GM_ROW_BYTES + at;
  const uint32_t scale_at = G::SG * 16 * n + (G::SG == 2 ? (n >> 3) * 16 : 0);
  w.scale_a = G::SG * 16 * arow + scale_at, w.scale_b = G::SG * 16 * brow + scale_at;

  // tile `id`. Workgroups go round-robin over the 8 XCDs: XCD x takes a contiguous run of the tiles.
  const auto piece_of = [&](int id) {
    Piece j;
    const int xcds = 8, x = id % xcds, q = total / xcds, r = total % xcds;
    int t = x * q + min(x, r) + id / xcds, tm, tn;  // bijective for any total
    j.e = j.from = 0, j.end = p.M, j.nb = (int)blocks_of(p.K);
    int first = 0, tiles_m = p.tiles_m;
    if constexpr (MODE == ROWS) {
      j.e = group_of(units, p.groups.E, t / p.tiles_n, w.lane);
      const int before = uniform(units[j.e]);
      t -= before * p.tiles_n;
      tiles_m = uniform(units[j.e + 1]) - before;
      first = uniform(start[j.e]), j.end = uniform(start[j.e + 1]);
    } else if constexpr (MODE == DEPTH) {
      const int tiles = p.tiles_m * p.tiles_n;
      j.e = t / tiles;
      t -= j.e * tiles;
      j.nb = (uniform(start[j.e + 1]) - uniform(start[j.e]) + BLOCK - 1) / BLOCK;
      j.from = uniform(units[j.e]) * (UNIT / BLOCK);
    }
    walk(t, tiles_m, p.tiles_n, tm, tn);
    j.m0 = first + tm * BM, j.n0 = tn * BN;
    j.s1 = (j.nb + GM_STAGE_BLOCKS - 1) / GM_STAGE_BLOCKS;
    return j;
  };
  const auto load_from = [&](const Piece& j) {
    const int ma = min(j.end - j.m0, BM), mb = min(N - j.n0, BN), sbytes = (j.nb + 3) & ~3;
    const int64_t qa = j.m0 * p.a.ldq + j.from * BLOCK_BYTES, sa = j.m0 * p.a.lds + j.from;
    int64_t qb = j.n0 * p.b.ldq + j.from * BLOCK_BYTES, sb = j.n0 * p.b.lds + j.from;
    if constexpr (MODE == ROWS) qb += j.e * p.step_q, sb += j.e * p.step_s;
    w.src.aq = fp4::make_rsrc(static_cast<const uint8_t*>(p.a.q) + qa, (uint32_t)((ma - 1) * (int)p.a.ldq + j.nb * 16));
    w.src.as = fp4::make_rsrc(static_cast<const uint8_t*>(p.a.s) + sa, (uint32_t)((ma - 1) * (int)p.a.lds + sbytes));
    w.src.bq = fp4::make_rsrc(static_cast<const uint8_t*>(p.b.q) + qb, (uint32_t)((mb - 1) * (int)p.b.ldq + j.nb * 16));
    w.src.bs = fp4::make_rsrc(static_cast<const uint8_t*>(p.b.s) + sb, (uint32_t)((mb - 1) * (int)p.b.lds + sbytes));
    if constexpr (MODE == DEPTH) set_depth(j.nb);
  };
  if constexpr (MODE != DEPTH) set_depth((int)blocks_of(p.K));
  const auto codes_from = [](int st, int end) { return st < end ? (uint32_t)st * GM_ROW_BYTES : NOTHING; };
  const auto scales_from = [](int st, int end) { return st < end ? (uint32_t)((st >> 1) / G::SG * G::SG) * 16 : NOTHING; };

  int id = blockIdx.x;
  Piece job = piece_of(id);
  load_from(job);
#pragma unroll
  for (int i = 0; i < NBUF; ++i) {
    const int ring = w.ring_of(i >> 1);
    issue_codes<G, 0, G::SLOTS>(w.src, w.codes(ring, i & 1), codes_from(i, job.s1), w.wave, w.lane);
    if (!(i & 1) && (G::SG == 1 || i == 0)) issue_scales<G>(w.src, w.scales(i >> 1), scales_from(i, job.s1), w.wave, w.lane);
  }
  wait_and_meet<G::BEHIND + G::SLOTS>();
#pragma unroll
  for (int i = 0; i < G::OPS; ++i) {
    w.op[0][i] = w.read_op(0, 0, 0, i);
    w.raw[i] = w.read_raw(0, i);
  }
#pragma unroll
  for (int i = 0; i < G::OPS; ++i) w.sc[0][i] = w.pick(i, 0);

  for (;;) {
#pragma unroll
    for (int i = 0; i < G::TM; ++i)
#pragma unroll
      for (int j = 0; j < G::TN; ++j) w.acc[i][j] = f32x4{0, 0, 0, 0};
    __builtin_amdgcn_sched_barrier(0);
    Piece next = job;
    id += gridDim.x;
    // As gemm_kernel's loop: two stages (one group of scales) at a time, one tile's last stages loading the next tile's first.
    // The scales of the stages at hand have been picked when the sources, and with them the depth's mask, change.
    int st = 0;
    do {
      int ahead = st + NBUF, end = job.s1, next_group = (st >> 1) + 1;
      if (st + 2 >= job.s1) {
        if (STREAMED<G> && id < total) {
          next = piece_of(id);
          load_from(next);
          ahead = 0, end = next.s1;
        }
        next_group = 0;
      }
      w.template chunk<0, 0, 0>(st >> 1, next_group, 0, 0);
      w.template chunk<1, 0, 0>(st >> 1, next_group, codes_from(ahead, end), scales_from(ahead, end));
      w.template chunk<2, 0, 0>(st >> 1, next_group, 0, 0);
      w.template chunk<3, 0, 0>(st >> 1, next_group, codes_from(ahead + 1, end), 0);
#pragma unroll
      for (int i = 0; i < G::OPS; ++i) w.sc[0][i] = w.sc[1][i];
      __builtin_amdgcn_sched_barrier(0);
      st += 2;
    } while (st < job.s1);

    // the MFMAs' sums are there behind these waits, as in gemm_kernel
    wait_for_sums<G>(w.acc);
#pragma unroll
    for (int i = 0; i < G::TM; ++i)
#pragma unroll
      for (int j = 0; j < G::TN; ++j) asm volatile("" : "+a"(w.acc[i][j]));
    uint8_t* stage = lds + G::RING + w.wave * G::STAGE;
    if constexpr (!STREAMED<G>) {
      // the ring is free: every wave's reads of it are done and no direct load is on its way
      wait_and_meet<0>();
      stage = lds + w.wave * (16 * (64 * G::TN + 16));
    }
    void* const y = MODE == DEPTH ? static_cast<uint8_t*>(p.y) + (int64_t)job.e * p.M * p.ldy * elem_bytes(OUT) : p.y;
    store_epilogue<OUT, G>(w.acc, p.epi, (int64_t)job.e * N, y, p.ldy, job.m0 + arow, job.end, job.n0 + brow - BM, N, w.lane, stage);
    if (!STREAMED<G> || id >= total) break;
    job = next;
  }
  // no direct load may be on its way when the workgroup ends and its LDS goes to another
  __builtin_amdgcn_s_waitcnt(0);
}

// `tiles`: the most tiles there can be.
template <class G, int OUT, Mode MODE>
static int launch_product(const Args& p, int64_t tiles, hipStream_t st) {
  static Fp4LdsLimit limit;
  const int lds = G::LDS + (MODE == DENSE ? 0 : group_table_bytes(p.groups.E));
  limit.ensure(reinterpret_cast<const void*>(&product_kernel<G, OUT, MODE>), G::LDS + (MODE == DENSE ? 0 : group_table_bytes(MAX_GROUPS)));
  const int units = fp4_device_cus() & ~7;  // a multiple of the 8 XCDs: a workgroup's tiles stay on its XCD
  const int64_t wgs = STREAMED<G> && units > 0 && tiles > units ? units : tiles;
  if (tiles > (1LL << 30) || !fits_launch(wgs, G::THREADS)) return FP4_ERR_UNSUPPORTED;
  return fp4_launch(product_kernel<G, OUT, MODE>, dim3((unsigned)wgs), dim3(G::THREADS), lds, st, p);
}

using Tile256 = Tile<256, 256, 2, 2, 2, 1>;
using Tile128 = Tile<128, 128, 2, 2, 2, 1>;
using Tile64 = Tile<64, 64, 2, 2, 4, 2>;
static_assert(Tile256::STAGE >= 16 * (64 * 4 + 16), "a wave's staging rows of 64 FP32 sums");
static_assert(Tile256::LDS + group_table_bytes(MAX_GROUPS) <= 160 * 1024, "");

template <int OUT, Mode MODE>
static int launch_tile(int tile, const Args& p, int64_t tiles, hipStream_t st) {
  if (tile == 256) return launch_product<Tile256, OUT, MODE>(p, tiles, st);
  if (tile == 128) return launch_product<Tile128, OUT, MODE>(p, tiles, st);
  return launch_product<Tile64, OUT, MODE>(p, tiles, st);
}
template <Mode MODE>
static int launch_out(int out_type, int tile, const Args& p, int64_t tiles, hipStream_t st) {
  if (out_type == FP4_TYPE_F32) return launch_tile<FP4_TYPE_F32, MODE>(tile, p, tiles, st);
  if (out_type == FP4_TYPE_BF16) return launch_tile<FP4_TYPE_BF16, MODE>(tile, p, tiles, st);
  return launch_tile<FP4_TYPE_F16, MODE>(tile, p, tiles, st);
}

}  // namespace mx
