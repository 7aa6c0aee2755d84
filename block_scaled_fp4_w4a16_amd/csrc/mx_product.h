// Tiles of MXFP4 products with an epilogue, of products whose rows are in groups with operands of their own, and of products
// that contract each group's rows: the stages of mx_tile.h, fed by other jobs and followed by another way out.
//
// The sums leave through LDS as FP32 (y's rounding comes behind the residual), 16 rows of a wave's columns at a time: a lane then
// holds 8 neighbouring columns of a row (4 of FP32), so that residual, z and y move in whole lines, and bias and activation
// are taken in between.
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
  int whole;              // as store_epilogue takes it
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

__device__ __forceinline__ uint32_t lds_address(const uint8_t* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)p;
}

// LDS accesses of the way out are written out: with LDS that direct loads write to, the compiler has every read and write of
// LDS wait for all of a wave's memory accesses, stores included, a thousand cycles each. A wave's LDS accesses stay in order.
// Part S of a wave's sums, 16 rows and the columns of a half, to its LDS. (The part's number in the text keeps the branches
// of stage_any apart: branches alike would be made one again, with the sums in memory.)
template <int S, class G, int SPLIT>
__device__ __forceinline__ void stage_sums(const f32x4 (&acc)[G::TM][G::TN], uint32_t in) {
  constexpr int I = S / SPLIT, J = S % SPLIT * (G::TN / SPLIT);
  if constexpr (G::TN / SPLIT == 4)
    asm volatile("ds_write_b128 %0, %1\n\tds_write_b128 %0, %2 offset:64\n\tds_write_b128 %0, %3 offset:128\n\t"
                 "ds_write_b128 %0, %4 offset:192 ; part %5"
                 :
                 : "v"(in), "a"(acc[I][J]), "a"(acc[I][J + 1]), "a"(acc[I][J + 2]), "a"(acc[I][J + 3]), "n"(S)
                 : "memory");
  else
    asm volatile("ds_write_b128 %0, %1\n\tds_write_b128 %0, %2 offset:64 ; part %3"
                 :
                 : "v"(in), "a"(acc[I][J]), "a"(acc[I][J + 1]), "n"(S)
                 : "memory");
}
// The same for s = FROM, FROM + BY, .. < TO: registers have no index, so branches find them.
template <int FROM, int TO, int BY, class G, int SPLIT>
__device__ __forceinline__ void stage_any(int s, const f32x4 (&acc)[G::TM][G::TN], uint32_t in) {
  if constexpr (TO - FROM <= BY) {
    stage_sums<FROM, G, SPLIT>(acc, in);
  } else {
    constexpr int MID = FROM + (TO - FROM) / BY / 2 * BY;
    if (s < MID) stage_any<FROM, MID, BY, G, SPLIT>(s, acc, in);
    else stage_any<MID, TO, BY, G, SPLIT>(s, acc, in);
  }
}
// A lane's share of a part back from LDS: 16 bytes at each of two (N 2) or four places.
template <int N, int O1, int O2, int O3>
__device__ __forceinline__ void read_part(uint32_t out, f32x4 (&v)[N]) {
  static_assert(N == 2 || N == 4, "");
  if constexpr (N == 4)
    asm volatile("ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:%5\n\tds_read_b128 %2, %4 offset:%6\n\t"
                 "ds_read_b128 %3, %4 offset:%7\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
                 : "v"(out), "n"(O1), "n"(O2), "n"(O3)
                 : "memory");
  else
    asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %2 offset:%3\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(v[0]), "=&v"(v[1])
                 : "v"(out), "n"(O1)
                 : "memory");
}

// How a wave's sums leave: in parts of 16 rows and COLS columns.
template <int OUT, class G>
struct Way {
  static constexpr int SPLIT = G::NBUF == 2 ? 2 : 1, COLS = 16 * G::TN / SPLIT, STRIDE = COLS * 4 + 16, ALL = G::TM * SPLIT;
  static constexpr int W = OUT == FP4_TYPE_F32 ? 4 : 8;                     // columns of a lane
  static constexpr int PER = COLS / W, ROWS = 64 / PER, STEPS = 16 / ROWS;  // lanes per row, rows per step
  static constexpr int READS = STEPS * W / 4;                               // of 16 bytes, per lane and part
  static constexpr int offset(int r) { return r / (W / 4) * ROWS * STRIDE + r % (W / 4) * 16; }
  static __device__ __forceinline__ void read(uint32_t out, f32x4 (&v)[READS]) {
    read_part<READS, offset(1), offset(2), offset(3)>(out, v);
  }
};

// W values of a 16-bit type (32-bit, if F32) by a buffer access, whose descriptor drops what lies behind its last row.
template <bool F32, int W>
__device__ __forceinline__ Raw<W> buffer_raw(__amdgpu_buffer_rsrc_t r, uint32_t at) {
  Raw<W> v{};
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(r, at + 16 * i, 0, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) v.v[4 * i + j] = x[j];
    }
  } else if constexpr (W == 8) {
    const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) v.v[j] = x[j];
  } else {
    const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0);
    v.v[0] = x[0], v.v[1] = x[1];
  }
  return v;
}
// 16 bytes out; `past`: marked as not to be kept in the caches.
__device__ __forceinline__ void put(__amdgpu_buffer_rsrc_t r, uint32_t at, const u32x4& x, bool past) {
  if (past) __builtin_amdgcn_raw_buffer_store_b128(x, r, at, 0, 2);
  else __builtin_amdgcn_raw_buffer_store_b128(x, r, at, 0, 0);
}
template <int OUT, int W>
__device__ __forceinline__ void buffer_store(__amdgpu_buffer_rsrc_t r, uint32_t at, const float (&f)[W], bool past) {
  if constexpr (OUT == FP4_TYPE_F32) {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      u32x4 x;
      __builtin_memcpy(&x, f + 4 * i, 16);
      put(r, at + 16 * i, x, past);
    }
  } else {
    static_assert(W == 8, "");
    put(r, at, u32x4{pack2<OUT>(f[0], f[1]), pack2<OUT>(f[2], f[3]), pack2<OUT>(f[4], f[5]), pack2<OUT>(f[6], f[7])}, past);
  }
}

// This wave's sums to y where all their columns exist, rows are aligned to 4 bytes and not too far apart for a descriptor.
// RES: 0 no residual, 1 of 16 bits, 2 of 32; Z: z is kept. Nothing branches around a memory access, so the compiler knows how
// many a residual has behind it: it is asked for U parts ahead and waits for no store that is younger.
template <int OUT, class G, int RES, bool Z>
__device__ __forceinline__ void store_whole(const f32x4 (&acc)[G::TM][G::TN], const fp4_epilogue& epi, int64_t bias_at, void* y,
                                            int64_t ldy, int row0, int rows, int col0, int lane, uint8_t* stage, bool past) {
  using P = Way<OUT, G>;
  constexpr int W = P::W, U = P::ALL < 4 ? P::ALL : 4, EB = elem_bytes(OUT), RB = RES == 2 ? 4 : 2, WIDTH = P::COLS * P::SPLIT;
  const int n = lane & 15, g = lane >> 4, r = lane / P::PER, c = lane % P::PER * W;
  const uint32_t in = lds_address(stage) + n * P::STRIDE + 16 * g, out = lds_address(stage) + r * P::STRIDE + 4 * c;
  const auto descriptor = [&](const void* p, int64_t ld, int eb) {
    return fp4::make_rsrc(static_cast<const uint8_t*>(p) + (row0 * ld + col0) * eb, (uint32_t)(((rows - 1) * (int)ld + WIDTH) * eb));
  };
  const auto place = [&](int s, int k, int64_t ld, int eb) {
    return (uint32_t)(((16 * (s / P::SPLIT) + k * P::ROWS + r) * (int)ld + s % P::SPLIT * P::COLS + c) * eb);
  };
  const auto to = descriptor(y, ldy, EB);
  auto from = to, keep = to;
  if constexpr (RES != 0) from = descriptor(epi.residual, epi.ldr, RB);
  if constexpr (Z) keep = descriptor(epi.z, epi.ldz, 4);
  const int res_type = RES == 2 ? FP4_TYPE_F32 : epi.residual_type == FP4_TYPE_BF16 ? FP4_TYPE_BF16 : FP4_TYPE_F16;

  float bias[P::SPLIT][W] = {};
  if (epi.bias) load_pieces(epi.bias_type, epi.bias, bias_at + col0 + c, P::COLS, bias);
  Raw<W> ahead[U][P::STEPS];
  if constexpr (RES != 0)
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < P::STEPS; ++k) ahead[u][k] = buffer_raw<RES == 2, W>(from, place(u, k, epi.ldr, RB));
  const int all = min(P::ALL, (rows + 15) / 16 * P::SPLIT);
#pragma unroll 1
  for (int s0 = 0; s0 < all; s0 += U) {  // parts without rows in the last round: their stores are dropped
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = s0 + u;
      if (u == 0) stage_any<0, P::ALL, U, G, P::SPLIT>(s, acc, in);
      else if (u == 1) stage_any<1, P::ALL + 1, U, G, P::SPLIT>(s, acc, in);
      else if (u == 2) stage_any<2, P::ALL + 2, U, G, P::SPLIT>(s, acc, in);
      else stage_any<3, P::ALL + 3, U, G, P::SPLIT>(s, acc, in);
      f32x4 v[P::READS];
      P::read(out, v);
#pragma unroll
      for (int k = 0; k < P::STEPS; ++k) {
        float f[W];
        __builtin_memcpy(f, v + k * (W / 4), 4 * W);
#pragma unroll
        for (int i = 0; i < W; ++i) f[i] += bias[u % P::SPLIT][i];
        if constexpr (Z) buffer_store<FP4_TYPE_F32>(keep, place(s, k, epi.ldz, 4), f, false);
        activate(epi.activation, f);
        if constexpr (RES != 0) {
          float add[W];
          values_of(res_type, ahead[u][k], add);
#pragma unroll
          for (int i = 0; i < W; ++i) f[i] += add[i];
          ahead[u][k] = buffer_raw<RES == 2, W>(from, place(s + U, k, epi.ldr, RB));  // past the tile: nothing
        }
        buffer_store<OUT>(to, place(s, k, ldy, EB), f, past);
      }
    }
  }
}

// Row tile I of a wave's sums to v (a branch finds it, as in stage_any).
template <int I, class G>
__device__ __forceinline__ void take_sums(const f32x4 (&acc)[G::TM][G::TN], f32x4 (&v)[G::TN]) {
#pragma unroll
  for (int j = 0; j < G::TN; ++j) {
    v[j] = acc[I][j];
    asm volatile("; row tile %1" : "+v"(v[j]) : "n"(I));
  }
}
template <int FROM, int TO, class G>
__device__ __forceinline__ void take_any(int i, const f32x4 (&acc)[G::TM][G::TN], f32x4 (&v)[G::TN]) {
  if constexpr (TO - FROM == 1) {
    take_sums<FROM, G>(acc, v);
  } else {
    constexpr int MID = (FROM + TO) / 2;
    if (i < MID) take_any<FROM, MID, G>(i, acc, v);
    else take_any<MID, TO, G>(i, acc, v);
  }
}

// store_whole for 16-bit y without residual and z: everything is done where the sums are, four columns of a row to a lane, and
// goes through LDS rounded, whole rows of the wave's columns at a time.
template <int OUT, class G>
__device__ __forceinline__ void store_rounded(const f32x4 (&acc)[G::TM][G::TN], const fp4_epilogue& epi, int64_t bias_at, void* y,
                                              int64_t ldy, int row0, int rows, int col0, int lane, uint8_t* stage, bool past) {
  constexpr int COLS = 16 * G::TN, STRIDE = COLS * 2 + 16, PER = COLS / 8, ROWS = 64 / PER, STEPS = 16 / ROWS, TN = G::TN;
  const int n = lane & 15, g = lane >> 4, r = lane / PER, c = lane % PER * 8;
  const uint32_t in = lds_address(stage) + n * STRIDE + 8 * g, out = lds_address(stage) + r * STRIDE + 2 * c;
  const auto to = fp4::make_rsrc(static_cast<uint8_t*>(y) + (row0 * ldy + col0) * 2, (uint32_t)(((rows - 1) * (int)ldy + COLS) * 2));
  float bias[TN][4] = {};
  if (epi.bias) load_pieces(epi.bias_type, epi.bias, bias_at + col0 + 4 * g, 16, bias);
  const int all = min(G::TM, (rows + 15) / 16);
#pragma unroll 1
  for (int i = 0; i < all; ++i) {
    f32x4 v[TN];
    take_any<0, G::TM, G>(i, acc, v);
    float f[4 * TN];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) f[4 * j + e] = v[j][e] + bias[j][e];
    activate(epi.activation, f);
    u32x2 h[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) h[j] = u32x2{pack2<OUT>(f[4 * j], f[4 * j + 1]), pack2<OUT>(f[4 * j + 2], f[4 * j + 3])};
    asm volatile("ds_write_b64 %0, %1\n\tds_write_b64 %0, %2 offset:32" : : "v"(in), "v"(h[0]), "v"(h[1]) : "memory");
    if constexpr (TN >= 4) asm volatile("ds_write_b64 %0, %1 offset:64\n\tds_write_b64 %0, %2 offset:96" : : "v"(in), "v"(h[2]), "v"(h[3]) : "memory");
    if constexpr (TN == 8)
      asm volatile("ds_write_b64 %0, %1 offset:128\n\tds_write_b64 %0, %2 offset:160\n\tds_write_b64 %0, %3 offset:192\n\t"
                   "ds_write_b64 %0, %4 offset:224"
                   :
                   : "v"(in), "v"(h[4]), "v"(h[5]), "v"(h[6]), "v"(h[7])
                   : "memory");
    const uint32_t at = (uint32_t)(((16 * i + r) * (int)ldy + c) * 2), step = ROWS * (int)ldy * 2;
    if constexpr (STEPS == 1) {
      f32x4 o;
      asm volatile("ds_read_b128 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(o) : "v"(out) : "memory");
      put(to, at, __builtin_bit_cast(u32x4, o), past);
    } else {
      f32x4 o[STEPS];
      read_part<STEPS, ROWS * STRIDE, 2 * ROWS * STRIDE, 3 * ROWS * STRIDE>(out, o);
#pragma unroll
      for (int k = 0; k < STEPS; ++k) {
        const f32x4 x = o[k];
        put(to, at + k * step, __builtin_bit_cast(u32x4, x), past);
      }
    }
  }
}

// The same where columns end inside the tile, or rows lie at any alignment: accesses of what is there.
template <int OUT, class G>
__device__ __forceinline__ void store_part(const f32x4 (&acc)[G::TM][G::TN], const fp4_epilogue& epi, int64_t bias_at, void* y,
                                           int64_t ldy, int row0, int rows, int col0, int N, int lane, uint8_t* stage) {
  using P = Way<OUT, G>;
  constexpr int W = P::W;
  const int n = lane & 15, g = lane >> 4, r = lane / P::PER;
  const uint32_t in = lds_address(stage) + n * P::STRIDE + 16 * g, out = lds_address(stage) + r * P::STRIDE + lane % P::PER * (4 * W);
  const int all = min(P::ALL, (rows + 15) / 16 * P::SPLIT);
#pragma unroll 1
  for (int s = 0; s < all; ++s) {
    stage_any<0, P::ALL, 1, G, P::SPLIT>(s, acc, in);
    f32x4 v[P::READS];
    P::read(out, v);
    const int col = col0 + s % P::SPLIT * P::COLS + lane % P::PER * W, left = N - col;
    float bias[W] = {};
    if (epi.bias && left > 0) values_of(epi.bias_type, load_raw<W>(epi.bias_type, epi.bias, bias_at + col, left), bias);
#pragma unroll
    for (int k = 0; k < P::STEPS; ++k) {
      const int in_rows = 16 * (s / P::SPLIT) + k * P::ROWS + r;
      const int64_t row = row0 + in_rows;
      const bool there = in_rows < rows && left > 0;
      float f[W], add[W] = {};
      __builtin_memcpy(f, v + k * (W / 4), 4 * W);
      if (epi.residual && there) values_of(epi.residual_type, load_raw<W>(epi.residual_type, epi.residual, row * epi.ldr + col, left), add);
#pragma unroll
      for (int i = 0; i < W; ++i) f[i] += bias[i];
      if (epi.z && there) store_values<FP4_TYPE_F32>(epi.z, row * epi.ldz + col, f, left);
      activate(epi.activation, f);
      if (epi.residual)
#pragma unroll
        for (int i = 0; i < W; ++i) f[i] += add[i];
      if (there) store_values<OUT>(y, row * ldy + col, f, left);
    }
  }
}

// This wave's sums, rows row0 + 16 i .., columns col0 + 16 j .., to y; rows from `end` on and columns from N on are not there.
// `whole`: 0 where rows of y, z and the residual do not suit store_whole, 2 where y is not to be kept in the caches.
template <int OUT, class G>
__device__ __forceinline__ void store_epilogue(const f32x4 (&acc)[G::TM][G::TN], const fp4_epilogue& epi, int64_t bias_at, void* y,
                                               int64_t ldy, int row0, int end, int col0, int N, int lane, uint8_t* stage, int whole) {
  const int rows = min(end - row0, 16 * G::TM);
  if (rows <= 0 || col0 >= N) return;
#define MX_WHOLE(RES, Z) store_whole<OUT, G, RES, Z>(acc, epi, bias_at, y, ldy, row0, rows, col0, lane, stage, whole > 1)
  if (!whole || col0 + 16 * G::TN > N) {
    store_part<OUT, G>(acc, epi, bias_at, y, ldy, row0, rows, col0, N, lane, stage);
  } else if (!epi.residual) {
    if (epi.z) MX_WHOLE(0, true);
    else if constexpr (OUT == FP4_TYPE_F32) MX_WHOLE(0, false);
    else store_rounded<OUT, G>(acc, epi, bias_at, y, ldy, row0, rows, col0, lane, stage, whole > 1);
  } else if (epi.residual_type == FP4_TYPE_F32) {
    if (epi.z) MX_WHOLE(2, true);
    else MX_WHOLE(2, false);
  } else {
    if (epi.z) MX_WHOLE(1, true);
    else MX_WHOLE(1, false);
  }
#undef MX_WHOLE
}

// Rows of no group: the residual, or zero.
template <int OUT>
__device__ __forceinline__ void fill_row(const fp4_epilogue& epi, void* y, int64_t ldy, int64_t row, int N, int thread, int threads) {
  for (int c = 8 * thread; c < N; c += 8 * threads) {
    float f[8] = {};
    if (epi.residual) values_of(epi.residual_type, load_raw<8>(epi.residual_type, epi.residual, row * epi.ldr + c, N - c), f);
    store_values<OUT>(y, row * ldy + c, f, N - c);
  }
}

// Whether a workgroup takes several tiles, one's last stages loading the next one's first: with two buffers, which every tile
// begins alike.
template <class G>
constexpr bool STREAMED = G::NBUF == 2;
template <class G>
constexpr int PER_UNIT = G::LDS > 80 * 1024 ? 1 : 2;  // workgroups that fit a compute unit

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
  int total = p.tiles_m * p.tiles_n;
  if constexpr (MODE != DENSE) {
    if (w.wave == 0) start[p.groups.E + 1] = read_groups<MODE == ROWS ? BM : UNIT>(p.groups, MODE == ROWS ? p.M : p.K, start, nullptr, w.lane);
    __syncthreads();
    if constexpr (MODE == DEPTH) total *= p.groups.E;
    if constexpr (MODE == ROWS) {
      total = uniform(start[p.groups.E + 1]) * p.tiles_n;
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
    const int xcds = 8, x = id % xcds, whole = p.tiles_m * p.tiles_n, q = total / xcds, r = total % xcds;
    int t = x * q + min(x, r) + id / xcds, tm, tn;  // bijective for any total
    if constexpr (MODE == DEPTH) {
      // groups differ in their tiles' work: each one's are spread over the XCDs, in runs where they divide evenly
      t = id;
      if (whole % xcds == 0) {
        const int run = whole / xcds, e = id / whole;
        t = e * whole + x * run + (id - e * whole) / xcds;
      }
    }
    j.e = j.from = 0, j.end = p.M, j.nb = (int)blocks_of(p.K);
    int first = 0, tiles_m = p.tiles_m;
    if constexpr (MODE == ROWS) {
      const Found f = find_group<BM>(start, p.groups.E, t / p.tiles_n, w.lane);
      j.e = f.e;
      t -= f.before * p.tiles_n;
      first = uniform(start[j.e]), j.end = uniform(start[j.e + 1]);
      tiles_m = (j.end - first + BM - 1) / BM;
    } else if constexpr (MODE == DEPTH) {
      j.e = t / whole;
      t -= j.e * whole;
      j.nb = (uniform(start[j.e + 1]) - uniform(start[j.e]) + BLOCK - 1) / BLOCK;
      j.from = units_before<UNIT>(start, j.e, w.lane) * (UNIT / BLOCK);
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
    store_epilogue<OUT, G>(w.acc, p.epi, (int64_t)job.e * N, y, p.ldy, job.m0 + arow, job.end, job.n0 + brow - BM, N, w.lane, stage, p.whole);
    if (!STREAMED<G> || id >= total) break;
    job = next;
  }
  // no direct load may be on its way when the workgroup ends and its LDS goes to another
  __builtin_amdgcn_s_waitcnt(0);
}

// A tensor whose rows store_whole can take: at most 2^31 bytes in 256 of them, each aligned to 4.
static inline bool suits(const void* p, int64_t ld, int eb) { return !p || (fp4_aligned(p, 4) && ld * eb % 4 == 0 && ld * eb < (1 << 23)); }

// `tiles`: the most tiles there can be.
template <class G, int OUT, Mode MODE>
static int launch_product(Args p, int64_t tiles, hipStream_t st) {
  p.whole = suits(p.y, p.ldy, elem_bytes(OUT)) && suits(p.epi.residual, p.epi.ldr, elem_bytes(p.epi.residual_type)) && suits(p.epi.z, p.epi.ldz, 4);
  // An output that the L2s cannot hold goes past them: kept, its lines would be written back in the next tiles' way, whose
  // stores then wait for memory while the matrix core idles. 8192 x 14336 x 4096 with gelu 375 -> 330 us, weight gradients of
  // 16 experts of 4096 x 2560 195 -> 150 us with their quantisation. z, which the backward pass comes back to, is kept as far
  // as the last-level cache goes: a training step of 8192 x 9728 x 2560 takes 591 us with both kept, 562 with y past them, 620
  // with both.
  const int64_t bytes = (int64_t)p.M * p.N * elem_bytes(OUT) * (MODE == DEPTH ? p.groups.E : 1);
  if (p.whole && bytes > (32 << 20)) p.whole = 2;
  static Fp4LdsLimit limit;
  const int lds = G::LDS + (MODE == DENSE ? 0 : group_table_bytes(p.groups.E));
  limit.ensure(reinterpret_cast<const void*>(&product_kernel<G, OUT, MODE>), G::LDS + (MODE == DENSE ? 0 : group_table_bytes(MAX_GROUPS)));
  const int units = PER_UNIT<G> * (fp4_device_cus() & ~7);  // a multiple of the 8 XCDs: a workgroup's tiles stay on its XCD
  const int64_t wgs = STREAMED<G> && units > 0 && tiles > units ? units : tiles;
  if (tiles > (1LL << 30) || !fits_launch(wgs, G::THREADS)) return FP4_ERR_UNSUPPORTED;
  return fp4_launch(product_kernel<G, OUT, MODE>, dim3((unsigned)wgs), dim3(G::THREADS), lds, st, p);
}

using Tile256 = Tile<256, 256, 2, 2, 2, 1>;
using Tile128 = Tile<128, 128, 2, 2, 2, 1>;
using Tile64 = Tile<64, 64, 2, 2, 4, 2>;
using TileWide = Tile<64, 128, 2, 2, 2, 1>;
static_assert(Tile256::STAGE >= 16 * (64 * 4 + 16) && Tile128::STAGE >= 16 * (32 * 4 + 16), "a wave's staging rows of FP32 sums");
static_assert(Tile256::LDS + group_table_bytes(MAX_GROUPS) <= 160 * 1024, "");
static_assert(Tile128::LDS + group_table_bytes(MAX_GROUPS) <= 80 * 1024 && Tile64::LDS + group_table_bytes(MAX_GROUPS) <= 80 * 1024 &&
                  TileWide::LDS + group_table_bytes(MAX_GROUPS) <= 80 * 1024,
              "two workgroups to a compute unit (PER_UNIT)");

template <int OUT, Mode MODE>
static int launch_tile(int tile, const Args& p, int64_t tiles, hipStream_t st) {
  if (tile == 256) return launch_product<Tile256, OUT, MODE>(p, tiles, st);
  if constexpr (MODE != DEPTH)
    if (tile == 64) return launch_product<Tile64, OUT, MODE>(p, tiles, st);
  if constexpr (MODE == ROWS)
    if (tile == WIDE) return launch_product<TileWide, OUT, MODE>(p, tiles, st);
  return launch_product<Tile128, OUT, MODE>(p, tiles, st);
}
template <Mode MODE>
static int launch_out(int out_type, int tile, const Args& p, int64_t tiles, hipStream_t st) {
  if (out_type == FP4_TYPE_F32) return launch_tile<FP4_TYPE_F32, MODE>(tile, p, tiles, st);
  if (out_type == FP4_TYPE_BF16) return launch_tile<FP4_TYPE_BF16, MODE>(tile, p, tiles, st);
  return launch_tile<FP4_TYPE_F16, MODE>(tile, p, tiles, st);
}

}  // namespace mx
