// MXFP4 x MXFP4 product with many rows, y[m][n] = sum_k A[m][k] B[n][k], on the scaled matrix instruction, and the
// entry points of the products.
//
// A workgroup of 4 waves (2 x 2) computes a BM x BN tile of y. Stages of 256 positions (one 128-byte line of codes
// per row) go global -> LDS by 16-byte direct loads into two buffers; the scales of two stages (16 bytes per row)
// travel with the even one. Each row's eight 16-byte blocks are XOR-swizzled by the row, so that the operand reads
// (16 rows, one block each) touch every bank once. The codes are MFMA operands as they stand.
// A wave holds one chunk's operands of both matrices and the next chunk's of B: after the MFMAs of row tile i it
// reads row tile i of the next chunk into the registers just freed, so an operand is read about a chunk ahead. In a
// stage's second chunk every LDS read of the stage has been issued, so the barrier that ends the stage stands at
// that chunk's start and the matrix core works through the reads and loads behind it.
// Blocks past K: their scale bytes are replaced by 0 on both sides, which makes every product at most
// 36 2^-254 = 0 in FP32, whatever the codes are. Rows past M or N load nothing and are not stored.
#include "mx.h"

namespace mx {

constexpr int GM_STAGE_BLOCKS = 8, GM_ROW_BYTES = 128;

template <int BM, int BN>
struct Tile {
  static constexpr int TM = BM / 32, TN = BN / 32;         // 16-row tiles per wave
  static constexpr int ROWS = BM + BN;                     // rows of both operands, A's first
  static constexpr int CODES = ROWS * GM_ROW_BYTES;        // bytes per stage
  static constexpr int SCALES = ROWS * 16;                 // bytes per two stages
  static constexpr int LDS = 2 * CODES + 2 * SCALES;
  static constexpr int SLOTS = CODES / 16 / 256;           // 16-byte direct loads per thread and stage
  static constexpr int SSLOTS = SCALES / 16 / 256;         // the same of the scales, per two stages
  static_assert(TN <= TM && ROWS % 256 == 0, "");
};

__device__ __forceinline__ int swizzle(int row) { return (row & 7) ^ ((row >> 3) & 1); }

// Every memory operation of this wave is done, and so is every wave's of the workgroup.
__device__ __forceinline__ void wait_all_and_meet() {
  __builtin_amdgcn_s_waitcnt(0);
  asm volatile("s_barrier" ::: "memory");
}

struct Sources {
  __amdgpu_buffer_rsrc_t aq, as, bq, bs;
  int ldqa, ldqb, ldsa, ldsb;
};

// Direct load I of one stage's codes: instruction I of wave w brings rows 8 (4 I + w) .. + 7, eight lanes a row.
// `from` (128 times the stage) is part of the range-checked offset: past the operand's last byte nothing is read.
// NOTHING lies past every operand's last byte (an operand's tile has at most 2^30 bytes).
constexpr uint32_t NOTHING = 1u << 31;

template <int BM, int BN, int I>
__device__ __forceinline__ void issue_codes_part(const Sources& src, uint8_t* buf, uint32_t from, int wave, int lane) {
  const int first = (4 * I + wave) * 8;
  const int row = first + (lane >> 3);
  const uint32_t at = from + ((lane & 7) ^ swizzle(row)) * 16;
  auto* to = (__attribute__((address_space(3))) void*)(buf + first * GM_ROW_BYTES);
  if constexpr (32 * I < BM)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src.aq, to, 16, (uint32_t)(row * src.ldqa) + at, 0, 0, 0);
  else
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src.bq, to, 16, (uint32_t)((row - BM) * src.ldqb) + at, 0, 0, 0);
}

template <int BM, int BN, int I0, int I1>
__device__ __forceinline__ void issue_codes(const Sources& src, uint8_t* buf, uint32_t from, int wave, int lane) {
  if constexpr (I0 < I1) {
    issue_codes_part<BM, BN, I0>(src, buf, from, wave, lane);
    issue_codes<BM, BN, I0 + 1, I1>(src, buf, from, wave, lane);
  }
}

// The direct loads of two stages' scales (`from`: 16 times the group): 64 rows per instruction, dealt to the waves.
template <int BM, int BN>
__device__ __forceinline__ void issue_scales(const Sources& src, uint8_t* buf, uint32_t from, int wave, int lane) {
  using G = Tile<BM, BN>;
#pragma unroll
  for (int i = 0; i < G::SSLOTS; ++i) {
    const int first = (4 * i + wave) * 64;
    const int row = first + lane;
    auto* to = (__attribute__((address_space(3))) void*)(buf + first * 16);
    if (first < BM) __builtin_amdgcn_raw_ptr_buffer_load_lds(src.as, to, 16, (uint32_t)(row * src.ldsa) + from, 0, 0, 0);
    else __builtin_amdgcn_raw_ptr_buffer_load_lds(src.bs, to, 16, (uint32_t)((row - BM) * src.ldsb) + from, 0, 0, 0);
  }
}

// acc += A B^T with scale byte C of both scale registers, as fp4 mfma() but written out so that the sum stays in the
// accumulation registers that it came from: with the compiler's builtin, whose result is a new register, a tile of
// 256 sums per lane is copied and spilled in the loop. The s_nop covers the two wait states between a vector
// instruction that writes an operand and the MFMA that reads it, which the compiler does not see here.
template <int C>
__device__ __forceinline__ void mfma_acc(f32x4& acc, const u32x4& a, uint32_t sa, const u32x4& b, uint32_t sb) {
#define MX_MFMA(SEL)                                                                                     \
  asm volatile("s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 " SEL " cbsz:4 blgp:4" \
               : "+a"(acc)                                                                               \
               : "v"(a), "v"(b), "v"(sa), "v"(sb))
  if constexpr (C == 0) MX_MFMA("op_sel:[0,0,0] op_sel_hi:[0,0,0]");
  else if constexpr (C == 1) MX_MFMA("op_sel:[1,1,0] op_sel_hi:[0,0,0]");
  else if constexpr (C == 2) MX_MFMA("op_sel:[0,0,0] op_sel_hi:[1,1,0]");
  else MX_MFMA("op_sel:[1,1,0] op_sel_hi:[1,1,0]");
#undef MX_MFMA
}

// Four dwords of a row's scales (four chunks of four blocks) -> byte c is block g of chunk c.
__device__ __forceinline__ uint32_t pick_scales(const u32x4& w, int g) {
  const uint32_t sel = (uint32_t)g | (uint32_t)(4 + g) << 8;
  const uint32_t lo = __builtin_amdgcn_perm(w[1], w[0], sel);
  const uint32_t hi = __builtin_amdgcn_perm(w[3], w[2], sel);
  return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}

// Workgroup -> (tile row, tile column, part of K). Workgroups go round-robin over the 8 XCDs, each of which has its
// own L2: XCD x takes a contiguous run of the tiles, walked in columns of `BAND` tile rows so that the tiles in
// flight on one XCD share rows of both operands.
__device__ __forceinline__ void place(int id, int total, int tiles_m, int tiles_n, int& tm, int& tn, int& part) {
  const int xcds = 8, x = id % xcds, i = id / xcds;
  const int q = total / xcds, r = total % xcds;
  int t = x * q + min(x, r) + i;  // bijective for any total
  const int tiles = tiles_m * tiles_n;
  part = t / tiles;
  t -= part * tiles;
  constexpr int BAND = 4;
  const int per = BAND * tiles_n, band = t / per, in = t - band * per;
  const int h = min(BAND, tiles_m - band * BAND);
  tn = in / h;
  tm = band * BAND + in - tn * h;
}

// A wave's state.
template <int BM, int BN>
struct Wave {
  using G = Tile<BM, BN>;
  f32x4 acc[G::TM][G::TN];
  u32x4 a[G::TM], b[2][G::TN];          // operands; B's of even chunks in b[0], of odd ones in b[1]
  uint32_t sa[2][G::TM], sb[2][G::TN];  // scales of two groups: byte c is this lane's block of chunk c
  Sources src;
  uint8_t* lds;
  int wave, lane;
  uint32_t frag_a, frag_b;    // LDS offsets of this lane's block of chunk 0, row tile 0; ^ 64 leads to chunk 1
  uint32_t scale_a, scale_b;  // LDS offsets of this lane's row of scales, row tile 0
  int last_group;
  uint32_t tail;              // mask of the last group's scales

  __device__ __forceinline__ uint8_t* codes(int buf) const { return lds + buf * G::CODES; }
  __device__ __forceinline__ uint8_t* scales(int buf) const { return lds + 2 * G::CODES + buf * G::SCALES; }
  __device__ __forceinline__ u32x4 read_codes(uint32_t at, int buf, int chunk, int t) const {
    return *reinterpret_cast<const u32x4*>(codes(buf) + (chunk ? at ^ 64u : at) + t * 16 * GM_ROW_BYTES);
  }
  __device__ __forceinline__ uint32_t read_scale(uint32_t at, int group) const {
    return pick_scales(*reinterpret_cast<const u32x4*>(scales(group & 1) + at), lane >> 4) &
           (group == last_group ? tail : ~0u);
  }
  template <int S>
  __device__ __forceinline__ void read_scales(int i, int group) {
    sa[S][i] = read_scale(scale_a + 256 * i, group);
    if (i < G::TN) sb[S][i] = read_scale(scale_b + 256 * i, group);
  }

  // Row tile I's MFMAs of chunk C of a group (its scales are in set 0).
  template <int C, int I>
  __device__ __forceinline__ void mult() {
#pragma unroll
    for (int j = 0; j < G::TN; ++j) mfma_acc<C>(acc[I][j], b[C & 1][j], sb[0][j], a[I], sa[0][I]);
  }
  // After row tile I of chunk C: A's row tile I of the next chunk, and two of B's in the first half of the rows.
  template <int C, int I>
  __device__ __forceinline__ void fetch() {
    constexpr int NC = (C + 1) & 1, NB = ((C + 1) >> 1) & 1;
    a[I] = read_codes(frag_a, NB, NC, I);
    if constexpr (2 * I < G::TN) b[NC][2 * I] = read_codes(frag_b, NB, NC, 2 * I);
    if constexpr (2 * I + 1 < G::TN) b[NC][2 * I + 1] = read_codes(frag_b, NB, NC, 2 * I + 1);
  }

  // A stage's first chunk, from row tile I on.
  template <int C, int I>
  __device__ __forceinline__ void first_chunk() {
    if constexpr (I < G::TM) {
      mult<C, I>();
      fetch<C, I>();
      __builtin_amdgcn_sched_barrier(0);
      first_chunk<C, I + 1>();
    }
  }

  // A stage's second chunk, from row tile I on. After row tile 0 the stage ends; the direct loads of the stage after
  // the next (from byte `codes_from` of the codes, `scales_from` of the scales) are spread over the rows. `group` is
  // the group of the next stage.
  template <int C, int I>
  __device__ __forceinline__ void second_chunk(uint32_t codes_from, uint32_t scales_from, int group) {
    if constexpr (I < G::TM) {
      mult<C, I>();
      if constexpr (I == 0) {
        __builtin_amdgcn_sched_barrier(0);
        wait_all_and_meet();
      }
      fetch<C, I>();
      if constexpr (C == 3) read_scales<1>(I, group);
      issue_codes<BM, BN, G::SLOTS * I / G::TM, G::SLOTS*(I + 1) / G::TM>(src, codes(C >> 1), codes_from, wave, lane);
      if constexpr (C == 1 && I == G::TM - 1) issue_scales<BM, BN>(src, scales((group + 1) & 1), scales_from, wave, lane);
      __builtin_amdgcn_sched_barrier(0);
      second_chunk<C, I + 1>(codes_from, scales_from, group);
    }
  }
};

// parts > 1: part p sums stages [p per, (p + 1) per) into plane p of `y` (FP32, M x N), else all of K into y.
template <int BM, int BN>
__global__ void __launch_bounds__(256, BM * BN > 128 * 128 ? 1 : 2)
    gemm_kernel(fp4_mx a, fp4_mx b, void* __restrict__ y, int64_t ldy, int M, int N, int K, int out_type, int vec, int tiles_m,
                int tiles_n, int parts, int per) {
  using G = Tile<BM, BN>;
  extern __shared__ uint8_t lds[];
  Wave<BM, BN> w;
  w.lds = lds;
  w.lane = threadIdx.x & 63;
  w.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = w.lane & 15, g = w.lane >> 4;
  int tm, tn, part;
  place(blockIdx.x, gridDim.x, tiles_m, tiles_n, tm, tn, part);
  const int m0 = tm * BM, n0 = tn * BN;
  const int nb = (int)blocks_of(K), stages_all = (nb + GM_STAGE_BLOCKS - 1) / GM_STAGE_BLOCKS;
  const int s0 = part * per, s1 = min(stages_all, s0 + per);  // s0 is even: no part begins inside a scale group

  const int ma = min(M - m0, BM), mb = min(N - n0, BN);
  w.src.ldqa = (int)a.ldq, w.src.ldqb = (int)b.ldq, w.src.ldsa = (int)a.lds, w.src.ldsb = (int)b.lds;
  const int sbytes = (nb + 3) & ~3;
  w.src.aq = fp4::make_rsrc(static_cast<const uint8_t*>(a.q) + (int64_t)m0 * a.ldq, (uint32_t)((ma - 1) * (int)a.ldq + nb * 16));
  w.src.as = fp4::make_rsrc(static_cast<const uint8_t*>(a.s) + (int64_t)m0 * a.lds, (uint32_t)((ma - 1) * (int)a.lds + sbytes));
  w.src.bq = fp4::make_rsrc(static_cast<const uint8_t*>(b.q) + (int64_t)n0 * b.ldq, (uint32_t)((mb - 1) * (int)b.ldq + nb * 16));
  w.src.bs = fp4::make_rsrc(static_cast<const uint8_t*>(b.s) + (int64_t)n0 * b.lds, (uint32_t)((mb - 1) * (int)b.lds + sbytes));

  // this lane's valid blocks of the last group of four chunks
  w.last_group = (stages_all - 1) >> 1;
  w.tail = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (16 * w.last_group + 4 * c + g < nb) w.tail |= 0xffu << (8 * c);

  const int arow = (w.wave >> 1) * (BM / 2), brow = BM + (w.wave & 1) * (BN / 2);  // this wave's first rows in LDS
  const uint32_t at = n * GM_ROW_BYTES + ((g ^ swizzle(n)) << 4);                  // (multiples of 16)
  w.frag_a = arow * GM_ROW_BYTES + at, w.frag_b = brow * GM_ROW_BYTES + at;
  w.scale_a = (arow + n) * 16, w.scale_b = (brow + n) * 16;
#pragma unroll
  for (int i = 0; i < G::TM; ++i)
#pragma unroll
    for (int j = 0; j < G::TN; ++j) w.acc[i][j] = f32x4{0, 0, 0, 0};

  const auto codes_from = [&](int st) { return st < s1 ? (uint32_t)st * GM_ROW_BYTES : NOTHING; };
  issue_codes<BM, BN, 0, G::SLOTS>(w.src, w.codes(0), codes_from(s0), w.wave, w.lane);
  issue_scales<BM, BN>(w.src, w.scales((s0 >> 1) & 1), (uint32_t)(s0 >> 1) * 16, w.wave, w.lane);
  wait_all_and_meet();
  issue_codes<BM, BN, 0, G::SLOTS>(w.src, w.codes(1), codes_from(s0 + 1), w.wave, w.lane);
#pragma unroll
  for (int i = 0; i < G::TM; ++i) {
    w.a[i] = w.read_codes(w.frag_a, 0, 0, i);
    if (i < G::TN) w.b[0][i] = w.read_codes(w.frag_b, 0, 0, i);
    w.template read_scales<0>(i, s0 >> 1);
  }
  // Two stages (one group of scales) at a time. Past the last stage nothing is loaded: its look ahead reads what is
  // in LDS and is not used, and the second half of an odd count multiplies by the zero scales of blocks past K. One
  // loop body without branches serves every stage.
  for (int st = s0; st < s1; st += 2) {
    const int group = st >> 1;
    w.template first_chunk<0, 0>();
    w.template second_chunk<1, 0>(codes_from(st + 2), st + 2 < s1 ? (uint32_t)(group + 1) * 16 : NOTHING, group);
    w.template first_chunk<2, 0>();
    w.template second_chunk<3, 0>(codes_from(st + 3), 0, group + 1);
#pragma unroll
    for (int i = 0; i < G::TM; ++i) w.sa[0][i] = w.sa[1][i];
#pragma unroll
    for (int j = 0; j < G::TN; ++j) w.sb[0][j] = w.sb[1][j];
  }
  // no direct load may be on its way when the workgroup ends and its LDS goes to another
  __builtin_amdgcn_s_waitcnt(0);

  // the last MFMAs' results: 18 wait states before anything but an MFMA reads them, then every read of a sum is
  // ordered behind the wait
  asm volatile("s_nop 15\n\ts_nop 15");
#pragma unroll
  for (int i = 0; i < G::TM; ++i)
#pragma unroll
    for (int j = 0; j < G::TN; ++j) asm volatile("" : "+a"(w.acc[i][j]));

  if (parts > 1) y = static_cast<float*>(y) + (int64_t)part * M * ldy;
  const int row0 = m0 + arow + n, col0 = n0 + brow - BM + 4 * g;
  if (vec && m0 + BM <= M && n0 + BN <= N) {
    if (out_type == FP4_TYPE_F32) {
      float* p = static_cast<float*>(y) + (int64_t)row0 * ldy + col0;
#pragma unroll
      for (int i = 0; i < G::TM; ++i)
#pragma unroll
        for (int j = 0; j < G::TN; ++j) *reinterpret_cast<f32x4*>(p + (int64_t)16 * i * ldy + 16 * j) = w.acc[i][j];
    } else {
      uint16_t* p = static_cast<uint16_t*>(y) + (int64_t)row0 * ldy + col0;
#pragma unroll
      for (int i = 0; i < G::TM; ++i)
#pragma unroll
        for (int j = 0; j < G::TN; ++j) {
          const f32x4 v = w.acc[i][j];
          *reinterpret_cast<u32x2*>(p + (int64_t)16 * i * ldy + 16 * j) =
              u32x2{to16(out_type, v[0]) | to16(out_type, v[1]) << 16, to16(out_type, v[2]) | to16(out_type, v[3]) << 16};
        }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < G::TM; ++i)
#pragma unroll
    for (int j = 0; j < G::TN; ++j) {
      const int row = row0 + 16 * i, col = col0 + 16 * j;
      if (row < M && col < N) store4(out_type, y, (int64_t)row * ldy + col, w.acc[i][j], N - col, vec);
    }
}

// y = the sum of the K parts' planes, in the order of the parts. Planes have rows of `ldp` floats (a multiple of 4).
__global__ void __launch_bounds__(256) combine_kernel(const float* __restrict__ planes, void* __restrict__ y, int64_t ldy, int M,
                                                      int N, int64_t ldp, int parts, int out_type, int vec) {
  const int64_t quads = ldp >> 2, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= quads * M) return;
  const int64_t row = i / quads, col = 4 * (i - row * quads);
  f32x4 sum = *reinterpret_cast<const f32x4*>(planes + row * ldp + col);
  for (int p = 1; p < parts; ++p) sum += *reinterpret_cast<const f32x4*>(planes + ((int64_t)p * M + row) * ldp + col);
  store4(out_type, y, row * ldy + col, sum, (int)(N - col), vec);
}

// How a product is run.
struct Plan {
  int rows;    // 1: rows_kernel, else gemm_kernel
  int tile;    // 256 or 128
  int parts;   // K parts
  int per;     // stages per part (even)
  int64_t ldp; // floats per row of a plane
};

static Plan plan_of(int64_t M, int64_t N, int64_t K) {
  Plan p{};
  p.ldp = (N + 3) / 4 * 4;
  p.parts = 1;
  const int stages = (int)((blocks_of(K) + 7) / 8);
  p.per = (stages + 1) & ~1;
  if (M <= 64) {
    p.rows = 1;
    return p;
  }
  const int cus = fp4_device_cus();
  auto tiles = [&](int t) { return ((M + t - 1) / t) * ((N + t - 1) / t); };
  p.tile = tiles(256) >= cus ? 256 : 128;
  const int64_t grid = tiles(p.tile);
  if (p.tile == 128 && grid < cus && stages >= 4) {
    int64_t want = 2 * cus / grid;
    if (want > 16) want = 16;
    int per = (int)((stages + want - 1) / want);
    per = (per + 1) & ~1;
    p.parts = (stages + per - 1) / per;
    p.per = per;
  }
  return p;
}

static int64_t plane_bytes(const Plan& p, int64_t M) { return p.parts > 1 ? p.parts * M * p.ldp * 4 : 0; }

template <int B>
static int launch_gemm(const Plan& p, int out_type, int M, int N, int K, const fp4_mx& a, const fp4_mx& b, void* y, int64_t ldy,
                       void* ws, hipStream_t st) {
  using G = Tile<B, B>;
  static Fp4LdsLimit limit;
  limit.ensure(reinterpret_cast<const void*>(&gemm_kernel<B, B>), G::LDS);
  const int tm = (M + B - 1) / B, tn = (N + B - 1) / B;
  const int64_t grid = (int64_t)tm * tn * p.parts;
  if (grid > 0x7fffffffLL) return FP4_ERR_UNSUPPORTED;
  const int vec = fp4_aligned(y, 4 * elem_bytes(out_type)) && ldy % 4 == 0;
  if (p.parts == 1)
    return fp4_launch(gemm_kernel<B, B>, dim3((unsigned)grid), dim3(256), G::LDS, st, a, b, y, ldy, M, N, K, out_type, vec, tm,
                      tn, 1, p.per);
  if (int rc = fp4_launch(gemm_kernel<B, B>, dim3((unsigned)grid), dim3(256), G::LDS, st, a, b, ws, p.ldp, M, N, K, FP4_TYPE_F32,
                          1, tm, tn, p.parts, p.per))
    return rc;
  const int64_t quads = (p.ldp >> 2) * M;
  return fp4_launch(combine_kernel, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, st, ws, y, ldy, M, N, p.ldp, p.parts,
                    out_type, vec);
}

static int run_product(Plan p, int out_type, int64_t M, int64_t N, int64_t K, const fp4_mx& a, const fp4_mx& b, void* y,
                       int64_t ldy, void* ws, size_t ws_bytes, hipStream_t st) {
  if (p.rows) return launch_rows(0, out_type, (int)M, (int)N, (int)K, nullptr, 0, &a, b, y, ldy, st);
  if (p.parts > 1 && (!ws || ws_bytes < (size_t)plane_bytes(p, M))) {
    p.parts = 1;
    p.per = ((int)((blocks_of(K) + 7) / 8) + 1) & ~1;
  }
  return p.tile == 256 ? launch_gemm<256>(p, out_type, (int)M, (int)N, (int)K, a, b, y, ldy, ws, st)
                       : launch_gemm<128>(p, out_type, (int)M, (int)N, (int)K, a, b, y, ldy, ws, st);
}

static int check_product(int out_type, int64_t M, int64_t N, int64_t K) {
  if (!valid_type(out_type)) return FP4_ERR_ARG;
  if (N < 1) return FP4_ERR_SHAPE;
  if (int rc = check_dims(M, K)) return rc;
  if (N > MAX_ROWS) return FP4_ERR_UNSUPPORTED;
  return FP4_OK;
}

static int check_output(int out_type, int64_t N, const void* y, int64_t ldy) {
  if (!y) return FP4_ERR_ARG;
  if (ldy < N) return FP4_ERR_SHAPE;
  if (ldy > (1LL << 40)) return FP4_ERR_UNSUPPORTED;
  return fp4_aligned(y, (uintptr_t)elem_bytes(out_type)) ? FP4_OK : FP4_ERR_ALIGN;
}

// Dense activations are quantised inside the product up to this many rows, into the workspace above it.
constexpr int FUSED_ROWS = 16;

struct LinearSpace {
  int64_t q, s, planes;  // bytes, each a multiple of 256
};
static int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }
static LinearSpace linear_space(const Plan& p, int64_t M, int64_t K) {
  const int64_t nb = blocks_of(K);
  return {round256(M * nb * 16), round256(M * ((nb + 3) / 4 * 4)), plane_bytes(p, M)};
}

}  // namespace mx

using namespace mx;

extern "C" int64_t w4a4_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (int rc = check_product(FP4_TYPE_F32, M, N, K)) return rc;
  return M == 0 ? 0 : plane_bytes(plan_of(M, N, K), M);
}

extern "C" int w4a4_matmul(int out_type, int64_t M, int64_t N, int64_t K, const fp4_mx* a, const fp4_mx* b, void* y,
                           int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  if (int rc = check_product(out_type, M, N, K)) return rc;
  if (M == 0) return FP4_OK;
  if (int rc = check_operand(a, K)) return rc;
  if (int rc = check_operand(b, K)) return rc;
  if (int rc = check_output(out_type, N, y, ldy)) return rc;
  if (workspace && !fp4_aligned(workspace, 16)) return FP4_ERR_ALIGN;
  return run_product(plan_of(M, N, K), out_type, M, N, K, *a, *b, y, ldy, workspace, workspace_bytes,
                     static_cast<hipStream_t>(stream));
}

extern "C" int64_t w4a4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (int rc = check_product(FP4_TYPE_F32, M, N, K)) return rc;
  if (M <= FUSED_ROWS) return 0;
  const LinearSpace sp = linear_space(plan_of(M, N, K), M, K);
  return sp.q + sp.s + sp.planes;
}

extern "C" int w4a4_linear(int x_type, int out_type, int64_t M, int64_t N, int64_t K, const void* x, int64_t ldx,
                           const fp4_mx* b, void* y, int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_type(x_type)) return FP4_ERR_ARG;
  if (int rc = check_product(out_type, M, N, K)) return rc;
  if (M == 0) return FP4_OK;
  if (!x) return FP4_ERR_ARG;
  if (ldx < K) return FP4_ERR_SHAPE;
  if (ldx > (1LL << 40)) return FP4_ERR_UNSUPPORTED;
  if (!fp4_aligned(x, (uintptr_t)elem_bytes(x_type))) return FP4_ERR_ALIGN;
  if (int rc = check_operand(b, K)) return rc;
  if (int rc = check_output(out_type, N, y, ldy)) return rc;
  if (workspace && !fp4_aligned(workspace, 16)) return FP4_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (M <= FUSED_ROWS) return launch_rows(x_type, out_type, (int)M, (int)N, (int)K, x, ldx, nullptr, *b, y, ldy, st);
  const Plan p = plan_of(M, N, K);
  const LinearSpace sp = linear_space(p, M, K);
  if (!workspace || workspace_bytes < (size_t)(sp.q + sp.s)) return FP4_ERR_ARG;
  auto* w = static_cast<uint8_t*>(workspace);
  const int64_t nb = blocks_of(K);
  const fp4_mx a = {w, w + sp.q, nb * 16, (nb + 3) / 4 * 4};
  if (int rc = launch_quantize_rows(x_type, M, K, x, ldx, a, st)) return rc;
  return run_product(p, out_type, M, N, K, a, *b, y, ldy, w + sp.q + sp.s, workspace_bytes - (size_t)(sp.q + sp.s), st);
}
