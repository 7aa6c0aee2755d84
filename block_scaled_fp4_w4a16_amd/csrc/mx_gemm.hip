// MXFP4 x MXFP4 product with many rows, y[m][n] = sum_k A[m][k] B[n][k], on the scaled matrix instruction, and the
// entry points of the products.
//
// A workgroup of 4 waves (2 x 2) computes a BM x BN tile of y. Stages of 256 positions (one 128-byte line of codes
// per row) go global -> LDS by 16-byte direct loads into a ring of buffers; the scales of two or four stages (16 or 32
// bytes per row) travel with the first of them. Each row's eight 16-byte blocks are XOR-swizzled by the row's last three
// bits, so that the operand reads (16 rows, one block each) are as fast as reads of consecutive bytes: 1.75 ns per
// instruction and compute unit; with rows 8 .. 15 swizzled differently from 0 .. 7 they take 3.5. The codes are MFMA
// operands as they stand.
// A wave holds the operands of two chunks of 128 positions, of both matrices, in two sets of registers. While one chunk's
// MFMAs run from one set, the next chunk's operands are read into the other, B's first, dealt out behind the MFMAs of the
// first three quarters of the row tiles. That set is free by then: the chunk before used it, and an MFMA issued in order
// has taken its operands before a later read can return. In a stage's second chunk every LDS read of the stage has
// been issued, so the barrier that ends the stage stands behind that chunk's first MFMA, and the matrix core works through
// the reads and loads behind it.
// Blocks past K: their scale bytes are replaced by 0 on both sides, which makes every product at most
// 36 2^-254 = 0 in FP32, whatever the codes are. Rows past M or N load nothing and are not stored.
// Tiles of 256 (64 KB of codes a stage, one workgroup per compute unit): 8192 x 14336 x 4096 takes 240 us, 4.0 PFLOP/s, with
// FP32 output 300 us (its epilogue spills). A stage takes 3350 to 3600 cycles against 2048 of matrix instructions, which
// run for 47 % of the kernel's cycles at 2.1 GHz; the same instructions on random operands in registers alone reach 6.5
// to 7.2 PFLOP/s at 1.6 to 1.7 GHz.
// Smaller tiles are for fewer outputs and are bound by their loads: 16 KB a stage of 64 x 64 outputs take 0.26 us on a
// compute unit (64 bytes per ns), 0.41 for two workgroups at once; 333 x 2560 x 9728 13.3 us, 64 x 14336 x 4096 8.1 us
// (33 MB, 4.1 TB/s), from weights that stay in the caches; 15.1 and 11.2 us from cold ones.

#include "mx_tile.h"

namespace mx {

// Stores a wave's sums: acc[i][j][e] is row `row0` + 16 i (+ lane % 16), column `col0` + 16 j + 4 (lane / 16) + e. Whole
// tiles (`full`: every row and column exists and 16-byte stores are aligned) go 16 rows at a time through `stage` (this
// wave's LDS), so that a store instruction writes long runs of a few rows, whole lines, and not 64 bytes of each of 16
// rows, which take several times as long to issue.
template <int OUT, class G>
__device__ __forceinline__ void store_tile(const f32x4 (&acc)[G::TM][G::TN], void* y, int64_t ldy, int M, int N, int row0, int col0,
                                           int lane, bool full, bool vec, uint8_t* stage) {
  const int n = lane & 15, g = lane >> 4;
  if (full) {
    constexpr int EB = elem_bytes(OUT), SPLIT = OUT == FP4_TYPE_F32 && G::TN > 1 ? 2 : 1;  // column halves of FP32
    constexpr int TJ = G::TN / SPLIT, RUN = TJ * 16 * EB, STRIDE = RUN + 16;
    constexpr int PER = RUN / 16, ROWS = 64 / PER;  // lanes per row and rows per store
    uint8_t* const in = stage + n * STRIDE + 4 * g * EB;
    const uint8_t* const out = stage + lane / PER * STRIDE + lane % PER * 16;
    uint8_t* p = static_cast<uint8_t*>(y) + ((int64_t)(row0 + lane / PER) * ldy + col0) * EB + lane % PER * 16;
#pragma unroll
    for (int i = 0; i < G::TM; ++i) {
#pragma unroll
      for (int h = 0; h < SPLIT; ++h) {
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
          const f32x4 v = acc[i][h * TJ + j];
          if constexpr (OUT == FP4_TYPE_F32) *reinterpret_cast<f32x4*>(in + j * 64) = v;
          else *reinterpret_cast<u32x2*>(in + j * 32) = u32x2{pack2<OUT>(v[0], v[1]), pack2<OUT>(v[2], v[3])};
        }
        asm volatile("" ::: "memory");  // one wave's LDS accesses stay in order: no barrier
#pragma unroll
        for (int r = 0; r < 16; r += ROWS)
          *reinterpret_cast<u32x4*>(p + (int64_t)(16 * i + r) * ldy * EB + h * RUN) = *reinterpret_cast<const u32x4*>(out + r * STRIDE);
        asm volatile("" ::: "memory");
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < G::TM; ++i)
#pragma unroll
      for (int j = 0; j < G::TN; ++j) {
        const int row = row0 + 16 * i + n, col = col0 + 16 * j + 4 * g;
        if (row < M && col < N) store4(OUT, y, (int64_t)row * ldy + col, acc[i][j], N - col, vec);
      }
  }
}

// One tile's work: its first row and column, its part of K and the stages [s0, s1) of that part.
struct Job {
  int m0, n0, part, s0, s1;
};

// parts > 1: part p sums stages [p per, (p + 1) per) into plane p of `y` (FP32, M x N), else all of K into y. A workgroup
// takes tiles blockIdx.x, + gridDim.x, ... as one stream of stages: behind a tile's last stages the next tile's first ones
// are loaded, and its first operands are read, as if K went on, so that between two tiles only the sums are stored.
template <class G, int OUT>
__global__ void __launch_bounds__(G::THREADS, G::LDS > 80 * 1024 ? G::WAVES / 4 : G::WAVES / 2)
    gemm_kernel(fp4_mx a, fp4_mx b, void* __restrict__ y, int64_t ldy, int M, int N, int K, int vec, int tiles_m, int tiles_n,
                int parts, int per) {
  constexpr int BM = G::BM, BN = G::BN, NBUF = G::NBUF;
  extern __shared__ uint8_t lds[];
  Wave<G> w;
  w.lds = lds;
  w.lane = threadIdx.x & 63;
  w.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = w.lane & 15, g = w.lane >> 4;
  const int nb = (int)blocks_of(K), stages_all = (nb + GM_STAGE_BLOCKS - 1) / GM_STAGE_BLOCKS;
  const int total = tiles_m * tiles_n * parts;
  w.src.ldqa = (int)a.ldq, w.src.ldqb = (int)b.ldq, w.src.ldsa = (int)a.lds, w.src.ldsb = (int)b.lds;

  // this lane's valid blocks of the last group of four chunks
  w.last_group = (stages_all - 1) >> 1;
  w.tail = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    if (16 * w.last_group + 4 * c + g < nb) w.tail |= 0xffu << (8 * c);

  // this wave's first rows in LDS (multiples of 16)
  const int arow = w.wave / G::WN * (BM / G::WM), brow = BM + w.wave % G::WN * (BN / G::WN);
  const uint32_t at = n * GM_ROW_BYTES + ((g ^ swizzle(n)) << 4);
  w.frag_a = arow * GM_ROW_BYTES + at, w.frag_b = brow * GM_ROW_BYTES + at;
  const uint32_t scale_at = G::SG * 16 * n + (G::SG == 2 ? (n >> 3) * 16 : 0);
  w.scale_a = G::SG * 16 * arow + scale_at, w.scale_b = G::SG * 16 * brow + scale_at;

  // tile `id`: its place, and the sources of its loads
  const auto job_of = [&](int id) {
    Job j;
    int tm, tn;
    place(id, total, tiles_m, tiles_n, tm, tn, j.part);
    j.m0 = tm * BM, j.n0 = tn * BN;
    j.s0 = j.part * per, j.s1 = min(stages_all, j.s0 + per);  // s0 is even: no part begins inside a scale group
    return j;
  };
  const auto load_from = [&](const Job& j) {
    const int ma = min(M - j.m0, BM), mb = min(N - j.n0, BN), sbytes = (nb + 3) & ~3;
    w.src.aq = fp4::make_rsrc(static_cast<const uint8_t*>(a.q) + j.m0 * a.ldq, (uint32_t)((ma - 1) * (int)a.ldq + nb * 16));
    w.src.as = fp4::make_rsrc(static_cast<const uint8_t*>(a.s) + j.m0 * a.lds, (uint32_t)((ma - 1) * (int)a.lds + sbytes));
    w.src.bq = fp4::make_rsrc(static_cast<const uint8_t*>(b.q) + j.n0 * b.ldq, (uint32_t)((mb - 1) * (int)b.ldq + nb * 16));
    w.src.bs = fp4::make_rsrc(static_cast<const uint8_t*>(b.s) + j.n0 * b.lds, (uint32_t)((mb - 1) * (int)b.lds + sbytes));
  };
  const auto codes_from = [](int st, int end) { return st < end ? (uint32_t)st * GM_ROW_BYTES : NOTHING; };
  const auto scales_from = [](int st, int end) { return st < end ? (uint32_t)((st >> 1) / G::SG * G::SG) * 16 : NOTHING; };

  int id = blockIdx.x;
  Job job = job_of(id);
  load_from(job);
#pragma unroll
  for (int i = 0; i < NBUF; ++i) {
    const int st = job.s0 + i, ring = w.ring_of(st >> 1);
    issue_codes<G, 0, G::SLOTS>(w.src, w.codes(ring, i & 1), codes_from(st, job.s1), w.wave, w.lane);
    if (!(i & 1) && (G::SG == 1 || i == 0 || !(st >> 1 & 1)))
      issue_scales<G>(w.src, w.scales(st >> 1), scales_from(st, job.s1), w.wave, w.lane);
  }
  wait_and_meet<G::BEHIND + G::SLOTS>();
#pragma unroll
  for (int i = 0; i < G::OPS; ++i) {
    w.op[0][i] = w.read_op(w.ring_of(job.s0 >> 1), 0, 0, i);
    w.raw[i] = w.read_raw(job.s0 >> 1, i);
  }
#pragma unroll
  for (int i = 0; i < G::OPS; ++i) w.sc[0][i] = w.pick(i, job.s0 >> 1);

  for (;;) {
#pragma unroll
    for (int i = 0; i < G::TM; ++i)
#pragma unroll
      for (int j = 0; j < G::TN; ++j) w.acc[i][j] = f32x4{0, 0, 0, 0};
    __builtin_amdgcn_sched_barrier(0);
    Job next = job;
    id += gridDim.x;
    // Two stages (one group of scales) at a time; the stages NBUF ahead are loaded. Past the workgroup's last stage
    // nothing is: the look ahead reads what is in LDS and is not used. The second half of an odd count multiplies by
    // the zero scales of blocks past K. One loop body without branches serves every stage.
    int st = job.s0;
    do {  // a tile has a stage at least: the sums have one way out of the loop, with no copies of them before the wait
      int ahead = st + NBUF, end = job.s1, next_group = (st >> 1) + 1;
      if (st + 2 >= job.s1) {
        if (id < total) {  // only with NBUF = 2
          next = job_of(id);
          load_from(next);
          ahead = next.s0, end = next.s1;
        }
        next_group = next.s0 >> 1;
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

    // An MFMA's result needs eight wait states (4 passes) before anything but an MFMA reads it, and the compiler does not see
    // these MFMAs. The last eight's sums go through the wait itself, so that no copy of them can come before it (a copy
    // that the compiler made in front of a bare wait came after seven); every read of another sum is ordered behind it.
    wait_for_sums<G>(w.acc);
#pragma unroll
    for (int i = 0; i < G::TM; ++i)
#pragma unroll
      for (int j = 0; j < G::TN; ++j) asm volatile("" : "+a"(w.acc[i][j]));
    void* const yp = parts > 1 ? static_cast<float*>(y) + (int64_t)job.part * M * ldy : y;
    store_tile<OUT, G>(w.acc, yp, ldy, M, N, job.m0 + arow, job.n0 + brow - BM, w.lane,
                       vec && job.m0 + BM <= M && job.n0 + BN <= N, vec, lds + G::RING + w.wave * G::STAGE);
    if (id >= total) break;
    job = next;
  }
  // no direct load may be on its way when the workgroup ends and its LDS goes to another
  __builtin_amdgcn_s_waitcnt(0);
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

template <class G, int OUT>
static int launch_tiles(const Plan& p, int M, int N, int K, const fp4_mx& a, const fp4_mx& b, void* y, int64_t ldy,
                        hipStream_t st) {
  static Fp4LdsLimit limit;
  limit.ensure(reinterpret_cast<const void*>(&gemm_kernel<G, OUT>), G::LDS);
  const int tm = (M + G::BM - 1) / G::BM, tn = (N + G::BN - 1) / G::BN;
  const int64_t grid = (int64_t)tm * tn * p.parts;
  const int vec = fp4_aligned(y, 16) && ldy % (OUT == FP4_TYPE_F32 ? 4 : 8) == 0;
  // one workgroup per compute unit takes several tiles where only one fits (a multiple of the 8 XCDs, so that a
  // workgroup's tiles stay on its XCD); smaller tiles overlap by sharing a unit
  const int units = fp4_device_cus() & ~7;
  const int64_t wgs = G::NBUF == 2 && G::LDS > 80 * 1024 && units > 0 && grid > units ? units : grid;
  if (grid > (1LL << 30) || !fits_launch(wgs, G::THREADS)) return FP4_ERR_UNSUPPORTED;
  return fp4_launch(gemm_kernel<G, OUT>, dim3((unsigned)wgs), dim3(G::THREADS), G::LDS, st, a, b, y, ldy, M, N, K, vec, tm, tn,
                    p.parts, p.per);
}

template <class G>
static int launch_gemm(const Plan& p, int out_type, int M, int N, int K, const fp4_mx& a, const fp4_mx& b, void* y, int64_t ldy,
                       void* ws, hipStream_t st) {
  if (p.parts > 1) {
    if (int rc = launch_tiles<G, FP4_TYPE_F32>(p, M, N, K, a, b, ws, p.ldp, st)) return rc;
    const int vec = fp4_aligned(y, 4 * elem_bytes(out_type)) && ldy % 4 == 0;
    const int64_t quads = (p.ldp >> 2) * M;
    return fp4_launch(combine_kernel, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, st, ws, y, ldy, M, N, p.ldp, p.parts,
                      out_type, vec);
  }
  if (out_type == FP4_TYPE_F32) return launch_tiles<G, FP4_TYPE_F32>(p, M, N, K, a, b, y, ldy, st);
  if (out_type == FP4_TYPE_BF16) return launch_tiles<G, FP4_TYPE_BF16>(p, M, N, K, a, b, y, ldy, st);
  return launch_tiles<G, FP4_TYPE_F16>(p, M, N, K, a, b, y, ldy, st);
}

static int run_product(Plan p, int out_type, int64_t M, int64_t N, int64_t K, const fp4_mx& a, const fp4_mx& b, void* y,
                       int64_t ldy, void* ws, size_t ws_bytes, hipStream_t st) {
  if (p.tile == 0) return launch_rows(0, out_type, (int)M, (int)N, (int)K, nullptr, 0, &a, b, y, ldy, st);
  if (p.parts > 1 && (!ws || ws_bytes < (size_t)plane_bytes(p, M))) {
    p.parts = 1;
    p.per = (stages_of(K) + 1) & ~1;
  }
  if (p.first_n > 0) {
    const int64_t n = p.first_n;
    p.first_n = 0;
    if (int rc = run_product(p, out_type, M, n, K, a, b, y, ldy, nullptr, 0, st)) return rc;
    const fp4_mx rest = {static_cast<uint8_t*>(b.q) + n * b.ldq, static_cast<uint8_t*>(b.s) + n * b.lds, b.ldq, b.lds};
    return run_product(plan_of(M, N - n, K, fp4_device_cus(), false), out_type, M, N - n, K, a, rest,
                       static_cast<uint8_t*>(y) + n * elem_bytes(out_type), ldy, nullptr, 0, st);
  }
  const auto launch = [&](auto fn) { return fn(p, out_type, (int)M, (int)N, (int)K, a, b, y, ldy, ws, st); };
  if (p.tile == 256) return launch(launch_gemm<Tile<256, 256, 2, 2, 2, 1>>);
  if (p.tile == 128) return launch(launch_gemm<Tile<128, 128, 2, 2, 2, 1>>);
  return launch(launch_gemm<Tile<64, 64, 2, 2, 4, 2>>);
}

// K parts' planes alone, in tiles of 64 or 128 (parts have no others).
int launch_planes(int tile, int parts, int per, int64_t ldp, int M, int N, int K, const fp4_mx& a, const fp4_mx& b, void* planes,
                  hipStream_t st) {
  Plan p{};
  p.parts = parts, p.per = per;
  if (tile == 128) return launch_tiles<Tile<128, 128, 2, 2, 2, 1>, FP4_TYPE_F32>(p, M, N, K, a, b, planes, ldp, st);
  return launch_tiles<Tile<64, 64, 2, 2, 4, 2>, FP4_TYPE_F32>(p, M, N, K, a, b, planes, ldp, st);
}

}  // namespace mx

using namespace mx;

extern "C" int w4a4_matmul(int out_type, int64_t M, int64_t N, int64_t K, const fp4_mx* a, const fp4_mx* b, void* y,
                           int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  if (int rc = check_product(out_type, M, N, K)) return rc;
  if (M == 0) return FP4_OK;
  if (int rc = check_operand(a, K)) return rc;
  if (int rc = check_operand(b, K)) return rc;
  if (int rc = check_output(out_type, N, y, ldy)) return rc;
  if (workspace && !fp4_aligned(workspace, 16)) return FP4_ERR_ALIGN;
  return run_product(plan_of(M, N, K, fp4_device_cus()), out_type, M, N, K, *a, *b, y, ldy, workspace, workspace_bytes,
                     static_cast<hipStream_t>(stream));
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
  if (fused(M, N, K)) return launch_rows(x_type, out_type, (int)M, (int)N, (int)K, x, ldx, nullptr, *b, y, ldy, st);
  const Plan p = plan_of(M, N, K, fp4_device_cus());
  const LinearSpace sp = linear_space(p, M, K);
  if (!workspace || workspace_bytes < (size_t)(sp.q + sp.s)) return FP4_ERR_ARG;
  auto* w = static_cast<uint8_t*>(workspace);
  const int64_t nb = blocks_of(K);
  const fp4_mx a = {w, w + sp.q, nb * 16, (nb + 3) / 4 * 4};
  if (int rc = launch_quantize_rows(x_type, M, K, x, ldx, a, st)) return rc;
  return run_product(p, out_type, M, N, K, a, *b, y, ldy, w + sp.q + sp.s, workspace_bytes - (size_t)(sp.q + sp.s), st);
}
