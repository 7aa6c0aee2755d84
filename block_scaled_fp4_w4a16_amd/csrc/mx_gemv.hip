// MXFP4 products with few rows of activations (decode, drafted tokens, small batches):
//   y[m][n] = sum_k A[m][k] B[n][k],  A in MXFP4 or dense and quantised on the way, B the weights in MXFP4.
//
// Bound by the bytes of B (17 per 32 weights). A workgroup owns 16 rows of B and all of A; its waves split K in
// pairs of 128-position chunks (a pair is one 128-byte line of a weight row), which go through LDS in whole lines. A lane
// reads 16-byte blocks of codes that are MFMA operands as they stand: nothing is decoded, and the scaled matrix
// instruction applies the block scales. The waves' sums meet in LDS in a fixed order.
// One row of 9728 x 2560 (13.2 MB) takes 5.5 us from cold weights, 2.4 TB/s, of 8192 x 28672 (125 MB) 25.1 us, 5.0 TB/s, and 3.4
// and 20.4 us where the same weights come again (replayed in a graph): the small ones are bound by a launch (1.8 us) and one
// round trip to memory. The figures below are of weights that come again.
#include "mx_epilogue.h"
#include "mx_groups.h"

namespace mx {

constexpr int GV_MAX_WAVES = 10;

// One lane's block of a dense row: 32 values from `k0` on (zeros past K) -> 16 bytes of codes and the scale byte.
template <int T>
__device__ __forceinline__ void quantize_block(const uint8_t* row, int k0, int K, u32x4& codes, uint32_t& sb) {
  constexpr int R = T == FP4_TYPE_F32 ? 32 : 16;
  uint32_t v[R];
  const uint8_t* p = row + (int64_t)k0 * elem_bytes(T);
  if (k0 + BLOCK <= K) {
#pragma unroll
    for (int i = 0; i < R / 4; ++i) {
      const u32x4 w = load16(p + 16 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * i + j] = w[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] = 0;
#pragma unroll
    for (int i = 0; i < BLOCK; ++i)
      if (k0 + i < K) {
        if constexpr (T == FP4_TYPE_F32) v[i] = reinterpret_cast<const uint32_t*>(p)[i];
        else v[i >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
      }
  }
  uint32_t m = 0;
  if constexpr (T == FP4_TYPE_F32) {
#pragma unroll
    for (int i = 0; i < 32; ++i) m = max(m, v[i] & 0x7fffffffu);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max_u16x2(m, v[i] & 0x7fff7fffu);
    m = amax_bits16<T>(max(m & 0xffffu, m >> 16));
  }
  sb = scale_byte(m);
  const float sc = scale_value(sb);
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    uint32_t c = 0;
    if constexpr (T == FP4_TYPE_F32) {
      c = cvt_pair32<0>(c, v[8 * d], v[8 * d + 1], sc);
      c = cvt_pair32<1>(c, v[8 * d + 2], v[8 * d + 3], sc);
      c = cvt_pair32<2>(c, v[8 * d + 4], v[8 * d + 5], sc);
      c = cvt_pair32<3>(c, v[8 * d + 6], v[8 * d + 7], sc);
    } else {
      c = cvt_pair16<T, 0>(c, v[4 * d], sc);
      c = cvt_pair16<T, 1>(c, v[4 * d + 1], sc);
      c = cvt_pair16<T, 2>(c, v[4 * d + 2], sc);
      c = cvt_pair16<T, 3>(c, v[4 * d + 3], sc);
    }
    codes[d] = c & code_mask(sb);
  }
}

// A pair of chunks of 16 operand rows (of 8, if `half`) into a wave's LDS: 128 bytes of codes per row at `codes`, the row's
// eight blocks XOR-swizzled by its last three bits, and 8 bytes of scales per row at `scales` (256 bytes, the second half
// unused). Neighbouring lanes read neighbouring bytes: the address unit takes a line per cycle, so that MFMA operands
// loaded as they are used, 16 rows at once, take four times as long (38 against 152 bytes per ns and compute unit, with
// everything in the L2). What lies past the operand's last byte is not read.
__device__ __forceinline__ void load_pair(__amdgpu_buffer_rsrc_t q, __amdgpu_buffer_rsrc_t s, int ldq, int lds, int p, bool half,
                                          uint8_t* codes, uint8_t* scales, int lane) {
  const uint32_t from = (lane >> 3) * ldq + (((lane & 7) ^ (lane >> 3)) << 4) + p * 128;
  const uint32_t sfrom = lane < 32 ? (uint32_t)((lane >> 1) * lds + (lane & 1) * 4 + p * 8) : 1u << 31;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(q, (__attribute__((address_space(3))) void*)codes, 16, from, 0, 0, 0);
  if (!half)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(q, (__attribute__((address_space(3))) void*)(codes + 1024), 16, from + 8 * ldq, 0, 0, 0);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(s, (__attribute__((address_space(3))) void*)scales, 4, sfrom, 0, 0, 0);
}

// Block g of chunk h of row n.
__device__ __forceinline__ u32x4 read_block(const uint8_t* codes, int n, int g, int h) {
  return *reinterpret_cast<const u32x4*>(codes + n * 128 + (((4 * h + g) ^ (n & 7)) << 4));
}

// LDS of a wave, in bytes: the weights' codes, both operands' scales and A's codes (of 8 rows where M allows); its sums
// take the same place at the end.
constexpr int GV_W = 0, GV_WS = 2048, GV_AS = 2304, GV_A = 2560;
static __host__ __device__ __forceinline__ int wave_lds(bool dense, int M) { return dense ? GV_AS : M <= 8 ? GV_A + 1024 : GV_A + 2048; }

// The sums of 16 columns from n0 on, in the first wave: lane l = 16 g + n has row n, columns n0 + 4 g .. + 3.
// XT: 0 for A in MXFP4, else the type of dense A. A wave takes the pairs wave, wave + waves, ... one after the other: loads
// of several pairs at once, or of the next one ahead, took as long or longer at every size (the waves of a compute unit
// cover each other). `each`: LDS bytes of a wave; A of `half` has 8 rows there.
template <int XT>
__device__ __forceinline__ f32x4 rows_sum(uint8_t* space, int each, bool half, int waves, int n0, const uint8_t* bq, const uint8_t* bs,
                                          int N, int K, int ldq, int lds, int M, const void* a, const uint8_t* as, int64_t lda, int las) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int nb = (int)blocks_of(K), pairs = (nb + 7) >> 3;
  const int rows = min(16, N - n0);
  const auto wq = fp4::make_rsrc(bq + (int64_t)n0 * ldq, (uint32_t)((rows - 1) * ldq + nb * BLOCK_BYTES));
  const auto ws = fp4::make_rsrc(bs + (int64_t)n0 * lds, (uint32_t)((rows - 1) * lds + ((nb + 3) & ~3)));
  uint8_t* const mine = space + wave * each;

  f32x4 acc = {0, 0, 0, 0};
  for (int p = wave; p < pairs; p += waves) {
    load_pair(wq, ws, ldq, lds, p, false, mine + GV_W, mine + GV_WS, lane);
    __builtin_amdgcn_sched_barrier(0);
    u32x4 av[2];
    uint32_t asc[2];
    if constexpr (XT == 0) {
      // rows of A past M: what is there, for sums that are not stored
      const auto aq = fp4::make_rsrc(a, (uint32_t)((M - 1) * (int)lda + nb * BLOCK_BYTES));
      const auto ar = fp4::make_rsrc(as, (uint32_t)((M - 1) * las + ((nb + 3) & ~3)));
      load_pair(aq, ar, (int)lda, las, p, half, mine + GV_A, mine + GV_AS, lane);
    } else {
      const uint8_t* row = static_cast<const uint8_t*>(a) + (int64_t)min(n, M - 1) * lda * elem_bytes(XT);
#pragma unroll
      for (int h = 0; h < 2; ++h) quantize_block<XT>(row, min(8 * p + 4 * h + g, nb - 1) * BLOCK, K, av[h], asc[h]);
    }
    __builtin_amdgcn_s_waitcnt(0xf70);  // the direct loads are there (vmcnt 0)
    asm volatile("" ::: "memory");
    const u32x2 wsc = *reinterpret_cast<const u32x2*>(mine + GV_WS + n * 8);
    if constexpr (XT == 0) {
      const int an = half ? n & 7 : n;
      const u32x2 s = *reinterpret_cast<const u32x2*>(mine + GV_AS + n * 8);
      av[0] = read_block(mine + GV_A, an, g, 0);
      av[1] = read_block(mine + GV_A, an, g, 1);
      asc[0] = s[0] >> (8 * g), asc[1] = s[1] >> (8 * g);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // a block past K: both scales 0, whose products are 36 2^-254 = 0 in FP32 whatever the codes are
      const bool in = 8 * p + 4 * h + g < nb;
      acc = mfma<0, 0>(read_block(mine + GV_W, n, g, h), in ? wsc[h] >> (8 * g) : 0u, av[h], in ? asc[h] : 0u, acc);
    }
    // every read is done before the next pair's loads overwrite what was read
    __builtin_amdgcn_s_waitcnt(0xc07f);
    asm volatile("" ::: "memory");
  }

  *reinterpret_cast<f32x4*>(mine + lane * 16) = acc;
  __syncthreads();
  f32x4 sum = acc;
  if (threadIdx.x < 64)
    for (int v = 1; v < waves; ++v) sum += *reinterpret_cast<const f32x4*>(space + v * each + lane * 16);
  return sum;
}

// The arguments that the weights' loads need come first: they are preloaded into scalar registers.
template <int XT>
__global__ void __launch_bounds__(64 * GV_MAX_WAVES)
    rows_kernel(const uint8_t* __restrict__ bq, const uint8_t* __restrict__ bs, int N, int K, int ldq, int lds, int m_waves,
                const void* __restrict__ a, const uint8_t* __restrict__ as, int64_t lda, int las, void* __restrict__ y,
                int64_t ldy, int out_type, int vec) {
  extern __shared__ uint8_t space[];
  const int waves = m_waves >> 8, M = m_waves & 255, n0 = blockIdx.x * 16;
  const f32x4 sum = rows_sum<XT>(space, wave_lds(XT != 0, M), M <= 8, waves, n0, bq, bs, N, K, ldq, lds, M, a, as, lda, las);
  const int lane = threadIdx.x, n = lane & 15, c = n0 + 4 * (lane >> 4);
  if (threadIdx.x < 64 && n < M && c < N) store4(out_type, y, n * ldy + c, sum, N - c, vec);
}

// The same with an epilogue.
template <int XT>
__global__ void __launch_bounds__(64 * GV_MAX_WAVES)
    rows_epilogue_kernel(const uint8_t* __restrict__ bq, const uint8_t* __restrict__ bs, int N, int K, int ldq, int lds, int m_waves,
                         const void* a, const uint8_t* as, int64_t lda, int las, void* y, int64_t ldy, int out_type, fp4_epilogue epi) {
  extern __shared__ uint8_t space[];
  const int waves = m_waves >> 8, M = m_waves & 255, n0 = blockIdx.x * 16;
  const f32x4 sum = rows_sum<XT>(space, wave_lds(XT != 0, M), M <= 8, waves, n0, bq, bs, N, K, ldq, lds, M, a, as, lda, las);
  const int lane = threadIdx.x, n = lane & 15, c = n0 + 4 * (lane >> 4);
  if (threadIdx.x < 64 && n < M && c < N) finish4(epi, out_type, y, ldy, n, c, c, sum, N - c);
}

// Up to 16 rows in groups, each with rows of B and a bias of its own. Workgroups in y take the groups that have rows, in order
// (as many as there are rows at most); those past the last one leave.
template <int XT>
__global__ void __launch_bounds__(64 * GV_MAX_WAVES)
    rows_grouped_kernel(const uint8_t* __restrict__ bq, const uint8_t* __restrict__ bs, int N, int K, int ldq, int lds, int m_waves,
                        Groups groups, int64_t step_q, int64_t step_s, const void* a, const uint8_t* as, int64_t lda, int las, void* y,
                        int64_t ldy, int out_type, int fill, fp4_epilogue epi) {
  extern __shared__ uint8_t space[];
  const int waves = m_waves >> 8, T = m_waves & 255, n0 = blockIdx.x * 16;
  const int lane = threadIdx.x & 63;
  int seen = 0, most = 0, first = 0, e = -1, row0 = 0, M = 0;
  for (int base = 0; base < groups.E; base += 64) {
    // bounds that decrease count as the largest in front of them (read_groups)
    const int i = base + lane;
    int lo = i < groups.E ? bound_at(groups, i, T) : 0, hi = i < groups.E ? bound_at(groups, i + 1, T) : 0;
    if (base == 0) first = uniform(lo);
    lo = max(scan_max(lo), most), hi = max(scan_max(hi), lo);
    const bool here = i < groups.E && hi > lo;
    const uint64_t some = __builtin_amdgcn_ballot_w64(here);
    const int rank = seen + __builtin_popcountll(some & ((1ull << lane) - 1));
    const uint64_t mine = __builtin_amdgcn_ballot_w64(here && rank == (int)blockIdx.y);
    if (mine) {
      const int from = __builtin_ctzll(mine);
      e = base + from;
      row0 = __builtin_amdgcn_readlane(lo, from), M = __builtin_amdgcn_readlane(hi, from) - row0;
    }
    seen += __builtin_popcountll(some);
    most = __builtin_amdgcn_readlane(hi, 63);
  }
  if (fill && blockIdx.y == 0) {
    for (int i = threadIdx.x; i < 16 * (first + T - most); i += blockDim.x) {
      const int c = n0 + (i & 15);
      if (c >= N) continue;
      const int64_t row = row_outside(i >> 4, first, most);
      float f[1] = {0};
      if (epi.residual) values_of(epi.residual_type, load_raw<1>(epi.residual_type, epi.residual, row * epi.ldr + c, 1), f);
      store_values(out_type, y, row * ldy + c, f, 1);
    }
  }
  if (M == 0) return;
  const uint8_t* const ar = static_cast<const uint8_t*>(a) + (int64_t)row0 * lda * (XT == 0 ? 1 : elem_bytes(XT));
  const f32x4 sum = rows_sum<XT>(space, wave_lds(XT != 0, T), T <= 8, waves, n0, bq + e * step_q, bs + e * step_s, N, K, ldq, lds, M, ar,
                                 as + (int64_t)row0 * las, lda, las);
  const int n = lane & 15, c = n0 + 4 * (lane >> 4);
  if (threadIdx.x < 64 && n < M && c < N)
    finish4(epi, out_type, y, ldy, row0 + n, c, (int64_t)e * N + c, sum, N - c);
}

// A product of few rows: what launch_rows takes, and what comes behind the sums.
struct Rows {
  int x_type, out_type, M, N, K;
  const void* x;
  int64_t ldx;
  const fp4_mx* a;
  const fp4_mx& b;
  void* y;
  int64_t ldy;
  const fp4_epilogue* epi;
  const Groups* groups;
  int64_t step_q, step_s;
  int fill;
};

template <int XT>
static int launch_variant(const Rows& r, int waves, hipStream_t st) {
  const int eb = elem_bytes(r.out_type), m_waves = r.M | waves << 8;
  const int vec = fp4_aligned(r.y, 4 * eb) && r.ldy % 4 == 0;
  const dim3 grid((unsigned)((r.N + 15) / 16), r.groups ? (unsigned)(r.M < r.groups->E ? r.M : r.groups->E) : 1), block(64 * waves);
  if (!fits_launch((int64_t)grid.x * grid.y, 64 * waves)) return FP4_ERR_UNSUPPORTED;
  const size_t lds = (size_t)waves * wave_lds(XT != 0, r.M);
  const void *x = XT ? r.x : r.a->q, *s = XT ? nullptr : r.a->s;
  const int64_t ldx = XT ? r.ldx : r.a->ldq, las = XT ? 0 : r.a->lds;
  if (r.groups)
    return fp4_launch(rows_grouped_kernel<XT>, grid, block, lds, st, r.b.q, r.b.s, r.N, r.K, r.b.ldq, r.b.lds, m_waves, *r.groups,
                      r.step_q, r.step_s, x, s, ldx, las, r.y, r.ldy, r.out_type, r.fill, r.epi ? *r.epi : fp4_epilogue{});
  if (r.epi)
    return fp4_launch(rows_epilogue_kernel<XT>, grid, block, lds, st, r.b.q, r.b.s, r.N, r.K, r.b.ldq, r.b.lds, m_waves, x, s, ldx, las,
                      r.y, r.ldy, r.out_type, *r.epi);
  return fp4_launch(rows_kernel<XT>, grid, block, lds, st, r.b.q, r.b.s, r.N, r.K, r.b.ldq, r.b.lds, m_waves, x, s, ldx, las, r.y, r.ldy,
                    r.out_type, vec);
}

static int launch_any_rows(const Rows& r, hipStream_t st) {
  const int pairs = (int)((blocks_of(r.K) + 7) / 8);
  const int64_t tiles = (int64_t)((r.N + 15) / 16) * (r.groups ? (r.M < r.groups->E ? r.M : r.groups->E) : 1);
  // Ten waves where a compute unit gets one workgroup (2560 x 9728: 4.7 us, with 8 waves 5.4; 4096 x 4096: 2.8 and 3.0),
  // eight where it gets several, of which more then fit (9728 x 2560: 4.3 us, with 10 waves 4.6; 8192 x 28672: 22.5 and 23.8).
  const int most = tiles > fp4_device_cus() ? 8 : 10, waves = pairs < most ? pairs : most;
  if (r.x_type == FP4_TYPE_F32) return launch_variant<FP4_TYPE_F32>(r, waves, st);
  if (r.x_type == FP4_TYPE_BF16) return launch_variant<FP4_TYPE_BF16>(r, waves, st);
  if (r.x_type == FP4_TYPE_F16) return launch_variant<FP4_TYPE_F16>(r, waves, st);
  return launch_variant<0>(r, waves, st);
}

// M <= 16.
int launch_rows(int x_type, int out_type, int M, int N, int K, const void* x, int64_t ldx, const fp4_mx* a,
                const fp4_mx& b, void* y, int64_t ldy, hipStream_t st, const fp4_epilogue* epi) {
  return launch_any_rows({x_type, out_type, M, N, K, x, ldx, a, b, y, ldy, epi, nullptr, 0, 0, 0}, st);
}

// The same with the rows in groups.
int launch_rows_grouped(int x_type, int out_type, int T, int N, int K, const Groups& groups, const void* x, int64_t ldx, const fp4_mx* a,
                        const fp4_mx& b, int64_t step_q, int64_t step_s, const fp4_epilogue* epi, void* y, int64_t ldy, int fill,
                        hipStream_t st) {
  return launch_any_rows({x_type, out_type, T, N, K, x, ldx, a, b, y, ldy, epi, &groups, step_q, step_s, fill}, st);
}

}  // namespace mx
