// MXFP4 products with few rows of activations (decode, drafted tokens, small batches):
//   y[m][n] = sum_k A[m][k] B[n][k],  A in MXFP4 or dense and quantised on the way, B the weights in MXFP4.
//
// Bound by the bytes of B (17 per 32 weights). A workgroup owns 16 rows of B and all of A; its waves split K in
// pairs of 128-position chunks (a pair is one 128-byte line of a weight row), each lane reading 16-byte blocks of
// codes that are MFMA operands as they stand: nothing is decoded, and the scaled matrix instruction applies the
// block scales. The waves' sums meet in LDS in a fixed order.
#include "mx.h"

namespace mx {

constexpr int GV_MAX_WAVES = 16;

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

// Blocks of operand rows by buffer loads: bytes past the operand come back as zeros.
__device__ __forceinline__ u32x4 load_codes(__amdgpu_buffer_rsrc_t r, uint32_t at) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0);
}
__device__ __forceinline__ u32x2 load_scales(__amdgpu_buffer_rsrc_t r, uint32_t at) {
  return __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0);
}

// XT: 0 for A in MXFP4, else the type of dense A. A wave takes the pairs wave, wave + waves, ... one after the other: loads
// of several pairs at once, or of the next one ahead, took as long or longer at every size (the waves of a compute unit
// cover each other), while more registers mean fewer waves. The arguments that the weights' loads need come first: they
// are preloaded into scalar registers.
template <int XT>
__global__ void __launch_bounds__(64 * GV_MAX_WAVES)
    rows_kernel(const uint8_t* __restrict__ bq, const uint8_t* __restrict__ bs, int N, int K, int ldq, int lds, int m_waves,
                const void* __restrict__ a, const uint8_t* __restrict__ as, int64_t lda, int las, void* __restrict__ y,
                int64_t ldy, int out_type, int vec) {
  extern __shared__ f32x4 red[];  // [waves][64]
  const int lane = threadIdx.x & 63, waves = m_waves >> 8, M = m_waves & 255;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int nb = (int)blocks_of(K), pairs = (nb + 7) >> 3;
  const int n0 = blockIdx.x * 16, rows = min(16, N - n0);
  const auto wq = fp4::make_rsrc(bq + (int64_t)n0 * ldq, (uint32_t)((rows - 1) * ldq + nb * BLOCK_BYTES));
  const auto ws = fp4::make_rsrc(bs + (int64_t)n0 * lds, (uint32_t)((rows - 1) * lds + ((nb + 3) & ~3)));
  const uint32_t wq0 = n * ldq + g * BLOCK_BYTES, ws0 = n * lds;

  f32x4 acc = {0, 0, 0, 0};
  for (int p = wave; p < pairs; p += waves) {
    const u32x4 w[2] = {load_codes(wq, wq0 + p * 128), load_codes(wq, wq0 + p * 128 + 64)};
    const u32x2 wsc = load_scales(ws, ws0 + p * 8);
    __builtin_amdgcn_sched_barrier(0);
    u32x4 av[2];
    uint32_t asc[2];
    if constexpr (XT == 0) {
      // rows of A past M read nothing
      const auto aq = fp4::make_rsrc(a, (uint32_t)((M - 1) * (int)lda + nb * BLOCK_BYTES));
      const auto ar = fp4::make_rsrc(as, (uint32_t)((M - 1) * las + ((nb + 3) & ~3)));
      const uint32_t at = n * (int)lda + g * BLOCK_BYTES + p * 128;
      av[0] = load_codes(aq, at);
      av[1] = load_codes(aq, at + 64);
      const u32x2 s = load_scales(ar, n * las + p * 8);
      asc[0] = s[0] >> (8 * g), asc[1] = s[1] >> (8 * g);
    } else {
      const uint8_t* row = static_cast<const uint8_t*>(a) + (int64_t)min(n, M - 1) * lda * elem_bytes(XT);
#pragma unroll
      for (int h = 0; h < 2; ++h) quantize_block<XT>(row, min(8 * p + 4 * h + g, nb - 1) * BLOCK, K, av[h], asc[h]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // a block past K: both scales 0, whose products are 36 2^-254 = 0 in FP32 whatever the codes are
      const bool in = 8 * p + 4 * h + g < nb;
      acc = mfma<0, 0>(w[h], in ? wsc[h] >> (8 * g) : 0u, av[h], in ? asc[h] : 0u, acc);
    }
  }

  red[wave * 64 + lane] = acc;
  __syncthreads();
  if (threadIdx.x < 64) {
    f32x4 sum = red[lane];
    for (int v = 1; v < waves; ++v) sum += red[v * 64 + lane];
    const int c = n0 + 4 * g;
    if (n < M && c < N) store4(out_type, y, n * ldy + c, sum, N - c, vec);
  }
}

template <int XT>
static int launch_variant(int waves, int out_type, int M, int N, int K, const void* x, int64_t ldx, const fp4_mx* a,
                          const fp4_mx& b, void* y, int64_t ldy, hipStream_t st) {
  const int eb = elem_bytes(out_type);
  const int vec = fp4_aligned(y, 4 * eb) && ldy % 4 == 0;
  const dim3 grid((unsigned)((N + 15) / 16));
  if (!fits_launch(grid.x, 64 * waves)) return FP4_ERR_UNSUPPORTED;
  return fp4_launch(rows_kernel<XT>, grid, dim3(64 * waves), (size_t)waves * 1024, st, b.q, b.s, N, K, b.ldq, b.lds,
                    M | waves << 8, XT ? x : a->q, XT ? nullptr : a->s, XT ? ldx : a->ldq, XT ? 0 : a->lds, y, ldy, out_type, vec);
}

// M <= 16.
int launch_rows(int x_type, int out_type, int M, int N, int K, const void* x, int64_t ldx, const fp4_mx* a,
                const fp4_mx& b, void* y, int64_t ldy, hipStream_t st) {
  const int pairs = (int)((blocks_of(K) + 7) / 8);
  // ten waves, or one per pair: at 4096 x 4096 (16 pairs) 3.6 us, with 8 waves 3.7 and with 16 3.9; at 2560 x 9728 (38
  // pairs) 5.3 us, 5.5 and 5.7; at 9728 x 2560 (10 pairs) 4.7 us, with 8 waves 4.9
  const int waves = pairs < 10 ? pairs : 10;
#define MX_GV(XT) return launch_variant<XT>(waves, out_type, M, N, K, x, ldx, a, b, y, ldy, st)
  if (x_type == FP4_TYPE_F32) MX_GV(FP4_TYPE_F32);
  if (x_type == FP4_TYPE_BF16) MX_GV(FP4_TYPE_BF16);
  if (x_type == FP4_TYPE_F16) MX_GV(FP4_TYPE_F16);
  MX_GV(0);
#undef MX_GV
}

}  // namespace mx
