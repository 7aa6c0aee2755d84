// MXFP4 products with few rows of activations (decode, drafted tokens, small batches):
//   y[m][n] = sum_k A[m][k] B[n][k],  A in MXFP4 or dense and quantised on the way, B the weights in MXFP4.
//
// Bound by the bytes of B (17 per 32 weights). A workgroup owns 16 T rows of B and all of A; its waves split K in
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

// XT: 0 for A in MXFP4, else the type of dense A. MB blocks of 16 rows of A, T tiles of 16 rows of B, U chunk
// pairs in flight.
template <int XT, int MB, int T, int U>
__global__ void __launch_bounds__(64 * GV_MAX_WAVES)
    rows_kernel(const uint8_t* __restrict__ bq, const uint8_t* __restrict__ bs, int ldq, int lds, const void* __restrict__ a,
                const uint8_t* __restrict__ as, int64_t lda, int las, int M, int N, int K, void* __restrict__ y, int64_t ldy,
                int out_type, int vec) {
  extern __shared__ float red[];  // [waves][MB][T][64][4]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int n = lane & 15, g = lane >> 4;
  const int nb = (int)blocks_of(K), pairs = (nb + 7) >> 3;
  const int n0 = blockIdx.x * 16 * T;

  const uint8_t* qrow[T];
  const uint8_t* srow[T];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const int64_t r = min(n0 + 16 * t + n, N - 1);
    qrow[t] = bq + r * ldq;
    srow[t] = bs + r * lds;
  }
  const uint8_t* arow[MB];
  const uint8_t* asrow[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    const int64_t r = min(16 * b + n, M - 1);
    arow[b] = static_cast<const uint8_t*>(a) + r * lda * (XT ? elem_bytes(XT) : 1);
    asrow[b] = XT ? nullptr : as + r * las;
  }

  f32x4 acc[MB][T];
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[b][t] = f32x4{0, 0, 0, 0};

  for (int p0 = wave; p0 < pairs; p0 += waves * U) {
    u32x4 w[U][2][T];
    uint32_t ws[U][2][T];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int blk = 8 * (p0 + u * waves) + 4 * h + g;
        const int at = min(blk, nb - 1);  // past the end: the last block again, with scale 2^-127 on both sides
#pragma unroll
        for (int t = 0; t < T; ++t) {
          w[u][h][t] = *reinterpret_cast<const u32x4*>(qrow[t] + (int64_t)at * BLOCK_BYTES);
          ws[u][h][t] = srow[t][at];
        }
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int blk = 8 * (p0 + u * waves) + 4 * h + g;
        const int at = min(blk, nb - 1);
#pragma unroll
        for (int b = 0; b < MB; ++b) {
          u32x4 av;
          uint32_t sv;
          if constexpr (XT != 0) {
            quantize_block<XT>(arow[b], at * BLOCK, K, av, sv);
          } else {
            av = *reinterpret_cast<const u32x4*>(arow[b] + (int64_t)at * BLOCK_BYTES);
            sv = asrow[b][at];
          }
          if (blk >= nb) sv = 0;
#pragma unroll
          for (int t = 0; t < T; ++t)
            acc[b][t] = mfma<0, 0>(w[u][h][t], blk < nb ? ws[u][h][t] : 0u, av, sv, acc[b][t]);
        }
      }
  }

#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int t = 0; t < T; ++t)
      *reinterpret_cast<f32x4*>(red + ((size_t)(wave * MB + b) * T + t) * 256 + lane * 4) = acc[b][t];
  __syncthreads();
  for (int e = threadIdx.x; e < MB * T * 64; e += blockDim.x) {
    f32x4 sum = *reinterpret_cast<const f32x4*>(red + (size_t)e * 4);
    for (int v = 1; v < waves; ++v) sum += *reinterpret_cast<const f32x4*>(red + ((size_t)v * MB * T * 64 + e) * 4);
    const int l = e & 63, bt = e >> 6, b = bt / T, t = bt % T;
    const int m = 16 * b + (l & 15), c = n0 + 16 * t + 4 * (l >> 4);
    if (m < M && c < N) store4(out_type, y, (int64_t)m * ldy + c, sum, N - c, vec);
  }
}

template <int XT, int MB, int T, int U>
static int launch_variant(int waves, int out_type, int M, int N, int K, const void* x, int64_t ldx, const fp4_mx* a,
                          const fp4_mx& b, void* y, int64_t ldy, hipStream_t st) {
  const int eb = elem_bytes(out_type);
  const int vec = fp4_aligned(y, 4 * eb) && ldy % 4 == 0;
  const dim3 grid((unsigned)((N + 16 * T - 1) / (16 * T)));
  const size_t lds = (size_t)waves * MB * T * 1024;
  return fp4_launch(rows_kernel<XT, MB, T, U>, grid, dim3(64 * waves), lds, st, b.q, b.s, b.ldq, b.lds, XT ? x : a->q,
                    XT ? nullptr : a->s, XT ? ldx : a->ldq, XT ? 0 : a->lds, M, N, K, y, ldy, out_type, vec);
}

// M <= 64; dense A (x_type != 0): M <= 16.
int launch_rows(int x_type, int out_type, int M, int N, int K, const void* x, int64_t ldx, const fp4_mx* a,
                const fp4_mx& b, void* y, int64_t ldy, hipStream_t st) {
  const int pairs = (int)((blocks_of(K) + 7) / 8);
  int waves = pairs < 8 ? pairs : 8;
#define MX_GV(XT, MB, T, U) return launch_variant<XT, MB, T, U>(waves, out_type, M, N, K, x, ldx, a, b, y, ldy, st)
  if (x_type == FP4_TYPE_F32) MX_GV(FP4_TYPE_F32, 1, 1, 2);
  if (x_type == FP4_TYPE_BF16) MX_GV(FP4_TYPE_BF16, 1, 1, 2);
  if (x_type == FP4_TYPE_F16) MX_GV(FP4_TYPE_F16, 1, 1, 2);
  if (M <= 16) MX_GV(0, 1, 1, 2);
  if (M <= 32) MX_GV(0, 2, 1, 2);
  MX_GV(0, 4, 1, 2);
#undef MX_GV
}

}  // namespace mx
