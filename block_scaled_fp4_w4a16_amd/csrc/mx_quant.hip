// MXFP4 quantisation and its inverse.
//
// A block is 32 consecutive values along the axis that a product contracts. With a = max |x_i|,
//   s = max(floor(log2 a) - 2, -127),  code_i = E2M1 nearest to x_i / 2^s (halves to even, at most 6),
// so every step is exact but the one rounding to E2M1, which the hardware conversion does. All kernels read each
// value once and are bound by memory.
#include "mx.h"

namespace mx {

// ---------------------------------------------------------------------------------------- along the rows
// A lane holds 8 consecutive values of a row, a quad of lanes one block (its maximum: two lane exchanges), 16 lanes
// four blocks (whose scale bytes one lane stores as a dword). Loads and code stores are contiguous over the wave.
// A workgroup covers 2^ct_shift groups of 8 columns and 256 >> ct_shift rows, U times over.
template <int T, int U>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const void* __restrict__ x, int64_t ldx, uint8_t* __restrict__ q,
                                                            uint8_t* __restrict__ s, int64_t ldq, int64_t lds, int M, int K,
                                                            int ct_shift) {
  const int oct = (blockIdx.x << ct_shift) + (threadIdx.x & ((1 << ct_shift) - 1));
  const int rows_wg = 256 >> ct_shift;
  const int64_t row0 = (int64_t)blockIdx.y * (rows_wg * U) + (threadIdx.x >> ct_shift);
  const int nb = (int)blocks_of(K);
  const int c = 8 * oct;
  constexpr int R = T == FP4_TYPE_F32 ? 8 : 4;  // dwords per 8 values
  uint32_t v[U][R];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = row0 + (int64_t)u * rows_wg;
    const uint8_t* p = static_cast<const uint8_t*>(x) + (row * ldx + c) * elem_bytes(T);
#pragma unroll
    for (int i = 0; i < R; ++i) v[u][i] = 0;
    if (row < M && c + 8 <= K) {
      const u32x4 a = load16(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[u][i] = a[i];
      if constexpr (R == 8) {
        const u32x4 b = load16(p + 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u][4 + i] = b[i];
      }
    } else if (row < M && c < K) {  // the last, partial group of a row
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < K) {
          if constexpr (R == 8) v[u][i] = reinterpret_cast<const uint32_t*>(p)[i];
          else v[u][i >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
        }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = row0 + (int64_t)u * rows_wg;
    uint32_t m = 0;
    if constexpr (R == 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, v[u][i] & 0x7fffffffu);
      m = quad_max(m);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) m = max_u16x2(m, v[u][i] & 0x7fff7fffu);
      m = amax_bits16<T>(quad_max(max(m & 0xffffu, m >> 16)));
    }
    const uint32_t sb = scale_byte(m);
    const float sc = scale_value(sb);
    uint32_t code = 0;
    if constexpr (R == 8) {
      code = cvt_pair32<0>(code, v[u][0], v[u][1], sc);
      code = cvt_pair32<1>(code, v[u][2], v[u][3], sc);
      code = cvt_pair32<2>(code, v[u][4], v[u][5], sc);
      code = cvt_pair32<3>(code, v[u][6], v[u][7], sc);
    } else {
      code = cvt_pair16<T, 0>(code, v[u][0], sc);
      code = cvt_pair16<T, 1>(code, v[u][1], sc);
      code = cvt_pair16<T, 2>(code, v[u][2], sc);
      code = cvt_pair16<T, 3>(code, v[u][3], sc);
    }
    code &= code_mask(sb);
    const uint32_t four = sb | dpp<dpp_row_shl(4)>(sb) << 8 | dpp<dpp_row_shl(8)>(sb) << 16 | dpp<dpp_row_shl(12)>(sb) << 24;
    if (row < M && oct < 4 * nb) {
      *reinterpret_cast<uint32_t*>(q + row * ldq + 4 * oct) = code;
      if ((oct & 15) == 0) *reinterpret_cast<uint32_t*>(s + row * lds + (oct >> 2)) = four;
    }
  }
}

int launch_quantize_rows(int type, int64_t M, int64_t K, const void* x, int64_t ldx, const fp4_mx& rows, hipStream_t st) {
  const int64_t octs = 4 * blocks_of(K);
  // widest tile of columns (16 to 256 groups of 8) that leaves at most an eighth of its lanes past the row's end
  int sh = 8;
  while (sh > 4 && ((octs + (1 << sh) - 1) >> sh << sh) * 8 > octs * 9) --sh;
  const int64_t gx = (octs + (1 << sh) - 1) >> sh;
  const int rows_wg = 256 >> sh;
  auto* q = static_cast<uint8_t*>(rows.q);
  auto* s = static_cast<uint8_t*>(rows.s);
  // four rows per lane once that still leaves a few workgroups per compute unit
  const bool four = gx * M >= (int64_t)16 * rows_wg * fp4_device_cus();
  const int64_t per = (int64_t)rows_wg * (four ? 4 : 1);
  // a grid has at most 65535 rows of workgroups: longer inputs go in several launches
  const int64_t most = 65535 * per;
  for (int64_t r = 0; r < M; r += most) {
    const int64_t m = M - r < most ? M - r : most;
    const dim3 grid((unsigned)gx, (unsigned)((m + per - 1) / per));
    const uint8_t* xr = static_cast<const uint8_t*>(x) + r * ldx * elem_bytes(type);
    uint8_t* qr = q + r * rows.ldq;
    uint8_t* sr = s + r * rows.lds;
    int rc;
#define MX_ROWS(T)                                                                                                      \
  rc = four ? fp4_launch(quantize_rows_kernel<T, 4>, grid, dim3(256), 0, st, xr, ldx, qr, sr, rows.ldq, rows.lds, m, K, sh) \
            : fp4_launch(quantize_rows_kernel<T, 1>, grid, dim3(256), 0, st, xr, ldx, qr, sr, rows.ldq, rows.lds, m, K, sh)
    if (type == FP4_TYPE_F32) MX_ROWS(FP4_TYPE_F32);
    else if (type == FP4_TYPE_BF16) MX_ROWS(FP4_TYPE_BF16);
    else MX_ROWS(FP4_TYPE_F16);
#undef MX_ROWS
    if (rc) return rc;
  }
  return FP4_OK;
}

// ---------------------------------------------------------------------- along the columns, or along both axes
// A lane holds a patch of 32 rows x C columns in registers (C = 16 bytes of a row: 8 or 4 values). Down its columns
// every block is the lane's own: no exchange. Along its rows a block is 4 (16-bit types) or 8 (FP32) neighbouring
// lanes. A wave covers 4 patches down and 16 across: 128 rows x 128 (64) columns. Both results come from the one
// reading of x.
template <int T, bool ROWS>
__global__ void __launch_bounds__(256) quantize_cols_kernel(const void* __restrict__ x, int64_t ldx, fp4_mx rows, fp4_mx cols,
                                                            int M, int K, int tiles_k, int64_t tiles) {
  constexpr int EB = elem_bytes(T), C = 16 / EB, WC = 16 * C;
  const int lane = threadIdx.x & 63;
  const int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (tile >= tiles) return;
  const int tm = (int)(tile / tiles_k), tk = (int)(tile % tiles_k);
  const int cg = lane & 15, mb = lane >> 4;
  const int col0 = tk * WC, col = col0 + cg * C;
  const int row0 = tm * 128 + mb * 32;
  const uint8_t* p = static_cast<const uint8_t*>(x) + ((int64_t)row0 * ldx + col) * EB;
  u32x4 v[32];
  if (tm * 128 + 128 <= M && col0 + WC <= K) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = load16(p + (int64_t)i * ldx * EB);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      u32x4 w = {0, 0, 0, 0};
      if (row0 + i < M) {
        const uint8_t* r = p + (int64_t)i * ldx * EB;
#pragma unroll
        for (int j = 0; j < C; ++j)
          if (col + j < K) {
            if constexpr (T == FP4_TYPE_F32) w[j] = reinterpret_cast<const uint32_t*>(r)[j];
            else w[j >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(r)[j] << (16 * (j & 1));
          }
      }
      v[i] = w;
    }
  }

  // down the columns
  {
    auto* q = static_cast<uint8_t*>(cols.q);
    auto* s = static_cast<uint8_t*>(cols.s);
    const int bm = tm * 4 + mb;
    const bool live = row0 < M;
#pragma unroll
    for (int p4 = 0; p4 < 4; ++p4) {
      uint32_t m = 0;
      if constexpr (T == FP4_TYPE_F32) {
#pragma unroll
        for (int i = 0; i < 32; ++i) m = max(m, v[i][p4] & 0x7fffffffu);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) m = max_u16x2(m, v[i][p4] & 0x7fff7fffu);
      }
#pragma unroll
      for (int h = 0; h < (T == FP4_TYPE_F32 ? 1 : 2); ++h) {
        const int cc = T == FP4_TYPE_F32 ? p4 : 2 * p4 + h;
        uint32_t bits;
        if constexpr (T == FP4_TYPE_F32) bits = m;
        else bits = amax_bits16<T>(h ? m >> 16 : m & 0xffffu);
        const uint32_t sb = scale_byte(bits);
        const float sc = scale_value(sb);
        u32x4 out;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          uint32_t code = 0;
          if constexpr (T == FP4_TYPE_F32) {
            code = cvt_pair32<0>(code, v[8 * d][p4], v[8 * d + 1][p4], sc);
            code = cvt_pair32<1>(code, v[8 * d + 2][p4], v[8 * d + 3][p4], sc);
            code = cvt_pair32<2>(code, v[8 * d + 4][p4], v[8 * d + 5][p4], sc);
            code = cvt_pair32<3>(code, v[8 * d + 6][p4], v[8 * d + 7][p4], sc);
          } else {
            const uint32_t sel = h ? 0x07060302u : 0x05040100u;
            code = cvt_pair16<T, 0>(code, __builtin_amdgcn_perm(v[8 * d + 1][p4], v[8 * d][p4], sel), sc);
            code = cvt_pair16<T, 1>(code, __builtin_amdgcn_perm(v[8 * d + 3][p4], v[8 * d + 2][p4], sel), sc);
            code = cvt_pair16<T, 2>(code, __builtin_amdgcn_perm(v[8 * d + 5][p4], v[8 * d + 4][p4], sel), sc);
            code = cvt_pair16<T, 3>(code, __builtin_amdgcn_perm(v[8 * d + 7][p4], v[8 * d + 6][p4], sel), sc);
          }
          out[d] = code & code_mask(sb);
        }
        if (live && col + cc < K) {
          *reinterpret_cast<u32x4*>(q + (int64_t)(col + cc) * cols.ldq + 16 * bm) = out;
          s[(int64_t)(col + cc) * cols.lds + bm] = (uint8_t)sb;
        }
      }
    }
  }

  // along the rows
  if constexpr (ROWS) {
    auto* q = static_cast<uint8_t*>(rows.q);
    auto* s = static_cast<uint8_t*>(rows.s);
    const bool live = col < (int)blocks_of(K) * BLOCK;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      uint32_t m;
      uint32_t code = 0;
      uint32_t sb;
      if constexpr (T == FP4_TYPE_F32) {
        m = max(max(v[i][0] & 0x7fffffffu, v[i][1] & 0x7fffffffu), max(v[i][2] & 0x7fffffffu, v[i][3] & 0x7fffffffu));
        m = quad_max(m);
        m = max(m, dpp<DPP_HALF_MIRROR>(m));
        sb = scale_byte(m);
        const float sc = scale_value(sb);
        code = cvt_pair32<0>(code, v[i][0], v[i][1], sc);
        code = cvt_pair32<1>(code, v[i][2], v[i][3], sc);
        code &= code_mask(sb);
        code |= dpp<DPP_XOR1>(code) << 16;  // the even lane of a pair stores both halves
      } else {
        m = max_u16x2(max_u16x2(v[i][0] & 0x7fff7fffu, v[i][1] & 0x7fff7fffu),
                      max_u16x2(v[i][2] & 0x7fff7fffu, v[i][3] & 0x7fff7fffu));
        sb = scale_byte(amax_bits16<T>(quad_max(max(m & 0xffffu, m >> 16))));
        const float sc = scale_value(sb);
        code = cvt_pair16<T, 0>(code, v[i][0], sc);
        code = cvt_pair16<T, 1>(code, v[i][1], sc);
        code = cvt_pair16<T, 2>(code, v[i][2], sc);
        code = cvt_pair16<T, 3>(code, v[i][3], sc);
        code &= code_mask(sb);
      }
      if (row0 + i < M && live) {
        uint8_t* qr = q + (int64_t)(row0 + i) * rows.ldq + (col >> 1);
        if constexpr (T == FP4_TYPE_F32) {
          if (!(lane & 1)) *reinterpret_cast<uint32_t*>(qr) = code;
          if (!(lane & 7)) s[(int64_t)(row0 + i) * rows.lds + (col >> 5)] = (uint8_t)sb;
        } else {
          *reinterpret_cast<uint32_t*>(qr) = code;
          if (!(lane & 3)) s[(int64_t)(row0 + i) * rows.lds + (col >> 5)] = (uint8_t)sb;
        }
      }
    }
  }
}

static int launch_quantize_cols(int type, int64_t M, int64_t K, const void* x, int64_t ldx, const fp4_mx* rows,
                                const fp4_mx& cols, hipStream_t st) {
  const int wc = 16 * 16 / elem_bytes(type);
  const int64_t tk = (K + wc - 1) / wc, tm = (M + 127) / 128, tiles = tk * tm;
  if ((tiles + 3) / 4 > 0x7fffffffLL) return FP4_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)((tiles + 3) / 4));
  const fp4_mx r = rows ? *rows : fp4_mx{};
#define MX_COLS(T)                                                                                                     \
  return rows ? fp4_launch(quantize_cols_kernel<T, true>, grid, dim3(256), 0, st, x, ldx, r, cols, M, K, tk, tiles)    \
              : fp4_launch(quantize_cols_kernel<T, false>, grid, dim3(256), 0, st, x, ldx, r, cols, M, K, tk, tiles)
  if (type == FP4_TYPE_F32) MX_COLS(FP4_TYPE_F32);
  if (type == FP4_TYPE_BF16) MX_COLS(FP4_TYPE_BF16);
  MX_COLS(FP4_TYPE_F16);
#undef MX_COLS
}

// --------------------------------------------------------------------------------------------------- inverse
// A lane turns 4 bytes of codes into 8 values; same tiling as quantize_rows_kernel.
template <int T, int U>
__global__ void __launch_bounds__(256) dequant_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s, int64_t ldq,
                                                      int64_t lds, void* __restrict__ out, int64_t ldo, int M, int K,
                                                      int ct_shift) {
  const int oct = (blockIdx.x << ct_shift) + (threadIdx.x & ((1 << ct_shift) - 1));
  const int rows_wg = 256 >> ct_shift;
  const int64_t row0 = (int64_t)blockIdx.y * (rows_wg * U) + (threadIdx.x >> ct_shift);
  const int c = 8 * oct;
  uint32_t w[U], sb[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = row0 + (int64_t)u * rows_wg;
    w[u] = sb[u] = 0;
    if (row < M && c < K) {
      w[u] = *reinterpret_cast<const uint32_t*>(q + row * ldq + 4 * oct);
      sb[u] = s[row * lds + (oct >> 2)];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = row0 + (int64_t)u * rows_wg;
    if (row >= M || c >= K) continue;
    const float sc = sb[u] == 255u ? __builtin_nanf("") : scale_value(sb[u]);
    const bool nan = sb[u] == 255u;
    uint8_t* p = static_cast<uint8_t*>(out) + (row * ldo + c) * elem_bytes(T);
    if constexpr (T == FP4_TYPE_F32) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const auto r = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u] >> (8 * i), sc, 0);
        f[2 * i] = nan ? __builtin_nanf("") : r[0];
        f[2 * i + 1] = nan ? __builtin_nanf("") : r[1];
      }
      if (c + 8 <= K) {
        __builtin_memcpy(p, f, 32);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + i < K) reinterpret_cast<float*>(p)[i] = f[i];
      }
    } else {
      uint32_t f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const auto r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[u] >> (8 * i), sc, 0);
        f[i] = nan ? 0x7fc07fc0u : __builtin_bit_cast(uint32_t, r);
      }
      if (c + 8 <= K) {
        __builtin_memcpy(p, f, 16);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + i < K) reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(f[i >> 1] >> (16 * (i & 1)));
      }
    }
  }
}

}  // namespace mx

using namespace mx;

extern "C" int fp4_quantize_mxfp4(int type, int64_t M, int64_t K, const void* x, int64_t ldx, const fp4_mx* rows,
                                  const fp4_mx* cols, void* stream) {
  if (!valid_type(type)) return FP4_ERR_ARG;
  if (!rows && !cols) return FP4_ERR_ARG;
  if (int rc = check_dims(M, K)) return rc;
  if (M == 0) return FP4_OK;
  if (!x) return FP4_ERR_ARG;
  if (ldx < K) return FP4_ERR_SHAPE;
  if (ldx > (1LL << 40)) return FP4_ERR_UNSUPPORTED;
  if (!fp4_aligned(x, (uintptr_t)elem_bytes(type))) return FP4_ERR_ALIGN;
  if (rows)
    if (int rc = check_operand(rows, K)) return rc;
  if (cols) {
    if (M > MAX_DEPTH) return FP4_ERR_UNSUPPORTED;
    if (int rc = check_operand(cols, M)) return rc;
  }
  hipStream_t st = static_cast<hipStream_t>(stream);
  return cols ? launch_quantize_cols(type, M, K, x, ldx, rows, *cols, st)
              : launch_quantize_rows(type, M, K, x, ldx, *rows, st);
}

extern "C" int fp4_dequant_mxfp4(int type, int64_t M, int64_t K, const fp4_mx* a, void* out, int64_t ldo, void* stream) {
  if (type != FP4_TYPE_F32 && type != FP4_TYPE_BF16) return FP4_ERR_ARG;
  if (int rc = check_dims(M, K)) return rc;
  if (M == 0) return FP4_OK;
  if (!out) return FP4_ERR_ARG;
  if (int rc = check_operand(a, K)) return rc;
  if (ldo < K) return FP4_ERR_SHAPE;
  if (ldo > (1LL << 40)) return FP4_ERR_UNSUPPORTED;
  if (!fp4_aligned(out, (uintptr_t)elem_bytes(type))) return FP4_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t octs = (K + 7) / 8;
  int sh = 8;
  while (sh > 4 && ((octs + (1 << sh) - 1) >> sh << sh) * 8 > octs * 9) --sh;
  const int64_t gx = (octs + (1 << sh) - 1) >> sh;
  const int rows_wg = 256 >> sh;
  const bool four = gx * M >= (int64_t)16 * rows_wg * fp4_device_cus();
  const int64_t per = (int64_t)rows_wg * (four ? 4 : 1), most = 65535 * per;
  for (int64_t r = 0; r < M; r += most) {
    const int64_t m = M - r < most ? M - r : most;
    const dim3 grid((unsigned)gx, (unsigned)((m + per - 1) / per));
    const uint8_t* q = static_cast<const uint8_t*>(a->q) + r * a->ldq;
    const uint8_t* s = static_cast<const uint8_t*>(a->s) + r * a->lds;
    uint8_t* o = static_cast<uint8_t*>(out) + r * ldo * elem_bytes(type);
    int rc;
#define MX_DQ(T)                                                                                                      \
  rc = four ? fp4_launch(dequant_kernel<T, 4>, grid, dim3(256), 0, st, q, s, a->ldq, a->lds, o, ldo, m, K, sh)        \
            : fp4_launch(dequant_kernel<T, 1>, grid, dim3(256), 0, st, q, s, a->ldq, a->lds, o, ldo, m, K, sh)
    if (type == FP4_TYPE_F32) MX_DQ(FP4_TYPE_F32);
    else MX_DQ(FP4_TYPE_BF16);
#undef MX_DQ
    if (rc) return rc;
  }
  return FP4_OK;
}
