// MXFP4 quantisation and its inverse.
//
// A block is 32 consecutive values along the axis that a product contracts. With a = max |x_i|,
//   s = max(floor(log2 a) - 2, -127),  code_i = E2M1 nearest to x_i / 2^s (halves to even, at most 6),
// so every step is exact but the one rounding to E2M1, which the hardware conversion does. All kernels read each
// value once and are bound by memory (a copy moves 4.8 TB/s): 2048 x 9728 bf16 along the rows takes 9.1 us (50 MB, part of
// them in the last-level cache), its inverse 9.2 us, 4095 x 9728 bf16 both ways 32 us (122 MB, 3.8 TB/s), 9728 x 2560 FP32
// both ways 30 us (126 MB, 4.2 TB/s).
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
// A lane holds a patch of 32 rows x 4 columns in registers, a wave 32 rows x 256 columns, the W waves of a workgroup
// 32 W rows. Down its columns every block is a lane's own, with no exchange; the results (16 bytes per column and wave)
// meet in LDS, so that a column's 16 W bytes leave as whole lines. Along the rows a block is 8 neighbouring lanes; a
// 4 x 4 exchange within each quad of lanes turns four rows' 2 bytes per lane into 8 bytes of one row, so that a store
// writes 128 bytes of each of four rows. Both results come from the one reading of x.
template <int T>
struct Patch {
  static constexpr int R = T == FP4_TYPE_F32 ? 4 : 2;  // registers per row
  uint32_t v[32][R];
  // the largest magnitude of column c (a 16-bit type: as amax_bits16 takes it)
  __device__ __forceinline__ void column_max(uint32_t (&m)[4]) const {
    if constexpr (T == FP4_TYPE_F32) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        m[c] = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) m[c] = max(m[c], v[i][c] & 0x7fffffffu);
      }
    } else {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) w = max_u16x2(w, v[i][p] & 0x7fff7fffu);
        m[2 * p] = amax_bits16<T>(w & 0xffffu);
        m[2 * p + 1] = amax_bits16<T>(w >> 16);
      }
    }
  }
  // codes of rows 2 i and 2 i + 1 of column C into byte B of `code`
  template <int C, int B>
  __device__ __forceinline__ uint32_t column_pair(uint32_t code, int i, float scale) const {
    if constexpr (T == FP4_TYPE_F32) return cvt_pair32<B>(code, v[2 * i][C], v[2 * i + 1][C], scale);
    else
      return cvt_pair16<T, B>(code, __builtin_amdgcn_perm(v[2 * i + 1][C >> 1], v[2 * i][C >> 1], C & 1 ? 0x07060302u : 0x05040100u),
                              scale);
  }
  template <int C>
  __device__ __forceinline__ u32x4 column(float scale, uint32_t mask) const {
    u32x4 out;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      uint32_t code = column_pair<C, 0>(0, 4 * d, scale);
      code = column_pair<C, 1>(code, 4 * d + 1, scale);
      code = column_pair<C, 2>(code, 4 * d + 2, scale);
      code = column_pair<C, 3>(code, 4 * d + 3, scale);
      out[d] = code & mask;
    }
    return out;
  }
  // row i: the scale byte of its block (8 lanes) and this lane's four codes; FINITE: the patch has no infinity or NaN
  template <bool FINITE>
  __device__ __forceinline__ void row(int i, uint32_t& sb, uint32_t& code) const {
    uint32_t m;
    if constexpr (T == FP4_TYPE_F32) {
      m = max(max(v[i][0] & 0x7fffffffu, v[i][1] & 0x7fffffffu), max(v[i][2] & 0x7fffffffu, v[i][3] & 0x7fffffffu));
    } else {  // the largest of the four in both halves
      m = max_u16x2(v[i][0] & 0x7fff7fffu, v[i][1] & 0x7fff7fffu);
      m = max_u16x2(m, __builtin_amdgcn_alignbit(m, m, 16));
    }
    m = quad_max(m);
    m = max(m, dpp<DPP_HALF_MIRROR>(m));
    if constexpr (T == FP4_TYPE_F16) m = amax_bits16<T>(m & 0xffffu);
    if constexpr (T == FP4_TYPE_BF16 && !FINITE) m &= 0xffff0000u;
    sb = FINITE ? finite_scale_byte(m) : scale_byte(m);
    const float sc = FINITE ? finite_scale_value(sb) : scale_value(sb);
    if constexpr (T == FP4_TYPE_F32) code = cvt_pair32<1>(cvt_pair32<0>(0, v[i][0], v[i][1], sc), v[i][2], v[i][3], sc);
    else code = cvt_pair16<T, 1>(cvt_pair16<T, 0>(0, v[i][0], sc), v[i][1], sc);
    if constexpr (!FINITE) code &= code_mask(sb);
  }
};

// A wave's rows, four at a time (rows and blocks past the input's are not stored): their codes, and their scales into LDS
// as [row][block] bytes.
template <int T, bool FINITE>
__device__ __forceinline__ void quantize_patch_rows(const Patch<T>& p, const fp4_mx& rows, uint8_t* scales, int row0, int col0, int lane,
                                                    int M, int nb) {
  const int quad = lane & 3, at = (col0 >> 1) + 8 * (lane >> 2);
  const bool live = at < 16 * nb;
  uint8_t* const q = static_cast<uint8_t*>(rows.q) + (int64_t)(row0 + quad) * rows.ldq + at;
  uint32_t mine = 0;  // the scales of rows 4 (lane % 8) .. + 3 of this lane's block, one byte each
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    __builtin_amdgcn_sched_barrier(0);  // four rows at a time: every row's exchange at once does not fit the registers
    uint32_t sb[4], c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p.template row<FINITE>(4 * g + i, sb[i], c[i]);
    if ((lane & 7) == g) mine = sb[0] | sb[1] << 8 | sb[2] << 16 | sb[3] << 24;
    // lane q of a quad takes row 4 g + q: first rows {0, 1} against {2, 3} with the lane two away, then the rows of
    // a pair with the neighbour
    const uint32_t lo = c[0] | c[1] << 16, hi = c[2] | c[3] << 16;
    const uint32_t keep = quad & 2 ? hi : lo, got = dpp<DPP_XOR2>(quad & 2 ? lo : hi);
    const uint32_t sel = quad & 1 ? 0x07060302u : 0x05040100u, other = quad & 1 ? 0x05040100u : 0x07060302u;
    const uint32_t own = __builtin_amdgcn_perm(got, keep, sel);  // this lane's and the far lane's codes of its row
    const uint32_t nbr = dpp<DPP_XOR1>(__builtin_amdgcn_perm(got, keep, other));
    // halves of own: (this lane, lane ^ 2); of nbr: (lane ^ 1, lane ^ 3)
    const uint32_t even = quad & 1 ? nbr : own, odd = quad & 1 ? own : nbr;
    const uint32_t first = __builtin_amdgcn_perm(odd, even, 0x05040100u), second = __builtin_amdgcn_perm(odd, even, 0x07060302u);
    const u32x2 out = quad & 2 ? u32x2{second, first} : u32x2{first, second};
    if (live && row0 + 4 * g + quad < M) *reinterpret_cast<u32x2*>(q + (int64_t)(4 * g) * rows.ldq) = out;
  }
#pragma unroll
  for (int b = 0; b < 4; ++b) scales[(4 * (lane & 7) + b) * 8 + (lane >> 3)] = (uint8_t)(mine >> (8 * b));
}

template <int T, int W, bool ROWS>
__global__ void __launch_bounds__(64 * W) quantize_cols_kernel(const void* __restrict__ x, int64_t ldx, fp4_mx rows, fp4_mx cols,
                                                               int M, int K, int tiles_k) {
  constexpr int EB = elem_bytes(T), R = Patch<T>::R;
  __shared__ u32x4 col_codes[256 * W];
  __shared__ uint8_t col_scales[256 * W];
  __shared__ uint8_t row_scales[ROWS ? W * 256 : 16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tm = blockIdx.x / tiles_k, tk = blockIdx.x - tm * tiles_k;
  const int col0 = 256 * tk, col = col0 + 4 * lane;
  const int row0 = 32 * (W * tm + wave);

  Patch<T> p;
  // row addresses are the wave's, columns the lane's
  const uint8_t* base = static_cast<const uint8_t*>(x) + (int64_t)min(row0, M - 1) * ldx * EB;
  const uint32_t off = (uint32_t)col * EB;
  const int64_t step = ldx * EB;
  const int last = M - 1 - row0;  // rows past the last one read it again
  if (col + 4 <= K) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      __builtin_memcpy(p.v[i], base + off, 4 * EB);
      if (i < last) base += step;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const uint8_t* r = base + off;
#pragma unroll
      for (int j = 0; j < R; ++j) p.v[i][j] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (col + j < K) {
          if constexpr (T == FP4_TYPE_F32) p.v[i][j] = reinterpret_cast<const uint32_t*>(r)[j];
          else p.v[i][j >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(r)[j] << (16 * (j & 1));
        }
      if (i < last) base += step;
    }
  }
  if (row0 + 32 > M) {  // and count as zeros
#pragma unroll
    for (int i = 0; i < 32; ++i)
#pragma unroll
      for (int j = 0; j < R; ++j) p.v[i][j] = row0 + i < M ? p.v[i][j] : 0u;
  }

  // down the columns: block `wave` of column c sits in slot wave ^ (c / 4 % W) of its 16 W bytes of LDS, so that
  // neither the writes (one slot of columns 4 lane + j) nor the reads (all slots of a column) meet in a bank
  uint32_t m[4], sb[4];
  p.column_max(m);
  // an infinity or NaN in the wave's patch shows in a column's maximum
  const bool finite = __builtin_amdgcn_ballot_w64((max(max(m[0], m[1]), max(m[2], m[3])) >> 23) == 255u) == 0;
  const int slot = 4 * W * lane + (wave ^ (lane & (W - 1)));
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    sb[c] = scale_byte(m[c]);
    col_scales[(4 * lane + c) * W + wave] = (uint8_t)sb[c];
  }
  col_codes[slot] = p.template column<0>(scale_value(sb[0]), code_mask(sb[0]));
  col_codes[slot + W] = p.template column<1>(scale_value(sb[1]), code_mask(sb[1]));
  col_codes[slot + 2 * W] = p.template column<2>(scale_value(sb[2]), code_mask(sb[2]));
  col_codes[slot + 3 * W] = p.template column<3>(scale_value(sb[3]), code_mask(sb[3]));

  if constexpr (ROWS) {
    // the column pass's magnitudes are not kept for the rows: that would double the registers
#pragma unroll
    for (int i = 0; i < 32; ++i)
#pragma unroll
      for (int j = 0; j < R; ++j) asm volatile("" : "+v"(p.v[i][j]));
    uint8_t* const s = row_scales + wave * 256;
    if (finite) quantize_patch_rows<T, true>(p, rows, s, row0, col0, lane, M, (int)blocks_of(K));
    else quantize_patch_rows<T, false>(p, rows, s, row0, col0, lane, M, (int)blocks_of(K));
  }
  __syncthreads();
  if constexpr (ROWS) {
    // lane: row lane / 2, four blocks
    const int row = row0 + (lane >> 1), blk = (col0 >> 5) + 4 * (lane & 1);
    if (row < M && blk < (int)blocks_of(K))
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(rows.s) + (int64_t)row * rows.lds + blk) =
          *reinterpret_cast<const uint32_t*>(row_scales + wave * 256 + lane * 4);
  }
  const int nbm = (int)blocks_of(M);
  auto* q = static_cast<uint8_t*>(cols.q);
  auto* s = static_cast<uint8_t*>(cols.s);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = i * 64 * W + threadIdx.x, c = e / W, b = e % W;
    if (col0 + c < K && W * tm + b < nbm)
      *reinterpret_cast<u32x4*>(q + (int64_t)(col0 + c) * cols.ldq + 16 * (W * tm + b)) = col_codes[c * W + (b ^ ((c >> 2) & (W - 1)))];
  }
  for (int e = threadIdx.x; e < 64 * W; e += 64 * W) {
    const int c = e / (W / 4), b = 4 * (e % (W / 4));
    if (col0 + c < K && W * tm + b < nbm)
      *reinterpret_cast<uint32_t*>(s + (int64_t)(col0 + c) * cols.lds + W * tm + b) = *reinterpret_cast<const uint32_t*>(col_scales + c * W + b);
  }
}

static int launch_quantize_cols(int type, int64_t M, int64_t K, const void* x, int64_t ldx, const fp4_mx* rows,
                                const fp4_mx& cols, hipStream_t st) {
  const int64_t tk = (K + 255) / 256;
  const bool tall = tk * ((M + 255) / 256) >= 2 * fp4_device_cus();
  const int w = tall ? 8 : 4;
  const int64_t tiles = tk * ((M + 32 * w - 1) / (32 * w));
  if (!fits_launch(tiles, 64 * w)) return FP4_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)tiles), block(64 * w);
  const fp4_mx r = rows ? *rows : fp4_mx{};
#define MX_COLS(T, W)                                                                                            \
  return rows ? fp4_launch(quantize_cols_kernel<T, W, true>, grid, block, 0, st, x, ldx, r, cols, M, K, tk)      \
              : fp4_launch(quantize_cols_kernel<T, W, false>, grid, block, 0, st, x, ldx, r, cols, M, K, tk)
#define MX_COLS_W(T)       \
  if (tall) MX_COLS(T, 8); \
  MX_COLS(T, 4)
  if (type == FP4_TYPE_F32) { MX_COLS_W(FP4_TYPE_F32); }
  if (type == FP4_TYPE_BF16) { MX_COLS_W(FP4_TYPE_BF16); }
  MX_COLS_W(FP4_TYPE_F16);
#undef MX_COLS_W
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
