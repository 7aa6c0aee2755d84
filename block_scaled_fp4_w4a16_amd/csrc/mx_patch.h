// A wave's patch of 32 rows x 256 columns, from which MXFP4 blocks are made along either axis (mx_quant.hip describes it).
#pragma once
#include "mx.h"

namespace mx {

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

}  // namespace mx
