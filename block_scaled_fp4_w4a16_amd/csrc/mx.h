// Shared definitions of the MXFP4 operators: element types, the block scale, conversions and argument checks.
#pragma once
#include "common.h"
#include "fp4w4a16.h"
#include "launch.h"

namespace mx {

using fp4::u32x2;
using fp4::u32x4;

constexpr int BLOCK = 32;        // values that share one E8M0 scale
constexpr int BLOCK_BYTES = 16;  // their codes
constexpr int CHUNK = 128;       // positions one 16x16x128 MFMA contracts: four blocks

__host__ __device__ constexpr int64_t blocks_of(int64_t k) { return (k + BLOCK - 1) / BLOCK; }
__host__ __device__ constexpr int elem_bytes(int type) { return type == FP4_TYPE_F32 ? 4 : 2; }

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// E8M0 byte of a block whose largest magnitude has the FP32 bit pattern `amax` (sign clear): the exponent
// field is floor(log2) + 127, E2M1's largest level has exponent 2, so the byte is field - 2, at least 0 (zeros
// and FP32 subnormals have field 0). An infinity or NaN (field 255) makes the whole block NaN: byte 255.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const uint32_t f = amax >> 23;
  return f == 255u ? 255u : (f > 2u ? f - 2u : 0u);
}

// 2^(s - 127) as FP32; byte 0 is the subnormal 2^-127, byte 255 gives infinity (see code_mask).
__device__ __forceinline__ float scale_value(uint32_t s) {
  return __builtin_bit_cast(float, s ? s << 23 : 0x00400000u);
}

// The same for a block known to be finite, in one instruction each: the exponent field less 2, held at 0; and a scale
// operand of the conversions, which use its exponent field alone (the mantissa bit makes byte 0 a 2^-127).
__device__ __forceinline__ uint32_t finite_scale_byte(uint32_t amax) { return __builtin_elementwise_sub_sat(amax >> 23, 2u); }
__device__ __forceinline__ float finite_scale_value(uint32_t s) { return __builtin_bit_cast(float, s << 23 | 0x00400000u); }

// Codes of a NaN block are zeros: only its scale byte says what it holds.
__device__ __forceinline__ uint32_t code_mask(uint32_t s) { return s == 255u ? 0u : ~0u; }

// Largest magnitude of 16-bit values as the FP32 pattern that scale_byte takes. `m` is the integer maximum
// of the sign-cleared patterns, which orders bf16 and FP16 values alike, NaN above infinity.
template <int T>
__device__ __forceinline__ uint32_t amax_bits16(uint32_t m) {
  if constexpr (T == FP4_TYPE_BF16) return m << 16;
  else return __builtin_bit_cast(uint32_t, (float)__builtin_bit_cast(_Float16, (uint16_t)m));
}

// Two values -> two E2M1 codes in byte SEL of `old`: x / scale rounded to nearest, halves to the even code,
// saturating at 6 (v_cvt_scalef32_pk_fp4_*; the scale's exponent divides exactly, subnormal 2^-127 included).
template <int T, int SEL>
__device__ __forceinline__ uint32_t cvt_pair16(uint32_t old, uint32_t pair, float scale) {
  if constexpr (T == FP4_TYPE_BF16)
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2, pair), scale, SEL);
  else
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, __builtin_bit_cast(f16x2, pair), scale, SEL);
}
template <int SEL>
__device__ __forceinline__ uint32_t cvt_pair32(uint32_t old, uint32_t a, uint32_t b, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, __builtin_bit_cast(float, a), __builtin_bit_cast(float, b), scale,
                                                  SEL);
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t,
                            __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
constexpr int DPP_XOR1 = 0xB1, DPP_XOR2 = 0x4E;  // quad_perm [1,0,3,2] and [2,3,0,1]
constexpr int DPP_HALF_MIRROR = 0x141;           // lane i <- lane 7 - i of its group of 8
constexpr int dpp_row_shl(int n) { return 0x100 + n; }  // lane i <- lane i + n of its row of 16, 0 past the end

// Maximum over the 4 lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, dpp<DPP_XOR1>(v));
  return max(v, dpp<DPP_XOR2>(v));
}

// Loads of `n` bytes at any alignment of the element type (gfx950 takes unaligned vector loads).
__device__ __forceinline__ u32x4 load16(const void* p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// FP32 -> bits of the output type, round to nearest even.
__device__ __forceinline__ uint32_t to16(int type, float v) {
  if (type == FP4_TYPE_BF16) return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v);
  return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v);
}

// Two FP32 sums -> two outputs of a 16-bit type in one register, rounded to nearest even.
template <int OUT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (OUT == FP4_TYPE_BF16) return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
  else return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
}

// Four consecutive outputs y[0 .. n - 1], n <= 4, of the given type; one vector store where all four exist and
// the address allows it.
__device__ __forceinline__ void store4(int type, void* y, int64_t at, const f32x4& v, int n, bool vec) {
  if (type == FP4_TYPE_F32) {
    float* p = static_cast<float*>(y) + at;
    if (vec && n >= 4) {
      *reinterpret_cast<f32x4*>(p) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) p[i] = v[i];
    }
    return;
  }
  uint16_t* p = static_cast<uint16_t*>(y) + at;
  const uint32_t a = to16(type, v[0]), b = to16(type, v[1]), c = to16(type, v[2]), d = to16(type, v[3]);
  if (vec && n >= 4) {
    *reinterpret_cast<u32x2*>(p) = u32x2{a | b << 16, c | d << 16};
  } else {
    if (n > 0) p[0] = (uint16_t)a;
    if (n > 1) p[1] = (uint16_t)b;
    if (n > 2) p[2] = (uint16_t)c;
    if (n > 3) p[3] = (uint16_t)d;
  }
}

// D (16 x 16) += A (16 x 128) B (16 x 128)^T on the scaled matrix instruction, both operands E2M1 with one E8M0
// byte per 32 positions. Lane l = 16 g + n gives block g of row n of A and of B: 16 bytes of codes and byte SA /
// SB of its scale register; it receives D[4 g + i][n]. Products are exact, the sum is kept in FP32.
template <int SA, int SB>
__device__ __forceinline__ f32x4 mfma(const u32x4& a, uint32_t sa, const u32x4& b, uint32_t sb, const f32x4& c) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, SA, (int)sa, SB, (int)sb);
}

// ------------------------------------------------------------------------------------------------ host side

static inline bool valid_type(int t) { return t == FP4_TYPE_F32 || t == FP4_TYPE_BF16 || t == FP4_TYPE_F16; }

constexpr int64_t MAX_ROWS = 1LL << 30, MAX_DEPTH = 1LL << 22, MAX_STRIDE = 1LL << 22;

// An MXFP4 operand of `rows` rows and depth `k` (both at least 1): null, stride and alignment checks.
static inline int check_operand(const fp4_mx* a, int64_t k) {
  if (!a || !a->q || !a->s) return FP4_ERR_ARG;
  const int64_t nb = blocks_of(k);
  if (a->ldq < nb * BLOCK_BYTES || a->lds < nb) return FP4_ERR_SHAPE;
  if (a->ldq > MAX_STRIDE || a->lds > MAX_STRIDE) return FP4_ERR_UNSUPPORTED;
  if (!fp4_aligned(a->q, 16) || a->ldq % 16 || !fp4_aligned(a->s, 4) || a->lds % 4) return FP4_ERR_ALIGN;
  return FP4_OK;
}

static inline int check_dims(int64_t rows, int64_t k) {
  if (rows < 0 || k < 1) return FP4_ERR_SHAPE;
  if (rows > MAX_ROWS || k > MAX_DEPTH) return FP4_ERR_UNSUPPORTED;
  return FP4_OK;
}

static inline int check_product(int out_type, int64_t M, int64_t N, int64_t K) {
  if (!valid_type(out_type)) return FP4_ERR_ARG;
  if (N < 1) return FP4_ERR_SHAPE;
  if (int rc = check_dims(M, K)) return rc;
  if (N > MAX_ROWS) return FP4_ERR_UNSUPPORTED;
  return FP4_OK;
}

static inline int check_output(int out_type, int64_t N, const void* y, int64_t ldy) {
  if (!y) return FP4_ERR_ARG;
  if (ldy < N) return FP4_ERR_SHAPE;
  if (ldy > (1LL << 40)) return FP4_ERR_UNSUPPORTED;
  return fp4_aligned(y, (uintptr_t)elem_bytes(out_type)) ? FP4_OK : FP4_ERR_ALIGN;
}

// Dense activations x[M][K] (M at least 1).
static inline int check_dense(int type, int64_t K, const void* x, int64_t ldx) {
  if (!x) return FP4_ERR_ARG;
  if (ldx < K) return FP4_ERR_SHAPE;
  if (ldx > (1LL << 40)) return FP4_ERR_UNSUPPORTED;
  return fp4_aligned(x, (uintptr_t)elem_bytes(type)) ? FP4_OK : FP4_ERR_ALIGN;
}

// Whether a launch stays below the 2^32 work items that one can have.
static inline bool fits_launch(int64_t workgroups, int threads) { return workgroups * threads < (1LL << 32); }

// Products of already checked arguments (mx_gemv.hip, mx_gemm.hip).
int launch_rows(int x_type, int out_type, int M, int N, int K, const void* x, int64_t ldx, const fp4_mx* a,
                const fp4_mx& b, void* y, int64_t ldy, hipStream_t st, const fp4_epilogue* epi = nullptr);
int launch_planes(int tile, int parts, int per, int64_t ldp, int M, int N, int K, const fp4_mx& a, const fp4_mx& b, void* planes,
                  hipStream_t st);
int launch_quantize_rows(int type, int64_t M, int64_t K, const void* x, int64_t ldx, const fp4_mx& rows, hipStream_t st);

}  // namespace mx
