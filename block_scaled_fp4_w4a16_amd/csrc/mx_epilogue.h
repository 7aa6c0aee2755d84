// What follows an MXFP4 product in the same kernel: y = f(z + bias) + residual with z the FP32 sum, rounded once to y's type;
// z + bias kept in FP32 where the backward pass needs it.
#pragma once
#include "mx.h"

namespace mx {

constexpr float LOG2E = 1.44269504f;
constexpr float TANH_1 = 1.59576912f, TANH_3 = 0.0713548163f;  // 2 sqrt(2 / pi), and that times 0.044715

// 1 / (1 + 2^u), and its limits 0 and 1 at infinities.
__device__ __forceinline__ float sigmoid2(float u) { return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u)); }

// What z is multiplied by in silu, and in gelu by tanh: s(2 sqrt(2 / pi) (z + 0.044715 z^3)), where z^2 is held below what makes
// s 0 or 1 anyway, so that no infinity less infinity arises.
__device__ __forceinline__ float silu_factor(float z) { return sigmoid2(z * -LOG2E); }
__device__ __forceinline__ float tanh_factor(float z) { return sigmoid2(z * (-LOG2E * TANH_1 - LOG2E * TANH_3 * fminf(z * z, 1e4f))); }

// The normal distribution's upper tail at |z|, and e = exp(-z^2 / 2) for its density. With a = |z| / sqrt 2 and
// t = 1 / (1 + 0.33 a), erfc(a) = t P(t) exp(-a^2), P a polynomial fitted to erfc(a) exp(a^2) / t for a up to 10.5 with relative
// weights: 1.25e-7 off at most, about a step of FP32, so that the tail has its relative accuracy. At infinities both are 0.
__device__ __forceinline__ float normal_tail(float z, float& e) {
  const float t = __builtin_amdgcn_rcpf(1.0f + (0.33f * 0.707106781f) * fabsf(z));
  float p = -0.5f * 0.134472281f;
  p = p * t + 0.5f * 0.456568509f;
  p = p * t - 0.5f * 0.344742447f;
  p = p * t + 0.5f * 0.402482688f;
  p = p * t + 0.5f * 0.0504948199f;
  p = p * t + 0.5f * 0.200193852f;
  p = p * t + 0.5f * 0.183129117f;
  p = p * t + 0.5f * 0.186345816f;
  e = __builtin_amdgcn_exp2f(z * z * (-0.5f * LOG2E));
  return p * t * e;
}

// f(z) of W values in place; `act` is the same for the whole wave. A NaN stays; f(infinity) is infinity; f(-infinity) is 0 for
// relu and gelu and NaN for silu and gelu by tanh (minus infinity times 0).
template <int W>
__device__ __forceinline__ void activate(int act, float (&z)[W]) {
  if (act == FP4_ACT_NONE) return;
  if (act == FP4_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < W; ++i) z[i] = z[i] < 0 ? 0.0f : z[i];
  } else if (act == FP4_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < W; ++i) {  // max(z, 0) - |z| tail: the maximum drops a NaN, the tail brings it back
      float e;
      const float tail = normal_tail(z[i], e);
      z[i] = fmaf(-fminf(fabsf(z[i]), 1e30f), tail, fmaxf(z[i], 0.0f));
    }
  } else if (act == FP4_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < W; ++i) z[i] *= silu_factor(z[i]);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) z[i] *= tanh_factor(z[i]);
  }
}

// f'(z). |z| is held where f' has long been 0 or 1 in FP32 (a NaN stays), so that infinities get their limits. With s the logistic
// function, 1 - s is taken as 2^u s: by a subtraction, an s that rounds to 1 less a bit or two would be z times that off.
__device__ __forceinline__ float slope(int act, float z) {
  if (act == FP4_ACT_RELU) return z > 0 ? 1.0f : z <= 0 ? 0.0f : z;
  z = z > 128.0f ? 128.0f : z < -128.0f ? -128.0f : z;
  if (act == FP4_ACT_SILU || act == FP4_ACT_GELU_TANH) {
    const bool silu = act == FP4_ACT_SILU;
    const float zz = z * z, u = z * (silu ? -LOG2E : -LOG2E * TANH_1 - LOG2E * TANH_3 * zz);
    const float e = __builtin_amdgcn_exp2f(fminf(u, 120.0f)), s = __builtin_amdgcn_rcpf(1.0f + e);
    const float d = z * s * (e * s) * (silu ? 1.0f : TANH_1 + 3.0f * TANH_3 * zz);
    return s + d;
  }
  if (act == FP4_ACT_GELU) {
    float e;
    const float tail = normal_tail(z, e);
    return (z < 0 ? tail : 1.0f - tail) + z * e * 0.398942280f;
  }
  return 1.0f;
}

// W values as they lie in memory at element `at` of a tensor of the given type, n of them (those past n: zeros).
template <int W>
struct Raw {
  uint32_t v[W];
};
template <int W>
__device__ __forceinline__ Raw<W> load_raw(int type, const void* p, int64_t at, int n) {
  Raw<W> r;
#pragma unroll
  for (int i = 0; i < W; ++i) r.v[i] = 0;
  if (type == FP4_TYPE_F32) {
    const uint8_t* q = static_cast<const uint8_t*>(p) + at * 4;
    if (n >= W) __builtin_memcpy(r.v, q, 4 * W);
    else
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (i < n) r.v[i] = reinterpret_cast<const uint32_t*>(q)[i];
  } else {
    const uint8_t* q = static_cast<const uint8_t*>(p) + at * 2;
    if (n >= W) __builtin_memcpy(r.v, q, 2 * W);
    else
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (i < n) r.v[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(q)[i] << (16 * (i & 1));
  }
  return r;
}
template <int W>
__device__ __forceinline__ void values_of(int type, const Raw<W>& r, float (&f)[W]) {
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const uint32_t half = r.v[i / 2] >> (16 * (i & 1));
    if (type == FP4_TYPE_F32) f[i] = __builtin_bit_cast(float, r.v[i]);
    else if (type == FP4_TYPE_BF16) f[i] = __builtin_bit_cast(float, half << 16);
    else f[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)half);
  }
}

// P pieces of W values, every one there, `step` elements apart: all are asked for before the first is waited for.
template <int P, int W>
__device__ __forceinline__ void load_pieces(int type, const void* p, int64_t at, int step, float (&f)[P][W]) {
  Raw<W> r[P] = {};
  if (type == FP4_TYPE_F32) {
#pragma unroll
    for (int i = 0; i < P; ++i) __builtin_memcpy(r[i].v, static_cast<const uint8_t*>(p) + (at + i * step) * 4, 4 * W);
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) __builtin_memcpy(r[i].v, static_cast<const uint8_t*>(p) + (at + i * step) * 2, 2 * W);
  }
#pragma unroll
  for (int i = 0; i < P; ++i) values_of(type, r[i], f[i]);
}

// W values, n of them, to element `at` of y.
template <int OUT, int W>
__device__ __forceinline__ void store_values(void* y, int64_t at, const float (&f)[W], int n) {
  if constexpr (OUT == FP4_TYPE_F32) {
    float* const p = static_cast<float*>(y) + at;
    if (n >= W) __builtin_memcpy(p, f, 4 * W);
    else
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (i < n) p[i] = f[i];
  } else {
    uint16_t* const p = static_cast<uint16_t*>(y) + at;
    uint16_t h[W];
#pragma unroll
    for (int i = 0; i < W; ++i) h[i] = (uint16_t)to16(OUT, f[i]);
    if (n >= W) __builtin_memcpy(p, h, 2 * W);
    else
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (i < n) p[i] = h[i];
  }
}
template <int W>
__device__ __forceinline__ void store_values(int type, void* y, int64_t at, const float (&f)[W], int n) {
  if (type == FP4_TYPE_F32) store_values<FP4_TYPE_F32>(y, at, f, n);
  else if (type == FP4_TYPE_BF16) store_values<FP4_TYPE_BF16>(y, at, f, n);
  else store_values<FP4_TYPE_F16>(y, at, f, n);
}

// Four sums of one row, n of them columns that exist, to y: for the kernels whose sums are not in tiles. `bias_at`: the first
// one's place in the bias.
__device__ __forceinline__ void finish4(const fp4_epilogue& e, int out_type, void* y, int64_t ldy, int64_t row, int64_t col, int64_t bias_at,
                                        const f32x4& sum, int n) {
  float f[4] = {sum[0], sum[1], sum[2], sum[3]}, add[4];
  if (e.bias) {
    values_of(e.bias_type, load_raw<4>(e.bias_type, e.bias, bias_at, n), add);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] += add[i];
  }
  if (e.z) store_values<FP4_TYPE_F32>(e.z, row * e.ldz + col, f, n);
  activate(e.activation, f);
  if (e.residual) {
    values_of(e.residual_type, load_raw<4>(e.residual_type, e.residual, row * e.ldr + col, n), add);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] += add[i];
  }
  store_values(out_type, y, row * ldy + col, f, n);
}

// ------------------------------------------------------------------------------------------------ host side

// e of a product with N columns: types, strides, alignments.
static inline int check_epilogue(const fp4_epilogue* e, int64_t N) {
  if (!e) return FP4_ERR_ARG;
  if (e->activation < FP4_ACT_NONE || e->activation > FP4_ACT_GELU_TANH) return FP4_ERR_ARG;
  if (e->bias) {
    if (!valid_type(e->bias_type)) return FP4_ERR_ARG;
    if (!fp4_aligned(e->bias, (uintptr_t)elem_bytes(e->bias_type))) return FP4_ERR_ALIGN;
  }
  if (e->residual) {
    if (!valid_type(e->residual_type)) return FP4_ERR_ARG;
    if (e->ldr < N) return FP4_ERR_SHAPE;
    if (e->ldr > (1LL << 40)) return FP4_ERR_UNSUPPORTED;
    if (!fp4_aligned(e->residual, (uintptr_t)elem_bytes(e->residual_type))) return FP4_ERR_ALIGN;
  }
  if (e->z) {
    if (e->ldz < N) return FP4_ERR_SHAPE;
    if (e->ldz > (1LL << 40)) return FP4_ERR_UNSUPPORTED;
    if (!fp4_aligned(e->z, 4)) return FP4_ERR_ALIGN;
  }
  return FP4_OK;
}

}  // namespace mx
