// MXFP4 products with an epilogue, y = f(A B^T + bias) + residual: the entry points, and the K parts' way out.
#include <algorithm>

#include "mx_product.h"

namespace mx {

// y from the sum of the K parts' planes, in the order of the parts. Planes have rows of `ldp` floats (a multiple of 4).
__global__ void __launch_bounds__(256) combine_epilogue_kernel(const float* __restrict__ planes, void* y, int64_t ldy, int M, int N,
                                                               int64_t ldp, int parts, int out_type, fp4_epilogue epi) {
  const int64_t quads = ldp >> 2, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= quads * M) return;
  const int64_t row = i / quads, col = 4 * (i - row * quads);
  f32x4 sum = *reinterpret_cast<const f32x4*>(planes + row * ldp + col);
  for (int p = 1; p < parts; ++p) sum += *reinterpret_cast<const f32x4*>(planes + ((int64_t)p * M + row) * ldp + col);
  finish4(epi, out_type, y, ldy, row, col, col, sum, (int)(N - col));
}

static void* ahead(const void* p, int64_t n, int type) {
  return p ? const_cast<uint8_t*>(static_cast<const uint8_t*>(p) + n * elem_bytes(type)) : nullptr;
}

// The plan of a product with an epilogue whose K parts' planes have `room` bytes.
static Plan plan_with(int64_t M, int64_t N, int64_t K, const fp4_epilogue& e, int64_t room, bool split = true) {
  const bool erf = e.activation == FP4_ACT_GELU, other = !erf && e.activation > FP4_ACT_RELU;
  return plan_of(M, N, K, fp4_device_cus(), split, epilogue_costs(erf, other, e.residual, e.z).of, room);
}

static int64_t room_of(const void* workspace, size_t bytes) {
  return workspace ? (int64_t)(bytes < (size_t)INT64_MAX ? bytes : (size_t)INT64_MAX) : 0;
}

// `p`: the plan of the product, whose planes `ws` holds. Columns that are a product of their own (p.first_n) have the epilogue's columns with them.
static int run_epilogue(Plan p, int out_type, int64_t M, int64_t N, int64_t K, const fp4_mx& a, const fp4_mx& b, const fp4_epilogue& e,
                        void* y, int64_t ldy, void* ws, hipStream_t st) {
  if (p.tile == 0) return launch_rows(0, out_type, (int)M, (int)N, (int)K, nullptr, 0, &a, b, y, ldy, st, &e);
  if (p.parts > 1) {
    if (int rc = launch_planes(p.tile, p.parts, p.per, p.ldp, (int)M, (int)N, (int)K, a, b, ws, st)) return rc;
    const int64_t quads = (p.ldp >> 2) * M;
    return fp4_launch(combine_epilogue_kernel, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, st, ws, y, ldy, M, N, p.ldp, p.parts,
                      out_type, e);
  }
  if (p.first_n > 0) {
    const int64_t n = p.first_n;
    p.first_n = 0;
    if (int rc = run_epilogue(p, out_type, M, n, K, a, b, e, y, ldy, nullptr, st)) return rc;
    const fp4_mx rest = {static_cast<uint8_t*>(b.q) + n * b.ldq, static_cast<uint8_t*>(b.s) + n * b.lds, b.ldq, b.lds};
    fp4_epilogue behind = e;
    behind.bias = ahead(e.bias, n, e.bias_type);
    behind.residual = ahead(e.residual, n, e.residual_type);
    behind.z = static_cast<float*>(ahead(e.z, n, FP4_TYPE_F32));
    return run_epilogue(plan_with(M, N - n, K, e, 0, false), out_type, M, N - n, K, a, rest, behind, ahead(y, n, out_type), ldy, nullptr,
                        st);
  }
  Args g{};
  g.a = a, g.b = b, g.y = y, g.ldy = ldy, g.M = (int)M, g.N = (int)N, g.K = (int)K, g.epi = e;
  g.tiles_m = (int)((M + p.tile - 1) / p.tile), g.tiles_n = (int)((N + p.tile - 1) / p.tile);
  return launch_out<DENSE>(out_type, p.tile, g, (int64_t)g.tiles_m * g.tiles_n, st);
}

}  // namespace mx

using namespace mx;

// Bytes of the planes with this epilogue, without one (null).
static int64_t planes_with(int64_t M, int64_t N, int64_t K, const fp4_epilogue* e) {
  return plane_bytes(e ? plan_with(M, N, K, *e, INT64_MAX) : plan_of(M, N, K, fp4_device_cus()), M);
}

// The most of them that any epilogue's plan has, or the plan without one.
static int64_t most_planes(int64_t M, int64_t N, int64_t K) {
  static const float there = 0;  // stands for a residual and a kept z: neither is read here
  int64_t most = planes_with(M, N, K, nullptr);
  for (const int act : {FP4_ACT_NONE, FP4_ACT_SILU, FP4_ACT_GELU})
    for (const bool residual : {false, true})
      for (const bool z : {false, true}) {
        fp4_epilogue e{};
        e.activation = act, e.residual = residual ? &there : nullptr, e.z = z ? const_cast<float*>(&there) : nullptr;
        most = std::max(most, planes_with(M, N, K, &e));
      }
  return most;
}

extern "C" int64_t w4a4_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (int rc = check_product(FP4_TYPE_F32, M, N, K)) return rc;
  return M == 0 ? 0 : most_planes(M, N, K);
}

extern "C" int64_t w4a4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (int rc = check_product(FP4_TYPE_F32, M, N, K)) return rc;
  if (M == 0 || fused(M, N, K)) return 0;
  const LinearSpace sp = linear_space(Plan{}, M, K);
  return sp.q + sp.s + most_planes(M, N, K);
}

extern "C" int64_t w4a4_matmul_epilogue_workspace_bytes(int64_t M, int64_t N, int64_t K, const fp4_epilogue* epilogue) {
  if (int rc = check_product(FP4_TYPE_F32, M, N, K)) return rc;
  if (epilogue)
    if (int rc = check_epilogue(epilogue, N)) return rc;
  return M == 0 ? 0 : planes_with(M, N, K, epilogue);
}

extern "C" int64_t w4a4_linear_epilogue_workspace_bytes(int64_t M, int64_t N, int64_t K, const fp4_epilogue* epilogue) {
  if (int rc = check_product(FP4_TYPE_F32, M, N, K)) return rc;
  if (epilogue)
    if (int rc = check_epilogue(epilogue, N)) return rc;
  if (M == 0 || fused(M, N, K)) return 0;
  const LinearSpace sp = linear_space(Plan{}, M, K);
  return sp.q + sp.s + planes_with(M, N, K, epilogue);
}

extern "C" int w4a4_matmul_epilogue(int out_type, int64_t M, int64_t N, int64_t K, const fp4_mx* a, const fp4_mx* b,
                                    const fp4_epilogue* epilogue, void* y, int64_t ldy, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  if (int rc = check_product(out_type, M, N, K)) return rc;
  if (int rc = check_epilogue(epilogue, N)) return rc;
  if (M == 0) return FP4_OK;
  if (int rc = check_operand(a, K)) return rc;
  if (int rc = check_operand(b, K)) return rc;
  if (int rc = check_output(out_type, N, y, ldy)) return rc;
  if (workspace && !fp4_aligned(workspace, 16)) return FP4_ERR_ALIGN;
  return run_epilogue(plan_with(M, N, K, *epilogue, room_of(workspace, workspace_bytes)), out_type, M, N, K, *a, *b, *epilogue, y, ldy,
                      workspace, static_cast<hipStream_t>(stream));
}

extern "C" int w4a4_linear_epilogue(int x_type, int out_type, int64_t M, int64_t N, int64_t K, const void* x, int64_t ldx,
                                    const fp4_mx* b, const fp4_epilogue* epilogue, void* y, int64_t ldy, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  if (!valid_type(x_type)) return FP4_ERR_ARG;
  if (int rc = check_product(out_type, M, N, K)) return rc;
  if (int rc = check_epilogue(epilogue, N)) return rc;
  if (M == 0) return FP4_OK;
  if (int rc = check_dense(x_type, K, x, ldx)) return rc;
  if (int rc = check_operand(b, K)) return rc;
  if (int rc = check_output(out_type, N, y, ldy)) return rc;
  if (workspace && !fp4_aligned(workspace, 16)) return FP4_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (fused(M, N, K)) return launch_rows(x_type, out_type, (int)M, (int)N, (int)K, x, ldx, nullptr, *b, y, ldy, st, epilogue);
  const LinearSpace sp = linear_space(Plan{}, M, K);
  if (!workspace || workspace_bytes < (size_t)(sp.q + sp.s)) return FP4_ERR_ARG;
  const Plan p = plan_with(M, N, K, *epilogue, room_of(workspace, workspace_bytes - (size_t)(sp.q + sp.s)));
  auto* w = static_cast<uint8_t*>(workspace);
  const int64_t nb = blocks_of(K);
  const fp4_mx a = {w, w + sp.q, nb * 16, (nb + 3) / 4 * 4};
  if (int rc = launch_quantize_rows(x_type, M, K, x, ldx, a, st)) return rc;
  return run_epilogue(p, out_type, M, N, K, a, *b, *epilogue, y, ldy, w + sp.q + sp.s, st);
}
