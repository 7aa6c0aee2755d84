// MXFP4 products of rows in groups (a mixture of experts): the entry points. The tiles' kernel finds the groups' sizes on the
// device (mx_groups.h): every workgroup reads the bounds, so that neither the host nor a kernel in front has to.
#include "mx_product.h"

namespace mx {

static int check_grouped(int out_type, int64_t T, int64_t N, int64_t K, const fp4_groups* groups) {
  if (int rc = check_product(out_type, T, N, K)) return rc;
  if (int rc = check_groups(groups)) return rc;
  return groups->count * N > MAX_ROWS ? FP4_ERR_UNSUPPORTED : FP4_OK;
}

// B's groups lie `step_q` bytes of codes and `step_s` of scales apart.
static int run_grouped(int out_type, int64_t T, int64_t N, int64_t K, const fp4_groups& groups, const fp4_mx& a, const fp4_mx& b,
                       int64_t step_q, int64_t step_s, const fp4_epilogue* e, int fill, void* y, int64_t ldy, hipStream_t st) {
  const Groups g = groups_of(groups);
  const int tile = grouped_tile(T, N, K, g.E, fp4_device_cus());
  if (tile == 0)
    return launch_rows_grouped(0, out_type, (int)T, (int)N, (int)K, g, nullptr, 0, &a, b, step_q, step_s, e, y, ldy, fill, st);
  Args p{};
  p.a = a, p.b = b, p.y = y, p.ldy = ldy, p.M = (int)T, p.N = (int)N, p.K = (int)K, p.fill = fill, p.groups = g;
  p.step_q = step_q, p.step_s = step_s;
  if (e) p.epi = *e;
  p.tiles_n = (int)((N + tile_columns(tile) - 1) / tile_columns(tile));
  return launch_out<ROWS>(out_type, tile, p, most_tiles(T, g.E, tile_rows(tile)) * p.tiles_n, st);
}

static bool grouped_fused(int64_t T, int64_t N, int64_t K, int64_t E) {
  const int64_t some = E < T ? E : T;
  return T <= 16 && (N + 15) / 16 * stages_of(K) * some * (T / some + 3) <= 32768;
}

}  // namespace mx

using namespace mx;

extern "C" int w4a4_grouped_matmul(int out_type, int64_t T, int64_t N, int64_t K, const fp4_groups* groups, const fp4_mx* a,
                                   const fp4_mx* b, const fp4_epilogue* epilogue, int fill, void* y, int64_t ldy, void* stream) {
  if (int rc = check_grouped(out_type, T, N, K, groups)) return rc;
  if (epilogue)
    if (int rc = check_epilogue(epilogue, N)) return rc;
  if (T == 0) return FP4_OK;
  if (int rc = check_operand(a, K)) return rc;
  if (int rc = check_operand(b, K)) return rc;
  if (int rc = check_output(out_type, N, y, ldy)) return rc;
  return run_grouped(out_type, T, N, K, *groups, *a, *b, N * b->ldq, N * b->lds, epilogue, fill, y, ldy, static_cast<hipStream_t>(stream));
}

extern "C" int64_t w4a4_grouped_linear_workspace_bytes(int64_t T, int64_t N, int64_t K, int64_t count) {
  if (int rc = check_product(FP4_TYPE_F32, T, N, K)) return rc;
  if (count < 1) return FP4_ERR_SHAPE;
  if (count > MAX_GROUPS) return FP4_ERR_UNSUPPORTED;
  if (T == 0 || grouped_fused(T, N, K, count)) return 0;
  const LinearSpace sp = linear_space(Plan{}, T, K);
  return sp.q + sp.s;
}

extern "C" int w4a4_grouped_linear(int x_type, int out_type, int64_t T, int64_t N, int64_t K, const fp4_groups* groups, const void* x,
                                   int64_t ldx, const fp4_mx* b, const fp4_epilogue* epilogue, int fill, void* y, int64_t ldy,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_type(x_type)) return FP4_ERR_ARG;
  if (int rc = check_grouped(out_type, T, N, K, groups)) return rc;
  if (epilogue)
    if (int rc = check_epilogue(epilogue, N)) return rc;
  if (T == 0) return FP4_OK;
  if (int rc = check_dense(x_type, K, x, ldx)) return rc;
  if (int rc = check_operand(b, K)) return rc;
  if (int rc = check_output(out_type, N, y, ldy)) return rc;
  if (workspace && !fp4_aligned(workspace, 16)) return FP4_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (grouped_fused(T, N, K, groups->count))
    return launch_rows_grouped(x_type, out_type, (int)T, (int)N, (int)K, groups_of(*groups), x, ldx, nullptr, *b, N * b->ldq, N * b->lds,
                               epilogue, y, ldy, fill, st);
  const LinearSpace sp = linear_space(Plan{}, T, K);
  if (!workspace || workspace_bytes < (size_t)(sp.q + sp.s)) return FP4_ERR_ARG;
  auto* w = static_cast<uint8_t*>(workspace);
  const int64_t nb = blocks_of(K);
  const fp4_mx a = {w, w + sp.q, nb * 16, (nb + 3) / 4 * 4};
  if (int rc = launch_quantize_rows(x_type, T, K, x, ldx, a, st)) return rc;
  return run_grouped(out_type, T, N, K, *groups, a, *b, N * b->ldq, N * b->lds, epilogue, fill, y, ldy, st);
}

extern "C" int w4a4_grouped_matmul_t(int out_type, int64_t T, int64_t N, int64_t K, const fp4_groups* groups, const fp4_mx* a,
                                     const fp4_mx* b, int fill, void* y, int64_t ldy, void* stream) {
  if (int rc = check_grouped(out_type, T, K, N, groups)) return rc;
  if (T == 0) return FP4_OK;
  const int64_t depth = most_tiles(groups->count * N, groups->count, UNIT) * UNIT, step = (N + UNIT - 1) / UNIT * UNIT;
  if (depth > MAX_DEPTH) return FP4_ERR_UNSUPPORTED;
  if (int rc = check_operand(a, N)) return rc;
  if (int rc = check_operand(b, depth)) return rc;
  if (int rc = check_output(out_type, K, y, ldy)) return rc;
  return run_grouped(out_type, T, K, N, *groups, *a, *b, step / 2, step / BLOCK, nullptr, fill, y, ldy, static_cast<hipStream_t>(stream));
}

extern "C" int w4a4_grouped_gradient(int out_type, int64_t T, int64_t N, int64_t K, const fp4_groups* groups, const fp4_mx* a,
                                     const fp4_mx* b, void* dw, int64_t ldw, void* stream) {
  if (int rc = check_grouped(out_type, T, N, K, groups)) return rc;
  const int64_t E = groups->count, depth = most_tiles(T, E, UNIT) * UNIT;
  if (depth > MAX_DEPTH) return FP4_ERR_UNSUPPORTED;
  if (int rc = check_output(out_type, K, dw, ldw)) return rc;
  if (T > 0) {
    if (int rc = check_operand(a, depth)) return rc;
    if (int rc = check_operand(b, depth)) return rc;
  }
  const int tile = gradient_tile(T, N, K, E, fp4_device_cus());
  Args p{};
  if (T > 0) p.a = *a, p.b = *b;
  p.y = dw, p.ldy = ldw, p.M = (int)N, p.N = (int)K, p.K = (int)T, p.groups = groups_of(*groups);
  p.tiles_m = (int)((N + tile - 1) / tile), p.tiles_n = (int)((K + tile - 1) / tile);
  return launch_out<DEPTH>(out_type, tile, p, E * p.tiles_m * p.tiles_n, static_cast<hipStream_t>(stream));
}
