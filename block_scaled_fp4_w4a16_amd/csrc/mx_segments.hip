// MXFP4 quantisation of rows in groups, along the rows and along the columns, of a dense matrix or of D = x f'(z), the gradient
// behind an activation, with its sums down the columns (the bias's gradient).
//
// Down the columns a block's 32 rows are of one group: each group begins anew at a multiple of 256 positions of the operand, a
// stage of the products that contract it. A workgroup takes 32 W rows of one unit of 256 and 256 columns, as
// quantize_cols_kernel does, from one reading of x and z; blocks behind the group's last row are written as zeros.
// The sums of 32 rows are a lane's, those of the workgroup meet in LDS, those of a group's workgroups lie in memory, one row
// of FP32 sums per tile of rows, and a second kernel adds them up in FP64 in the order of the rows: no atomics.
#include "mx_epilogue.h"
#include "mx_groups.h"
#include "mx_patch.h"

namespace mx {

struct Segments {
  const void* x;
  const float* z;
  fp4_mx rows, cols;  // q null: not wanted
  float* sums;        // null: not wanted
  int64_t ldx, ldz;
  Groups groups;
  int M, K, tiles_k, each_units;  // each_units: units per group where the groups are alike, else 0
};

// One row's four values of a lane -> x f'(z), the sums first, then rounded to x's type.
template <int T, int ACT, int R>
__device__ __forceinline__ void gradient_row(uint32_t (&v)[R], const u32x4& z, bool there, const bool (&in)[4], float (&sum)[4]) {
  float f[4];
  Raw<4> raw;
#pragma unroll
  for (int i = 0; i < R; ++i) raw.v[i] = v[i];
  values_of(T, raw, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t bits = z[i];  // (a bit cast of a vector's element itself takes the first one)
    const float d = f[i] * slope(ACT, __builtin_bit_cast(float, bits));
    f[i] = there && in[i] ? d : 0.0f;
    sum[i] += f[i];
    asm volatile("" : "+v"(sum[i]));  // added here: where the sums are wanted or not, later, every value would have to be kept
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if constexpr (T == FP4_TYPE_F32) v[i] = __builtin_bit_cast(uint32_t, f[i]);
    else v[i] = pack2<T>(f[2 * i], f[2 * i + 1]);
    asm volatile("" : "+v"(v[i]));  // a pair stays one register: what is taken apart later would be kept apart from here on
  }
}

// ACT: the activation whose derivative is taken, FP4_ACT_NONE where x is quantised as it is. (Told apart at each value, the four
// would take 199 registers and a branch a value.)
template <int T, int W, int ACT>
__global__ void __launch_bounds__(64 * W) quantize_grouped_kernel(Segments p) {
  constexpr int EB = elem_bytes(T), R = Patch<T>::R, PARTS = UNIT / (32 * W);
  __shared__ u32x4 col_codes[256 * W];
  __shared__ uint8_t col_scales[256 * W];
  __shared__ uint8_t row_scales[W * 256];
  __shared__ int table[2 * (MAX_GROUPS + 1)];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tm = blockIdx.x / p.tiles_k, tk = blockIdx.x - tm * p.tiles_k;
  const int unit = tm / PARTS;
  const int M = p.M, K = p.K;
  int begin, end;
  if (p.each_units) {
    const int e = unit / p.each_units;
    begin = e * p.groups.each, end = begin + p.groups.each;
    begin += (unit - e * p.each_units) * UNIT;
  } else {
    int* const start = table;
    int* const units = table + p.groups.E + 1;
    if (wave == 0) read_groups<UNIT>(p.groups, M, start, units, lane);
    __syncthreads();
    if (unit >= uniform(units[p.groups.E])) return;
    const int e = group_of(units, p.groups.E, unit, lane);
    begin = uniform(start[e]) + (unit - uniform(units[e])) * UNIT, end = uniform(start[e + 1]);
  }
  const int col0 = 256 * tk, col = col0 + 4 * lane;
  const int row0 = begin + 32 * (W * (tm % PARTS) + wave);

  Patch<T> patch;
  // row addresses are the wave's, columns the lane's; rows past the group's last one read it again (or, in a wave that has
  // none, the matrix's last) and count as zeros
  const int from = min(row0, end - 1), last = end - 1 - from;
  const uint8_t* base = static_cast<const uint8_t*>(p.x) + (int64_t)from * p.ldx * EB;
  const uint32_t off = (uint32_t)col * EB;
  const int64_t step = p.ldx * EB;
  if (col + 4 <= K) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      __builtin_memcpy(patch.v[i], base + off, 4 * EB);
      if (i < last) base += step;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const uint8_t* r = base + off;
#pragma unroll
      for (int j = 0; j < R; ++j) patch.v[i][j] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (col + j < K) {
          if constexpr (T == FP4_TYPE_F32) patch.v[i][j] = reinterpret_cast<const uint32_t*>(r)[j];
          else patch.v[i][j >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(r)[j] << (16 * (j & 1));
        }
      if (i < last) base += step;
    }
  }
  float sum[4] = {0, 0, 0, 0};
  if constexpr (ACT != FP4_ACT_NONE) {
    // four rows of z at a time, the next four on their way meanwhile: all 32 do not fit the registers. Rows behind the last
    // one are not read; a lane at the matrix's edge reads into the next row, which `in` drops. z is marked as not to be kept
    // in the caches, where the operands made here will be read from (8192 x 9728: a step of 613 us takes 591).
    const auto zr = fp4::make_rsrc(p.z + (int64_t)from * p.ldz, (uint32_t)(min(last, 31) * (int)p.ldz + K) * 4);
    const bool in[4] = {col < K, col + 1 < K, col + 2 < K, col + 3 < K};
    u32x4 z[2][4];
    const auto ask = [&](int b) {
#pragma unroll
      for (int i = 0; i < 4; ++i) z[b & 1][i] = __builtin_amdgcn_raw_buffer_load_b128(zr, ((4 * b + i) * (int)p.ldz + col) * 4, 0, 2);
    };
    ask(0);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      if (b < 7) ask(b + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 4; ++i) gradient_row<T, ACT>(patch.v[4 * b + i], z[b & 1][i], row0 + 4 * b + i < end, in, sum);
      __builtin_amdgcn_sched_barrier(0);
    }
  } else {
    if (row0 + 32 > end) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
#pragma unroll
        for (int j = 0; j < R; ++j) patch.v[i][j] = row0 + i < end ? patch.v[i][j] : 0u;
    }
    if (p.sums) {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        float f[4];
        Raw<4> raw;
#pragma unroll
        for (int j = 0; j < R; ++j) raw.v[j] = patch.v[i][j];
        values_of(T, raw, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] += f[j];
      }
    }
  }
  if (p.sums) {
    // the columns' codes come later: their place takes the waves' sums first
    auto* const all = reinterpret_cast<f32x4*>(col_codes);
    all[wave * 64 + lane] = f32x4{sum[0], sum[1], sum[2], sum[3]};
    __syncthreads();
    const int c = threadIdx.x;
    if (c < 64 && col0 + 4 * c < K) {
      f32x4 s = all[c];
#pragma unroll
      for (int v = 1; v < W; ++v) s += all[v * 64 + c];
      const float f[4] = {s[0], s[1], s[2], s[3]};
      store_values<FP4_TYPE_F32>(p.sums, (int64_t)tm * K + col0 + 4 * c, f, K - col0 - 4 * c);
    }
    __syncthreads();
  }
  if (!p.rows.q && !p.cols.q) return;

  // from here on as quantize_cols_kernel, the groups' own bounds in place of the matrix's
  uint32_t m[4], sb[4];
  patch.column_max(m);
  const bool finite = __builtin_amdgcn_ballot_w64((max(max(m[0], m[1]), max(m[2], m[3])) >> 23) == 255u) == 0;
  if (p.cols.q) {
    const int slot = 4 * W * lane + (wave ^ (lane & (W - 1)));
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      sb[c] = scale_byte(m[c]);
      col_scales[(4 * lane + c) * W + wave] = (uint8_t)sb[c];
    }
    col_codes[slot] = patch.template column<0>(scale_value(sb[0]), code_mask(sb[0]));
    col_codes[slot + W] = patch.template column<1>(scale_value(sb[1]), code_mask(sb[1]));
    col_codes[slot + 2 * W] = patch.template column<2>(scale_value(sb[2]), code_mask(sb[2]));
    col_codes[slot + 3 * W] = patch.template column<3>(scale_value(sb[3]), code_mask(sb[3]));
  }
  if (p.rows.q) {
    // the column pass's magnitudes are not kept for the rows: that would double the registers
#pragma unroll
    for (int i = 0; i < 32; ++i)
#pragma unroll
      for (int j = 0; j < R; ++j) asm volatile("" : "+v"(patch.v[i][j]));
    uint8_t* const s = row_scales + wave * 256;
    if (finite) quantize_patch_rows<T, true>(patch, p.rows, s, row0, col0, lane, end, (int)blocks_of(K));
    else quantize_patch_rows<T, false>(patch, p.rows, s, row0, col0, lane, end, (int)blocks_of(K));
  }
  __syncthreads();
  if (p.rows.q) {
    // lane: row lane / 2, four blocks
    const int row = row0 + (lane >> 1), blk = (col0 >> 5) + 4 * (lane & 1);
    if (row < end && blk < (int)blocks_of(K))
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.rows.s) + (int64_t)row * p.rows.lds + blk) =
          *reinterpret_cast<const uint32_t*>(row_scales + wave * 256 + lane * 4);
  }
  if (!p.cols.q) return;
  auto* q = static_cast<uint8_t*>(p.cols.q) + (int64_t)tm * (16 * W);
  auto* s = static_cast<uint8_t*>(p.cols.s) + (int64_t)tm * W;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = i * 64 * W + threadIdx.x, c = e / W, b = e % W;
    if (col0 + c < K) *reinterpret_cast<u32x4*>(q + (int64_t)(col0 + c) * p.cols.ldq + 16 * b) = col_codes[c * W + (b ^ ((c >> 2) & (W - 1)))];
  }
  for (int e = threadIdx.x; e < 64 * W; e += 64 * W) {
    const int c = e / (W / 4), b = 4 * (e % (W / 4));
    if (col0 + c < K)
      *reinterpret_cast<uint32_t*>(s + (int64_t)(col0 + c) * p.cols.lds + b) = *reinterpret_cast<const uint32_t*>(col_scales + c * W + b);
  }
}

// dbias[e][k] = the sum of group e's tiles.
__global__ void __launch_bounds__(256) add_sums_kernel(const float* __restrict__ sums, Groups groups, int M, int K, int parts,
                                                       int each_units, void* __restrict__ out, int type) {
  __shared__ int table[2 * (MAX_GROUPS + 1)];
  const int e = blockIdx.y, k = blockIdx.x * 256 + threadIdx.x;
  int first, last;
  if (each_units) {
    first = e * each_units, last = first + each_units;
  } else {
    int* const units = table + groups.E + 1;
    if (threadIdx.x < 64) read_groups<UNIT>(groups, M, table, units, threadIdx.x);
    __syncthreads();
    first = units[e], last = units[e + 1];
  }
  if (k >= K) return;
  double sum = 0;
  const float* p = sums + (int64_t)first * parts * K + k;
#pragma unroll 8
  for (int t = first * parts; t < last * parts; ++t, p += K) sum += *p;
  const float f[1] = {(float)sum};
  store_values(type, out, (int64_t)e * K + k, f, 1);
}

static int64_t sums_bytes(int64_t T, int64_t K, int64_t E) { return most_tiles(T, E, UNIT) * (UNIT / 128) * K * 4; }

}  // namespace mx

using namespace mx;

static int check_counts(int64_t T, int64_t count) {
  if (T < 0 || count < 1) return FP4_ERR_SHAPE;
  if (T > MAX_ROWS || count > MAX_GROUPS) return FP4_ERR_UNSUPPORTED;
  return FP4_OK;
}

extern "C" int64_t fp4_grouped_depth(int64_t T, int64_t count) {
  if (int rc = check_counts(T, count)) return rc;
  return most_tiles(T, count, UNIT) * UNIT;
}

extern "C" int64_t fp4_grouped_sums_bytes(int64_t T, int64_t K, int64_t count) {
  if (int rc = check_counts(T, count)) return rc;
  if (int rc = check_dims(T, K)) return rc;
  return sums_bytes(T, K, count);
}

extern "C" int fp4_quantize_mxfp4_grouped(int type, int64_t T, int64_t K, const void* x, int64_t ldx, const fp4_groups* groups,
                                          const fp4_mx* rows, const fp4_mx* cols, const fp4_gradient* gradient, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  if (!valid_type(type) || !groups) return FP4_ERR_ARG;
  if (int rc = check_dims(T, K)) return rc;
  if (int rc = check_counts(T, groups->count)) return rc;
  const bool alike = !groups->offsets;
  if (alike) {
    if (T % groups->count) return FP4_ERR_SHAPE;
  } else if (int rc = check_groups(groups)) {
    return rc;
  }
  const bool sums = gradient && gradient->dbias, z = gradient && gradient->z;
  if (!rows && !cols && !sums) return FP4_ERR_ARG;
  if (gradient) {
    if (gradient->activation < FP4_ACT_NONE || gradient->activation > FP4_ACT_GELU_TANH) return FP4_ERR_ARG;
    if (sums) {
      if (!valid_type(gradient->dbias_type)) return FP4_ERR_ARG;
      if (!fp4_aligned(gradient->dbias, (uintptr_t)elem_bytes(gradient->dbias_type))) return FP4_ERR_ALIGN;
    }
    if (z) {
      if (gradient->ldz < K) return FP4_ERR_SHAPE;
      if (gradient->ldz > (1LL << 23)) return FP4_ERR_UNSUPPORTED;  // 32 rows of it are addressed with 32 bits
      if (!fp4_aligned(gradient->z, 4)) return FP4_ERR_ALIGN;
    }
  }
  const int64_t E = groups->count, depth = most_tiles(T, E, UNIT) * UNIT;
  const int64_t need = sums ? sums_bytes(T, K, E) : 0;
  if (T > 0) {
    if (int rc = check_dense(type, K, x, ldx)) return rc;
    if (rows)
      if (int rc = check_operand(rows, K)) return rc;
    if (cols) {
      if (depth > MAX_DEPTH) return FP4_ERR_UNSUPPORTED;
      if (int rc = check_operand(cols, depth)) return rc;
    }
    if (sums && (!workspace || workspace_bytes < (size_t)need)) return FP4_ERR_ARG;
    if (workspace && !fp4_aligned(workspace, 16)) return FP4_ERR_ALIGN;
  }
  hipStream_t st = static_cast<hipStream_t>(stream);
  Groups g = groups_of(*groups);
  int each_units = 0, parts = 1;
  if (alike) g.each = (int)(T / E), each_units = (g.each + UNIT - 1) / UNIT;
  if (T > 0) {
    const int64_t tk = (K + 255) / 256, units = alike ? E * each_units : most_tiles(T, E, UNIT);
    // half units where whole ones would leave compute units idle
    const int w = tk * units >= 2 * fp4_device_cus() ? 8 : 4;
    parts = UNIT / (32 * w);
    if (!fits_launch(tk * units * parts, 64 * w)) return FP4_ERR_UNSUPPORTED;
    Segments p{};
    p.x = x, p.ldx = ldx, p.groups = g, p.M = (int)T, p.K = (int)K, p.tiles_k = (int)tk, p.each_units = each_units;
    if (rows) p.rows = *rows;
    if (cols) p.cols = *cols;
    if (sums) p.sums = static_cast<float*>(workspace);
    if (z) p.z = gradient->z, p.ldz = gradient->ldz;
    const dim3 grid((unsigned)(tk * units * parts)), block(64 * w);
    const int act = z ? gradient->activation : FP4_ACT_NONE;
    int rc;
#define MX_SEG(T_, W_, ACT_) rc = fp4_launch(quantize_grouped_kernel<T_, W_, ACT_>, grid, block, 0, st, p)
#define MX_SEG_ACT(T_, W_)                                              \
  if (act == FP4_ACT_NONE) MX_SEG(T_, W_, FP4_ACT_NONE);                \
  else if (act == FP4_ACT_RELU) MX_SEG(T_, W_, FP4_ACT_RELU);           \
  else if (act == FP4_ACT_SILU) MX_SEG(T_, W_, FP4_ACT_SILU);           \
  else if (act == FP4_ACT_GELU) MX_SEG(T_, W_, FP4_ACT_GELU);           \
  else MX_SEG(T_, W_, FP4_ACT_GELU_TANH)
#define MX_SEG_W(T_)                  \
  if (w == 8) { MX_SEG_ACT(T_, 8); }  \
  else { MX_SEG_ACT(T_, 4); }
    if (type == FP4_TYPE_F32) { MX_SEG_W(FP4_TYPE_F32) }
    else if (type == FP4_TYPE_BF16) { MX_SEG_W(FP4_TYPE_BF16) }
    else { MX_SEG_W(FP4_TYPE_F16) }
#undef MX_SEG_W
#undef MX_SEG_ACT
#undef MX_SEG
    if (rc) return rc;
  }
  if (!sums) return FP4_OK;
  return fp4_launch(add_sums_kernel, dim3((unsigned)((K + 255) / 256), (unsigned)E), dim3(256), 0, st, static_cast<const float*>(workspace), g,
                    T, K, parts, each_units, gradient->dbias, gradient->dbias_type);
}
