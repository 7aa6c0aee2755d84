// Native half of the Python binding of the MXFP4 operators: argument checks, allocation through torch and the calls of
// the C entry points, and the trainable layer's autograd node. A decode-sized product runs for a few microseconds;
// the same checks written in Python took 23 to 30 microseconds a call.
#include <ATen/ATen.h>
#include <ATen/MemoryOverlap.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/jit/frontend/tracer.h>
#include <torch/csrc/utils/pybind.h>

#include "fp4w4a16.h"

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace {

template <typename... A>
[[noreturn]] void type_error(const A&... a) {
  throw py::type_error(c10::str(a...));
}
template <typename... A>
[[noreturn]] void value_error(const A&... a) {
  throw py::value_error(c10::str(a...));
}

// A trace records what goes through torch's dispatcher, of these calls only the allocations: replayed, it would return
// memory that nothing has written.
void refuse_tracing() {
  if (torch::jit::tracer::isTracing() ||
      c10::impl::TorchDispatchModeTLS::get_mode(c10::impl::TorchDispatchModeKey::PROXY).has_value())
    throw std::runtime_error("MXFP4 calls cannot be traced (torch.jit.trace, make_fx): their kernels would be missing from the graph");
}

int64_t blocks_of(int64_t k) { return (k + 31) / 32; }

int dense_type(const Tensor& t, const char* what, bool half = true) {
  switch (t.scalar_type()) {
    case at::kFloat: return FP4_TYPE_F32;
    case at::kBFloat16: return FP4_TYPE_BF16;
    case at::kHalf:
      if (half) return FP4_TYPE_F16;
      [[fallthrough]];
    default: type_error(what, " must be float32", half ? ", bfloat16 or float16" : " or bfloat16", ", not ", t.scalar_type());
  }
}

// Row stride (in elements) of a rows x cols matrix whose rows are contiguous and do not overlap.
int64_t rows_of(const Tensor& t, int64_t rows, int64_t cols, const char* what) {
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    value_error(what, " must have shape [", rows, ", ", cols, "], not ", t.sizes());
  if (t.is_neg()) value_error(what, " is a lazily negated view, whose memory has the other sign: resolve_neg() it first");
  if (cols > 1 && t.stride(1) != 1) value_error(what, ": the elements of a row must be contiguous");
  if (rows > 1 && t.stride(0) < cols) value_error(what, ": rows overlap");
  return rows > 1 ? t.stride(0) : std::max<int64_t>(cols, 1);
}

// These calls run outside autograd. Rounding to codes has no gradient, as any conversion to whole numbers, but a dense
// factor of a product has one, which must not get lost unseen, and neither must that of a tensor written over.
void no_gradient(const Tensor& t, const char* what) {
  if (at::GradMode::is_enabled() && t.requires_grad())
    throw std::runtime_error(c10::str(what, " requires a gradient, which this call does not compute: detach it, call under "
                                      "torch.no_grad(), or use mx_linear"));
}

// A kernel is about to write t's memory, which autograd does not see: a graph that saved t has to notice.
void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

fp4_mx operand(const Tensor& q, const Tensor& s, int64_t rows, int64_t k, const char* what) {
  if (q.scalar_type() != at::kByte || s.scalar_type() != at::kByte) type_error(what, ": codes and scales must be uint8");
  const int64_t nb = blocks_of(k), padded = (nb + 3) / 4 * 4;
  const int64_t ldq = rows_of(q, rows, 16 * nb, what);
  int64_t lds = rows_of(s, rows, nb, what);
  if (rows == 1) lds = padded;
  // rows of scales are read and, by the quantisation, written in whole dwords
  if (rows > 0 && s.storage_offset() + (rows - 1) * lds + padded > (int64_t)s.storage().nbytes())
    value_error(what, ": the last row of scales must own its memory up to a multiple of 4 bytes");
  return {q.data_ptr(), s.data_ptr(), ldq, lds};
}

c10::Device one_device(std::initializer_list<const Tensor*> ts) {
  const c10::Device d = (*ts.begin())->device();
  for (const Tensor* t : ts)
    if (t->device() != d) value_error("tensors must all live on one GPU (got ", d, " and ", t->device(), ")");
  if (!d.is_cuda()) value_error("tensors must live on the GPU");
  return d;
}

void check(int64_t rc, const char* what) {
  if (rc < 0) throw std::runtime_error(c10::str(what, ": ", fp4_status_string((int)rc), " (status ", rc, ")"));
}

void* current(c10::Device d) { return c10::hip::getCurrentHIPStream(d.index()).stream(); }

// Makes the caller's stream (a torch stream or a raw handle; None: leaves it alone) the device's current one for the length
// of a call, so that the copies, outputs and workspaces the call makes are in the stream's order too.
struct OnStream {
  std::optional<c10::hip::HIPStream> before;
  OnStream(const py::handle& stream, c10::Device d) {
    if (stream.is_none()) return;
    py::object h = py::reinterpret_borrow<py::object>(stream);
    if (py::hasattr(stream, "cuda_stream")) {
      // a kernel runs on its stream's GPU, which may not reach the tensors' memory
      const py::object on = py::getattr(py::getattr(stream, "device", py::none()), "index", py::none());
      if (!on.is_none() && on.cast<int64_t>() != d.index())
        value_error("the stream belongs to GPU ", on.cast<int64_t>(), ", the tensors live on ", d);
      h = stream.attr("cuda_stream");
    }
    const auto raw = reinterpret_cast<hipStream_t>(h.cast<uintptr_t>());
    before = c10::hip::getCurrentHIPStream(d.index());
    c10::hip::setCurrentHIPStream(c10::hip::getStreamFromExternal(raw, d.index()));
  }
  OnStream(const OnStream&) = delete;
  ~OnStream() {
    if (before) c10::hip::setCurrentHIPStream(*before);
  }
};

struct Workspace {
  Tensor hold;
  void* p = nullptr;
  size_t bytes = 0;
};
// The given workspace, or one of `need` bytes from torch's allocator.
Workspace workspace_of(const OptTensor& given, int64_t need, c10::Device d) {
  Workspace w;
  if (given) {
    if (given->device() != d) value_error("the workspace must live on the tensors' GPU");
    if (!given->is_contiguous()) value_error("tensors must be contiguous");
    w.hold = *given;
    written(w.hold);
  } else if (need > 0) {
    w.hold = at::empty({need}, at::TensorOptions().dtype(at::kByte).device(d));
  } else {
    return w;
  }
  w.p = w.hold.data_ptr();
  w.bytes = w.hold.nbytes();
  return w;
}

// What follows a product (none of it: an empty Epilogue), and what keeps its memory.
struct Epilogue {
  OptTensor bias, residual;
  int activation = FP4_ACT_NONE;
  bool any() const { return bias || residual || activation != FP4_ACT_NONE; }
};

Epilogue epilogue_of(const OptTensor& bias, const std::optional<std::string>& activation, const OptTensor& residual) {
  Epilogue e{bias, residual};
  if (!activation) return e;
  static const char* const names[] = {"relu", "silu", "gelu", "gelu_tanh"};
  for (int i = 0; i < 4; ++i)
    if (*activation == names[i]) e.activation = FP4_ACT_RELU + i;
  if (e.activation == FP4_ACT_NONE) value_error("activation must be None, 'relu', 'silu', 'gelu' or 'gelu_tanh', not '", *activation, "'");
  return e;
}

// A bias of `groups` x N values (groups 0: one vector of N), contiguous.
Tensor bias_of(const Tensor& b, int64_t groups, int64_t N) {
  dense_type(b, "bias");
  const bool ok = groups == 0 ? b.dim() == 1 && b.size(0) == N : b.dim() == 2 && b.size(0) == groups && b.size(1) == N;
  if (!ok && groups == 0) value_error("bias must have shape [", N, "], not ", b.sizes());
  if (!ok) value_error("bias must have shape [", groups, ", ", N, "], not ", b.sizes());
  return b.resolve_neg().contiguous();
}

// Whether two M x N matrices with contiguous rows share memory: by their places where they have the same row stride and element
// size, else as far as torch can tell (it cannot of rows with gaps).
bool share_memory(const Tensor& a, const Tensor& b, int64_t M, int64_t N, int64_t lda, int64_t ldb) {
  if (M < 1 || N < 1) return false;
  const int64_t eb = a.element_size();
  if (lda != ldb || eb != (int64_t)b.element_size()) {
    const auto s = at::get_overlap_status(a, b);
    return s == at::MemOverlapStatus::Full || s == at::MemOverlapStatus::Partial;
  }
  // b lies `rows` rows and `at` bytes behind a, 0 <= at < a row's stride
  const int64_t row = lda * eb, far = (int64_t)b.data_ptr() - (int64_t)a.data_ptr();
  const int64_t rows = far >= 0 ? far / row : -((-far + row - 1) / row), at = far - rows * row;
  return (at < N * eb && std::abs(rows) < M) || (at + N * eb > row && std::abs(rows + 1) < M);
}

// `e` as the library takes it, for y [M, N]; `bias` receives what the bias's pointer points to.
fp4_epilogue native(const Epilogue& e, const Tensor& y, int64_t M, int64_t N, int64_t groups, c10::Device d, Tensor& bias) {
  fp4_epilogue n{};
  n.activation = e.activation;
  if (e.bias) {
    if (e.bias->device() != d) value_error("tensors must all live on one GPU (got ", d, " and ", e.bias->device(), ")");
    bias = bias_of(*e.bias, groups, N);
    n.bias = bias.data_ptr(), n.bias_type = dense_type(bias, "bias");
  }
  if (e.residual) {
    const Tensor& r = *e.residual;
    if (r.device() != d) value_error("tensors must all live on one GPU (got ", d, " and ", r.device(), ")");
    n.residual_type = dense_type(r, "residual");
    n.ldr = rows_of(r, M, N, "residual");
    n.residual = r.data_ptr();
    const int64_t ldy = rows_of(y, M, N, "y");
    const bool same = r.data_ptr() == y.data_ptr();
    if (M > 0 && same && (r.scalar_type() != y.scalar_type() || n.ldr != ldy))
      value_error("a residual that is the output has to be so in type and strides too");
    if (!same && share_memory(r, y, M, N, n.ldr, ldy)) value_error("the residual and the output share a part of their memory: one would change the other");
  }
  return n;
}

void no_gradient(const Epilogue& e) {
  if (e.bias) no_gradient(*e.bias, "bias");
  if (e.residual) no_gradient(*e.residual, "residual");
}

// ------------------------------------------------------------------------------------------------ operators

void quantize_into(int64_t M, int64_t K, const Tensor& x, const Tensor* q, const Tensor* s, const Tensor* qt, const Tensor* st_,
                   c10::Device d) {
  const int type = dense_type(x, "x");
  const int64_t ldx = rows_of(x, M, K, "x");
  fp4_mx rows{}, cols{};
  if (q) rows = operand(*q, *s, M, K, "rows");
  if (qt) cols = operand(*qt, *st_, K, M, "columns");
  c10::DeviceGuard guard(d);
  check(fp4_quantize_mxfp4(type, M, K, x.data_ptr(), ldx, q ? &rows : nullptr, qt ? &cols : nullptr, current(d)),
        "fp4_quantize_mxfp4");
}

void quantize(int64_t M, int64_t K, const Tensor& x, const OptTensor& q, const OptTensor& s, const OptTensor& qt,
              const OptTensor& st_, const py::object& stream) {
  refuse_tracing();
  dense_type(x, "x");
  if (q.has_value() != s.has_value() || qt.has_value() != st_.has_value()) value_error("codes and scales come in pairs");
  rows_of(x, M, K, "x");
  const c10::Device d = one_device({&x, q ? &*q : &x, s ? &*s : &x, qt ? &*qt : &x, st_ ? &*st_ : &x});
  const OnStream on(stream, d);
  for (const OptTensor* t : {&q, &s, &qt, &st_})
    if (*t) written(**t);
  quantize_into(M, K, x, q ? &*q : nullptr, s ? &*s : nullptr, qt ? &*qt : nullptr, st_ ? &*st_ : nullptr, d);
}

struct Operand {
  Tensor codes, scales;
};

Operand new_operand(int64_t rows, int64_t k, c10::Device d) {
  if (rows < 0 || k < 1) value_error("an MXFP4 operand needs rows >= 0 and K >= 1, not ", rows, " and ", k);
  const auto opt = at::TensorOptions().dtype(at::kByte).device(d);
  const int64_t nb = blocks_of(k), padded = (nb + 3) / 4 * 4;
  Operand o{at::empty({rows, 16 * nb}, opt), at::empty({rows, padded}, opt)};
  if (padded != nb) o.scales = o.scales.narrow(1, 0, nb);
  return o;
}

// x [..., K] as a matrix whose rows are contiguous (a copy only where the strides or a lazy negation ask for one).
Tensor as_rows(const Tensor& given) {
  if (given.dim() < 1) value_error("a tensor with at least one axis expected");
  const Tensor x = given.is_neg() ? given.resolve_neg() : given;
  Tensor m = x.dim() == 2 ? x : x.size(-1) > 0 ? x.reshape({x.numel() / x.size(-1), x.size(-1)}) : x.reshape({-1, 0});
  const bool ok = (m.size(1) <= 1 || m.stride(1) == 1) && (m.size(0) <= 1 || m.stride(0) >= m.size(1));
  return ok ? m : m.contiguous();
}

using Quantized = std::pair<Operand, Operand>;

Quantized quantize_new(const Tensor& m, bool rows, bool cols, c10::Device d) {
  Quantized r;
  if (rows) r.first = new_operand(m.size(0), m.size(1), d);
  if (cols) r.second = new_operand(m.size(1), m.size(0), d);
  quantize_into(m.size(0), m.size(1), m, rows ? &r.first.codes : nullptr, rows ? &r.first.scales : nullptr,
                cols ? &r.second.codes : nullptr, cols ? &r.second.scales : nullptr, d);
  return r;
}

// (rows, K, codes, scales, codes along the columns, their scales)
py::tuple quantize_py(const Tensor& x, bool rows, bool cols, const py::object& stream) {
  refuse_tracing();
  dense_type(x, "x");
  const c10::Device d = one_device({&x});
  const OnStream on(stream, d);
  const Tensor m = as_rows(x);
  const Quantized r = quantize_new(m, rows, cols, d);
  return py::make_tuple(m.size(0), m.size(1), r.first.codes, r.first.scales, r.second.codes, r.second.scales);
}

void dequant(int64_t M, int64_t K, const Tensor& q, const Tensor& s, const Tensor& out, const py::object& stream) {
  refuse_tracing();
  const int type = dense_type(out, "out", false);
  no_gradient(out, "the output");
  const int64_t ldo = rows_of(out, M, K, "out");
  const c10::Device d = one_device({&q, &s, &out});
  const fp4_mx a = operand(q, s, M, K, "operand");
  const OnStream on(stream, d);
  c10::DeviceGuard guard(d);
  written(out);
  check(fp4_dequant_mxfp4(type, M, K, &a, out.data_ptr(), ldo, current(d)), "fp4_dequant_mxfp4");
}

void product_into(int64_t M, int64_t N, int64_t K, const fp4_mx& a, const fp4_mx& b, const Tensor& y, const OptTensor& ws,
                  c10::Device d, const fp4_epilogue* after = nullptr) {
  const int type = dense_type(y, "y");
  const int64_t ldy = rows_of(y, M, N, "y");
  c10::DeviceGuard guard(d);
  const int64_t need = ws ? 0 : w4a4_matmul_epilogue_workspace_bytes(M, N, K, after);
  check(need, "w4a4_matmul");
  const Workspace w = workspace_of(ws, need, d);
  if (after)
    check(w4a4_matmul_epilogue(type, M, N, K, &a, &b, after, y.data_ptr(), ldy, w.p, w.bytes, current(d)), "w4a4_matmul_epilogue");
  else
    check(w4a4_matmul(type, M, N, K, &a, &b, y.data_ptr(), ldy, w.p, w.bytes, current(d)), "w4a4_matmul");
}

void matmul(int64_t M, int64_t N, int64_t K, const Tensor& aq, const Tensor& as, const Tensor& bq, const Tensor& bs,
            const Tensor& y, const py::object& stream, const OptTensor& ws, const OptTensor& bias,
            const std::optional<std::string>& activation, const OptTensor& residual) {
  refuse_tracing();
  no_gradient(y, "the output");
  const Epilogue e = epilogue_of(bias, activation, residual);
  no_gradient(e);
  const c10::Device d = one_device({&aq, &as, &bq, &bs, &y});
  const OnStream on(stream, d);
  Tensor held;
  const fp4_epilogue after = native(e, y, M, N, 0, d, held);
  const fp4_mx a = operand(aq, as, M, K, "A"), b = operand(bq, bs, N, K, "B");
  written(y);
  product_into(M, N, K, a, b, y, ws, d, e.any() ? &after : nullptr);
}

void linear_into(int64_t M, int64_t N, int64_t K, const Tensor& x, const Operand& B, const Tensor& y,
                 const OptTensor& ws, c10::Device d, const fp4_epilogue* after) {
  const int tx = dense_type(x, "x"), ty = dense_type(y, "y");
  const int64_t ldx = rows_of(x, M, K, "x"), ldy = rows_of(y, M, N, "y");
  const fp4_mx b = operand(B.codes, B.scales, N, K, "B");
  c10::DeviceGuard guard(d);
  const int64_t need = ws ? 0 : w4a4_linear_epilogue_workspace_bytes(M, N, K, after);
  check(need, "w4a4_linear");
  const Workspace w = workspace_of(ws, need, d);
  if (after)
    check(w4a4_linear_epilogue(tx, ty, M, N, K, x.data_ptr(), ldx, &b, after, y.data_ptr(), ldy, w.p, w.bytes, current(d)),
          "w4a4_linear_epilogue");
  else
    check(w4a4_linear(tx, ty, M, N, K, x.data_ptr(), ldx, &b, y.data_ptr(), ldy, w.p, w.bytes, current(d)), "w4a4_linear");
}

void linear(int64_t M, int64_t N, int64_t K, const Tensor& x, const Tensor& bq, const Tensor& bs, const Tensor& y,
            const py::object& stream, const OptTensor& ws, const OptTensor& bias, const std::optional<std::string>& activation,
            const OptTensor& residual) {
  refuse_tracing();
  no_gradient(x, "x");
  no_gradient(y, "the output");
  const Epilogue e = epilogue_of(bias, activation, residual);
  no_gradient(e);
  const c10::Device d = one_device({&x, &bq, &bs, &y});
  const OnStream on(stream, d);
  Tensor held;
  const fp4_epilogue after = native(e, y, M, N, 0, d, held);
  written(y);
  linear_into(M, N, K, x, {bq, bs}, y, ws, d, e.any() ? &after : nullptr);
}

// ---- rows in groups

struct Groups {
  Tensor offsets;  // contiguous
  fp4_groups g;
};

Groups groups_of(const Tensor& offsets, c10::Device d) {
  if (offsets.scalar_type() != at::kInt && offsets.scalar_type() != at::kLong)
    type_error("offsets must be int32 or int64, not ", offsets.scalar_type());
  if (offsets.dim() != 1 || offsets.size(0) < 2) value_error("offsets must be a vector of at least two bounds, not ", offsets.sizes());
  if (offsets.device() != d) value_error("tensors must all live on one GPU (got ", d, " and ", offsets.device(), ")");
  Groups r;
  r.offsets = offsets.resolve_neg().contiguous();
  r.g = {r.offsets.data_ptr(), offsets.size(0) - 1, offsets.scalar_type() == at::kInt ? 32 : 64};
  return r;
}

void grouped_matmul(int64_t T, int64_t N, int64_t K, const Tensor& aq, const Tensor& as, const Tensor& bq, const Tensor& bs,
                    const Tensor& offsets, const Tensor& y, const OptTensor& bias, const std::optional<std::string>& activation,
                    const OptTensor& residual, bool fill, const py::object& stream) {
  refuse_tracing();
  no_gradient(y, "the output");
  const Epilogue e = epilogue_of(bias, activation, residual);
  no_gradient(e);
  const int type = dense_type(y, "y");
  const c10::Device d = one_device({&aq, &as, &bq, &bs, &y});
  const OnStream on(stream, d);
  const Groups g = groups_of(offsets, d);
  Tensor held;
  const fp4_epilogue after = native(e, y, T, N, g.g.count, d, held);
  const fp4_mx a = operand(aq, as, T, K, "A"), b = operand(bq, bs, g.g.count * N, K, "B");
  const int64_t ldy = rows_of(y, T, N, "y");
  c10::DeviceGuard guard(d);
  written(y);
  check(w4a4_grouped_matmul(type, T, N, K, &g.g, &a, &b, &after, fill, y.data_ptr(), ldy, current(d)), "w4a4_grouped_matmul");
}

void grouped_linear(int64_t T, int64_t N, int64_t K, const Tensor& x, const Tensor& bq, const Tensor& bs, const Tensor& offsets,
                    const Tensor& y, const OptTensor& bias, const std::optional<std::string>& activation, const OptTensor& residual,
                    bool fill, const py::object& stream, const OptTensor& ws) {
  refuse_tracing();
  no_gradient(x, "x");
  no_gradient(y, "the output");
  const Epilogue e = epilogue_of(bias, activation, residual);
  no_gradient(e);
  const int tx = dense_type(x, "x"), ty = dense_type(y, "y");
  const c10::Device d = one_device({&x, &bq, &bs, &y});
  const OnStream on(stream, d);
  const Groups g = groups_of(offsets, d);
  Tensor held;
  const fp4_epilogue after = native(e, y, T, N, g.g.count, d, held);
  const fp4_mx b = operand(bq, bs, g.g.count * N, K, "B");
  const int64_t ldx = rows_of(x, T, K, "x"), ldy = rows_of(y, T, N, "y");
  c10::DeviceGuard guard(d);
  const int64_t need = ws ? 0 : w4a4_grouped_linear_workspace_bytes(T, N, K, g.g.count);
  check(need, "w4a4_grouped_linear");
  const Workspace w = workspace_of(ws, need, d);
  written(y);
  check(w4a4_grouped_linear(tx, ty, T, N, K, &g.g, x.data_ptr(), ldx, &b, &after, fill, y.data_ptr(), ldy, w.p, w.bytes, current(d)),
        "w4a4_grouped_linear");
}

// The MXTensor methods: the output is allocated here unless it is given.
Tensor output_of(const OptTensor& out, int64_t rows, int64_t cols, at::ScalarType dtype, c10::Device d) {
  return out ? *out : at::empty({rows, cols}, at::TensorOptions().dtype(dtype).device(d));
}

Tensor dequant_new(const Tensor& codes, const Tensor& scales, int64_t rows, int64_t K, at::ScalarType dtype,
                   const py::object& stream) {
  refuse_tracing();
  const OnStream on(stream, one_device({&codes, &scales}));
  Tensor out = output_of({}, rows, K, dtype, codes.device());
  dequant(rows, K, codes, scales, out, py::none());
  return out;
}

// A residual [M, N] whose rows are contiguous (a copy only where its strides ask for one).
OptTensor residual_rows(const OptTensor& residual, int64_t M, int64_t N) {
  if (!residual) return residual;
  if (residual->dim() != 2 || residual->size(0) != M || residual->size(1) != N)
    value_error("residual must have shape [", M, ", ", N, "], not ", residual->sizes());
  return as_rows(*residual);
}

Tensor matmul_new(const Tensor& aq, const Tensor& as, int64_t M, const Tensor& bq, const Tensor& bs, int64_t N, int64_t K,
                  const OptTensor& out, at::ScalarType dtype, const py::object& stream, const OptTensor& ws, const OptTensor& bias,
                  const std::optional<std::string>& activation, const OptTensor& residual) {
  refuse_tracing();
  if (out) no_gradient(*out, "the output");
  no_gradient(epilogue_of(bias, activation, residual));
  const OnStream on(stream, one_device({&bq, &bs}));
  const OptTensor r = residual_rows(residual, M, N);
  Tensor y = output_of(out, M, N, dtype, bq.device());
  matmul(M, N, K, aq, as, bq, bs, y, py::none(), ws, bias, activation, r);
  return y;
}

Tensor linear_new(const Tensor& x, const Tensor& bq, const Tensor& bs, int64_t N, int64_t K, const OptTensor& out,
                  at::ScalarType dtype, const py::object& stream, const OptTensor& ws, const OptTensor& bias,
                  const std::optional<std::string>& activation, const OptTensor& residual) {
  refuse_tracing();
  no_gradient(x, "x");
  if (out) no_gradient(*out, "the output");
  no_gradient(epilogue_of(bias, activation, residual));
  if (x.dim() != 2) value_error("x must be [M, K] with the weights' K");
  if (x.size(1) != K) value_error("depths differ: ", x.size(1), " and ", K);
  const OnStream on(stream, one_device({&x, &bq, &bs}));
  const OptTensor r = residual_rows(residual, x.size(0), N);
  Tensor y = output_of(out, x.size(0), N, dtype, bq.device());
  linear(x.size(0), N, K, as_rows(x), bq, bs, y, py::none(), ws, bias, activation, r);
  return y;
}

// The experts' weights are the rows of one operand, one expert after the other.
int64_t rows_per_group(int64_t rows, const Tensor& offsets) {
  const int64_t groups = offsets.dim() == 1 ? offsets.size(0) - 1 : 0;
  if (groups < 1) value_error("offsets must be a vector of at least two bounds, not ", offsets.sizes());
  if (rows % groups || rows == 0) value_error("an operand of ", rows, " rows does not hold ", groups, " experts' weights");
  return rows / groups;
}

Tensor grouped_matmul_new(const Tensor& aq, const Tensor& as, int64_t T, const Tensor& bq, const Tensor& bs, int64_t rows, int64_t K,
                          const Tensor& offsets, const OptTensor& out, at::ScalarType dtype, const py::object& stream,
                          const OptTensor& bias, const std::optional<std::string>& activation, const OptTensor& residual) {
  refuse_tracing();
  if (out) no_gradient(*out, "the output");
  no_gradient(epilogue_of(bias, activation, residual));
  const int64_t N = rows_per_group(rows, offsets);
  const OnStream on(stream, one_device({&bq, &bs}));
  const OptTensor r = residual_rows(residual, T, N);
  Tensor y = output_of(out, T, N, dtype, bq.device());
  grouped_matmul(T, N, K, aq, as, bq, bs, offsets, y, bias, activation, r, !out, py::none());
  return y;
}

Tensor grouped_linear_new(const Tensor& x, const Tensor& bq, const Tensor& bs, int64_t rows, int64_t K, const Tensor& offsets,
                          const OptTensor& out, at::ScalarType dtype, const py::object& stream, const OptTensor& ws, const OptTensor& bias,
                          const std::optional<std::string>& activation, const OptTensor& residual) {
  refuse_tracing();
  no_gradient(x, "x");
  if (out) no_gradient(*out, "the output");
  no_gradient(epilogue_of(bias, activation, residual));
  if (x.dim() != 2) value_error("x must be [T, K] with the weights' K");
  if (x.size(1) != K) value_error("depths differ: ", x.size(1), " and ", K);
  const int64_t N = rows_per_group(rows, offsets);
  const OnStream on(stream, one_device({&x, &bq, &bs}));
  const OptTensor r = residual_rows(residual, x.size(0), N);
  Tensor y = output_of(out, x.size(0), N, dtype, bq.device());
  grouped_linear(x.size(0), N, K, as_rows(x), bq, bs, offsets, y, bias, activation, r, !out, py::none(), ws);
  return y;
}

// Codes and scales used as they are where their rows are aligned (16 and 4 bytes), else copied.
py::tuple from_canonical(const Tensor& codes, const Tensor& scales, std::optional<int64_t> K) {
  if (codes.scalar_type() != at::kByte || scales.scalar_type() != at::kByte) type_error("codes and scales must be uint8");
  if (codes.dim() != 2 || scales.dim() != 2 || codes.size(0) != scales.size(0))
    value_error("codes and scales must be matrices with the same number of rows");
  const int64_t k = K ? *K : 2 * codes.size(1), rows = codes.size(0), nb = blocks_of(k), padded = (nb + 3) / 4 * 4;
  if (k < 1 || codes.size(1) != 16 * nb || scales.size(1) != nb)
    value_error("K = ", k, " needs ", 16 * nb, " bytes of codes and ", nb, " scales a row, not ", codes.size(1), " and ",
                scales.size(1));
  const c10::Device d = one_device({&codes, &scales});
  const auto aligned = [&](const Tensor& t, int64_t cols, uintptr_t a) {
    return (cols <= 1 || t.stride(1) == 1) && (rows <= 1 || (t.stride(0) % (int64_t)a == 0 && t.stride(0) >= cols)) &&
           (uintptr_t)t.data_ptr() % a == 0;
  };
  const auto opt = at::TensorOptions().dtype(at::kByte).device(d);
  Tensor q = codes, s = scales;
  if (!aligned(q, 16 * nb, 16)) q = at::empty({rows, 16 * nb}, opt).copy_(codes);
  const int64_t end = s.storage_offset() + std::max<int64_t>(rows - 1, 0) * s.stride(0) + padded;
  if (!aligned(s, nb, 4) || end > (int64_t)s.storage().nbytes())
    s = at::empty({rows, padded}, opt).narrow(1, 0, nb).copy_(scales);
  return py::make_tuple(q, s, rows, k);
}

// ------------------------------------------------------------------------------------------- trainable layer

// y = Q(x) Q(w)^T. Rounding to MXFP4 counts as the identity in the backward pass, whose products are MXFP4 too:
// dx = Q(g) Q(w^T)^T contracts N, dw = Q(g^T) Q(x^T)^T contracts the rows of x, each operand quantised along the axis
// contracted. The transposed operands are made with the forward ones, from one reading of x and of w.
// An operand in one allocation (each costs over a microsecond): its codes, then its scales.
struct Held {
  Tensor memory;
  fp4_mx a{};
};

fp4_mx in_memory(const Tensor& memory, int64_t rows, int64_t k) {
  const int64_t nb = blocks_of(k);
  auto* p = static_cast<uint8_t*>(memory.data_ptr());
  return {p, p + rows * 16 * nb, 16 * nb, (nb + 3) / 4 * 4};
}

Held new_held(int64_t rows, int64_t k, c10::Device d) {
  const int64_t nb = blocks_of(k);
  Held h;
  h.memory = at::empty({rows * (16 * nb + (nb + 3) / 4 * 4)}, at::TensorOptions().dtype(at::kByte).device(d));
  h.a = in_memory(h.memory, rows, k);
  return h;
}

// m along its rows and, if asked, along its columns.
void quantize_held(const Tensor& m, Held* rows, Held* cols, c10::Device d) {
  if (rows) *rows = new_held(m.size(0), m.size(1), d);
  if (cols) *cols = new_held(m.size(1), m.size(0), d);
  c10::DeviceGuard guard(d);
  check(fp4_quantize_mxfp4(dense_type(m, "x"), m.size(0), m.size(1), m.data_ptr(), rows_of(m, m.size(0), m.size(1), "x"),
                           rows ? &rows->a : nullptr, cols ? &cols->a : nullptr, current(d)),
        "fp4_quantize_mxfp4");
}

struct MxLinear : torch::autograd::Function<MxLinear> {
  static Tensor forward(torch::autograd::AutogradContext* ctx, const Tensor& x, const Tensor& w, bool need_dx, bool need_dw) {
    const c10::Device d = x.device();
    const Tensor xm = as_rows(x), wm = as_rows(w);
    const int64_t m = xm.size(0), k = xm.size(1), n = wm.size(0);
    std::vector<int64_t> shape = x.sizes().vec();
    shape.back() = n;
    Tensor y = at::empty(shape, x.options().requires_grad(false).memory_format(at::MemoryFormat::Contiguous));
    Held xt, wt;
    if (m > 0) {
      Held wq, xq;
      quantize_held(wm, &wq, need_dx ? &wt : nullptr, d);
      quantize_held(xm, &xq, need_dw ? &xt : nullptr, d);
      product_into(m, n, k, xq.a, wq.a, y.view({m, n}), {}, d);
    }
    ctx->save_for_backward({xt.memory, wt.memory});
    ctx->saved_data["shape"] = x.sizes().vec();
    ctx->saved_data["types"] = std::vector<int64_t>{(int64_t)x.scalar_type(), (int64_t)w.scalar_type()};
    return y;
  }

  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx, torch::autograd::variable_list grads) {
    const bool need_dx = ctx->needs_input_grad(0), need_dw = ctx->needs_input_grad(1);
    const auto shape = ctx->saved_data["shape"].toIntVector();
    const auto types = ctx->saved_data["types"].toIntVector();
    const Tensor g = as_rows(grads[0]);
    const int64_t m = g.size(0), n = g.size(1), k = shape.back();
    const c10::Device d = g.device();
    const auto opt = at::TensorOptions().device(d);
    Tensor dx, dw;
    if (need_dx) dx = at::empty(shape, opt.dtype((at::ScalarType)types[0]));
    if (need_dw) dw = at::empty({n, k}, opt.dtype((at::ScalarType)types[1]));
    if (m == 0) {
      if (need_dw) dw.zero_();
    } else if (need_dx || need_dw) {
      Held rows, cols;
      quantize_held(g, need_dx ? &rows : nullptr, need_dw ? &cols : nullptr, d);
      const auto saved = ctx->get_saved_variables();
      if (need_dx) product_into(m, k, n, rows.a, in_memory(saved[1], k, n), dx.view({m, k}), {}, d);
      if (need_dw) product_into(n, k, m, cols.a, in_memory(saved[0], k, m), dw, {}, d);
    }
    torch::autograd::variable_list out{dx, dw, Tensor(), Tensor()};
    if (at::GradMode::is_enabled()) {  // create_graph: the gradients have no derivative, and asking for one is an error
      for (Tensor* t : {&dx, &dw})
        if (t->defined()) *t = t->detach().requires_grad_();
      const auto error = std::make_shared<torch::autograd::DelayedError>("mx_linear is differentiable once", 2);
      torch::autograd::variable_list both = error->apply({dx, dw});
      out[0] = both[0], out[1] = both[1];
    }
    return out;
  }
};

// ---- layers with an epilogue, and layers of experts

// The rows of m in groups, D = m f'(z) in m's place where there is a z, along its rows and / or along its columns, and the
// groups' sums into `dbias`. The operand along the columns has fp4_grouped_depth() positions.
void quantize_groups(const Tensor& m, const fp4_groups& groups, Held* rows, Held* cols, const Tensor* z, int activation,
                     const Tensor* dbias, c10::Device d) {
  const int64_t T = m.size(0), K = m.size(1), depth = fp4_grouped_depth(T, groups.count);
  check(depth, "fp4_quantize_mxfp4_grouped");
  if (rows) *rows = new_held(T, K, d);
  if (cols) *cols = new_held(K, std::max<int64_t>(depth, 1), d);
  fp4_gradient gradient{};
  if (z) gradient.z = z->data_ptr<float>(), gradient.ldz = K, gradient.activation = activation;
  Workspace w;
  c10::DeviceGuard guard(d);
  if (dbias) {
    gradient.dbias = dbias->data_ptr(), gradient.dbias_type = dense_type(*dbias, "bias");
    const int64_t need = fp4_grouped_sums_bytes(T, K, groups.count);
    check(need, "fp4_quantize_mxfp4_grouped");
    w = workspace_of({}, need, d);
  }
  check(fp4_quantize_mxfp4_grouped(dense_type(m, "x"), T, K, m.data_ptr(), rows_of(m, T, K, "x"), &groups, rows ? &rows->a : nullptr,
                                   cols ? &cols->a : nullptr, z || dbias ? &gradient : nullptr, w.p, w.bytes, current(d)),
        "fp4_quantize_mxfp4_grouped");
}

// Which gradients a call may be asked for; those of missing inputs are never.
enum { NEED_X = 1, NEED_W = 2, NEED_BIAS = 4, NEED_RESIDUAL = 8 };

int needed(const Tensor& x, const Tensor& w, const Epilogue& e) {
  if (!at::GradMode::is_enabled()) return 0;
  const auto asks = [](const OptTensor& t) { return t && t->requires_grad(); };
  return (x.requires_grad() ? NEED_X : 0) | (w.requires_grad() ? NEED_W : 0) | (asks(e.bias) ? NEED_BIAS : 0) |
         (asks(e.residual) ? NEED_RESIDUAL : 0);
}

// The gradients that the backward pass is asked for: edges are numbered over the inputs that are there.
int wanted(torch::autograd::AutogradContext* ctx, bool bias, bool residual) {
  int edge = 2, need = (ctx->needs_input_grad(0) ? NEED_X : 0) | (ctx->needs_input_grad(1) ? NEED_W : 0);
  if (bias && ctx->needs_input_grad(edge++)) need |= NEED_BIAS;
  if (residual && ctx->needs_input_grad(edge)) need |= NEED_RESIDUAL;
  return need;
}

// The backward pass's list: gradients of x, w, bias and residual, then nothing for `rest` inputs. Under create_graph they
// have no derivative, and asking for one is an error.
torch::autograd::variable_list gradients(torch::autograd::variable_list four, int rest, const char* what) {
  if (at::GradMode::is_enabled()) {
    for (Tensor& t : four)
      if (t.defined()) t = t.detach().requires_grad_();
    const auto error = std::make_shared<torch::autograd::DelayedError>(c10::str(what, " is differentiable once"), 4);
    four = error->apply(std::move(four));
  }
  four.resize(4 + rest);
  return four;
}

Tensor new_output(const Tensor& x, int64_t n) {
  std::vector<int64_t> shape = x.sizes().vec();
  shape.back() = n;
  return at::empty(shape, x.options().requires_grad(false).memory_format(at::MemoryFormat::Contiguous));
}

// y = f(Q(x) Q(w)^T + bias) + residual. Kept for the backward pass: the transposed operands in 4 bits and, with an activation,
// z in FP32. (z in y's type would be half of that, but f' at a z rounded to 8 bits moves a hundredth of D's values to another
// level of their 4 bits.) Without a group of its own the batch is one group.
struct MxLinearEpilogue : torch::autograd::Function<MxLinearEpilogue> {
  static Tensor forward(torch::autograd::AutogradContext* ctx, const Tensor& x, const Tensor& w, const OptTensor& bias,
                        const OptTensor& residual, int64_t activation, int64_t need) {
    const c10::Device d = x.device();
    const Tensor xm = as_rows(x), wm = as_rows(w);
    const int64_t m = xm.size(0), k = xm.size(1), n = wm.size(0);
    Tensor y = new_output(x, n), z, held;
    Held xt, wt;
    if (activation != FP4_ACT_NONE && (need & (NEED_X | NEED_W | NEED_BIAS)))
      z = at::empty({m, n}, at::TensorOptions().dtype(at::kFloat).device(d));
    if (m > 0) {
      Held wq, xq;
      quantize_held(wm, &wq, need & NEED_X ? &wt : nullptr, d);
      quantize_held(xm, &xq, need & NEED_W ? &xt : nullptr, d);
      const Tensor ym = y.view({m, n});
      const Epilogue e{bias, residual ? OptTensor(as_rows(*residual)) : residual, (int)activation};
      fp4_epilogue after = native(e, ym, m, n, 0, d, held);
      if (z.defined()) after.z = z.data_ptr<float>(), after.ldz = n;
      product_into(m, n, k, xq.a, wq.a, ym, {}, d, &after);
    }
    ctx->save_for_backward({xt.memory, wt.memory, z});
    ctx->saved_data["shape"] = x.sizes().vec();
    ctx->saved_data["w"] = (int64_t)w.scalar_type();
    ctx->saved_data["x"] = (int64_t)x.scalar_type();
    ctx->saved_data["bias"] = bias ? (int64_t)bias->scalar_type() : -1;
    ctx->saved_data["residual"] = residual ? (int64_t)residual->scalar_type() : -1;
    ctx->saved_data["activation"] = activation;
    return y;
  }

  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx, torch::autograd::variable_list grads) {
    const int64_t bias_type = ctx->saved_data["bias"].toInt(), residual_type = ctx->saved_data["residual"].toInt();
    const int need = wanted(ctx, bias_type >= 0, residual_type >= 0);
    const auto shape = ctx->saved_data["shape"].toIntVector();
    const Tensor g = as_rows(grads[0]);
    const int64_t m = g.size(0), n = g.size(1), k = shape.back();
    const c10::Device d = g.device();
    const auto opt = at::TensorOptions().device(d);
    Tensor dx, dw, db, dr;
    if (need & NEED_X) dx = at::empty(shape, opt.dtype((at::ScalarType)ctx->saved_data["x"].toInt()));
    if (need & NEED_W) dw = at::empty({n, k}, opt.dtype((at::ScalarType)ctx->saved_data["w"].toInt()));
    if (need & NEED_BIAS) db = at::empty({n}, opt.dtype((at::ScalarType)bias_type));
    if (need & NEED_RESIDUAL) dr = grads[0].to((at::ScalarType)residual_type);
    if (m == 0) {
      if (dw.defined()) dw.zero_();
      if (db.defined()) db.zero_();
    } else if (need & (NEED_X | NEED_W | NEED_BIAS)) {
      const auto saved = ctx->get_saved_variables();
      const Tensor& z = saved[2];
      Held rows, cols;
      Held *pr = need & NEED_X ? &rows : nullptr, *pc = need & NEED_W ? &cols : nullptr;
      if (z.defined() || db.defined())
        quantize_groups(g, {nullptr, 1, 0}, pr, pc, z.defined() ? &z : nullptr, (int)ctx->saved_data["activation"].toInt(),
                        db.defined() ? &db : nullptr, d);
      else
        quantize_held(g, pr, pc, d);
      if (need & NEED_X) product_into(m, k, n, rows.a, in_memory(saved[1], k, n), dx.view({m, k}), {}, d);
      if (need & NEED_W) product_into(n, k, m, cols.a, in_memory(saved[0], k, m), dw, {}, d);
    }
    return gradients({dx, dw, db, dr}, 2, "mx_linear");
  }
};

// The same with rows in groups, each with weights and a bias of its own.
struct MxGroupedLinear : torch::autograd::Function<MxGroupedLinear> {
  static Tensor forward(torch::autograd::AutogradContext* ctx, const Tensor& x, const Tensor& w, const OptTensor& bias,
                        const OptTensor& residual, const Tensor& offsets, int64_t activation, int64_t need) {
    const c10::Device d = x.device();
    const Groups g = groups_of(offsets, d);
    const int64_t experts = w.size(0), n = w.size(1), k = w.size(2);
    const Tensor xm = as_rows(x), wm = as_rows(w);
    const int64_t m = xm.size(0);
    Tensor y = new_output(x, n), z, held;
    Held xt, wt;
    if (activation != FP4_ACT_NONE && (need & (NEED_X | NEED_W | NEED_BIAS)))
      z = at::empty({m, n}, at::TensorOptions().dtype(at::kFloat).device(d));
    if (m > 0) {
      Held wq, xq;
      if (need & NEED_X) quantize_groups(wm, {nullptr, experts, 0}, &wq, &wt, nullptr, 0, nullptr, d);
      else quantize_held(wm, &wq, nullptr, d);
      if (need & NEED_W) quantize_groups(xm, g.g, &xq, &xt, nullptr, 0, nullptr, d);
      else quantize_held(xm, &xq, nullptr, d);
      const Tensor ym = y.view({m, n});
      const Epilogue e{bias, residual ? OptTensor(as_rows(*residual)) : residual, (int)activation};
      fp4_epilogue after = native(e, ym, m, n, experts, d, held);
      if (z.defined()) after.z = z.data_ptr<float>(), after.ldz = n;
      c10::DeviceGuard guard(d);
      check(w4a4_grouped_matmul(dense_type(ym, "y"), m, n, k, &g.g, &xq.a, &wq.a, &after, 1, ym.data_ptr(), n, current(d)),
            "w4a4_grouped_matmul");
    }
    ctx->save_for_backward({xt.memory, wt.memory, z, offsets});
    ctx->saved_data["shape"] = x.sizes().vec();
    ctx->saved_data["weights"] = w.sizes().vec();
    ctx->saved_data["w"] = (int64_t)w.scalar_type();
    ctx->saved_data["x"] = (int64_t)x.scalar_type();
    ctx->saved_data["bias"] = bias ? (int64_t)bias->scalar_type() : -1;
    ctx->saved_data["residual"] = residual ? (int64_t)residual->scalar_type() : -1;
    ctx->saved_data["activation"] = activation;
    return y;
  }

  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx, torch::autograd::variable_list grads) {
    const int64_t bias_type = ctx->saved_data["bias"].toInt(), residual_type = ctx->saved_data["residual"].toInt();
    const int need = wanted(ctx, bias_type >= 0, residual_type >= 0);
    const auto shape = ctx->saved_data["shape"].toIntVector(), weights = ctx->saved_data["weights"].toIntVector();
    const int64_t experts = weights[0], n = weights[1], k = weights[2];
    const Tensor g = as_rows(grads[0]);
    const int64_t m = g.size(0);
    const c10::Device d = g.device();
    const auto opt = at::TensorOptions().device(d);
    Tensor dx, dw, db, dr;
    if (need & NEED_X) dx = at::empty(shape, opt.dtype((at::ScalarType)ctx->saved_data["x"].toInt()));
    if (need & NEED_W) dw = at::empty(weights, opt.dtype((at::ScalarType)ctx->saved_data["w"].toInt()));
    if (need & NEED_BIAS) db = at::empty({experts, n}, opt.dtype((at::ScalarType)bias_type));
    if (need & NEED_RESIDUAL) dr = grads[0].to((at::ScalarType)residual_type);
    if (m == 0) {
      if (dw.defined()) dw.zero_();
      if (db.defined()) db.zero_();
    } else if (need & (NEED_X | NEED_W | NEED_BIAS)) {
      const auto saved = ctx->get_saved_variables();
      const Tensor& z = saved[2];
      const Groups groups = groups_of(saved[3], d);
      Held rows, cols;
      quantize_groups(g, groups.g, need & NEED_X ? &rows : nullptr, need & NEED_W ? &cols : nullptr, z.defined() ? &z : nullptr,
                      (int)ctx->saved_data["activation"].toInt(), db.defined() ? &db : nullptr, d);
      c10::DeviceGuard guard(d);
      if (need & NEED_X) {
        const fp4_mx b = in_memory(saved[1], k, fp4_grouped_depth(experts * n, experts));
        check(w4a4_grouped_matmul_t(dense_type(dx, "x"), m, n, k, &groups.g, &rows.a, &b, 1, dx.data_ptr(), k, current(d)),
              "w4a4_grouped_matmul_t");
      }
      if (need & NEED_W) {
        const fp4_mx b = in_memory(saved[0], k, fp4_grouped_depth(m, experts));
        check(w4a4_grouped_gradient(dense_type(dw, "w"), m, n, k, &groups.g, &cols.a, &b, dw.data_ptr(), k, current(d)),
              "w4a4_grouped_gradient");
      }
    }
    return gradients({dx, dw, db, dr}, 3, "mx_grouped_linear");
  }
};

// The layers' epilogue: on x's GPU, the residual of y's shape.
void check_after(const Epilogue& e, const Tensor& x, int64_t groups, int64_t n) {
  if (e.bias) {
    one_device({&x, &*e.bias});
    bias_of(*e.bias, groups, n);
  }
  if (!e.residual) return;
  one_device({&x, &*e.residual});
  dense_type(*e.residual, "residual");
  std::vector<int64_t> shape = x.sizes().vec();
  shape.back() = n;
  if (e.residual->sizes() != at::IntArrayRef(shape)) value_error("residual must have shape ", at::IntArrayRef(shape), ", not ", e.residual->sizes());
}

Tensor mx_linear(const Tensor& x, const Tensor& w, const OptTensor& bias, const std::optional<std::string>& activation,
                 const OptTensor& residual) {
  refuse_tracing();
  dense_type(x, "x");
  dense_type(w, "w");
  if (x.dim() < 1 || w.dim() != 2 || x.size(-1) != w.size(1))
    value_error("x [..., K] and w [N, K] expected, not ", x.sizes(), " and ", w.sizes());
  if (w.size(0) < 1 || w.size(1) < 1) value_error("w has no rows or no columns");
  one_device({&x, &w});
  const Epilogue e = epilogue_of(bias, activation, residual);
  check_after(e, x, 0, w.size(0));
  const int need = needed(x, w, e);
  py::gil_scoped_release release;
  if (e.any()) return MxLinearEpilogue::apply(x, w, bias, residual, (int64_t)e.activation, (int64_t)need);
  return MxLinear::apply(x, w, (need & NEED_X) != 0, (need & NEED_W) != 0);
}

Tensor mx_grouped_linear(const Tensor& x, const Tensor& w, const Tensor& offsets, const OptTensor& bias,
                         const std::optional<std::string>& activation, const OptTensor& residual) {
  refuse_tracing();
  dense_type(x, "x");
  dense_type(w, "w");
  if (x.dim() < 1 || w.dim() != 3 || x.size(-1) != w.size(2))
    value_error("x [..., K] and w [E, N, K] expected, not ", x.sizes(), " and ", w.sizes());
  if (w.numel() < 1) value_error("w has no experts, no rows or no columns");
  const c10::Device d = one_device({&x, &w});
  groups_of(offsets, d);
  if (offsets.size(0) != w.size(0) + 1) value_error(w.size(0), " experts have ", w.size(0) + 1, " bounds, not ", offsets.size(0));
  const Epilogue e = epilogue_of(bias, activation, residual);
  check_after(e, x, w.size(0), w.size(1));
  const int need = needed(x, w, e);
  py::gil_scoped_release release;
  return MxGroupedLinear::apply(x, w, bias, residual, offsets, (int64_t)e.activation, (int64_t)need);
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
  m.def("quantize", &quantize);
  m.def("quantize_new", &quantize_py);
  m.def("dequant", &dequant);
  m.def("matmul", &matmul);
  m.def("linear", &linear);
  m.def("dequant_new", &dequant_new);
  m.def("matmul_new", &matmul_new);
  m.def("linear_new", &linear_new);
  m.def("from_canonical", &from_canonical);
  m.def("grouped_matmul", &grouped_matmul);
  m.def("grouped_linear", &grouped_linear);
  m.def("grouped_matmul_new", &grouped_matmul_new);
  m.def("grouped_linear_new", &grouped_linear_new);
  m.def("mx_linear", &mx_linear);
  m.def("mx_grouped_linear", &mx_grouped_linear);
}
