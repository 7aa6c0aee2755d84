// Native half of the Python binding of the MXFP4 operators: argument checks, allocation through torch and the calls of
// the C entry points, and the trainable layer's autograd node. A decode-sized product runs for a few microseconds;
// the same checks written in Python took 23 to 30 microseconds a call.
#include <ATen/ATen.h>
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
                  c10::Device d) {
  const int type = dense_type(y, "y");
  const int64_t ldy = rows_of(y, M, N, "y");
  c10::DeviceGuard guard(d);
  const int64_t need = ws ? 0 : w4a4_matmul_workspace_bytes(M, N, K);
  check(need, "w4a4_matmul");
  const Workspace w = workspace_of(ws, need, d);
  check(w4a4_matmul(type, M, N, K, &a, &b, y.data_ptr(), ldy, w.p, w.bytes, current(d)), "w4a4_matmul");
}

void matmul(int64_t M, int64_t N, int64_t K, const Tensor& aq, const Tensor& as, const Tensor& bq, const Tensor& bs,
            const Tensor& y, const py::object& stream, const OptTensor& ws) {
  refuse_tracing();
  no_gradient(y, "the output");
  const c10::Device d = one_device({&aq, &as, &bq, &bs, &y});
  const OnStream on(stream, d);
  written(y);
  product_into(M, N, K, operand(aq, as, M, K, "A"), operand(bq, bs, N, K, "B"), y, ws, d);
}

void linear_into(int64_t M, int64_t N, int64_t K, const Tensor& x, const Operand& B, const Tensor& y,
                 const OptTensor& ws, c10::Device d) {
  const int tx = dense_type(x, "x"), ty = dense_type(y, "y");
  const int64_t ldx = rows_of(x, M, K, "x"), ldy = rows_of(y, M, N, "y");
  const fp4_mx b = operand(B.codes, B.scales, N, K, "B");
  c10::DeviceGuard guard(d);
  const int64_t need = ws ? 0 : w4a4_linear_workspace_bytes(M, N, K);
  check(need, "w4a4_linear");
  const Workspace w = workspace_of(ws, need, d);
  check(w4a4_linear(tx, ty, M, N, K, x.data_ptr(), ldx, &b, y.data_ptr(), ldy, w.p, w.bytes, current(d)), "w4a4_linear");
}

void linear(int64_t M, int64_t N, int64_t K, const Tensor& x, const Tensor& bq, const Tensor& bs, const Tensor& y,
            const py::object& stream, const OptTensor& ws) {
  refuse_tracing();
  no_gradient(x, "x");
  no_gradient(y, "the output");
  const c10::Device d = one_device({&x, &bq, &bs, &y});
  const OnStream on(stream, d);
  written(y);
  linear_into(M, N, K, x, {bq, bs}, y, ws, d);
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

Tensor matmul_new(const Tensor& aq, const Tensor& as, int64_t M, const Tensor& bq, const Tensor& bs, int64_t N, int64_t K,
                  const OptTensor& out, at::ScalarType dtype, const py::object& stream, const OptTensor& ws) {
  refuse_tracing();
  if (out) no_gradient(*out, "the output");
  const OnStream on(stream, one_device({&bq, &bs}));
  Tensor y = output_of(out, M, N, dtype, bq.device());
  matmul(M, N, K, aq, as, bq, bs, y, py::none(), ws);
  return y;
}

Tensor linear_new(const Tensor& x, const Tensor& bq, const Tensor& bs, int64_t N, int64_t K, const OptTensor& out,
                  at::ScalarType dtype, const py::object& stream, const OptTensor& ws) {
  refuse_tracing();
  no_gradient(x, "x");
  if (out) no_gradient(*out, "the output");
  if (x.dim() != 2) value_error("x must be [M, K] with the weights' K");
  if (x.size(1) != K) value_error("depths differ: ", x.size(1), " and ", K);
  const OnStream on(stream, one_device({&x, &bq, &bs}));
  Tensor y = output_of(out, x.size(0), N, dtype, bq.device());
  linear(x.size(0), N, K, as_rows(x), bq, bs, y, py::none(), ws);
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

Tensor mx_linear(const Tensor& x, const Tensor& w) {
  refuse_tracing();
  dense_type(x, "x");
  dense_type(w, "w");
  if (x.dim() < 1 || w.dim() != 2 || x.size(-1) != w.size(1))
    value_error("x [..., K] and w [N, K] expected, not ", x.sizes(), " and ", w.sizes());
  if (w.size(0) < 1 || w.size(1) < 1) value_error("w has no rows or no columns");
  one_device({&x, &w});
  const bool grad = at::GradMode::is_enabled();
  const bool need_dx = grad && x.requires_grad(), need_dw = grad && w.requires_grad();
  py::gil_scoped_release release;
  return MxLinear::apply(x, w, need_dx, need_dw);
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
  m.def("mx_linear", &mx_linear);
}
