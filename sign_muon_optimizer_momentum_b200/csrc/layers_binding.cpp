// Python binding of the per-worker training operators: argument checks,
// output and workspace allocation (PyTorch's caching allocator) and the call
// of the C ABI, for layers.py, which documents the functions.  It is C++ and
// not ctypes because these calls are made many times a training step: checks
// and marshalling in Python took two to four times as long as a small
// operator's kernels.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <algorithm>
#include <optional>
#include <string>
#include <tuple>
#include <vector>

#include "signmuon.h"

namespace {

namespace py = pybind11;
using at::Tensor;
using Splits = std::optional<std::vector<int64_t>>;
using MaybeTensor = std::optional<Tensor>;

// Raises SignMuonError for a status that is not SIGNMUON_OK.
void check_status(const char* name, signmuon_status status) {
  if (status != SIGNMUON_OK)
    py::module_::import("sign_muon_optimizer_momentum_b200._lib").attr("_check")(name, static_cast<int>(status));
}

signmuon_dtype dtype_code(at::ScalarType t) {
  if (t == at::kFloat) return SIGNMUON_F32;
  TORCH_CHECK_TYPE(t == at::kBFloat16, "unsupported dtype ", t, " (fp32 or bf16)");
  return SIGNMUON_BF16;
}

void check_cuda(const Tensor& t, const char* what) { TORCH_CHECK_VALUE(t.is_cuda(), what, " must be a CUDA tensor"); }
void check_cuda(const Tensor& t, const char* what, const Tensor& like) {
  check_cuda(t, what);
  TORCH_CHECK_VALUE(t.device() == like.device(), what, " is on ", t.device(), ", expected ", like.device());
}
void check_type(const Tensor& t, at::ScalarType dtype, const char* what) {
  TORCH_CHECK_TYPE(t.scalar_type() == dtype, what, ": expected ", dtype, ", got ", t.scalar_type());
}

// A tensor of rows in its last dimension.
struct RowsOf {
  int64_t n, cols, ld;
};
RowsOf rows_of(const Tensor& tensor, const char* what) {
  Tensor t = tensor;
  TORCH_CHECK_VALUE(t.dim() >= 1, what, ": expected rows in the last dimension");
  const int64_t cols = t.size(-1);
  TORCH_CHECK_VALUE(cols > 0, what, ": expected at least one column");
  if (t.is_contiguous()) return {t.numel() / cols, cols, cols};
  if (t.dim() != 2) {
    // One stride has to lead from each row to the next, over all leading
    // dimensions.
    int64_t ld = -1, rows = 1;
    for (int64_t d = t.dim() - 2; d >= 0; --d) {
      if (t.size(d) == 1) continue;
      if (ld < 0) ld = t.stride(d);
      TORCH_CHECK_VALUE(t.stride(d) == ld * rows, what, ": rows must have one stride");
      rows *= t.size(d);
    }
    t = t.as_strided({rows, cols}, {ld < 0 ? cols : ld, t.stride(-1)});
  }
  const int64_t n = t.size(0), ld = t.stride(0);
  TORCH_CHECK_VALUE((cols == 1 || t.stride(1) == 1) && (n <= 1 || ld >= cols), what,
                    ": columns must be adjacent and rows must not overlap");
  return {n, cols, ld > cols ? ld : cols};
}

// The row stride of an output of this shape and type.
int64_t check_out(const Tensor& t, at::IntArrayRef shape, at::ScalarType dtype, const char* what, const Tensor& like) {
  check_cuda(t, what, like);
  check_type(t, dtype, what);
  TORCH_CHECK_VALUE(t.sizes() == shape, what, ": expected shape ", shape, ", got ", t.sizes());
  return rows_of(t, what).ld;
}

// A tensor's memory: n pieces of `bytes` that start `step` apart.
struct Pieces {
  const char* p;
  int64_t n, bytes, step;
};
Pieces pieces_of(const Tensor& t) {
  const char* p = static_cast<const char*>(t.const_data_ptr());
  const int64_t all = (int64_t)t.nbytes(), size = (int64_t)t.element_size();
  if (!all || t.is_contiguous()) return {p, 1, all, all};
  const RowsOf r = rows_of(t, "tensor");
  return {p, r.n, r.cols * size, r.ld * size};
}
// Whether they have bytes in common.  (Of rows of two different strides this is
// not known: false.)
bool overlap(Pieces a, Pieces b) {
  if (!a.bytes || !b.bytes || a.p + (a.n - 1) * a.step + a.bytes <= b.p || b.p + (b.n - 1) * b.step + b.bytes <= a.p) return false;
  if (a.n == 1) std::swap(a, b);
  if (b.n == 1) {
    // The first piece of a that ends behind b's start.
    const int64_t before = b.p - a.p - a.bytes, k = before < 0 ? 0 : before / a.step + 1;
    return k < a.n && a.p + k * a.step < b.p + b.bytes;
  }
  if (a.step != b.step) return false;
  const int64_t off = ((b.p - a.p) % a.step + a.step) % a.step;
  return off < a.bytes || off + b.bytes > a.step;
}

// An output shares no memory with an input; or, where that is allowed, it is
// the same tensor.
void check_apart(const Tensor& out, const Tensor& in, const char* what, bool same = false) {
  const Pieces a = pieces_of(out), b = pieces_of(in);
  if (same && a.p == b.p && a.n == b.n && a.bytes == b.bytes && a.step == b.step) return;
  TORCH_CHECK_VALUE(!overlap(a, b), "out overlaps ", what);
}

// Tells autograd that a caller's tensor has been written to: a backward pass that
// saved it then fails instead of using the new values.
void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

bool check_ids(const Tensor& ids, const char* what, const Tensor& like) {
  check_cuda(ids, what, like);
  const bool wide = ids.scalar_type() == at::kLong;
  TORCH_CHECK_TYPE(wide || ids.scalar_type() == at::kInt, what, ": expected int32 or int64, got ", ids.scalar_type());
  TORCH_CHECK_VALUE(ids.is_contiguous(), what, " must be contiguous");
  return wide;
}

// The workers' row offsets.
std::vector<int64_t> shares(int64_t rows, int64_t n_workers, const Splits& splits) {
  TORCH_CHECK_VALUE(n_workers >= 1 && n_workers <= SIGNMUON_MAX_WORKERS, "n_workers must be in [1, ", SIGNMUON_MAX_WORKERS, "]");
  if (!splits) {
    TORCH_CHECK_VALUE(rows % n_workers == 0, rows, " rows do not divide into ", n_workers, " workers: give splits");
    std::vector<int64_t> even(n_workers + 1);
    for (int64_t m = 0; m <= n_workers; ++m) even[m] = m * (rows / n_workers);
    return even;
  }
  bool ok = (int64_t)splits->size() == n_workers + 1 && splits->front() == 0 && splits->back() == rows;
  for (size_t i = 1; ok && i < splits->size(); ++i) ok = (*splits)[i - 1] <= (*splits)[i];
  TORCH_CHECK_VALUE(ok, "splits must be ", n_workers + 1, " non-decreasing offsets from 0 to ", rows);
  return *splits;
}

// (Not by way of the dispatcher, which takes as long as the allocation.)
Tensor empty(at::IntArrayRef shape, at::ScalarType dtype, const Tensor& like) {
  return Tensor(at::detail::empty_cuda(shape, dtype, like.device(), std::nullopt));
}

// One tensor for each worker, each 16-byte aligned as the step wants them, in
// one allocation.
std::vector<Tensor> per_worker(int64_t n, at::IntArrayRef shape, at::ScalarType dtype, const Tensor& like) {
  int64_t elems = 1;
  std::vector<int64_t> strides(shape.size());
  for (size_t d = shape.size(); d-- > 0;) strides[d] = elems, elems *= shape[d];
  const int64_t granule = 16 / (int64_t)c10::elementSize(dtype), step = (elems + granule - 1) / granule * granule;
  const Tensor whole = empty({n * step}, dtype, like);
  std::vector<Tensor> out;
  out.reserve(n);
  for (int64_t i = 0; i < n; ++i) {
    auto view = c10::make_intrusive<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(whole.storage()), whole.key_set(),
                                                     whole.dtype());
    view->set_sizes_and_strides(shape, strides, i * step);
    out.emplace_back(std::move(view));
  }
  return out;
}
std::vector<void*> pointers(const Tensor* t, size_t n) {
  std::vector<void*> p(n);
  for (size_t i = 0; i < n; ++i) p[i] = t[i].data_ptr();
  return p;
}

// The tensors' device and its current stream for the length of a call.
struct Call {
  c10::cuda::OptionalCUDAGuard guard;
  void* stream;
  explicit Call(const Tensor& t) {
    if (t.device().index() != c10::cuda::current_device()) guard.set_device(t.device());
    stream = c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
  }
  Tensor workspace(size_t bytes, const Tensor& like) const { return empty({(int64_t)bytes}, at::kByte, like); }
};

signmuon_shape shape_of(int64_t rows, int64_t cols) {
  TORCH_CHECK_VALUE(rows <= INT32_MAX && cols <= INT32_MAX, "at most 2^31 - 1 rows and columns");
  return {(int32_t)rows, (int32_t)cols};
}

// ---------------------------------------------------------------- embedding
Tensor embedding_forward(const Tensor& table, const Tensor& ids, double scale, std::optional<at::ScalarType> dtype,
                         const MaybeTensor& out) {
  check_cuda(table, "table");
  TORCH_CHECK_VALUE(table.dim() == 2, "table must have two dimensions");
  const bool wide = check_ids(ids, "ids", table);
  const RowsOf t = rows_of(table, "table");
  TORCH_CHECK_VALUE(t.n > 0, "table must have at least one row");
  const at::ScalarType type = dtype.value_or(table.scalar_type());
  const signmuon_dtype table_code = dtype_code(table.scalar_type()), code = dtype_code(type);
  std::vector<int64_t> shape = ids.sizes().vec();
  shape.push_back(t.cols);
  const int64_t ld = out ? check_out(*out, shape, type, "out", table) : t.cols;
  if (out) check_apart(*out, table, "table"), check_apart(*out, ids, "ids");
  const Call call(table);
  const Tensor y = out ? *out : empty(shape, type, table);
  check_status("signmuon_embedding_forward",
               signmuon_embedding_forward(shape_of(t.n, t.cols), table_code, table.data_ptr(), t.ld, ids.numel(), wide,
                                          ids.data_ptr(), (float)scale, code, y.data_ptr(), ld, call.stream));
  if (out) written(*out);
  return y;
}

std::vector<Tensor> embedding_backward(const Tensor& ids, const Tensor& grad_out, int64_t vocab, int64_t n_workers,
                                       const Splits& splits, double scale, std::optional<at::ScalarType> dtype,
                                       const std::optional<std::vector<Tensor>>& out, bool accumulate) {
  check_cuda(grad_out, "grad_out");
  const bool wide = check_ids(ids, "ids", grad_out);
  const RowsOf dy = rows_of(grad_out, "grad_out");
  TORCH_CHECK_VALUE(ids.numel() == dy.n, ids.numel(), " ids for ", dy.n, " rows of grad_out");
  TORCH_CHECK_VALUE(vocab >= 1, "vocab must be >= 1");
  const signmuon_shape shape = shape_of(vocab, dy.cols);
  const at::ScalarType type = dtype.value_or(grad_out.scalar_type());
  const signmuon_dtype dy_code = dtype_code(grad_out.scalar_type()), code = dtype_code(type);
  const std::vector<int64_t> rows = shares(dy.n, n_workers, splits);
  if (out) {
    TORCH_CHECK_VALUE((int64_t)out->size() == n_workers, "expected ", n_workers, " gradient buffers, got ", out->size());
    for (size_t m = 0; m < out->size(); ++m) {
      const std::string what = "out[" + std::to_string(m) + "]";
      check_out((*out)[m], {vocab, dy.cols}, type, what.c_str(), grad_out);
      TORCH_CHECK_VALUE((*out)[m].is_contiguous(), what, " must be contiguous");
      check_apart((*out)[m], grad_out, "grad_out"), check_apart((*out)[m], ids, "ids");
    }
    std::vector<const char*> at;
    for (const Tensor& t : *out) at.push_back(static_cast<const char*>(t.data_ptr()));
    std::sort(at.begin(), at.end());
    for (size_t m = 1; m < at.size(); ++m)
      TORCH_CHECK_VALUE(at[m] - at[m - 1] >= (ptrdiff_t)(*out)[0].nbytes(), "gradient buffers overlap");
  } else {
    TORCH_CHECK_VALUE(!accumulate, "accumulate needs out");
  }
  const Call call(grad_out);
  std::vector<Tensor> grads = out ? *out : per_worker(n_workers, {vocab, dy.cols}, type, grad_out);
  const std::vector<void*> ptrs = pointers(grads.data(), grads.size());
  const Tensor ws = call.workspace(signmuon_embedding_backward_workspace_bytes(shape, (int)n_workers, rows.data()), grad_out);
  check_status("signmuon_embedding_backward",
               signmuon_embedding_backward(shape, (int)n_workers, rows.data(), wide, ids.data_ptr(), dy_code,
                                           grad_out.data_ptr(), dy.ld, (float)scale, accumulate, code, ptrs.data(),
                                           ws.data_ptr(), ws.nbytes(), call.stream));
  if (out)
    for (const Tensor& t : *out) written(t);
  return grads;
}

// --------------------------------------------------------------- layer norm
void check_vector(const Tensor& t, int64_t cols, const char* what, const Tensor& like) {
  check_cuda(t, what, like);
  TORCH_CHECK_VALUE(t.numel() == cols && t.dim() >= 1 && t.size(-1) == cols && t.is_contiguous(), what, ": expected ", cols,
                    " contiguous elements");
}

std::tuple<Tensor, Tensor, Tensor> layer_norm_forward(const Tensor& x, const Tensor& weight, const MaybeTensor& bias,
                                                      double eps, const MaybeTensor& out) {
  check_cuda(x, "x");
  const RowsOf r = rows_of(x, "x");
  check_vector(weight, r.cols, "weight", x);
  if (bias) {
    check_vector(*bias, r.cols, "bias", x);
    check_type(*bias, weight.scalar_type(), "bias");
  }
  TORCH_CHECK_VALUE(eps >= 0, "eps must be >= 0");
  const signmuon_dtype code = dtype_code(x.scalar_type()), w_code = dtype_code(weight.scalar_type());
  const signmuon_shape shape = shape_of(1, r.cols);
  const int64_t ld = out ? check_out(*out, x.sizes(), x.scalar_type(), "out", x) : r.cols;
  if (out) check_apart(*out, x, "x", true), check_apart(*out, weight, "weight");
  if (out && bias) check_apart(*out, *bias, "bias");
  const Call call(x);
  const Tensor y = out ? *out : empty(x.sizes(), x.scalar_type(), x);
  const at::IntArrayRef lead = x.sizes().slice(0, x.dim() - 1);
  const Tensor mean = empty(lead, at::kFloat, x), rstd = empty(lead, at::kFloat, x);
  check_status("signmuon_layer_norm_forward",
               signmuon_layer_norm_forward(r.n, shape.cols, code, x.data_ptr(), r.ld, w_code, weight.data_ptr(),
                                           bias ? bias->data_ptr() : nullptr, (float)eps, y.data_ptr(), ld,
                                           mean.data_ptr<float>(), rstd.data_ptr<float>(), call.stream));
  if (out) written(*out);
  return {y, mean, rstd};
}

std::tuple<Tensor, std::vector<Tensor>, std::optional<std::vector<Tensor>>> layer_norm_backward(
    const Tensor& grad_out, const Tensor& x, const Tensor& weight, const Tensor& mean, const Tensor& rstd, int64_t n_workers,
    const Splits& splits, bool bias, const MaybeTensor& out) {
  check_cuda(grad_out, "grad_out");
  check_cuda(x, "x", grad_out);
  const RowsOf dy = rows_of(grad_out, "grad_out");
  TORCH_CHECK_VALUE(x.sizes() == grad_out.sizes(), "x is ", x.sizes(), ", grad_out ", grad_out.sizes());
  check_type(x, grad_out.scalar_type(), "x");
  const RowsOf r = rows_of(x, "x");
  check_vector(weight, r.cols, "weight", x);
  for (const auto& [t, what] : {std::pair<const Tensor&, const char*>(mean, "mean"), {rstd, "rstd"}}) {
    check_cuda(t, what, x);
    check_type(t, at::kFloat, what);
    TORCH_CHECK_VALUE(t.numel() == r.n && t.is_contiguous(), what, ": expected ", r.n, " contiguous elements");
  }
  const signmuon_dtype code = dtype_code(x.scalar_type()), w_code = dtype_code(weight.scalar_type());
  const signmuon_shape shape = shape_of(1, r.cols);
  const std::vector<int64_t> rows = shares(r.n, n_workers, splits);
  const int64_t ld = out ? check_out(*out, x.sizes(), x.scalar_type(), "out", x) : r.cols;
  if (out) {
    check_apart(*out, grad_out, "grad_out", true);
    for (const auto& [t, what] : {std::pair<const Tensor&, const char*>(x, "x"), {weight, "weight"}, {mean, "mean"}, {rstd, "rstd"}})
      check_apart(*out, t, what);
  }
  const Call call(x);
  const Tensor dx = out ? *out : empty(x.sizes(), x.scalar_type(), x);
  std::vector<Tensor> dw = per_worker(n_workers * (bias ? 2 : 1), weight.sizes(), weight.scalar_type(), x);
  const std::vector<void*> ptrs = pointers(dw.data(), dw.size());
  const Tensor ws = call.workspace(signmuon_layer_norm_backward_workspace_bytes(shape.cols, (int)n_workers, rows.data()), x);
  check_status("signmuon_layer_norm_backward",
               signmuon_layer_norm_backward(shape.cols, (int)n_workers, rows.data(), code, grad_out.data_ptr(), dy.ld,
                                            x.data_ptr(), r.ld, w_code, weight.data_ptr(), mean.data_ptr<float>(),
                                            rstd.data_ptr<float>(), dx.data_ptr(), ld, ptrs.data(),
                                            bias ? ptrs.data() + n_workers : nullptr, ws.data_ptr(), ws.nbytes(),
                                            call.stream));
  if (out) written(*out);
  if (!bias) return {dx, std::move(dw), std::nullopt};
  std::vector<Tensor> db(dw.begin() + n_workers, dw.end());
  dw.resize(n_workers);
  return {dx, std::move(dw), std::move(db)};
}

// ------------------------------------------------------------- distillation
std::tuple<Tensor, Tensor, MaybeTensor> distill(const Tensor& logits, const Tensor& top_ids, const Tensor& top_logits,
                                                int64_t n_workers, const Splits& splits, double temperature,
                                                double grad_scale, bool with_grad, const MaybeTensor& out) {
  check_cuda(logits, "logits");
  const RowsOf z = rows_of(logits, "logits");
  const bool wide = check_ids(top_ids, "top_ids", logits);
  check_cuda(top_logits, "top_logits", logits);
  const at::IntArrayRef lead = logits.sizes().slice(0, logits.dim() - 1);
  TORCH_CHECK_VALUE(top_ids.dim() == logits.dim() && top_ids.sizes().slice(0, top_ids.dim() - 1) == lead &&
                        top_logits.sizes() == top_ids.sizes(),
                    "top_ids and top_logits must have one row of entries for each row of logits");
  const int64_t top = top_ids.size(-1);
  TORCH_CHECK_VALUE(top >= 1 && top <= 1024, "between 1 and 1024 top logits are supported");
  TORCH_CHECK_VALUE(top_logits.is_contiguous(), "top_logits must be contiguous");
  TORCH_CHECK_VALUE(temperature >= 1e-6 && temperature <= 1e6, "temperature must be in [1e-6, 1e6]");
  const signmuon_dtype code = dtype_code(logits.scalar_type()), top_code = dtype_code(top_logits.scalar_type());
  const signmuon_shape shape = shape_of(1, z.cols);
  const std::vector<int64_t> rows = shares(z.n, n_workers, splits);
  const int64_t ld = with_grad && out ? check_out(*out, logits.sizes(), logits.scalar_type(), "out", logits) : z.cols;
  if (with_grad && out) {
    check_apart(*out, logits, "logits", true);
    check_apart(*out, top_ids, "top_ids"), check_apart(*out, top_logits, "top_logits");
  }
  const Call call(logits);
  const Tensor loss = empty({n_workers}, at::kFloat, logits), row_loss = empty(lead, at::kFloat, logits);
  MaybeTensor dz;
  if (with_grad) dz = out ? *out : empty(logits.sizes(), logits.scalar_type(), logits);
  const Tensor ws = call.workspace(signmuon_distill_workspace_bytes(z.n, (int)top), logits);
  check_status("signmuon_distill_loss",
               signmuon_distill_loss(shape.cols, (int)n_workers, rows.data(), code, logits.data_ptr(), z.ld, (int)top, wide,
                                     top_ids.data_ptr(), top_code, top_logits.data_ptr(), (float)temperature,
                                     (float)grad_scale, loss.data_ptr<float>(), row_loss.data_ptr<float>(),
                                     dz ? dz->data_ptr() : nullptr, ld, ws.data_ptr(), ws.nbytes(), call.stream));
  if (with_grad && out) written(*out);
  return {loss, row_loss, dz};
}

}  // namespace

PYBIND11_MODULE(_layers_native, m) {
  m.doc() = "Binding of the per-worker training operators (see layers.py).";
  m.def("embedding_forward", &embedding_forward);
  m.def("embedding_backward", &embedding_backward);
  m.def("layer_norm_forward", &layer_norm_forward);
  m.def("layer_norm_backward", &layer_norm_backward);
  m.def("distill", &distill);
  // For tests.
  m.def("shares", &shares);
  m.def("overlap", [](const Tensor& a, const Tensor& b) { return overlap(pieces_of(a), pieces_of(b)); });
  m.def("rows_of", [](const Tensor& t) {
    const RowsOf r = rows_of(t, "t");
    return std::make_tuple(r.n, r.cols, r.ld);
  });
}
