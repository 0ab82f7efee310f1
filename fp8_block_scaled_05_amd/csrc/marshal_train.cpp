// The argument marshalling of the training step's operators (host code only).
//
// Tensors of a call must be on one device, which need not be the current one:
// the call makes it current, and goes on that device's current stream.  The
// last argument of every function gives a device's current stream's handle,
// called when the tensors have been checked.
#include "marshal.hpp"

#include <c10/core/DeviceGuard.h>

#include <vector>

#include "fp8bs_train.h"

namespace marshal {
namespace {

// All tensors of a call, one after the other.
class Place {
 public:
  void add(const Tensor& t) {
    on_gpu(t);
    if (!first_) first_ = &t;
    TORCH_CHECK_VALUE(t.device() == first_->device(), "all tensors must be on one device, got ", first_->device(), " and ", t.device());
  }
  void add(const Tensor* t) {
    if (t) add(*t);
  }
  c10::Device device() const { return first_->device(); }
  hipStream_t stream(PyObject* current) const {
    THPObjectPtr index(PyLong_FromLong(device().index()));
    if (!index) throw python_error();
    THPObjectPtr handle(PyObject_CallOneArg(current, index));
    if (!handle) throw python_error();
    void* p = PyLong_AsVoidPtr(handle);
    if (!p && PyErr_Occurred()) throw python_error();
    return static_cast<hipStream_t>(p);
  }

 private:
  const Tensor* first_ = nullptr;
};

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v;
}

struct Matrix {
  void* p = nullptr;
  int64_t ld = 0;
};
Matrix matrix(const Tensor& t, at::IntArrayRef shape, at::ScalarType dtype, const char* name) {
  need(t, shape, dtype, name);
  return {t.data_ptr(), pitch(t, name)};
}
// An output that is wanted: `given` checked, or a new dense tensor like `like`.
struct Out {
  Tensor t;
  Matrix m;
};
Out matrix_out(bool wanted, const Tensor* given, const Tensor& like, at::IntArrayRef shape, at::ScalarType dtype, const char* name) {
  Out o;
  if (!wanted) return o;
  o.t = given ? *given : output(nullptr, like, shape, dtype, name);
  o.m = matrix(o.t, shape, dtype, name);
  return o;
}
Tensor dense_out(bool wanted, const Tensor* given, const Tensor& like, at::IntArrayRef shape, at::ScalarType dtype, const char* name) {
  return wanted ? output(given, like, shape, dtype, name) : Tensor();
}
template <class T>
T* ptr(const Tensor& t) {
  return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}

// A norm's weight [cols] (bf16 or f32), or none.
struct Weight {
  const void* p = nullptr;
  int64_t dtype = FP8BS_BF16;
};
Weight weight_of(const Tensor* w, int64_t cols) {
  if (!w) return {};
  const int32_t dtype = dtype_code(*w, "weight");
  dense(*w, {cols}, w->scalar_type(), "weight");
  return {w->data_ptr(), dtype};
}

}  // namespace

// x, weight, residual, eps, quantize, with_y, residual_out, y, q, scale, stream
PyObject* rmsnorm_quant(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 11);
  const Tensor& x = tensor(a[0], "x");
  const Tensor *w = optional(a[1], "weight"), *residual = optional(a[2], "residual"), *given_r = optional(a[6], "residual_out"),
               *given_y = optional(a[7], "y"), *given_q = optional(a[8], "q"), *given_s = optional(a[9], "scale");
  Place place;
  place.add(x);
  for (const Tensor* t : {w, residual, given_r, given_y, given_q, given_s}) place.add(t);
  const int64_t ld = pitch(x, "x"), rows = x.size(0), cols = x.size(1);
  const int32_t dtype = dtype_code(x, "x");
  const bool quantize = truth(a[4]), with_y = truth(a[5]);
  TORCH_CHECK_VALUE(residual || !given_r, "residual_out needs a residual");
  TORCH_CHECK_VALUE(quantize || (!given_q && !given_s), "q and scale need quantize");
  const c10::DeviceGuard guard(place.device());
  const Weight weight = weight_of(w, cols);
  Matrix res;
  if (residual) res = matrix(*residual, {rows, cols}, x.scalar_type(), "residual");
  if (fp8_rmsnorm_backward_workspace(rows, cols) < 0) {                          // refused before anything is allocated, here and below
    const fp8bs_rmsnorm_args sizes{x.data_ptr(), res.p, weight.p, nullptr, nullptr, nullptr, nullptr, rows,         cols,
                                   ld,           res.ld, 0,       0,       0,       dtype,   weight.dtype, real(a[3])};
    return refused(fp8_rmsnorm_quant(&sizes, nullptr));
  }
  const Out sum = matrix_out(residual, given_r, x, {rows, cols}, x.scalar_type(), "residual_out");
  const Out y = matrix_out(with_y || given_y, given_y, x, {rows, cols}, x.scalar_type(), "y");
  const Out q = matrix_out(quantize, given_q, x, {rows, cols}, at::kByte, "q");
  const Tensor scale = dense_out(quantize, given_s, x, {rows, cols / 128}, at::kFloat, "scale");
  const fp8bs_rmsnorm_args args{x.data_ptr(), res.p,  weight.p, sum.m.p,  y.m.p,  static_cast<uint8_t*>(q.m.p), ptr<float>(scale), rows, cols,
                                ld,           res.ld, sum.m.ld, y.m.ld,   q.m.ld, dtype,                        weight.dtype,      real(a[3])};
  if (fp8bs_status st = fp8_rmsnorm_quant(&args, place.stream(a[10]))) return refused(st);
  return wrap({q.t, scale, y.t, sum.t});
  END_HANDLE_TH_ERRORS
}

// dy, h, weight, dresidual, eps, dx, dweight, stream
PyObject* rmsnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 8);
  const Tensor &dy = tensor(a[0], "dy"), &h = tensor(a[1], "h");
  const Tensor *w = optional(a[2], "weight"), *dres = optional(a[3], "dresidual"), *given_dx = optional(a[5], "dx"),
               *given_dw = optional(a[6], "dweight");
  Place place;
  place.add(h);
  place.add(dy);
  for (const Tensor* t : {w, dres, given_dx, given_dw}) place.add(t);
  const int64_t ld = pitch(h, "h"), rows = h.size(0), cols = h.size(1);
  const int32_t dtype = dtype_code(h, "h");
  TORCH_CHECK_VALUE(w || !given_dw, "dweight needs a weight");
  const c10::DeviceGuard guard(place.device());
  const Weight weight = weight_of(w, cols);
  const Matrix g = matrix(dy, {rows, cols}, h.scalar_type(), "dy");
  Matrix res;
  if (dres) res = matrix(*dres, {rows, cols}, h.scalar_type(), "dresidual");
  const int64_t workspace = fp8_rmsnorm_backward_workspace(rows, cols), bytes = w ? workspace : 0;
  fp8bs_rmsnorm_backward_args args{g.p,  h.data_ptr(), weight.p, res.p, nullptr, nullptr, nullptr,      0,         rows,
                                   cols, g.ld,         ld,       res.ld, 0,      dtype,   weight.dtype, real(a[4])};
  if (workspace < 0) return refused(fp8_rmsnorm_backward(&args, nullptr));
  const Out dx = matrix_out(true, given_dx, h, {rows, cols}, h.scalar_type(), "dx");
  const Tensor dw = dense_out(w, given_dw, h, {cols}, at::kFloat, "dweight");
  Tensor room;
  if (bytes > 0) room = output(nullptr, h, {bytes}, at::kByte, "workspace");
  args.dx = dx.m.p, args.ld_dx = dx.m.ld, args.dweight = ptr<float>(dw);
  args.workspace = ptr<void>(room), args.workspace_bytes = bytes;
  if (fp8bs_status st = fp8_rmsnorm_backward(&args, place.stream(a[7]))) return refused(st);
  return wrap({dx.t, dw});
  END_HANDLE_TH_ERRORS
}

// gate, up, quantize, with_y, y, q, scale, stream
PyObject* swiglu_quant(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 8);
  const Tensor &gate = tensor(a[0], "gate"), &up = tensor(a[1], "up");
  const Tensor *given_y = optional(a[4], "y"), *given_q = optional(a[5], "q"), *given_s = optional(a[6], "scale");
  Place place;
  place.add(gate);
  place.add(up);
  for (const Tensor* t : {given_y, given_q, given_s}) place.add(t);
  const int64_t ld = pitch(gate, "gate"), rows = gate.size(0), cols = gate.size(1);
  const int32_t dtype = dtype_code(gate, "gate");
  const Matrix u = matrix(up, {rows, cols}, gate.scalar_type(), "up");
  const bool quantize = truth(a[2]), with_y = truth(a[3]);
  TORCH_CHECK_VALUE(quantize || (!given_q && !given_s), "q and scale need quantize");
  const c10::DeviceGuard guard(place.device());
  if (cols % 128) {
    const fp8bs_swiglu_args sizes{gate.data_ptr(), u.p, nullptr, nullptr, nullptr, rows, cols, ld, u.ld, 0, 0, dtype};
    return refused(fp8_swiglu_quant(&sizes, nullptr));
  }
  const Out y = matrix_out(with_y || given_y, given_y, gate, {rows, cols}, gate.scalar_type(), "y");
  const Out q = matrix_out(quantize, given_q, gate, {rows, cols}, at::kByte, "q");
  const Tensor scale = dense_out(quantize, given_s, gate, {rows, cols / 128}, at::kFloat, "scale");
  const fp8bs_swiglu_args args{gate.data_ptr(), u.p, y.m.p, static_cast<uint8_t*>(q.m.p), ptr<float>(scale), rows, cols, ld, u.ld, y.m.ld, q.m.ld,
                               dtype};
  if (fp8bs_status st = fp8_swiglu_quant(&args, place.stream(a[7]))) return refused(st);
  return wrap({q.t, scale, y.t});
  END_HANDLE_TH_ERRORS
}

// dy, gate, up, quantize, with_d, d, q, scale, stream
PyObject* swiglu_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 9);
  const Tensor &dy = tensor(a[0], "dy"), &gate = tensor(a[1], "gate"), &up = tensor(a[2], "up");
  const Tensor *given_d = optional(a[5], "d"), *given_q = optional(a[6], "q"), *given_s = optional(a[7], "scale");
  Place place;
  place.add(gate);
  place.add(up);
  place.add(dy);
  for (const Tensor* t : {given_d, given_q, given_s}) place.add(t);
  const int64_t ld = pitch(gate, "gate"), rows = gate.size(0), cols = gate.size(1);
  const int32_t dtype = dtype_code(gate, "gate");
  const Matrix u = matrix(up, {rows, cols}, gate.scalar_type(), "up"), g = matrix(dy, {rows, cols}, gate.scalar_type(), "dy");
  const bool quantize = truth(a[3]), with_d = truth(a[4]);
  TORCH_CHECK_VALUE(quantize || (!given_q && !given_s), "q and scale need quantize");
  const c10::DeviceGuard guard(place.device());
  if (cols % 128) {
    const fp8bs_swiglu_backward_args sizes{g.p, gate.data_ptr(), u.p, nullptr, nullptr, nullptr, rows, cols, g.ld, ld, u.ld, 0, 0, dtype};
    return refused(fp8_swiglu_backward(&sizes, nullptr));
  }
  const Out d = matrix_out(with_d || given_d, given_d, gate, {rows, 2 * cols}, gate.scalar_type(), "d");
  const Out q = matrix_out(quantize, given_q, gate, {rows, 2 * cols}, at::kByte, "q");
  const Tensor scale = dense_out(quantize, given_s, gate, {rows, cols / 128 * 2}, at::kFloat, "scale");
  const fp8bs_swiglu_backward_args args{g.p,  gate.data_ptr(), u.p,  d.m.p,  static_cast<uint8_t*>(q.m.p), ptr<float>(scale), rows, cols,
                                        g.ld, ld,              u.ld, d.m.ld, q.m.ld,                       dtype};
  if (fp8bs_status st = fp8_swiglu_backward(&args, place.stream(a[8]))) return refused(st);
  return wrap({q.t, scale, d.t});
  END_HANDLE_TH_ERRORS
}

// x, offsets, order, top_k, q, scale, padded, stream
PyObject* quant_grouped_t(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 8);
  const Tensor &x = tensor(a[0], "x"), &offsets = tensor(a[1], "offsets");
  const Tensor *order = optional(a[2], "order"), *given_q = optional(a[4], "q"), *given_s = optional(a[5], "scale"),
               *given_p = optional(a[6], "padded");
  Place place;
  place.add(x);
  place.add(offsets);
  for (const Tensor* t : {order, given_q, given_s, given_p}) place.add(t);
  const int64_t ld = pitch(x, "x"), rows = x.size(0), cols = x.size(1);
  const int32_t dtype = dtype_code(x, "x"), top_k = narrow(a[3]);
  TORCH_CHECK_VALUE(offsets.dim() == 1 && offsets.size(0) >= 2 && offsets.size(0) <= 1025, "offsets must be int32 [experts + 1], got ", offsets.sizes());
  dense(offsets, offsets.sizes(), at::kInt, "offsets");
  const int32_t groups = static_cast<int32_t>(offsets.size(0) - 1);
  int64_t places = rows;
  if (order) {
    TORCH_CHECK_VALUE(order->dim() == 1, "order must be int32 [places], got ", order->sizes());
    dense(*order, order->sizes(), at::kInt, "order");
    places = order->size(0);
  }
  const int64_t least = fp8_quant_grouped_t_columns(places, groups);
  TORCH_CHECK_VALUE(least >= 0, "too many rows: ", places);
  int64_t columns = least;
  if (given_q) {
    TORCH_CHECK_VALUE(given_q->dim() == 2 && given_q->size(1) >= least && given_q->size(1) % 128 == 0, "q has shape ", given_q->sizes(),
                      ", expected [", cols, ", a multiple of 128 from ", least, " on]");
    columns = given_q->size(1);
  }
  const c10::DeviceGuard guard(place.device());
  if (cols % 16 || columns > (int64_t(1) << 22))
    return refused(fp8_quant_grouped_t(x.data_ptr(), dtype, rows, cols, ld, ptr<int32_t>(offsets), groups,
                                       order ? static_cast<int32_t*>(order->data_ptr()) : nullptr, places, top_k, nullptr, columns, nullptr, columns,
                                       nullptr, nullptr));
  const Out q = matrix_out(true, given_q, x, {cols, columns}, at::kByte, "q");
  const Tensor scale = dense_out(true, given_s, x, {cols, columns / 128}, at::kFloat, "scale");
  const Tensor padded = dense_out(true, given_p, offsets, {groups + int64_t(1)}, at::kInt, "padded");
  if (fp8bs_status st = fp8_quant_grouped_t(x.data_ptr(), dtype, rows, cols, ld, ptr<int32_t>(offsets), groups,
                                            order ? static_cast<int32_t*>(order->data_ptr()) : nullptr, places, top_k,
                                            static_cast<uint8_t*>(q.m.p), q.m.ld, ptr<float>(scale), columns, ptr<int32_t>(padded),
                                            place.stream(a[7])))
    return refused(st);
  return wrap({q.t, scale, padded});
  END_HANDLE_TH_ERRORS
}

// padded, a, a_scale, b, b_scale, out_dtype code or -1, y, accumulate, stream
PyObject* grouped_wgrad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 9);
  const Tensor &padded = tensor(a[0], "padded"), &x = tensor(a[1], "a"), &xs = tensor(a[2], "a_scale"), &z = tensor(a[3], "b"),
               &zs = tensor(a[4], "b_scale");
  const Tensor* given = optional(a[6], "y");
  Place place;
  for (const Tensor* t : {&x, &xs, &z, &zs, &padded, given}) place.add(t);
  TORCH_CHECK_VALUE(padded.dim() == 1 && padded.size(0) >= 2 && padded.size(0) <= 1025, "padded must be int32 [experts + 1], got ", padded.sizes());
  dense(padded, padded.sizes(), at::kInt, "padded");
  const int32_t groups = static_cast<int32_t>(padded.size(0) - 1);
  const int64_t lda = pitch(x, "a"), ldb = pitch(z, "b"), rows = x.size(0), cols = z.size(0), columns = x.size(1);
  need(x, {rows, columns}, at::kByte, "a");
  need(z, {cols, columns}, at::kByte, "b");
  dense(xs, {rows, columns / 128}, at::kFloat, "a_scale");
  dense(zs, {cols, columns / 128}, at::kFloat, "b_scale");
  const int32_t asked = narrow(a[5]);
  const bool accumulate = truth(a[7]);
  TORCH_CHECK_VALUE(given || !accumulate, "accumulate needs y");
  const int32_t dtype = given ? dtype_code(*given, "y") : (asked < 0 ? int32_t(FP8BS_F32) : asked);
  TORCH_CHECK_TYPE(asked < 0 || asked == dtype, "y is not of out_dtype");
  const c10::DeviceGuard guard(place.device());
  const bool far = columns > (int64_t(1) << 22) || std::max(rows, cols) > (int64_t(1) << 26);
  if (rows % 16 || cols % 16 || columns % 128 || (far && rows && cols))
    return refused(fp8_blockscaled_grouped_wgrad(rows, cols, columns, groups, ptr<int32_t>(padded), ptr<uint8_t>(x), lda, ptr<float>(xs),
                                                 ptr<uint8_t>(z), ldb, ptr<float>(zs), nullptr, dtype, accumulate, nullptr));
  const Tensor y = output(given, x, {groups, rows, cols}, dtype == FP8BS_BF16 ? at::kBFloat16 : at::kFloat, "y");
  if (fp8bs_status st = fp8_blockscaled_grouped_wgrad(rows, cols, columns, groups, ptr<int32_t>(padded), ptr<uint8_t>(x), lda, ptr<float>(xs),
                                                      ptr<uint8_t>(z), ldb, ptr<float>(zs), y.data_ptr(), dtype, accumulate, place.stream(a[8])))
    return refused(st);
  return THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

namespace {

// Whether two tensors of one shape have their elements in one order (the stride
// of a dimension of one element says nothing).
bool same_order(const Tensor& a, const Tensor& b) {
  for (int64_t d = 0; d < a.dim(); ++d)
    if (a.size(d) > 1 && a.stride(d) != b.stride(d)) return a.numel() == 0;
  return true;
}

// The tensors of a list, whose elements fill their memory in any order.
void read_grads(PyObject* list, const char* name, Place& place, std::vector<fp8bs_grad>& out, std::vector<const Tensor*>& tensors) {
  TORCH_CHECK_TYPE(PyList_Check(list) || PyTuple_Check(list), name, " must be a list or a tuple of tensors");
  const Py_ssize_t count = PySequence_Fast_GET_SIZE(list);
  out.reserve(count);
  tensors.reserve(count);
  for (Py_ssize_t i = 0; i < count; ++i) {
    const Tensor& t = tensor(PySequence_Fast_GET_ITEM(list, i), name);
    place.add(t);
    TORCH_CHECK_VALUE(t.is_non_overlapping_and_dense(), name, "[", i, "] must fill its memory (strides ", t.strides(), ")");
    out.push_back({t.data_ptr(), t.numel(), dtype_code(t, name)});
    tensors.push_back(&t);
  }
}

}  // namespace

// grads, norm, stream
PyObject* grad_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 3);
  const Tensor* given = optional(a[1], "norm");
  Place place;
  std::vector<fp8bs_grad> grads;
  std::vector<const Tensor*> tensors;
  read_grads(a[0], "grads", place, grads, tensors);
  place.add(given);
  TORCH_CHECK_VALUE(!tensors.empty(), "no gradients");
  TORCH_CHECK_VALUE(grads.size() <= 65536, "too many gradients: ", grads.size());
  const int32_t count = static_cast<int32_t>(grads.size());
  const c10::DeviceGuard guard(place.device());
  const int64_t bytes = fp8_grad_norm_workspace(grads.data(), count);
  if (bytes < 0) return refused(fp8_grad_norm(grads.data(), count, nullptr, nullptr, 0, nullptr));
  const Tensor norm = output(given, *tensors[0], {1}, at::kFloat, "norm");
  Tensor room;
  if (bytes > 0) room = output(nullptr, *tensors[0], {bytes}, at::kByte, "workspace");
  if (fp8bs_status st = fp8_grad_norm(grads.data(), count, ptr<float>(norm), ptr<void>(room), bytes, place.stream(a[2]))) return refused(st);
  return THPVariable_Wrap(norm);
  END_HANDLE_TH_ERRORS
}

// grads, norm, max_norm, outs, stream
PyObject* grad_clip(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 5);
  const Tensor& norm = tensor(a[1], "norm");
  Place place;
  std::vector<fp8bs_grad> grads, outs;
  std::vector<const Tensor*> tensors, written;
  read_grads(a[0], "grads", place, grads, tensors);
  place.add(norm);
  dense(norm, {1}, at::kFloat, "norm");
  const bool apart = a[3] != Py_None;
  if (apart) {
    read_grads(a[3], "outs", place, outs, written);
    TORCH_CHECK_VALUE(outs.size() == grads.size(), "outs has ", outs.size(), " tensors, grads ", grads.size());
    for (size_t i = 0; i < outs.size(); ++i) {
      need(*written[i], tensors[i]->sizes(), tensors[i]->scalar_type(), "outs");
      TORCH_CHECK_VALUE(same_order(*written[i], *tensors[i]), "outs[", i, "] has other strides than grads[", i, "]");
    }
  }
  TORCH_CHECK_VALUE(grads.size() <= 65536, "too many gradients: ", grads.size());
  const c10::DeviceGuard guard(place.device());
  if (fp8bs_status st = fp8_grad_clip(grads.data(), apart ? outs.data() : nullptr, static_cast<int32_t>(grads.size()), ptr<float>(norm),
                                      real(a[2]), place.stream(a[4])))
    return refused(st);
  PyObject* result = apart ? a[3] : a[0];
  Py_INCREF(result);
  return result;
  END_HANDLE_TH_ERRORS
}

}  // namespace marshal
