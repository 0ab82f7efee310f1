// _marshal: the argument marshalling of the decoder layer's operators for
// PyTorch, as a CPython module (host code only; the kernels are in
// libfp8bs.so, which this links).  A decode step makes these calls in every
// layer with kernels of 5 to 10 us, so reading a tensor's fields through
// Python attributes would cost as much as the work (13 us a call so,
// 5 to 9 us through this module).
//
// Every function takes its arguments by position, checks tensors as the
// binding's other functions do (TypeError and ValueError), allocates what is
// not given, and returns the outputs, or the library's status where that is
// not FP8BS_OK.  The last argument is a function that gives the current
// stream's handle, called when the tensors have been checked.
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "fp8bs_decoder.h"

namespace {

using at::Tensor;

const Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}
const Tensor* optional(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
int32_t narrow(PyObject* o) {
  const int64_t v = integer(o);
  TORCH_CHECK_VALUE(v >= INT32_MIN && v <= INT32_MAX, "an integer argument is out of range: ", v);
  return static_cast<int32_t>(v);
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
hipStream_t stream(PyObject* current) {
  THPObjectPtr handle(PyObject_CallNoArgs(current));
  if (!handle) throw python_error();
  void* p = PyLong_AsVoidPtr(handle);
  if (!p && PyErr_Occurred()) throw python_error();
  return static_cast<hipStream_t>(p);
}

void on_gpu(const Tensor& t) { TORCH_CHECK_VALUE(t.is_cuda(), "all tensors must be on the GPU"); }
void need(const Tensor& t, at::IntArrayRef shape, at::ScalarType dtype, const char* name) {
  TORCH_CHECK_VALUE(t.sizes() == shape, name, " has shape ", t.sizes(), ", expected ", shape);
  TORCH_CHECK_TYPE(t.scalar_type() == dtype, name, " must be ", dtype, ", got ", t.scalar_type());
}
void dense(const Tensor& t, at::IntArrayRef shape, at::ScalarType dtype, const char* name) {
  need(t, shape, dtype, name);
  TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
}
// `given` checked, or a new tensor.
Tensor output(const Tensor* given, const Tensor& like, at::IntArrayRef shape, at::ScalarType dtype, const char* name) {
  if (!given) return at::empty(shape, like.options().dtype(dtype).requires_grad(false));
  on_gpu(*given);
  dense(*given, shape, dtype, name);
  return *given;
}
int32_t dtype_code(const Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return FP8BS_BF16;
  TORCH_CHECK_TYPE(t.scalar_type() == at::kFloat, name, " must be bfloat16 or float32, got ", t.scalar_type());
  return FP8BS_F32;
}
// Pitch of a matrix with unit column stride.
int64_t pitch(const Tensor& t, const char* name) {
  TORCH_CHECK_VALUE(t.dim() == 2, name, " must have two dimensions");
  TORCH_CHECK_VALUE(t.size(1) <= 1 || t.stride(1) == 1, name, " must have unit column stride");
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

fp8bs_kv_cache read_cache(PyObject* const* a) {
  const Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &ks = tensor(a[2], "k_scale"), &vs = tensor(a[3], "v_scale");
  TORCH_CHECK_VALUE(k.dim() == 4, "k must be [pages, kv_heads, page_size, head_dim], got ", k.sizes());
  dense(k, k.sizes(), at::kByte, "k");
  dense(v, k.sizes(), at::kByte, "v");
  dense(ks, k.sizes().slice(0, 2), at::kFloat, "k_scale");
  dense(vs, k.sizes().slice(0, 2), at::kFloat, "v_scale");
  for (const Tensor* t : {&k, &v, &ks, &vs}) on_gpu(*t);
  return {static_cast<uint8_t*>(k.data_ptr()), static_cast<uint8_t*>(v.data_ptr()), static_cast<float*>(ks.data_ptr()),
          static_cast<float*>(vs.data_ptr()), k.size(0), k.size(1), k.size(2), k.size(3)};
}
// A KVCache's four tensors, whose storages and sizes are read at each call
// (resize_ and set_ change them under a tensor); or the header's struct as
// bytes, of a caller whose memory is no tensor's.
fp8bs_kv_cache unpack_cache(PyObject* o) {
  if (PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 4) return read_cache(&PyTuple_GET_ITEM(o, 0));
  fp8bs_kv_cache c;
  TORCH_CHECK_TYPE(PyBytes_Check(o) && PyBytes_GET_SIZE(o) == sizeof c, "cache must be a KVCache");
  std::memcpy(&c, PyBytes_AS_STRING(o), sizeof c);
  return c;
}
fp8bs_kv_batch read_batch(PyObject* cu_o, PyObject* lens_o, PyObject* table_o, int64_t tokens, int64_t max_new, int64_t max_len) {
  const Tensor &cu = tensor(cu_o, "cu"), &lens = tensor(lens_o, "seq_lens"), &table = tensor(table_o, "block_table");
  TORCH_CHECK_TYPE(cu.scalar_type() == at::kInt && lens.scalar_type() == at::kInt && table.scalar_type() == at::kInt,
                   "cu, seq_lens and block_table must be int32");
  TORCH_CHECK_VALUE(lens.dim() == 1 && cu.dim() == 1 && cu.size(0) == lens.size(0) + 1 && table.dim() == 2 && table.size(0) == lens.size(0),
                    "cu [B+1], seq_lens [B] and block_table [B, width] expected, got ", cu.sizes(), ", ", lens.sizes(), ", ", table.sizes());
  on_gpu(cu);
  on_gpu(lens);
  on_gpu(table);
  const int64_t n = lens.size(0), width = table.size(1);
  TORCH_CHECK_VALUE(cu.is_contiguous() && lens.is_contiguous() && (width <= 1 || table.stride(1) == 1),
                    "cu and seq_lens must be contiguous, block_table must have unit column stride");
  return {static_cast<const int32_t*>(cu.data_ptr()), static_cast<const int32_t*>(lens.data_ptr()),
          static_cast<const int32_t*>(table.data_ptr()), n > 1 ? table.stride(0) : width, width, n, tokens, max_new, max_len};
}

struct Rows {
  const void* p;
  int64_t ld, hs;
};
// A bfloat16 [tokens, heads, dim] tensor.
Rows rows(const Tensor& t, int64_t tokens, int64_t heads, int64_t dim, const char* name) {
  TORCH_CHECK_TYPE(t.scalar_type() == at::kBFloat16, name, " must be bfloat16, got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.dim() == 3 && t.size(0) == tokens && t.size(1) == heads && t.size(2) == dim, name, " has shape ", t.sizes(),
                    ", expected [", tokens, ", ", heads, ", ", dim, "]");
  on_gpu(t);
  TORCH_CHECK_VALUE(t.stride(2) == 1, name, " must have unit stride within a head");
  return {t.data_ptr(), tokens > 1 ? t.stride(0) : heads * dim, heads > 1 ? t.stride(1) : dim};
}

PyObject* wrap(std::initializer_list<Tensor> ts) {
  THPObjectPtr tuple(PyTuple_New(static_cast<Py_ssize_t>(ts.size())));
  if (!tuple) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) PyTuple_SET_ITEM(tuple.get(), i++, THPVariable_Wrap(t));
  return tuple.release();
}
PyObject* refused(fp8bs_status st) { return PyLong_FromLong(st); }
void arity(Py_ssize_t got, Py_ssize_t want) { TORCH_CHECK_TYPE(got == want, want, " arguments expected, got ", got); }

PyObject* cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 4);
  read_cache(a);
  return PyTuple_Pack(4, a[0], a[1], a[2], a[3]);
  END_HANDLE_TH_ERRORS
}

// q, k, v, cache, cu, seq_lens, block_table, max_new, rope, layout, q_weight, k_weight, eps, q_out, stream
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 15);
  const Tensor* q = optional(a[0], "q");
  const Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
  const fp8bs_kv_cache c = unpack_cache(a[3]);
  TORCH_CHECK_VALUE(k.dim() == 3, "k must be [tokens, heads, head_dim], got ", k.sizes());
  const int64_t tokens = k.size(0);
  fp8bs_kv_append_args args{};
  const Rows kr = rows(k, tokens, c.kv_heads, c.head_dim, "k"), vr = rows(v, tokens, c.kv_heads, c.head_dim, "v");
  args.k = kr.p, args.ld_k = kr.ld, args.hs_k = kr.hs;
  args.v = vr.p, args.ld_v = vr.ld, args.hs_v = vr.hs;
  if (const Tensor* rope = optional(a[8], "rope")) {
    TORCH_CHECK_VALUE(rope->scalar_type() == at::kFloat && rope->dim() == 2 && rope->is_contiguous(),
                      "rope must be a contiguous float32 [positions, rot] table");
    on_gpu(*rope);
    args.rope = static_cast<const float*>(rope->data_ptr());
    args.rope_rows = rope->size(0);
    args.rot = rope->size(1);
  }
  args.rope_layout = integer(a[9]);
  for (int i = 0; i < 2; ++i) {
    const char* name = i ? "k_weight" : "q_weight";
    if (const Tensor* w = optional(a[10 + i], name)) {
      on_gpu(*w);
      dense(*w, {c.head_dim}, at::kBFloat16, name);
      (i ? args.k_weight : args.q_weight) = w->data_ptr();
    }
  }
  args.eps = real(a[12]);
  const fp8bs_kv_batch batch = read_batch(a[4], a[5], a[6], tokens, integer(a[7]), int64_t(1) << 30);
  Tensor out;
  if (q) {
    TORCH_CHECK_VALUE(q->dim() == 3, "q must be [tokens, heads, head_dim], got ", q->sizes());
    args.q_heads = q->size(1);
    const Rows qr = rows(*q, tokens, args.q_heads, c.head_dim, "q");
    args.q = qr.p, args.ld_q = qr.ld, args.hs_q = qr.hs;
    out = output(optional(a[13], "q_out"), *q, {tokens, args.q_heads, c.head_dim}, at::kBFloat16, "q_out");
    args.q_out = out.data_ptr();
  }
  if (fp8bs_status st = fp8_kv_append(&c, &batch, &args, stream(a[14]))) return refused(st);
  if (q) return THPVariable_Wrap(out);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// q, cache, cu, seq_lens, block_table, max_new, max_len, window, softmax_scale or None, return_lse, out, stream
PyObject* kv_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 12);
  const Tensor& q = tensor(a[0], "q");
  const fp8bs_kv_cache c = unpack_cache(a[1]);
  TORCH_CHECK_VALUE(q.dim() == 3 && q.size(2) == c.head_dim, "q has shape ", q.sizes(), ", the cache head_dim ", c.head_dim);
  const int64_t tokens = q.size(0), heads = q.size(1);
  const Rows r = rows(q, tokens, heads, c.head_dim, "q");
  const fp8bs_kv_batch batch = read_batch(a[2], a[3], a[4], tokens, integer(a[5]), integer(a[6]));
  fp8bs_kv_attention_args args{};
  args.q = r.p, args.ld_q = r.ld, args.hs_q = r.hs;
  args.q_heads = heads;
  args.window = integer(a[7]);
  args.softmax_scale = a[8] == Py_None ? 1.0 / std::sqrt(double(c.head_dim)) : real(a[8]);
  const int with_lse = PyObject_IsTrue(a[9]);
  if (with_lse < 0) throw python_error();
  const Tensor out = output(optional(a[10], "out"), q, {tokens, heads, c.head_dim}, at::kBFloat16, "out");
  args.out = out.data_ptr();
  Tensor lse, room;
  if (with_lse) {
    lse = output(nullptr, q, {tokens, heads}, at::kFloat, "lse");
    args.lse = static_cast<float*>(lse.data_ptr());
  }
  const int64_t bytes = fp8_kv_attention_workspace(&c, &batch, &args);
  if (bytes > 0) {
    room = output(nullptr, q, {bytes}, at::kByte, "workspace");
    args.workspace = room.data_ptr();
    args.workspace_bytes = bytes;
  }
  if (fp8bs_status st = fp8_kv_attention(&c, &batch, &args, stream(a[11]))) return refused(st);
  return with_lse ? wrap({out, lse}) : THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// logits, top_k, score, bias, groups, top_groups or None, renormalize, scale, ids, weights, stream
PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 11);
  const Tensor& x = tensor(a[0], "logits");
  on_gpu(x);
  const int64_t ld = pitch(x, "logits"), tokens = x.size(0), experts = x.size(1);
  const int32_t dtype = dtype_code(x, "logits"), top_k = narrow(a[1]), groups = narrow(a[4]);
  const float* bias = nullptr;
  if (const Tensor* b = optional(a[3], "bias")) {
    on_gpu(*b);
    dense(*b, {experts}, at::kFloat, "bias");
    bias = static_cast<const float*>(b->data_ptr());
  }
  const int renorm = PyObject_IsTrue(a[6]);
  if (renorm < 0) throw python_error();
  const int64_t k = std::clamp<int64_t>(top_k, 0, experts);     // more is refused below: nothing is allocated for it
  const Tensor ids = output(optional(a[8], "ids"), x, {tokens, k}, at::kInt, "ids");
  const Tensor w = output(optional(a[9], "weights"), x, {tokens, k}, at::kFloat, "weights");
  if (fp8bs_status st = fp8_moe_route(x.data_ptr(), dtype, tokens, experts, ld, narrow(a[2]), bias, groups,
                                      a[5] == Py_None ? groups : narrow(a[5]), top_k, renorm, real(a[7]),
                                      static_cast<int32_t*>(ids.data_ptr()), static_cast<float*>(w.data_ptr()), stream(a[10])))
    return refused(st);
  return wrap({ids, w});
  END_HANDLE_TH_ERRORS
}

// grad, logits, ids, score, renormalize, scale, dlogits, stream
PyObject* moe_route_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 8);
  const Tensor &g = tensor(a[0], "grad"), &x = tensor(a[1], "logits"), &ids = tensor(a[2], "ids");
  for (const Tensor* t : {&g, &x, &ids}) on_gpu(*t);
  const int64_t ld = pitch(x, "logits"), tokens = x.size(0), experts = x.size(1);
  const int32_t dtype = dtype_code(x, "logits");
  TORCH_CHECK_VALUE(ids.dim() == 2, "ids must be [tokens, top_k], got ", ids.sizes());
  const int64_t top_k = ids.size(1);
  dense(ids, {tokens, top_k}, at::kInt, "ids");
  dense(g, {tokens, top_k}, at::kFloat, "grad");
  const int renorm = PyObject_IsTrue(a[4]);
  if (renorm < 0) throw python_error();
  Tensor d;
  if (const Tensor* given = optional(a[6], "dlogits")) {
    on_gpu(*given);
    need(*given, {tokens, experts}, x.scalar_type(), "dlogits");
    d = *given;
  } else {
    d = output(nullptr, x, {tokens, experts}, x.scalar_type(), "dlogits");
  }
  TORCH_CHECK_VALUE(top_k <= INT32_MAX, "ids has too many columns");
  if (fp8bs_status st = fp8_moe_route_backward(static_cast<const float*>(g.data_ptr()), x.data_ptr(), dtype, tokens, experts, ld,
                                               static_cast<const int32_t*>(ids.data_ptr()), static_cast<int32_t>(top_k), narrow(a[3]), renorm,
                                               real(a[5]), d.data_ptr(), pitch(d, "dlogits"), stream(a[7])))
    return refused(st);
  return THPVariable_Wrap(d);
  END_HANDLE_TH_ERRORS
}

// x, ids, experts, q, scale, stream
PyObject* moe_dispatch(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 6);
  const Tensor &x = tensor(a[0], "x"), &ids = tensor(a[1], "ids");
  const int64_t ld = pitch(x, "x"), tokens = x.size(0), cols = x.size(1);
  TORCH_CHECK_VALUE(ids.dim() == 2 && ids.size(0) == tokens && ids.scalar_type() == at::kInt && ids.is_contiguous(),
                    "ids must be a contiguous int32 [T, top_k] tensor");
  on_gpu(x);
  on_gpu(ids);
  const int32_t dtype = dtype_code(x, "x"), experts = narrow(a[2]);
  const int64_t k = ids.size(1), rows = tokens * k;
  TORCH_CHECK_VALUE(k <= INT32_MAX, "ids has too many columns");
  auto i32 = [](const Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); };
  const int64_t bytes = fp8_moe_dispatch_workspace(tokens, experts, static_cast<int32_t>(k));
  if (bytes < 0)                                                // refused before anything is allocated
    return refused(fp8_moe_dispatch(x.data_ptr(), dtype, tokens, cols, ld, i32(ids), static_cast<int32_t>(k), experts, nullptr, nullptr, nullptr,
                                    nullptr, nullptr, nullptr, 0, stream(a[5])));
  const Tensor q = output(optional(a[3], "q"), x, {rows, cols}, at::kByte, "q");
  const Tensor scale = output(optional(a[4], "scale"), x, {rows, cols / 128}, at::kFloat, "scale");
  const Tensor offsets = output(nullptr, ids, {experts + int64_t(1)}, at::kInt, "offsets");
  const Tensor order = output(nullptr, ids, {rows}, at::kInt, "order");
  const Tensor position = output(nullptr, ids, {tokens, k}, at::kInt, "position");
  Tensor room;
  if (bytes > 0) room = output(nullptr, ids, {bytes}, at::kByte, "workspace");
  if (fp8bs_status st = fp8_moe_dispatch(x.data_ptr(), dtype, tokens, cols, ld, i32(ids), static_cast<int32_t>(k), experts,
                                         static_cast<uint8_t*>(q.data_ptr()), static_cast<float*>(scale.data_ptr()), i32(offsets), i32(order),
                                         i32(position), bytes > 0 ? room.data_ptr() : nullptr, std::max<int64_t>(bytes, 0), stream(a[5])))
    return refused(st);
  return wrap({q, scale, offsets, order, position});
  END_HANDLE_TH_ERRORS
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyMethodDef method(const char* name, Fast f) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {
    method("cache", cache),
    method("kv_append", kv_append),
    method("kv_attention", kv_attention),
    method("moe_route", moe_route),
    method("moe_route_backward", moe_route_backward),
    method("moe_dispatch", moe_dispatch),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
