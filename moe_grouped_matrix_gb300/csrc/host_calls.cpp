// The binding's short way to the MoE operators: for arguments that are right as
// they stand (dense CUDA tensors of the expected types and sizes, the current
// stream) one call from Python checks them, allocates the results and calls the C
// ABI.  At decoding sizes an operator is a few microseconds on the GPU, and this
// work done in Python costs more: combine() takes the host 10 us in Python, 3 here.
//
// Every function returns None for any other arguments, and moe.py then goes
// through them one by one and says what is wrong or handles the case; an int is
// the C ABI's status, not GMM_OK.  The C ABI's functions come from the library
// that the binding has loaded, by address.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "../../include/libgmm_moe.h"

namespace {

// In the order moe.py gives the addresses.
struct Calls {
  decltype(&gmm_route) route;
  decltype(&gmm_route_backward) route_backward;
  decltype(&gmm_sort_by_expert) sort;
  decltype(&gmm_dispatch) dispatch;
  decltype(&gmm_combine) combine;
  decltype(&gmm_combine_backward) combine_backward;
  decltype(&gmm_quantize_fp4) quantize;
  decltype(&gmm_dequantize_fp4) dequantize;
  decltype(&gmm_fp4) fp4;
} g_calls{};

using at::Tensor;
constexpr auto kF32 = at::kFloat;
constexpr auto kBF16 = at::kBFloat16;
constexpr auto kI32 = at::kInt;
constexpr auto kU8 = at::kByte;

// A tensor as it stands: not of a subclass, whose operations are its own.
const Tensor* tensor(PyObject* o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

bool dense(const Tensor* t, at::ScalarType type, at::IntArrayRef shape) {
  return t != nullptr && t->is_cuda() && t->scalar_type() == type && t->sizes() == shape && t->is_contiguous();
}

// Whether the tensors (NULL: none given) are the current device's: the C ABI launches there.
bool here(std::initializer_list<const Tensor*> all) {
  c10::DeviceIndex now = -1;
  if (c10::cuda::GetDevice(&now) != cudaSuccess) return false;
  for (const Tensor* t : all)
    if (t != nullptr && t->get_device() != now) return false;
  return true;
}

int code_of(const Tensor& t) { return t.scalar_type() == kF32 ? GMM_DTYPE_F32 : GMM_DTYPE_BF16; }
bool is_float(const Tensor& t) { return t.scalar_type() == kF32 || t.scalar_type() == kBF16; }

// The row pitch of a 2-D CUDA tensor of floats with dense rows; -1 for any other.
int64_t pitch(const Tensor* t) {
  if (t == nullptr || !t->is_cuda() || t->dim() != 2 || !is_float(*t)) return -1;
  const int64_t n = t->size(0), d = t->size(1);
  if (d > 1 && t->stride(1) != 1) return -1;
  if (n <= 1) return d;
  return t->stride(0) >= d ? t->stride(0) : -1;
}

// The CUDA allocation itself, without at::empty()'s way through the dispatcher (0.7 us a tensor).
Tensor empty(at::IntArrayRef shape, at::ScalarType type, const Tensor& like) {
  return Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}

void* stream_of(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

template <class T>
T* ptr(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
template <class T>
T* ptr_or_null(const Tensor* t) {
  return t == nullptr ? nullptr : static_cast<T*>(t->data_ptr());
}

PyObject* no_answer() { Py_RETURN_NONE; }

PyObject* answer(int status, std::initializer_list<Tensor> out) {
  if (status != GMM_OK) return PyLong_FromLong(status);
  if (out.size() == 1) return THPVariable_Wrap(*out.begin());
  PyObject* tuple = PyTuple_New(Py_ssize_t(out.size()));
  if (tuple == nullptr) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor& t : out) {
    PyObject* o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
    if (o == nullptr) {
      Py_DECREF(tuple);
      return nullptr;
    }
    PyTuple_SET_ITEM(tuple, i++, o);
  }
  return tuple;
}

// An int argument in [lo, hi]; `ok` turns false for any other.
int64_t integer(PyObject* o, int64_t lo, int64_t hi, bool* ok) {
  if (!PyLong_CheckExact(o)) {
    *ok = false;
    return 0;
  }
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &over);
  if (over != 0 || v < lo || v > hi) *ok = false;
  return v;
}

// No C++ exception (an allocation that fails) crosses into Python.  While a dispatch mode is on, which
// empty() below would pass by, there is no short way.
template <class F>
PyObject* guarded(F&& f) {
  try {
    if (c10::impl::TorchDispatchModeTLS::any_modes_set()) return no_answer();
    return f();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// route(logits, topk, score, renormalize, scale, select_bias, token_mask) -> (weights, experts)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 7) return no_answer();
    const Tensor *logits = tensor(a[0]), *bias = tensor(a[5]), *mask = tensor(a[6]);
    const int64_t ld = pitch(logits);
    if (ld < 0) return no_answer();
    const int64_t tokens = logits->size(0), experts = logits->size(1);
    bool ok = experts <= GMM_MAX_GROUPS && PyFloat_CheckExact(a[4]);
    const int64_t topk = integer(a[1], 1, experts < GMM_MAX_TOPK ? experts : GMM_MAX_TOPK, &ok);
    const int64_t score = integer(a[2], 0, GMM_SCORE_BIASED | 1, &ok), renormalize = integer(a[3], 0, 1, &ok);
    ok = ok && (a[5] == Py_None || dense(bias, kF32, {experts}));
    ok = ok && (a[6] == Py_None || dense(mask, at::kBool, {tokens}) || dense(mask, kU8, {tokens}));
    if (!ok || !here({logits, bias, mask})) return no_answer();
    Tensor weights = empty({tokens, topk}, kF32, *logits), chosen = empty({tokens, topk}, kI32, *logits);
    const int st = g_calls.route(logits->data_ptr(), code_of(*logits), tokens, int32_t(experts), ld, int32_t(topk),
                                 int(score), int(renormalize), float(PyFloat_AS_DOUBLE(a[4])),
                                 ptr_or_null<float>(bias), ptr_or_null<uint8_t>(mask), ptr<float>(weights),
                                 ptr<int32_t>(chosen), stream_of(*logits));
    return answer(st, {weights, chosen});
  });
}

// route_backward(dweights, experts, logits, score, renormalize, scale) -> dlogits
PyObject* route_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 6) return no_answer();
    const Tensor *dweights = tensor(a[0]), *chosen = tensor(a[1]), *logits = tensor(a[2]);
    const int64_t ld = pitch(logits);
    if (ld < 0 || chosen == nullptr || chosen->dim() != 2 || !PyFloat_CheckExact(a[5])) return no_answer();
    const int64_t tokens = logits->size(0), experts = logits->size(1), topk = chosen->size(1);
    bool ok = experts <= GMM_MAX_GROUPS && topk >= 1 && topk <= GMM_MAX_TOPK && topk <= experts;
    const int64_t score = integer(a[3], 0, 1, &ok), renormalize = integer(a[4], 0, 1, &ok);
    if (!ok || !dense(chosen, kI32, {tokens, topk}) || !dense(dweights, kF32, {tokens, topk}) ||
        !here({dweights, chosen, logits}))
      return no_answer();
    Tensor dlogits = empty({tokens, experts}, logits->scalar_type(), *logits);
    const int st = g_calls.route_backward(ptr<float>(*dweights), ptr<int32_t>(*chosen), logits->data_ptr(),
                                          code_of(*logits), tokens, int32_t(experts), ld, int32_t(topk), int(score),
                                          int(renormalize), float(PyFloat_AS_DOUBLE(a[5])), dlogits.data_ptr(),
                                          stream_of(*logits));
    return answer(st, {dlogits});
  });
}

// sort_by_expert(experts, num_experts) -> (group_sizes, rows, source)
PyObject* sort_by_expert(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 2) return no_answer();
    const Tensor* experts = tensor(a[0]);
    if (experts == nullptr || experts->dim() != 2) return no_answer();
    const int64_t tokens = experts->size(0), topk = experts->size(1);
    bool ok = dense(experts, kI32, {tokens, topk}) && topk >= 1 && topk <= GMM_MAX_TOPK;
    const int64_t num = integer(a[1], 1, GMM_MAX_GROUPS, &ok);
    if (!ok || !here({experts})) return no_answer();
    Tensor sizes = empty({num}, kI32, *experts), rows = empty({tokens, topk}, kI32, *experts),
           source = empty({tokens * topk}, kI32, *experts);
    const int st = g_calls.sort(ptr<int32_t>(*experts), tokens, int32_t(topk), int32_t(num), ptr<int32_t>(sizes),
                                ptr<int32_t>(rows), ptr<int32_t>(source), stream_of(*experts));
    return answer(st, {sizes, rows, source});
  });
}

// The tokens and slots of an order's rows and source; false where they are not one.
bool order_of(const Tensor* rows, const Tensor* source, int64_t* tokens, int64_t* topk) {
  if (rows == nullptr || rows->dim() != 2) return false;
  *tokens = rows->size(0), *topk = rows->size(1);
  return *topk >= 1 && *topk <= GMM_MAX_TOPK && dense(rows, kI32, {*tokens, *topk}) &&
         dense(source, kI32, {*tokens * *topk});
}

// dispatch(x, rows, source) -> rows of x
PyObject* dispatch(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 3) return no_answer();
    const Tensor *x = tensor(a[0]), *rows = tensor(a[1]), *source = tensor(a[2]);
    const int64_t ld = pitch(x);
    int64_t tokens, topk;
    if (ld < 0 || !order_of(rows, source, &tokens, &topk) || x->size(0) != tokens || !here({x, rows, source}))
      return no_answer();
    const int64_t d = x->size(1);
    Tensor out = empty({tokens * topk, d}, x->scalar_type(), *x);
    const int st = g_calls.dispatch(x->data_ptr(), code_of(*x), tokens, d, ld, int32_t(topk), ptr<int32_t>(*rows),
                                    ptr<int32_t>(*source), out.data_ptr(), stream_of(*x));
    return answer(st, {out});
  });
}

// combine(in, rows, source, weights) -> out
PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 4) return no_answer();
    const Tensor *in = tensor(a[0]), *rows = tensor(a[1]), *source = tensor(a[2]), *weights = tensor(a[3]);
    int64_t tokens, topk;
    if (!order_of(rows, source, &tokens, &topk) || in == nullptr || in->dim() != 2 || !is_float(*in))
      return no_answer();
    const int64_t d = in->size(1);
    if (!dense(in, in->scalar_type(), {tokens * topk, d}) ||
        (a[3] != Py_None && !dense(weights, kF32, {tokens, topk})) || !here({in, rows, source, weights}))
      return no_answer();
    Tensor out = empty({tokens, d}, in->scalar_type(), *in);
    const int st = g_calls.combine(in->data_ptr(), code_of(*in), tokens, d, int32_t(topk), ptr<int32_t>(*rows),
                                   ptr_or_null<float>(weights), out.data_ptr(), stream_of(*in));
    return answer(st, {out});
  });
}

// combine_backward(dout, in, rows, source, weights) -> (din, dweights)
PyObject* combine_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 5) return no_answer();
    const Tensor *dout = tensor(a[0]), *in = tensor(a[1]), *rows = tensor(a[2]), *source = tensor(a[3]),
                 *weights = tensor(a[4]);
    int64_t tokens, topk;
    if (!order_of(rows, source, &tokens, &topk) || in == nullptr || in->dim() != 2 || !is_float(*in))
      return no_answer();
    const int64_t d = in->size(1);
    if (!dense(in, in->scalar_type(), {tokens * topk, d}) || !dense(dout, in->scalar_type(), {tokens, d}) ||
        !dense(weights, kF32, {tokens, topk}) || !here({dout, in, rows, source, weights}))
      return no_answer();
    Tensor din = empty({tokens * topk, d}, in->scalar_type(), *in), dweights = empty({tokens, topk}, kF32, *in);
    const int st = g_calls.combine_backward(dout->data_ptr(), in->data_ptr(), code_of(*in), tokens, d, int32_t(topk),
                                            ptr<int32_t>(*rows), ptr<int32_t>(*source), ptr<float>(*weights),
                                            din.data_ptr(), ptr<float>(dweights), stream_of(*in));
    return answer(st, {din, dweights});
  });
}

int64_t windows_of(int64_t k, int64_t format) {
  const int64_t window = format == GMM_FP4_NVFP4 ? 256 : 512;
  return (k + window - 1) / window;
}

// quantize_fp4(x, format, rows, source) -> (codes, block_scale, row_scale or None); 2-D x
PyObject* quantize_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 4) return no_answer();
    const Tensor *x = tensor(a[0]), *rows = tensor(a[2]), *source = tensor(a[3]);
    const int64_t ld = pitch(x);
    if (ld < 0) return no_answer();
    bool ok = true;
    const int64_t format = integer(a[1], 0, 1, &ok), tokens = x->size(0), k = x->size(1);
    int64_t order_tokens = tokens, topk = 1;
    if (a[2] != Py_None) ok = ok && order_of(rows, source, &order_tokens, &topk) && order_tokens == tokens;
    if (!ok || k < 32 || k % 32 != 0 || !here({x, rows, source})) return no_answer();
    const int64_t out_rows = tokens * topk;
    Tensor codes = empty({out_rows, k / 2}, kU8, *x), scale = empty({windows_of(k, format), out_rows, 16}, kU8, *x), row;
    if (format == GMM_FP4_NVFP4) row = empty({out_rows}, kF32, *x);
    const int st = g_calls.quantize(x->data_ptr(), code_of(*x), 1, tokens, k, ld, int(format),
                                    ptr_or_null<int32_t>(rows), ptr_or_null<int32_t>(source), int32_t(topk),
                                    codes.data_ptr(), scale.data_ptr(),
                                    row.defined() ? ptr<float>(row) : nullptr, stream_of(*x));
    return answer(st, {codes, scale, row});
  });
}

// An Fp4Tensor's parts with `lead` leading dimensions: its sizes, or false.
bool fp4_of(const Tensor* codes, const Tensor* scale, const Tensor* row, bool has_row, int64_t format, int lead,
            int64_t* batch, int64_t* rows, int64_t* k) {
  if (codes == nullptr || codes->dim() != lead + 2) return false;
  *batch = lead != 0 ? codes->size(0) : 1;
  *rows = codes->size(lead), *k = 2 * codes->size(lead + 1);
  const int64_t w = windows_of(*k, format);
  if (*k < 32 || *k % 32 != 0 || has_row != (format == GMM_FP4_NVFP4)) return false;
  return lead != 0 ? dense(codes, kU8, {*batch, *rows, *k / 2}) && dense(scale, kU8, {*batch, w, *rows, 16}) &&
                         (!has_row || dense(row, kF32, {*batch, *rows}))
                   : dense(codes, kU8, {*rows, *k / 2}) && dense(scale, kU8, {w, *rows, 16}) &&
                         (!has_row || dense(row, kF32, {*rows}));
}

// dequantize_fp4(codes, block_scale, row_scale, format, out is f32) -> values; 2-D
PyObject* dequantize_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 5) return no_answer();
    const Tensor *codes = tensor(a[0]), *scale = tensor(a[1]), *row = tensor(a[2]);
    bool ok = true;
    const int64_t format = integer(a[3], 0, 1, &ok), f32 = integer(a[4], 0, 1, &ok);
    int64_t batch, rows, k;
    if (!ok || !fp4_of(codes, scale, row, a[2] != Py_None, format, 0, &batch, &rows, &k) || !here({codes, scale, row}))
      return no_answer();
    Tensor out = empty({rows, k}, f32 ? kF32 : kBF16, *codes);
    const int st = g_calls.dequantize(codes->data_ptr(), scale->data_ptr(), ptr_or_null<float>(row), int(format), 1,
                                      rows, k, out.data_ptr(), code_of(out), stream_of(*codes));
    return answer(st, {out});
  });
}

// gmm_fp4(lhs codes, scale, row, rhs codes, scale, row, format, group_sizes, group_offset, out is f32,
// workspace) -> out; no bias
PyObject* gmm_fp4_call(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 11) return no_answer();
    const Tensor *lc = tensor(a[0]), *ls = tensor(a[1]), *lr = tensor(a[2]), *rc = tensor(a[3]), *rs = tensor(a[4]),
                 *rr = tensor(a[5]), *sizes = tensor(a[7]), *ws = tensor(a[10]);
    bool ok = ws != nullptr && ws->is_cuda() && ws->scalar_type() == kU8 && ws->is_contiguous();
    const int64_t format = integer(a[6], 0, 1, &ok), offset = integer(a[8], 0, GMM_MAX_GROUPS, &ok),
                  f32 = integer(a[9], 0, 1, &ok);
    int64_t one, m, k, local, nn, kr;
    ok = ok && fp4_of(lc, ls, lr, a[2] != Py_None, format, 0, &one, &m, &k) &&
         fp4_of(rc, rs, rr, a[5] != Py_None, format, 1, &local, &nn, &kr) && k == kr;
    if (!ok || sizes == nullptr || sizes->dim() != 1 || !dense(sizes, kI32, {sizes->size(0)}) ||
        sizes->size(0) > GMM_MAX_GROUPS || local > GMM_MAX_GROUPS ||
        !here({lc, ls, lr, rc, rs, rr, sizes, ws}))
      return no_answer();
    Tensor out = empty({m, nn}, f32 ? kF32 : kBF16, *lc);
    const int st = g_calls.fp4(lc->data_ptr(), ls->data_ptr(), ptr_or_null<float>(lr), m, k, rc->data_ptr(),
                               rs->data_ptr(), ptr_or_null<float>(rr), int(format), int32_t(local), nn,
                               ptr<int32_t>(*sizes), int32_t(sizes->size(0)), int32_t(offset), nullptr,
                               GMM_DTYPE_BF16, out.data_ptr(), code_of(out), ws->data_ptr(), size_t(ws->numel()),
                               stream_of(*lc));
    return answer(st, {out});
  });
}

// bind(addresses of the C ABI's functions, in the order of Calls)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void** to = reinterpret_cast<void**>(&g_calls);
  if (n != Py_ssize_t(sizeof(Calls) / sizeof(void*))) {
    PyErr_SetString(PyExc_TypeError, "bind: wrong number of functions");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < n; ++i) {
    to[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  Py_RETURN_NONE;
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyMethodDef method(const char* name, Fast f) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method("bind", bind),
                           method("route", route),
                           method("route_backward", route_backward),
                           method("sort_by_expert", sort_by_expert),
                           method("dispatch", dispatch),
                           method("combine", combine),
                           method("combine_backward", combine_backward),
                           method("quantize_fp4", quantize_fp4),
                           method("dequantize_fp4", dequantize_fp4),
                           method("gmm_fp4", gmm_fp4_call),
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_host_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyObject* PyInit__host_calls(void) { return PyModule_Create(&g_module); }
