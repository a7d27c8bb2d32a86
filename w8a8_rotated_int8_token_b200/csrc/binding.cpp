// The checks and packing of the rope and cache calls of the Python binding, natively.
//
// A decoding step makes these calls once per layer, and in Python the checks of a
// dozen tensor arguments cost more than the launch. Each function here does what its
// namesake in __init__.py does for the plain case: every argument as it must be, on
// the current device and stream. It returns None for anything else, also for an error
// of the library: the caller then takes the Python path, which says what is wrong.
// The entry points come from the loaded library (bind), so this module links to
// nothing of it. Time of a call that the host bounds, checked in Python and here: rope
// 8.0 and 4.5 us, a read 12.0 and 6.4, an append with a read of what it wrote 19.9 and 10.0.

#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <string>

#include "convrot.h"

namespace {

using Status = convrot_status;
Status (*rope_fn)(const convrot_rope_args*, convrot_stream_t) = nullptr;
Status (*append_fn)(const convrot_cache_args*, convrot_stream_t) = nullptr;
Status (*read_fn)(const convrot_cache_args*, convrot_stream_t) = nullptr;
Status (*attention_fn)(const convrot_cache_attention_args*, int*, int64_t, convrot_stream_t) = nullptr;
size_t (*attention_bytes_fn)(int64_t, int64_t, int64_t, int64_t, int64_t) = nullptr;

constexpr float kScale = 0.08838834764831845f;  // 1 / sqrt(128)

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// CONVROT_DTYPE_* of head vectors, or -1.
int code_of(at::ScalarType t) {
  return t == at::kBFloat16 ? CONVROT_DTYPE_BF16 : t == at::kHalf ? CONVROT_DTYPE_F16 : -1;
}

int device_of(const at::Tensor* t) { return t != nullptr && t->is_cuda() ? t->get_device() : -1; }

// Head vectors [..., heads, D] of one type on `device` whose channels are contiguous.
bool heads(const at::Tensor* t, int device, int64_t dims, at::ScalarType type) {
  return t != nullptr && t->scalar_type() == type && device_of(t) == device && t->dim() == dims &&
         (t->stride(dims - 1) == 1 || t->size(dims - 1) <= 1);
}

// A contiguous tensor of a type, with these sizes, on `device`.
bool plain(const at::Tensor* t, int device, at::ScalarType type, at::IntArrayRef sizes) {
  return t != nullptr && t->scalar_type() == type && device_of(t) == device && t->sizes() == sizes && t->is_contiguous();
}

// An output like head vectors of `like`'s sizes, each element at an address of its own.
bool output(const at::Tensor* t, int device, at::ScalarType type, at::IntArrayRef sizes) {
  if (!heads(t, device, static_cast<int64_t>(sizes.size()), type) || t->sizes() != sizes) return false;
  for (int64_t i = 0; i < t->dim(); ++i)
    if (t->size(i) > 1 && t->stride(i) == 0) return false;
  return true;
}

// Tells autograd that a tensor of the caller's has been written, as torch's own operations do.
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

bool here(int device) { return device >= 0 && c10::cuda::current_device() == device; }

convrot_stream_t stream_of(int device) {
  return reinterpret_cast<convrot_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream());
}

bool cells(PyObject* const* a, int device, convrot_cells* c) {
  const at::Tensor *kc = tensor(a[0]), *vc = tensor(a[1]), *ks = tensor(a[2]), *vs = tensor(a[3]);
  if (kc == nullptr || kc->dim() != 4 || kc->size(3) != 128) return false;
  const at::IntArrayRef sizes = kc->sizes();
  if (!plain(kc, device, at::kChar, sizes) || !plain(vc, device, at::kChar, sizes) ||
      !plain(ks, device, at::kFloat, sizes.slice(0, 3)) || !plain(vs, device, at::kFloat, sizes.slice(0, 3)))
    return false;
  c->k_codes = static_cast<int8_t*>(kc->data_ptr());
  c->v_codes = static_cast<int8_t*>(vc->data_ptr());
  c->k_scale = static_cast<float*>(ks->data_ptr());
  c->v_scale = static_cast<float*>(vs->data_ptr());
  c->num_pages = sizes[0];
  c->H = sizes[1];
  c->page_size = sizes[2];
  c->D = 128;
  return true;
}

// A one-int status tensor or None.
bool status_word(PyObject* o, int device, int** to) {
  *to = nullptr;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o);
  if (!plain(t, device, at::kInt, {1})) return false;
  *to = static_cast<int*>(t->data_ptr());
  return true;
}

template <class Args, class... More, class... Same>
Status call(Status (*fn)(const Args*, More...), const Args& args, int device, Same... more) {
  if (fn == nullptr) return CONVROT_ERR_INVALID_ARG;
  const convrot_stream_t s = stream_of(device);
  Status st;
  Py_BEGIN_ALLOW_THREADS st = fn(&args, more..., s);
  Py_END_ALLOW_THREADS return st;
}

// A call that did not succeed: None for the Python form, which says what is wrong with it. An error of CUDA's is raised
// here: it may have come behind a launch, and heads must not be turned in place a second time.
PyObject* failed(PyObject* self, Status st, const char* name) {
  if (st != CONVROT_ERR_CUDA) Py_RETURN_NONE;
  const char* module_name = PyModule_GetName(self);
  if (module_name == nullptr) return nullptr;
  const char* dot = std::strrchr(module_name, '.');
  const std::string package(module_name, dot != nullptr ? dot - module_name : std::strlen(module_name));
  PyObject* home = PyImport_ImportModule(package.c_str());
  PyObject* type = home != nullptr ? PyObject_GetAttrString(home, "ConvRotError") : nullptr;
  PyObject* error = type != nullptr ? PyObject_CallFunction(type, "is", static_cast<int>(st), name) : nullptr;
  if (error != nullptr) PyErr_SetObject(type, error);
  Py_XDECREF(error);
  Py_XDECREF(type);
  Py_XDECREF(home);
  return nullptr;
}

// rope(X, positions, freq, axis, interleaved, inverse, Y or None)
PyObject* rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 7) Py_RETURN_NONE;
  const at::Tensor *x = tensor(a[0]), *pos = tensor(a[1]), *freq = tensor(a[2]), *axis = tensor(a[3]);
  const int device = device_of(x);
  if (!here(device) || pos == nullptr || freq == nullptr) Py_RETURN_NONE;
  const int64_t dims = x->dim();
  const int code = code_of(x->scalar_type());
  if (code < 0 || (dims != 3 && dims != 4) || !heads(x, device, dims, x->scalar_type())) Py_RETURN_NONE;
  convrot_rope_args r{};
  r.B = dims == 4 ? x->size(0) : 1;
  r.S = x->size(dims - 3), r.H = x->size(dims - 2), r.D = x->size(dims - 1);
  const int64_t pairs = freq->numel();
  // autograd's business is seen to in Python
  if (at::GradMode::is_enabled() && (x->requires_grad() || pos->requires_grad() || freq->requires_grad() ||
                                     (a[6] != Py_None && tensor(a[6]) != nullptr && tensor(a[6])->requires_grad())))
    Py_RETURN_NONE;
  if (2 * pairs > r.D || !plain(freq, device, at::kDouble, {pairs}) || !plain(axis, device, at::kInt, {pairs}))
    Py_RETURN_NONE;
  const int64_t pdims = pos->dim();
  if (device_of(pos) != device || (pos->scalar_type() != at::kInt && pos->scalar_type() != at::kFloat) ||
      (pdims != 2 && !(pdims == 3 && pos->size(1) == r.B)) || pos->size(0) < 1 || pos->size(pdims - 1) != r.S)
    Py_RETURN_NONE;
  const int inter = PyObject_IsTrue(a[4]), inverse = PyObject_IsTrue(a[5]);
  if (inter < 0 || inverse < 0) return nullptr;
  at::Tensor made;
  const at::Tensor* y = &made;
  if (a[6] == Py_None) {
    made = at::empty(x->sizes(), x->options().requires_grad(false));
  } else {
    y = tensor(a[6]);
    if (!output(y, device, x->scalar_type(), x->sizes())) Py_RETURN_NONE;
  }
  r.X = x->data_ptr();
  r.Y = y->data_ptr();
  r.positions = pos->data_ptr();
  r.freq = static_cast<const double*>(freq->data_ptr());
  r.axis = static_cast<const int32_t*>(axis->data_ptr());
  r.R = 2 * pairs;
  r.x_batch = dims == 4 ? x->stride(0) : 0, r.x_token = x->stride(dims - 3), r.x_head = x->stride(dims - 2);
  r.y_batch = dims == 4 ? y->stride(0) : 0, r.y_token = y->stride(dims - 3), r.y_head = y->stride(dims - 2);
  r.axes = pos->size(0), r.pos_axis = pos->stride(0), r.pos_batch = pdims == 3 ? pos->stride(1) : 0;
  r.pos_token = pos->stride(pdims - 1);
  r.dtype = code;
  r.pos_dtype = pos->scalar_type() == at::kInt ? CONVROT_POS_I32 : CONVROT_POS_F32;
  r.interleaved = inter, r.inverse = inverse;
  if (const Status st = call(rope_fn, r, device); st != CONVROT_OK) return failed(self, st, "convrot_rope");
  if (a[6] == Py_None) return THPVariable_Wrap(std::move(made));
  written(*y);
  Py_INCREF(a[6]);
  return a[6];
  END_HANDLE_TH_ERRORS
}

// append(K, V, slots, k_codes, v_codes, k_scale, v_scale, status or None) -> True or None
PyObject* append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8) Py_RETURN_NONE;
  const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]), *slots = tensor(a[2]);
  const int device = device_of(k);
  if (!here(device)) Py_RETURN_NONE;
  const int code = code_of(k->scalar_type());
  convrot_cache_args r{};
  if (code < 0 || !heads(k, device, 3, k->scalar_type()) || !heads(v, device, 3, k->scalar_type()) ||
      v->sizes() != k->sizes() || !cells(a + 3, device, &r.cells) || r.cells.H != k->size(1) || k->size(2) != 128 ||
      !plain(slots, device, at::kInt, {k->size(0)}) || !status_word(a[7], device, &r.status))
    Py_RETURN_NONE;
  r.K = k->data_ptr();
  r.V = v->data_ptr();
  r.slots = static_cast<const int32_t*>(slots->data_ptr());
  r.T = k->size(0);
  r.k_token = k->stride(0), r.k_head = k->stride(1), r.v_token = v->stride(0), r.v_head = v->stride(1);
  r.dtype = code;
  if (const Status st = call(append_fn, r, device); st != CONVROT_OK) return failed(self, st, "convrot_cache_append");
  Py_RETURN_TRUE;
  END_HANDLE_TH_ERRORS
}

// read(slots, k_codes, v_codes, k_scale, v_scale, dtype code, K or None, V or None, status or None) -> (K, V) or None
PyObject* read(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9) Py_RETURN_NONE;
  const at::Tensor* slots = tensor(a[0]);
  const int device = device_of(slots);
  if (!here(device)) Py_RETURN_NONE;
  const long code = PyLong_AsLong(a[5]);
  if (code == -1 && PyErr_Occurred()) return nullptr;
  convrot_cache_args r{};
  const int64_t T = slots->numel();
  if ((code != CONVROT_DTYPE_BF16 && code != CONVROT_DTYPE_F16) || !plain(slots, device, at::kInt, {T}) ||
      !cells(a + 1, device, &r.cells) || !status_word(a[8], device, &r.status))
    Py_RETURN_NONE;
  const at::ScalarType type = code == CONVROT_DTYPE_F16 ? at::kHalf : at::kBFloat16;
  const int64_t sizes[3] = {T, r.cells.H, 128};
  at::Tensor made[2];
  const at::Tensor* out[2];
  for (int i = 0; i < 2; ++i) {
    if (a[6 + i] == Py_None) {
      made[i] = at::empty(sizes, slots->options().dtype(type).requires_grad(false));
      out[i] = &made[i];
    } else {
      out[i] = tensor(a[6 + i]);
      if (!output(out[i], device, type, sizes)) Py_RETURN_NONE;
    }
  }
  r.K = out[0]->data_ptr();
  r.V = out[1]->data_ptr();
  r.slots = static_cast<const int32_t*>(slots->data_ptr());
  r.T = T;
  r.k_token = out[0]->stride(0), r.k_head = out[0]->stride(1);
  r.v_token = out[1]->stride(0), r.v_head = out[1]->stride(1);
  r.dtype = static_cast<int>(code);
  if (const Status st = call(read_fn, r, device); st != CONVROT_OK) return failed(self, st, "convrot_cache_read");
  PyObject* pair = PyTuple_New(2);
  if (pair == nullptr) return nullptr;
  for (int i = 0; i < 2; ++i) {
    PyObject* o = a[6 + i];
    if (o == Py_None) {
      o = THPVariable_Wrap(std::move(made[i]));
    } else {
      written(*out[i]);
      Py_INCREF(o);
    }
    if (o == nullptr) {
      Py_DECREF(pair);
      return nullptr;
    }
    PyTuple_SET_ITEM(pair, i, o);
  }
  return pair;
  END_HANDLE_TH_ERRORS
}

// attention(Q, k_codes, v_codes, k_scale, v_scale, pages, lengths, starts, tree, softmax_scale, O, ws, status); the
// last six may be None
PyObject* attention(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 13) Py_RETURN_NONE;
  const at::Tensor *q = tensor(a[0]), *pages = tensor(a[5]), *lengths = tensor(a[6]);
  const int device = device_of(q);
  if (!here(device) || pages == nullptr || lengths == nullptr) Py_RETURN_NONE;
  const int code = code_of(q->scalar_type());
  convrot_cache_attention_args r{};
  int* status = nullptr;
  if (code < 0 || !heads(q, device, 3, q->scalar_type()) || q->size(2) != 128 || !cells(a + 1, device, &r.cells))
    Py_RETURN_NONE;
  r.T = q->size(0), r.Hq = q->size(1), r.B = lengths->numel();
  if (r.cells.H == 0 || r.Hq == 0 || r.Hq % r.cells.H != 0 || !plain(lengths, device, at::kInt, {r.B})) Py_RETURN_NONE;
  if (pages->scalar_type() != at::kInt || device_of(pages) != device || pages->dim() != 2 || pages->size(0) != r.B ||
      (pages->stride(1) != 1 && pages->size(1) > 1))
    Py_RETURN_NONE;
  if (a[7] != Py_None) {
    const at::Tensor* starts = tensor(a[7]);
    if (!plain(starts, device, at::kInt, {r.B + 1})) Py_RETURN_NONE;
    r.starts = static_cast<const int32_t*>(starts->data_ptr());
  } else if (r.T != r.B) {
    Py_RETURN_NONE;
  }
  if (a[8] != Py_None) {
    const at::Tensor* tree = tensor(a[8]);
    if (!plain(tree, device, at::kLong, {r.T})) Py_RETURN_NONE;
    r.tree = static_cast<const int64_t*>(tree->data_ptr());
  }
  if (!status_word(a[12], device, &status)) Py_RETURN_NONE;
  r.softmax_scale = kScale;
  if (a[9] != Py_None) {
    const double scale = PyFloat_AsDouble(a[9]);
    if (scale == -1.0 && PyErr_Occurred()) return nullptr;
    if (!(std::fabs(scale) <= FLT_MAX)) Py_RETURN_NONE;
    r.softmax_scale = static_cast<float>(scale);
  }
  at::Tensor made, scratch;
  const at::Tensor* o = &made;
  if (a[10] != Py_None) {
    o = tensor(a[10]);
    if (!output(o, device, q->scalar_type(), q->sizes())) Py_RETURN_NONE;
  } else {
    made = at::empty(q->sizes(), q->options().requires_grad(false));
  }
  const at::Tensor* ws = &scratch;
  if (a[11] != Py_None) {
    ws = tensor(a[11]);
    if (device_of(ws) != device || !ws->is_contiguous()) Py_RETURN_NONE;
  } else {
    if (attention_bytes_fn == nullptr) Py_RETURN_NONE;
    const int64_t need = static_cast<int64_t>(attention_bytes_fn(r.T, r.B, r.Hq, r.cells.H, 128));
    scratch = at::empty({need < 256 ? 256 : need}, q->options().dtype(at::kByte).requires_grad(false));
  }
  r.Q = q->data_ptr();
  r.O = o->data_ptr();
  r.pages = static_cast<const int32_t*>(pages->data_ptr());
  r.lengths = static_cast<const int32_t*>(lengths->data_ptr());
  r.ws = ws->data_ptr();
  r.ws_bytes = static_cast<size_t>(ws->numel()) * ws->element_size();
  r.table_pages = pages->size(1), r.table_stride = pages->stride(0);
  r.q_token = q->stride(0), r.q_head = q->stride(1), r.o_token = o->stride(0), r.o_head = o->stride(1);
  r.dtype = code;
  if (const Status st = call(attention_fn, r, device, status, int64_t{0}); st != CONVROT_OK) return failed(self, st, "convrot_cache_attention");
  if (a[10] == Py_None) return THPVariable_Wrap(std::move(made));
  written(*o);
  Py_INCREF(a[10]);
  return a[10];
  END_HANDLE_TH_ERRORS
}

// bind(rope, append, read, attention_ex, attention_workspace_bytes): the addresses of the library's entry points
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "bind takes five addresses");
    return nullptr;
  }
  void* at[5];
  for (int i = 0; i < 5; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i]);
    if (at[i] == nullptr && PyErr_Occurred()) return nullptr;
  }
  rope_fn = reinterpret_cast<decltype(rope_fn)>(at[0]);
  append_fn = reinterpret_cast<decltype(append_fn)>(at[1]);
  read_fn = reinterpret_cast<decltype(read_fn)>(at[2]);
  attention_fn = reinterpret_cast<decltype(attention_fn)>(at[3]);
  attention_bytes_fn = reinterpret_cast<decltype(attention_bytes_fn)>(at[4]);
  Py_RETURN_NONE;
}

template <class F>
PyCFunction fast(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {{"rope", fast(rope), METH_FASTCALL, nullptr},
                         {"append", fast(append), METH_FASTCALL, nullptr},
                         {"read", fast(read), METH_FASTCALL, nullptr},
                         {"attention", fast(attention), METH_FASTCALL, nullptr},
                         {"bind", fast(bind), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
  PyObject* m = PyModule_Create(&module);
  // what the module may be used with: this torch, and a library compiled from the same convrot.h
  if (m != nullptr && (PyModule_AddStringConstant(m, "torch_version", BUILT_FOR_TORCH) != 0 ||
                       PyModule_AddStringConstant(m, "header", CONVROT_HEADER) != 0))
    Py_CLEAR(m);
  return m;
}
