// Native part of the Python binding: the calls over a paged cache, whose kernels
// take less time than their arguments' way through Python and ctypes. It checks
// and marshals tensors, allocates the outputs and workspaces that the caller did
// not bring, and calls the C ABI on the device's current stream. The library's
// functions are given to it by address (bind), so that there is one copy of the
// library in the process.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <string>

#include "tr_sparseconv.h"

namespace {

decltype(&tr_sparseconv_qk_norm_rope_append) append_fn = nullptr;
decltype(&tr_sparseconv_paged_attention_workspace_bytes) bytes_fn = nullptr;
decltype(&tr_sparseconv_paged_window_attention) attend_fn = nullptr;
decltype(&tr_sparseconv_shared_prefix_attention) prefix_fn = nullptr;
PyObject* check_fn = nullptr;   // check(code): raises for an error of the library
PyObject* stream_fn = nullptr;  // stream of a device index
PyObject* device_fn = nullptr;  // current device index

// A number past its C field would be taken modulo its range.
constexpr int64_t kFieldMost = int64_t(1) << 31;

[[noreturn]] void refuse(const std::string& what) {
  C10_THROW_ERROR(ValueError, what);
}

std::string text(PyObject* o) {
  PyObject* s = PyObject_Str(o);
  if (s == nullptr) throw python_error();
  const char* c = PyUnicode_AsUTF8(s);
  std::string out = c ? c : "?";
  Py_DECREF(s);
  return out;
}
std::string dtype_text(const at::Tensor& t) {
  const at::ScalarType s = t.scalar_type();
  return s == at::kFloat ? "torch.float32" : s == at::kBFloat16 ? "torch.bfloat16" : s == at::kHalf ? "torch.float16" : c10::toString(s);
}
std::string shape_text(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

const at::Tensor* tensor_or_null(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

int dtype_of(PyObject* o, const char* name) {
  const at::Tensor* t = tensor_or_null(o);
  if (t != nullptr) {
    if (t->scalar_type() == at::kBFloat16) return TR_SC_BF16;
    if (t->scalar_type() == at::kHalf) return TR_SC_F16;
    if (t->scalar_type() == at::kFloat) return TR_SC_F32;
  }
  refuse(std::string(name) + " has unsupported type " + (t ? dtype_text(*t) : text(reinterpret_cast<PyObject*>(Py_TYPE(o)))));
}

// A [tokens, heads, dim] tensor; tokens, heads -1: any.
tr_sc_heads heads_of(PyObject* o, const char* name, const at::Tensor* like = nullptr, int64_t tokens = -1, int64_t heads = -1) {
  const at::Tensor* t = tensor_or_null(o);
  if (t == nullptr || !t->is_cuda()) refuse(std::string(name) + " must be a GPU tensor");
  if (t->dim() != 3) refuse(std::string(name) + " must be [tokens, heads, dim], got " + shape_text(*t));
  const int64_t n = t->size(0), h = t->size(1), d = t->size(2);
  if (h >= kFieldMost || d >= kFieldMost)
    refuse(std::string(name) + " has " + std::to_string(h) + " heads of " + std::to_string(d) + " elements, past 2^31");
  if (like != nullptr) {
    if (d != like->size(2) || (tokens >= 0 && n != tokens) || (heads >= 0 && h != heads))
      refuse(std::string(name) + " must be [" + (tokens < 0 ? "*" : std::to_string(tokens)) + ", " +
             (heads < 0 ? "*" : std::to_string(heads)) + ", " + std::to_string(like->size(2)) + "], got " + shape_text(*t));
    if (t->scalar_type() != like->scalar_type() || t->device() != like->device())
      refuse(std::string(name) + " must be " + dtype_text(*like) + " on " + like->device().str() + ", got " +
             dtype_text(*t) + " on " + t->device().str());
  }
  if (d > 1 && t->stride(2) != 1) refuse(std::string("the elements of a row of ") + name + " must be adjacent");
  // a stride that is never taken may be anything
  return tr_sc_heads{n ? t->data_ptr() : nullptr, n > 1 ? t->stride(0) : 0, h > 1 ? t->stride(1) : 0, int(h)};
}

// A contiguous int32 vector of n elements (-1: any), or null for None.
const int32_t* ints_of(PyObject* o, const char* name, int64_t n, const at::Device& device) {
  if (o == Py_None) return nullptr;
  const at::Tensor* t = tensor_or_null(o);
  if (t == nullptr || t->device() != device || t->scalar_type() != at::kInt || t->dim() != 1 || !t->is_contiguous())
    refuse(std::string(name) + " must be a contiguous int32 vector on " + device.str());
  if (n >= 0 && t->size(0) != n)
    refuse(std::string(name) + " must have " + std::to_string(n) + " elements, got " + std::to_string(t->size(0)));
  return static_cast<const int32_t*>(t->data_ptr());
}

const float* gain_of(PyObject* o, const char* name, int64_t heads, int64_t dim, const at::Device& device, int* rows) {
  *rows = 1;
  if (o == Py_None) return nullptr;
  const at::Tensor* t = tensor_or_null(o);
  if (t == nullptr || t->device() != device || t->scalar_type() != at::kFloat || !t->is_contiguous())
    refuse(std::string(name) + " must be a contiguous fp32 tensor on " + device.str());
  if (t->dim() == 2 && t->size(0) == heads && t->size(1) == dim)
    *rows = int(heads);
  else if (t->dim() != 1 || t->size(0) != dim)
    refuse(std::string(name) + " must be [" + std::to_string(dim) + "] or [" + std::to_string(heads) + ", " +
           std::to_string(dim) + "], got " + shape_text(*t));
  return static_cast<const float*>(t->data_ptr());
}

tr_sc_pages pages_of(PyObject* ko, PyObject* vo, PyObject* to, PyObject* lo, const at::Tensor& like) {
  const at::Tensor *k = tensor_or_null(ko), *v = tensor_or_null(vo), *table = tensor_or_null(to);
  const at::Device device = like.device();
  int i = 0;
  for (const at::Tensor* t : {k, v}) {
    const char* name = i++ == 0 ? "k_pages" : "v_pages";
    if (t == nullptr || t->dim() != 4 || t->scalar_type() != like.scalar_type() || t->device() != device)
      refuse(std::string(name) + " must be a " + dtype_text(like) + " tensor [pages, page_size, heads, dim] on " + device.str());
    if (t->sizes() != k->sizes())
      refuse("k_pages " + shape_text(*k) + " and v_pages " + shape_text(*t) + " must have one shape");
    if (t->size(3) > 1 && t->stride(3) != 1) refuse(std::string("the elements of a row of ") + name + " must be adjacent");
  }
  const int64_t pages = k->size(0), size = k->size(1), heads = k->size(2), dim = like.size(2);
  if (k->size(3) != dim)
    refuse("the pages' heads have " + std::to_string(k->size(3)) + " elements, q's " + std::to_string(dim));
  if (table == nullptr || table->device() != device || table->scalar_type() != at::kInt || table->dim() != 2)
    refuse("page_table must be an int32 tensor [batch, pages] on " + device.str());
  const int64_t batch = table->size(0), width = table->size(1);
  if (width > 1 && table->stride(1) != 1) refuse("the entries of a row of page_table must be adjacent");
  if (batch < 1) refuse("page_table needs a sequence at least");
  if (lo == Py_None) refuse("k_len must be given");
  const int32_t* len = ints_of(lo, "k_len", batch, device);
  if (size >= kFieldMost || heads >= kFieldMost || width >= kFieldMost || batch >= kFieldMost)
    refuse("the pages or their table are too large");
  // a stride that is never taken may be anything
  const auto st = [](const at::Tensor& t, int d) { return t.size(d) > 1 ? t.stride(d) : int64_t(0); };
  tr_sc_pages p;
  p.k = pages ? k->data_ptr() : nullptr;
  p.v = pages ? v->data_ptr() : nullptr;
  p.k_page_stride = st(*k, 0);
  p.k_slot_stride = st(*k, 1);
  p.k_head_stride = st(*k, 2);
  p.v_page_stride = st(*v, 0);
  p.v_slot_stride = st(*v, 1);
  p.v_head_stride = st(*v, 2);
  p.pages = pages;
  p.page_size = int(size);
  p.heads = int(heads);
  p.table = width ? static_cast<const int32_t*>(table->data_ptr()) : nullptr;
  p.table_stride = batch > 1 ? table->stride(0) : 0;
  p.table_pages = int(width);
  p.len = len;
  p.batch = int(batch);
  return p;
}

int64_t integer(PyObject* o, const char* name) {
  int overflow = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &overflow);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  if (overflow) refuse(std::string(name) + " = " + text(o) + " is out of range");
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

// The output of the caller's, or a new contiguous one, owned by `made`.
tr_sc_heads out_of(PyObject* o, const char* name, const at::Tensor& like, int64_t tokens, int64_t heads, at::Tensor* made) {
  if (o != Py_None) return heads_of(o, name, &like, tokens, heads);
  *made = at::empty({tokens, heads, like.size(2)}, like.options().requires_grad(false));
  return tr_sc_heads{tokens ? made->data_ptr() : nullptr, tokens > 1 ? heads * like.size(2) : 0, heads > 1 ? like.size(2) : 0,
                     int(heads)};
}

int64_t call_int(PyObject* fn, PyObject* arg) {
  PyObject* r = arg ? PyObject_CallOneArg(fn, arg) : PyObject_CallNoArgs(fn);
  if (r == nullptr) throw python_error();
  const int64_t v = int64_t(PyLong_AsUnsignedLongLong(r));
  Py_DECREF(r);
  if (PyErr_Occurred()) throw python_error();
  return v;
}

// f(stream) on the device's current stream; raises for an error.
template <class F>
void call(const at::Device& device, const F& f) {
  PyObject* index = PyLong_FromLong(device.index());
  if (index == nullptr) throw python_error();
  int64_t stream = 0, current = 0;
  try {
    stream = call_int(stream_fn, index);
    current = call_int(device_fn, nullptr);
  } catch (...) {
    Py_DECREF(index);
    throw;
  }
  Py_DECREF(index);
  int code;
  {
    c10::OptionalDeviceGuard guard;
    if (current != device.index()) guard.reset_device(device);
    Py_BEGIN_ALLOW_THREADS code = f(reinterpret_cast<void*>(stream));
    Py_END_ALLOW_THREADS
  }
  if (code != TR_SC_OK) {
    PyObject* c = PyLong_FromLong(code);
    PyObject* r = c ? PyObject_CallOneArg(check_fn, c) : nullptr;
    Py_XDECREF(c);
    Py_XDECREF(r);
    if (r == nullptr) throw python_error();
  }
}

PyObject* given_or(PyObject* o, const at::Tensor& made) {
  if (o == Py_None) return THPVariable_Wrap(made);
  Py_INCREF(o);
  return o;
}

void need(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse("wrong number of arguments");
  if (append_fn == nullptr) refuse("the library is not bound");
}

// append(q, k, v, pos, freqs, k_pages, v_pages, page_table, k_len, cu_q, q_gain, k_gain, sections, interleaved, eps, norm,
// q_out)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need(n, 17);
  const int dt = dtype_of(a[0], "q");
  const tr_sc_heads q = heads_of(a[0], "q");
  const at::Tensor& like = *tensor_or_null(a[0]);
  const int64_t tokens = like.size(0), dim = like.size(2);
  const at::Device device = like.device();
  const tr_sc_heads k = heads_of(a[1], "k", &like, tokens), v = heads_of(a[2], "v", &like, tokens, k.heads);
  // the rotation
  const at::Tensor* pos = tensor_or_null(a[3]);
  if (pos == nullptr || pos->device() != device || pos->scalar_type() != at::kInt)
    refuse("pos must be an int32 tensor on " + device.str());
  const int64_t axes = pos->dim() == 1 ? 1 : pos->dim() == 2 ? pos->size(1) : 0;
  if (axes < 1 || axes > 3 || pos->size(0) != tokens)
    refuse("pos must be [" + std::to_string(tokens) + ", 1 .. 3 axes], got " + shape_text(*pos));
  if (axes > 1 && pos->stride(1) != 1) refuse("the axes of a position must be adjacent");
  const at::Tensor* freqs = tensor_or_null(a[4]);
  if (freqs == nullptr || freqs->device() != device || freqs->scalar_type() != at::kFloat || freqs->dim() != 1 ||
      freqs->size(0) != dim / 2 || !freqs->is_contiguous())
    refuse("freqs must be fp32 [" + std::to_string(dim / 2) + "] on " + device.str());
  tr_sc_rotation rot{tokens ? static_cast<const int32_t*>(pos->data_ptr()) : nullptr, tokens > 1 ? pos->stride(0) : 0,
                     static_cast<const float*>(freqs->data_ptr()), int(axes), {0, 0, 0}, 0};
  if (a[12] == Py_None) {
    for (int64_t i = 0; i < axes; ++i) rot.pairs[i] = int(dim / 2 / axes);
  } else {
    PyObject* s = PySequence_Fast(a[12], "sections must be a sequence");
    if (s == nullptr) throw python_error();
    bool fits = PySequence_Fast_GET_SIZE(s) == axes;
    for (int64_t i = 0; fits && i < axes; ++i) {
      int overflow = 0;
      const long long x = PyLong_AsLongLongAndOverflow(PySequence_Fast_GET_ITEM(s, i), &overflow);
      if (x == -1 && PyErr_Occurred()) {
        Py_DECREF(s);
        throw python_error();
      }
      fits = !overflow && x >= 0 && x <= dim;
      rot.pairs[i] = fits ? int(x) : 0;
    }
    Py_DECREF(s);
    if (!fits)
      refuse(std::to_string(axes) + " axes need " + std::to_string(axes) + " sections of pairs, got " + text(a[12]));
  }
  const int il = PyObject_IsTrue(a[13]), norm = PyObject_IsTrue(a[15]);
  if (il < 0 || norm < 0) throw python_error();
  rot.interleaved = il;
  int q_rows, k_rows;
  const float *qg = gain_of(a[10], "q_gain", q.heads, dim, device, &q_rows),
              *kg = gain_of(a[11], "k_gain", k.heads, dim, device, &k_rows);
  const float eps = float(number(a[14]));
  const tr_sc_pages pages = pages_of(a[5], a[6], a[7], a[8], like);
  const int32_t* cu = ints_of(a[9], "cu_q", int64_t(pages.batch) + 1, device);
  at::Tensor made;
  const tr_sc_heads out = out_of(a[16], "q_out", like, tokens, q.heads, &made);
  call(device, [&](void* stream) {
    return append_fn(&q, &k, &v, &rot, qg, q_rows, kg, k_rows, norm, eps, &out, &pages, cu, tokens, int(dim), dt, stream);
  });
  return given_or(a[16], made);
  END_HANDLE_TH_ERRORS
}

// attend(q, k_pages, v_pages, page_table, k_len, prefix_pages or None, prefix_len, cu_q, left, right, sinks, scale,
// return_lse, out, workspace)
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need(n, 15);
  const bool prefixed = a[5] != Py_None;
  const int64_t prefix_len = integer(a[6], "prefix_len");
  const at::Tensor *prefix_t = tensor_or_null(a[5]), *pool = tensor_or_null(a[1]);
  if (prefix_t != nullptr && prefix_t->dim() == 1 && pool != nullptr && pool->dim() == 4 &&
      prefix_t->size(0) * pool->size(1) < prefix_len)
    refuse(std::to_string(prefix_t->size(0)) + " pages of " + std::to_string(pool->size(1)) +
           " do not hold a prefix of " + std::to_string(prefix_len));
  const int dt = dtype_of(a[0], "q");
  const tr_sc_heads q = heads_of(a[0], "q");
  const at::Tensor& like = *tensor_or_null(a[0]);
  const int64_t tokens = like.size(0), dim = like.size(2);
  const at::Device device = like.device();
  const tr_sc_pages pages = pages_of(a[1], a[2], a[3], a[4], like);
  const int32_t* prefix = ints_of(a[5], "prefix_pages", -1, device);
  tr_sc_window win{};
  win.cu_q = ints_of(a[7], "cu_q", int64_t(pages.batch) + 1, device);
  win.batch = pages.batch;
  win.left = integer(a[8], "left");
  win.right = integer(a[9], "right");
  const int64_t sinks = integer(a[10], "sinks");
  if (win.left < -1 || win.right < -1 || sinks < 0 || sinks >= int64_t(1) << 31)
    refuse("window (" + text(a[8]) + ", " + text(a[9]) + ") with " + text(a[10]) +
           " sinks: sides are -1 or more, sinks 0 or more");
  win.sinks = int(sinks);
  win.scale = a[11] == Py_None ? float(1.0 / std::sqrt(double(dim))) : float(number(a[11]));
  const int want_lse = PyObject_IsTrue(a[12]);
  if (want_lse < 0) throw python_error();
  at::Tensor made, lse, space;
  const tr_sc_heads out = out_of(a[13], "out", like, tokens, q.heads, &made);
  if (want_lse) lse = at::empty({q.heads, tokens}, like.options().dtype(at::kFloat).requires_grad(false));
  size_t bytes = bytes_fn(&pages, &win, prefixed ? prefix_len : 0, tokens, q.heads, int(dim), dt);
  void* ws = nullptr;
  if (a[14] != Py_None) {  // a Workspace
    PyObject* size = PyObject_GetAttrString(a[14], "nbytes");
    if (size == nullptr) throw python_error();
    const int64_t have = PyLong_AsLongLong(size);
    Py_DECREF(size);
    if (PyErr_Occurred()) throw python_error();
    PyObject* buf = PyObject_GetAttrString(a[14], "buf");
    if (buf == nullptr) throw python_error();
    const at::Tensor* t = tensor_or_null(buf);
    if (t != nullptr) space = *t;  // the object may be made for this question alone
    Py_DECREF(buf);
    if (!space.defined()) refuse("workspace must be a Workspace");
    if (have < int64_t(bytes))
      refuse("workspace of " + std::to_string(have) + " bytes, " + std::to_string(bytes) + " needed");
    if (space.device() != device) refuse("the workspace is on " + space.device().str() + ", the tensors on " + device.str());
    const uintptr_t p = reinterpret_cast<uintptr_t>(space.data_ptr());
    ws = reinterpret_cast<void*>((p + 255) / 256 * 256);
    bytes = size_t(have);
  } else if (bytes > 0) {  // torch's own blocks are aligned to 256 bytes and more
    space = at::empty({int64_t(bytes)}, like.options().dtype(at::kByte).requires_grad(false));
    ws = space.data_ptr();
  }
  float* const lse_ptr = want_lse ? static_cast<float*>(lse.data_ptr()) : nullptr;
  call(device, [&](void* stream) {
    if (!prefixed) return attend_fn(&q, &pages, &win, &out, lse_ptr, tokens, int(dim), dt, ws, bytes, stream);
    return prefix_fn(&q, &pages, prefix, prefix_len, &win, &out, lse_ptr, tokens, int(dim), dt, ws, bytes, stream);
  });
  PyObject* o = given_or(a[13], made);
  if (!want_lse || o == nullptr) return o;
  PyObject* l = THPVariable_Wrap(lse);
  PyObject* pair = l ? PyTuple_Pack(2, o, l) : nullptr;
  Py_DECREF(o);
  Py_XDECREF(l);
  return pair;
  END_HANDLE_TH_ERRORS
}

// bind(append, bytes, attend, prefix: addresses; check, stream, device: callables)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 7) refuse("wrong number of arguments");
  void* at[4];
  for (int i = 0; i < 4; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) throw python_error();
  }
  append_fn = reinterpret_cast<decltype(append_fn)>(at[0]);
  bytes_fn = reinterpret_cast<decltype(bytes_fn)>(at[1]);
  attend_fn = reinterpret_cast<decltype(attend_fn)>(at[2]);
  prefix_fn = reinterpret_cast<decltype(prefix_fn)>(at[3]);
  PyObject** const to[3] = {&check_fn, &stream_fn, &device_fn};
  for (int i = 0; i < 3; ++i) {
    Py_INCREF(a[4 + i]);
    Py_XSETREF(*to[i], a[4 + i]);
  }
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(append)), METH_FASTCALL, nullptr},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(attend)), METH_FASTCALL, nullptr},
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(bind)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  // torch's C++ types have no stable layout: the package compares this before it binds
  if (m != nullptr && PyModule_AddStringConstant(m, "built_for", TR_SC_BUILT_FOR) != 0) Py_CLEAR(m);
  return m;
}
