// Native part of the Python binding: what a call on torch tensors does on the host,
// for calls whose time is the host's.  Checks, allocations and the call itself took
// 10 to 26 us from Python, a list's shapes, dtypes, devices, layouts and addresses
// 0.4 us per tensor.
//
// Every function here takes a usual call (plain tensors, contiguous or in rows of one
// layout, of one device that is the current one, the current stream, outputs to be
// allocated) and returns None for any other, and where the library returns an error: the binding's general
// path then goes through the call and says what is wrong.  The library's functions
// come as addresses from the binding, which has loaded it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstdint>

#include "triattn.h"

namespace {

decltype(&triattn_qk_norm_workspace_bytes) qk_bytes = nullptr;
decltype(&triattn_qk_norm_fwd) qk_fwd = nullptr;
decltype(&triattn_qk_norm_bwd) qk_bwd = nullptr;
decltype(&triattn_relpos_workspace_bytes) rel_bytes = nullptr;
decltype(&triattn_relpos_fwd) rel_fwd = nullptr;
decltype(&triattn_relpos_bwd) rel_bwd = nullptr;

// Allocations and calls run without the interpreter's lock, as torch's own do.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// A tensor argument, or null where it is not plainly one.
const at::Tensor* tensor(PyObject* o) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  return &THPVariable_Unpack(o);
}
bool none(PyObject* o) { return o == Py_None; }

// A tensor of the current device, which is `index` (-1: set it).
bool here(const at::Tensor& t, at::ScalarType type, c10::DeviceIndex& index) {
  if (t.scalar_type() != type || !t.is_cuda() || t.layout() != at::kStrided) return false;
  if (index < 0) {
    index = t.get_device();
    return c10::cuda::current_device() == index;
  }
  return t.get_device() == index;
}
bool plain(const at::Tensor& t, at::ScalarType type, c10::DeviceIndex& index) {
  return here(t, type, index) && t.is_contiguous();
}
bool sized(const at::Tensor& t, at::IntArrayRef sizes) { return t.sizes() == sizes; }
bool ints(const at::Tensor& t) {
  for (int64_t s : t.sizes())
    if (s > INT_MAX) return false;
  return true;
}
// Two [B, N_o, H, N, D] tensors of one layout of their rows (null: contiguous).
struct Rows {
  triattn_layout layout;
  const triattn_layout* at = nullptr;
  bool read(const at::Tensor& a, const at::Tensor& b, at::IntArrayRef sizes, c10::DeviceIndex& index) {
    if (!here(a, at::kBFloat16, index) || !here(b, at::kBFloat16, index) || !sized(a, sizes) || !sized(b, sizes))
      return false;
    if (a.is_contiguous() && b.is_contiguous()) return true;
    if (a.strides() != b.strides() || a.stride(4) != 1) return false;
    if (a.size(0) > 1 && a.stride(0) != a.size(1) * a.stride(1)) return false;
    layout = triattn_layout{a.stride(1), a.stride(2), a.stride(3)};
    at = &layout;
    return true;
  }
};
// Optional [B, N] int32 positions or chains.
bool tokens(PyObject* o, int64_t B, int64_t N, c10::DeviceIndex index, const int*& p) {
  p = nullptr;
  if (none(o)) return true;
  const at::Tensor* t = tensor(o);
  if (t == nullptr || !plain(*t, at::kInt, index) || !sized(*t, {B, N})) return false;
  p = static_cast<const int*>(t->const_data_ptr());
  return true;
}
at::Tensor bytes(size_t n, const at::Tensor& like) {
  return at::empty({static_cast<int64_t>(n)}, like.options().dtype(at::kByte));
}

// Numbers, once every tensor has passed; an error is a Python exception.
struct Args {
  PyObject* const* a;
  bool ok = true;
  long integer(int i) {
    const long v = PyLong_AsLong(a[i]);
    if (v == -1 && PyErr_Occurred()) ok = false;
    if (v > INT_MAX || v < INT_MIN) ok = false;
    return v;
  }
  double real(int i) {
    const double v = PyFloat_AsDouble(a[i]);
    if (v == -1.0 && PyErr_Occurred()) ok = false;
    return v;
  }
  // a call that is not plainly right goes to the general path
  bool good() {
    if (!ok) PyErr_Clear();
    return ok;
  }
};

struct QkNorm {
  const at::Tensor *q, *k, *wq, *wk;
  const int* pos;
  triattn_qk_norm_shape shape;
  Rows rows;
  c10::DeviceIndex index = -1;

  // q, k, w_q, w_k, positions, rotary, theta, eps from `a`
  bool read(PyObject* const* a, PyObject* positions, Args& n, int at) {
    q = tensor(a[0]);
    k = tensor(a[1]);
    wq = tensor(a[2]);
    wk = tensor(a[3]);
    if (q == nullptr || k == nullptr || wq == nullptr || wk == nullptr) return false;
    if (q->dim() != 5 || !ints(*q) || !rows.read(*q, *k, q->sizes(), index)) return false;
    if (!plain(*wq, at::kFloat, index) || !plain(*wk, at::kFloat, index) || !sized(*wk, wq->sizes())) return false;
    const int64_t B = q->size(0), No = q->size(1), H = q->size(2), N = q->size(3), D = q->size(4);
    const bool shared = wq->dim() == 1;
    if (!(shared ? sized(*wq, {D}) : sized(*wq, {H, D}))) return false;
    if (!tokens(positions, B, N, index, pos)) return false;
    shape = triattn_qk_norm_shape{};
    shape.B = static_cast<int>(B);
    shape.N_o = static_cast<int>(No);
    shape.N = static_cast<int>(N);
    shape.H = static_cast<int>(H);
    shape.D = static_cast<int>(D);
    shape.w_heads = shared ? 1 : shape.H;
    shape.rotary = static_cast<int>(n.integer(at));
    shape.theta = n.real(at + 1);
    shape.eps = static_cast<float>(n.real(at + 2));
    return n.good();
  }
};

PyObject* host_qk_norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args num{a};
  QkNorm c;
  if (n != 8 || !c.read(a, a[4], num, 5)) Py_RETURN_NONE;
  at::Tensor qo, ko;
  triattn_status code;
  {
    Unlocked unlocked;
    qo = at::empty(c.q->sizes(), c.q->options());
    ko = at::empty(c.q->sizes(), c.q->options());
    code = qk_fwd(&c.shape, c.q->const_data_ptr(), c.k->const_data_ptr(), c.rows.at,
                  static_cast<const float*>(c.wq->const_data_ptr()),
                  static_cast<const float*>(c.wk->const_data_ptr()), c.pos, qo.mutable_data_ptr(),
                  ko.mutable_data_ptr(), nullptr, c10::cuda::getCurrentCUDAStream(c.index).stream());
  }
  if (code != TRIATTN_OK) Py_RETURN_NONE;
  return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(qo)), THPVariable_Wrap(std::move(ko)));
  END_HANDLE_TH_ERRORS
}

PyObject* host_qk_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args num{a};
  QkNorm c;
  if (n != 10 || !c.read(a, a[6], num, 7)) Py_RETURN_NONE;
  const at::Tensor *dqo = tensor(a[4]), *dko = tensor(a[5]);
  Rows out_rows;
  if (dqo == nullptr || dko == nullptr || !out_rows.read(*dqo, *dko, c.q->sizes(), c.index)) Py_RETURN_NONE;
  const size_t need = qk_bytes(&c.shape);
  if (need == 0) Py_RETURN_NONE;
  at::Tensor dq, dk, dwq, dwk;
  triattn_status code;
  {
    Unlocked unlocked;
    const at::Tensor ws = bytes(need, *c.q);
    dq = at::empty(c.q->sizes(), c.q->options());
    dk = at::empty(c.q->sizes(), c.q->options());
    dwq = at::empty_like(*c.wq);
    dwk = at::empty_like(*c.wk);
    code = qk_bwd(&c.shape, c.q->const_data_ptr(), c.k->const_data_ptr(), c.rows.at,
                  static_cast<const float*>(c.wq->const_data_ptr()),
                  static_cast<const float*>(c.wk->const_data_ptr()), c.pos, dqo->const_data_ptr(),
                  dko->const_data_ptr(), out_rows.at, dq.mutable_data_ptr(), dk.mutable_data_ptr(), nullptr,
                  static_cast<float*>(dwq.mutable_data_ptr()), static_cast<float*>(dwk.mutable_data_ptr()),
                  ws.mutable_data_ptr(), need, c10::cuda::getCurrentCUDAStream(c.index).stream());
  }
  if (code != TRIATTN_OK) Py_RETURN_NONE;
  return Py_BuildValue("(NNNN)", THPVariable_Wrap(std::move(dq)), THPVariable_Wrap(std::move(dk)),
                       THPVariable_Wrap(std::move(dwq)), THPVariable_Wrap(std::move(dwk)));
  END_HANDLE_TH_ERRORS
}

// table, base, positions, chains, layout, kind, max_distance
PyObject* host_relpos_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args num{a};
  const at::Tensor* table = n == 7 ? tensor(a[0]) : nullptr;
  c10::DeviceIndex index = -1;
  if (table == nullptr || !plain(*table, at::kFloat, index) || table->dim() != 2 || !ints(*table)) Py_RETURN_NONE;
  const at::Tensor* base = none(a[1]) ? nullptr : tensor(a[1]);
  const at::Tensor* like = base != nullptr ? base : tensor(a[2]);
  if ((base == nullptr && !none(a[1])) || like == nullptr || like->dim() != (base != nullptr ? 4 : 2) || !ints(*like))
    Py_RETURN_NONE;
  const int64_t B = like->size(0), N = like->size(base != nullptr ? 2 : 1), F = table->size(1);
  triattn_relpos_shape s{};
  s.B = static_cast<int>(B);
  s.N = static_cast<int>(N);
  s.F = static_cast<int>(F);
  s.layout = static_cast<int>(num.integer(4));
  s.kind = static_cast<int>(num.integer(5));
  s.buckets = static_cast<int>(table->size(0));
  s.max_distance = static_cast<int>(num.integer(6));
  if (!num.good()) Py_RETURN_NONE;
  const std::array<int64_t, 4> sizes = s.layout == TRIATTN_RELPOS_HEADS ? std::array<int64_t, 4>{B, F, N, N}
                                                                        : std::array<int64_t, 4>{B, N, N, F};
  const int *pos, *chain;
  if ((base != nullptr && (!plain(*base, at::kBFloat16, index) || !sized(*base, sizes))) ||
      !tokens(a[2], B, N, index, pos) || !tokens(a[3], B, N, index, chain))
    Py_RETURN_NONE;
  if (base == nullptr && rel_bytes(&s) == 0) Py_RETURN_NONE;  // before an output of any size is allocated
  at::Tensor out;
  triattn_status code;
  {
    Unlocked unlocked;
    out = at::empty(sizes, table->options().dtype(at::kBFloat16));
    code = rel_fwd(&s, static_cast<const float*>(table->const_data_ptr()),
                   base != nullptr ? base->const_data_ptr() : nullptr, pos, chain, out.mutable_data_ptr(),
                   c10::cuda::getCurrentCUDAStream(index).stream());
  }
  if (code != TRIATTN_OK) Py_RETURN_NONE;
  return THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// d_out, buckets, positions, chains, layout, kind, max_distance
PyObject* host_relpos_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args num{a};
  const at::Tensor* d = n == 7 ? tensor(a[0]) : nullptr;
  if (d == nullptr || d->dim() != 4 || !ints(*d)) Py_RETURN_NONE;
  triattn_relpos_shape s{};
  s.layout = static_cast<int>(num.integer(4));
  s.kind = static_cast<int>(num.integer(5));
  s.buckets = static_cast<int>(num.integer(1));
  s.max_distance = static_cast<int>(num.integer(6));
  if (!num.good()) Py_RETURN_NONE;
  const bool heads = s.layout == TRIATTN_RELPOS_HEADS, fp32 = heads && d->scalar_type() == at::kFloat;
  c10::DeviceIndex index = -1;
  const int64_t B = d->size(0), N = d->size(2), F = d->size(heads ? 1 : 3);
  if (!plain(*d, fp32 ? at::kFloat : at::kBFloat16, index) || d->size(heads ? 3 : 1) != N) Py_RETURN_NONE;
  s.B = static_cast<int>(B);
  s.N = static_cast<int>(N);
  s.F = static_cast<int>(F);
  s.flags = fp32 ? TRIATTN_FLAG_DOUT_FP32 : 0u;
  const int *pos, *chain;
  if (!tokens(a[2], B, N, index, pos) || !tokens(a[3], B, N, index, chain)) Py_RETURN_NONE;
  const size_t need = rel_bytes(&s);
  if (need == 0) Py_RETURN_NONE;
  at::Tensor out;
  triattn_status code;
  {
    Unlocked unlocked;
    const at::Tensor ws = bytes(need, *d);
    out = at::empty({s.buckets, F}, d->options().dtype(at::kFloat));
    code = rel_bwd(&s, d->const_data_ptr(), pos, chain, static_cast<float*>(out.mutable_data_ptr()),
                   ws.mutable_data_ptr(), need, c10::cuda::getCurrentCUDAStream(index).stream());
  }
  if (code != TRIATTN_OK) Py_RETURN_NONE;
  return THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// The triattn_matrix array of a list of matrices of device `index`, BF16 or FP32
// (outputs: BF16), as bytes; null (no exception) where one is not plainly such a
// matrix or does not have the sizes of `of`.
PyObject* matrices(PyObject* list, long index, const triattn_matrix* of) {
  const Py_ssize_t n = PyList_GET_SIZE(list);
  PyObject* out = PyBytes_FromStringAndSize(nullptr, n * static_cast<Py_ssize_t>(sizeof(triattn_matrix)));
  if (out == nullptr) throw python_error();
  triattn_matrix* m = reinterpret_cast<triattn_matrix*>(PyBytes_AS_STRING(out));
  for (Py_ssize_t i = 0; i < n; ++i) {
    const at::Tensor* t = tensor(PyList_GET_ITEM(list, i));
    const bool fp32 = t != nullptr && of == nullptr && t->scalar_type() == at::kFloat;
    if (t == nullptr || (!fp32 && t->scalar_type() != at::kBFloat16) || !t->is_cuda() || t->layout() != at::kStrided ||
        t->get_device() != index || t->dim() != 2 || !t->is_contiguous() ||
        (of != nullptr && (t->size(0) != of[i].rows || t->size(1) != of[i].cols))) {
      Py_DECREF(out);
      return nullptr;
    }
    m[i] = triattn_matrix{};
    m[i].data = const_cast<void*>(t->const_data_ptr());
    m[i].rows = t->size(0);
    m[i].cols = m[i].stride = t->size(1);
    m[i].dtype = fp32 ? TRIATTN_DTYPE_FP32 : TRIATTN_DTYPE_BF16;
  }
  return out;
}

// list of matrices, list of outputs or None, device -> (bytes, bytes or None) or None
PyObject* host_matrix_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 3 || !PyList_Check(a[0]) || !(none(a[1]) || PyList_Check(a[1]))) Py_RETURN_NONE;
  Args num{a};
  const long index = num.integer(2);
  if (!num.good() || (!none(a[1]) && PyList_GET_SIZE(a[1]) != PyList_GET_SIZE(a[0]))) Py_RETURN_NONE;
  PyObject* in = matrices(a[0], index, nullptr);
  if (in == nullptr) Py_RETURN_NONE;
  if (none(a[1])) return Py_BuildValue("(NO)", in, Py_None);
  PyObject* out = matrices(a[1], index, reinterpret_cast<const triattn_matrix*>(PyBytes_AS_STRING(in)));
  if (out == nullptr) {
    Py_DECREF(in);
    Py_RETURN_NONE;
  }
  return Py_BuildValue("(NN)", in, out);
  END_HANDLE_TH_ERRORS
}

PyObject* host_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[6];
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "six addresses expected");
    return nullptr;
  }
  for (int i = 0; i < 6; ++i)
    if ((p[i] = PyLong_AsVoidPtr(a[i])) == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is null");
      return nullptr;
    }
  qk_bytes = reinterpret_cast<decltype(qk_bytes)>(p[0]);
  qk_fwd = reinterpret_cast<decltype(qk_fwd)>(p[1]);
  qk_bwd = reinterpret_cast<decltype(qk_bwd)>(p[2]);
  rel_bytes = reinterpret_cast<decltype(rel_bytes)>(p[3]);
  rel_fwd = reinterpret_cast<decltype(rel_fwd)>(p[4]);
  rel_bwd = reinterpret_cast<decltype(rel_bwd)>(p[5]);
  Py_RETURN_NONE;
}

#define HOST_FUNCTION(name) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(host_##name)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {HOST_FUNCTION(bind),          HOST_FUNCTION(qk_norm_fwd), HOST_FUNCTION(qk_norm_bwd),
                         HOST_FUNCTION(relpos_fwd),    HOST_FUNCTION(relpos_bwd),  HOST_FUNCTION(matrix_tables),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "triattn_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_triattn_host() { return PyModule_Create(&module); }
