// The 8-bit prefix operators on PyTorch tensors (the work behind int8.py):
// checks of the tensors, allocation of the results and the call into libpae,
// whose functions are handed over as addresses.  In Python, with ctypes, the
// same cost 10 us for a quantiser call and 15 us for an attention with fresh
// keys, more than the kernels take on small inputs (4 and 8 us); here the C call
// and the allocations are what is left.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pae.h"

namespace {

using at::Tensor;

struct Functions {
  decltype(&pae_quantize_rows) quantize_rows;
  decltype(&pae_linear_i8) linear_i8;
  decltype(&pae_kv8_write) kv8_write;
  decltype(&pae_kv8_read) kv8_read;
  decltype(&pae_kv8_attention) kv8_attention;
} g_f;
PyObject* g_check = nullptr;  // check(status): raises the package's error

constexpr int64_t kMost = 1 << 30;  // of a size: the library takes 32-bit integers

// A failed check: the message, as a ValueError (TypeError).
struct Refused {
  PyObject* type;
  std::string message;
};
[[noreturn]] void refuse(std::string message) { throw Refused{PyExc_ValueError, std::move(message)}; }

const Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, std::string(what) + " must be a tensor"};
  return THPVariable_Unpack(o);
}
// None: an undefined tensor
Tensor optional_tensor(PyObject* o, const char* what) { return o == Py_None ? Tensor() : tensor(o, what); }

int dtype_code(at::ScalarType t, const char* what) {
  if (t == at::kFloat) return PAE_FP32;
  if (t == at::kBFloat16) return PAE_BF16;
  refuse(std::string(what) + " must be torch.float32 or torch.bfloat16, not " + at::toString(t));
}
at::ScalarType dtype_of(PyObject* o) {
  if (!THPDtype_Check(o)) throw Refused{PyExc_TypeError, "dtype must be a torch.dtype"};
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

// All tensors that are there must be on CUDA device `device` (-1: the first
// one's); returns it.
int one_device(int device, std::initializer_list<const Tensor*> ts) {
  for (const Tensor* t : ts) {
    if (!t->defined()) continue;
    if (!t->is_cuda()) refuse("tensors must be on a CUDA device");
    if (device < 0) device = t->get_device();
    if (t->get_device() != device)
      refuse("tensors are on cuda:" + std::to_string(device) + " and cuda:" + std::to_string(t->get_device()) + ": one device is needed");
  }
  return device;
}

const void* vector(const Tensor& t, int64_t n, at::ScalarType type, const char* what) {
  if (t.scalar_type() != type || t.dim() != 1 || t.numel() != n || !t.is_contiguous())
    refuse(std::string(what) + " must be a contiguous " + at::toString(type) + " vector of " + std::to_string(n));
  return t.const_data_ptr();
}

// Runs f(stream) with `device` current, on its current stream.
template <typename F>
bool run(int device, F f) {
  c10::cuda::OptionalCUDAGuard guard;
  if (c10::cuda::current_device() != device) guard.set_index(static_cast<c10::DeviceIndex>(device));
  const auto stream = reinterpret_cast<pae_stream>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream());
  int status;
  Py_BEGIN_ALLOW_THREADS;
  status = static_cast<int>(f(stream));
  Py_END_ALLOW_THREADS;
  if (status == PAE_OK) return true;
  PyObject* r = PyObject_CallFunction(g_check, "i", status);
  if (r) {
    Py_DECREF(r);
    PyErr_SetString(PyExc_RuntimeError, "the library refused the call");
  }
  return false;
}

PyObject* pair(Tensor a, Tensor b) {
  PyObject *x = THPVariable_Wrap(std::move(a)), *y = THPVariable_Wrap(std::move(b));
  PyObject* t = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return t;
}

Tensor empty(at::IntArrayRef shape, const Tensor& like, at::ScalarType type) { return at::empty(shape, like.options().dtype(type)); }

// Every function: f(args) with `n` arguments, its refusals and C++ exceptions
// as Python errors.
#define ARGUMENTS(n)                                                                        \
  HANDLE_TH_ERRORS                                                                          \
  if (nargs != (n)) return PyErr_Format(PyExc_TypeError, "%d arguments expected", (int)(n)); \
  try {
#define END_ARGUMENTS                                 \
  }                                                   \
  catch (const Refused& r) {                          \
    PyErr_SetString(r.type, r.message.c_str());       \
    return nullptr;                                   \
  }                                                   \
  END_HANDLE_TH_ERRORS

// quantize_rows(x, rms_eps or None) -> codes, scale
PyObject* quantize_rows(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGUMENTS(2)
  const Tensor& x = tensor(a[0], "x");
  if (x.dim() != 2) refuse("x must be [rows, width]");
  const int64_t rows = x.size(0), width = x.size(1);
  if (width < 1) refuse("x must have width >= 1");
  if (rows > kMost || width > kMost) refuse("x must have at most 2^30 rows and columns");
  if (x.stride(1) != 1 && width > 1) refuse("x must be contiguous along width");
  const int code = dtype_code(x.scalar_type(), "x");
  double eps = 0.0;
  if (a[1] != Py_None) {
    eps = PyFloat_AsDouble(a[1]);
    if (eps == -1.0 && PyErr_Occurred()) return nullptr;
    if (!(eps > 1e-45)) refuse("rms_eps must be positive");  // (the library takes a float, 0 stands for no norm)
  }
  const int device = one_device(-1, {&x});
  Tensor codes = empty({rows, width}, x, at::kChar), scale = empty({rows}, x, at::kFloat);
  if (!run(device, [&](pae_stream s) {
        return g_f.quantize_rows(x.const_data_ptr(), rows > 1 ? x.stride(0) : width, (int)rows, (int)width, code, (float)eps,
                                 static_cast<signed char*>(codes.mutable_data_ptr()), static_cast<float*>(scale.mutable_data_ptr()), s);
      }))
    return nullptr;
  return pair(std::move(codes), std::move(scale));
  END_ARGUMENTS
}

// linear_i8(x, x_scale, w, w_scale, out_dtype, out or None) -> out
PyObject* linear_i8(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGUMENTS(6)
  const Tensor &x = tensor(a[0], "x"), &xs = tensor(a[1], "x_scale"), &w = tensor(a[2], "w"), &ws = tensor(a[3], "w_scale");
  Tensor out = optional_tensor(a[5], "out");
  if (x.dim() != 2 || w.dim() != 2) refuse("x must be [tokens, k] and w [n, k]");
  const int64_t tokens = x.size(0), k = x.size(1), n = w.size(0);
  if (k != w.size(1)) refuse("x [tokens, k] and w [n, k] must share k");
  if (tokens > kMost || n > kMost || k > kMost) refuse("tokens, n and k must be at most 2^30");
  if (x.scalar_type() != at::kChar || w.scalar_type() != at::kChar) refuse("x and w must be int8 codes");
  if (!x.is_contiguous() || !w.is_contiguous()) refuse("x and w must be contiguous");
  const auto* px = static_cast<const float*>(vector(xs, tokens, at::kFloat, "x_scale"));
  const auto* pw = static_cast<const float*>(vector(ws, n, at::kFloat, "w_scale"));
  const int device = one_device(-1, {&x, &xs, &w, &ws, &out});
  const int code = dtype_code(out.defined() ? out.scalar_type() : dtype_of(a[4]), "out");
  if (!out.defined())
    out = empty({tokens, n}, x, code == PAE_BF16 ? at::kBFloat16 : at::kFloat);
  else if (out.dim() != 2 || out.size(0) != tokens || out.size(1) != n || (out.stride(1) != 1 && n > 1))
    refuse("out must be [tokens, n], contiguous along n");
  if (!run(device, [&](pae_stream s) {
        return g_f.linear_i8(static_cast<const signed char*>(x.const_data_ptr()), px, static_cast<const signed char*>(w.const_data_ptr()),
                             pw, (int)tokens, (int)n, (int)k, out.mutable_data_ptr(), tokens > 1 ? out.stride(0) : n, code, s);
      }))
    return nullptr;
  return THPVariable_Wrap(std::move(out));
  END_ARGUMENTS
}

// The cache's first two arguments: its pae_kv8 as bytes, its device.
const pae_kv8* cache_of(PyObject* o) {
  if (!PyBytes_Check(o) || PyBytes_GET_SIZE(o) != (Py_ssize_t)sizeof(pae_kv8)) throw Refused{PyExc_TypeError, "not a cache"};
  return reinterpret_cast<const pae_kv8*>(PyBytes_AS_STRING(o));
}

int device_of(PyObject* o) {
  const long device = PyLong_AsLong(o);
  if (device < 0) refuse("the cache must be on a CUDA device");
  return (int)device;
}

struct Sequences {
  int n = 1;
  const int *cu = nullptr, *start = nullptr;
  Sequences(const pae_kv8* c, const Tensor& cu_rows, const Tensor& at) {
    if (cu_rows.defined()) {
      if (cu_rows.dim() != 1 || cu_rows.size(0) < 1) refuse("cu_rows must be a contiguous Int vector of n_seq + 1");
      if (cu_rows.size(0) - 1 > c->n_slots)
        refuse("cu_rows names " + std::to_string(cu_rows.size(0) - 1) + " sequences, the cache has " + std::to_string(c->n_slots) + " slots");
      n = (int)cu_rows.size(0) - 1;
      cu = static_cast<const int*>(vector(cu_rows, n + 1, at::kInt, "cu_rows"));
    }
    if (at.defined()) start = static_cast<const int*>(vector(at, n, at::kInt, "start"));
  }
};

// kv8_write(cache, device, k, v, cu_rows or None, start or None)
PyObject* kv8_write(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGUMENTS(6)
  const pae_kv8* c = cache_of(a[0]);
  const Tensor &k = tensor(a[2], "k"), &v = tensor(a[3], "v"), cu = optional_tensor(a[4], "cu_rows"), start = optional_tensor(a[5], "start");
  if (k.sizes() != v.sizes() || k.scalar_type() != v.scalar_type()) refuse("k and v must have the same shape and type");
  if (k.dim() != 3 || k.size(0) > kMost) refuse("k and v must be [rows, n_kv_heads, head_dim] with at most 2^30 rows");
  const int code = dtype_code(k.scalar_type(), "k and v");
  long long strides[2][2];
  for (int i = 0; i < 2; ++i) {
    const Tensor& t = i ? v : k;
    if (t.size(1) != c->n_kv_heads || t.size(2) != c->head_dim || t.stride(2) != 1)
      refuse("k and v must be [rows, " + std::to_string(c->n_kv_heads) + ", " + std::to_string(c->head_dim) +
             "], contiguous along the last dimension");
    strides[i][0] = t.size(0) > 1 ? t.stride(0) : 0;
    strides[i][1] = t.size(1) > 1 ? t.stride(1) : 0;
  }
  const Sequences s(c, cu, start);
  const int device = one_device(device_of(a[1]), {&k, &v, &cu, &start});
  if (!run(device, [&](pae_stream st) {
        return g_f.kv8_write(c, k.const_data_ptr(), v.const_data_ptr(), strides[0], strides[1], s.cu, s.start, s.n, (int)k.size(0), code, st);
      }))
    return nullptr;
  Py_RETURN_NONE;
  END_ARGUMENTS
}

// kv8_read(cache, device, cu_rows or None, start or None, n_rows, dtype) -> k, v
PyObject* kv8_read(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGUMENTS(6)
  const pae_kv8* c = cache_of(a[0]);
  const Tensor cu = optional_tensor(a[2], "cu_rows"), start = optional_tensor(a[3], "start");
  const int64_t rows = PyLong_AsLongLong(a[4]);
  if (rows == -1 && PyErr_Occurred()) return nullptr;
  if (rows < 0 || rows > kMost) refuse("n_rows must be in [0, 2^30]");
  const at::ScalarType type = dtype_of(a[5]);
  const int code = dtype_code(type, "dtype");
  const Sequences s(c, cu, start);
  const int device = one_device(device_of(a[1]), {&cu, &start});
  const auto options = at::TensorOptions().device(at::kCUDA, static_cast<c10::DeviceIndex>(device)).dtype(type);
  Tensor k = at::empty({rows, c->n_kv_heads, c->head_dim}, options), v = at::empty({rows, c->n_kv_heads, c->head_dim}, options);
  if (!run(device, [&](pae_stream st) {
        return g_f.kv8_read(c, k.mutable_data_ptr(), v.mutable_data_ptr(), nullptr, nullptr, s.cu, s.start, s.n, (int)rows, code, st);
      }))
    return nullptr;
  return pair(std::move(k), std::move(v));
  END_ARGUMENTS
}

void rows_of(const Tensor& t, int64_t heads, const pae_kv8* c, long long* strides, const char* what) {
  if (t.dim() != 4 || t.scalar_type() != at::kBFloat16 || t.size(2) != heads || t.size(3) != c->head_dim || t.stride(3) != 1)
    refuse(std::string(what) + " must be bfloat16 [n_seq, n, " + std::to_string(heads) + ", " + std::to_string(c->head_dim) +
           "], contiguous along the last dimension");
  for (int i = 0; i < 3; ++i) strides[i] = t.size(i) > 1 ? t.stride(i) : 0;
}

// kv8_attend(cache, device, q, lens, causal, k_new, v_new, scale, out, plan)
// (k_new .. out: or None; plan: (n_seq, n_q, n_q_heads, n_new, workspace or None)) -> out
PyObject* kv8_attend(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGUMENTS(10)
  const pae_kv8* c = cache_of(a[0]);
  const Tensor &q = tensor(a[2], "q"), &lens = tensor(a[3], "lens");
  const Tensor k = optional_tensor(a[5], "k_new"), v = optional_tensor(a[6], "v_new");
  Tensor out = optional_tensor(a[8], "out");
  const int causal = PyObject_IsTrue(a[4]);
  if (causal < 0) return nullptr;
  double scale = 0.0;
  if (a[7] != Py_None) {
    scale = PyFloat_AsDouble(a[7]);
    if (scale == -1.0 && PyErr_Occurred()) return nullptr;
    if ((float)scale == 0.0f) refuse("scale must not be 0");  // (0 stands for the default)
  }
  pae_kv8_query query{};
  if (q.dim() != 4) refuse("q must be [n_seq, n_q, n_q_heads, head_dim]");
  const int64_t n_seq = q.size(0), n_q = q.size(1), heads = q.size(2);
  if (n_seq > kMost || n_q > kMost || heads > kMost) refuse("q must have at most 2^30 rows and heads");
  if (k.defined() != v.defined()) refuse("k_new and v_new go together");
  const int device = one_device(device_of(a[1]), {&q, &lens, &k, &v, &out});
  query.lens = static_cast<const int*>(vector(lens, n_seq, at::kInt, "lens"));
  rows_of(q, heads, c, query.q_strides, "q");
  if (k.defined()) {
    if (k.sizes() != v.sizes() || k.dim() != 4 || k.size(0) != n_seq) refuse("k_new and v_new must be [n_seq, n_new, n_kv_heads, head_dim]");
    if (k.size(1) > kMost) refuse("k_new and v_new must have at most 2^30 rows");
    rows_of(k, c->n_kv_heads, c, query.k_new_strides, "k_new");
    rows_of(v, c->n_kv_heads, c, query.v_new_strides, "v_new");
    query.n_new = (int)k.size(1);
    query.k_new = k.const_data_ptr();
    query.v_new = v.const_data_ptr();
  }
  if (!PyTuple_Check(a[9]) || PyTuple_GET_SIZE(a[9]) != 5) throw Refused{PyExc_TypeError, "not a plan"};
  const int64_t key[4] = {n_seq, n_q, heads, query.n_new};
  for (int i = 0; i < 4; ++i)
    if (PyLong_AsLongLong(PyTuple_GET_ITEM(a[9], i)) != key[i])
      refuse("the plan is for another call: this one has n_seq " + std::to_string(n_seq) + ", n_q " + std::to_string(n_q) +
             ", n_q_heads " + std::to_string(heads) + ", fresh " + std::to_string(query.n_new));
  const Tensor ws = optional_tensor(PyTuple_GET_ITEM(a[9], 4), "workspace");
  if (ws.defined() && ws.get_device() != device) refuse("the plan is for another device");
  if (!out.defined()) out = empty(q.sizes(), q, at::kBFloat16);
  else if (out.sizes() != q.sizes()) refuse("out must have the shape of q");
  rows_of(out, heads, c, query.out_strides, "out");
  query.q = q.const_data_ptr();
  query.out = out.mutable_data_ptr();
  query.n_seq = (int)n_seq;
  query.n_q = (int)n_q;
  query.n_q_heads = (int)heads;
  query.causal = causal;
  query.scale = (float)scale;
  if (!run(device, [&](pae_stream s) {
        return g_f.kv8_attention(c, &query, ws.defined() ? ws.mutable_data_ptr() : nullptr, ws.defined() ? (size_t)ws.nbytes() : 0, s);
      }))
    return nullptr;
  return THPVariable_Wrap(std::move(out));
  END_ARGUMENTS
}

// bind((addresses of the five functions), check)
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long f[5];
  PyObject* check;
  if (!PyArg_ParseTuple(args, "(KKKKK)O", &f[0], &f[1], &f[2], &f[3], &f[4], &check)) return nullptr;
  g_f.quantize_rows = reinterpret_cast<decltype(g_f.quantize_rows)>(f[0]);
  g_f.linear_i8 = reinterpret_cast<decltype(g_f.linear_i8)>(f[1]);
  g_f.kv8_write = reinterpret_cast<decltype(g_f.kv8_write)>(f[2]);
  g_f.kv8_read = reinterpret_cast<decltype(g_f.kv8_read)>(f[3]);
  g_f.kv8_attention = reinterpret_cast<decltype(g_f.kv8_attention)>(f[4]);
  Py_INCREF(check);
  Py_XDECREF(g_check);
  g_check = check;
  Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr},
                         FAST(quantize_rows),
                         FAST(linear_i8),
                         FAST(kv8_write),
                         FAST(kv8_read),
                         FAST(kv8_attend),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_int8_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__int8_tensors() { return PyModule_Create(&module); }
