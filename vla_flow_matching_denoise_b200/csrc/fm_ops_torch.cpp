// Python module _ops: the calls of include/fm_ops.h on torch tensors.
//
// Checks shapes, types and devices, makes the outputs, and passes pointers to
// libfm_expert.so on the tensors' device and its current stream.  It is native
// because these calls are short: checking and allocating in Python through
// ctypes took 13-18 us of a 17-24 us call, several times its kernel.
// vla_flow_matching_denoise_b200/ops.py is the public face of it.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/grad_mode.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <optional>
#include <stdexcept>
#include <string>

#include "../../include/fm_ops.h"

namespace {

// A refusal with a ValueError's text.
struct Bad : std::runtime_error {
  using std::runtime_error::runtime_error;
};
// A failed library call.
struct Failed {
  const char* call;
  int status;
};

[[noreturn]] void bad(const char* fmt, ...) {
  char msg[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  throw Bad(msg);
}

std::string shape_of(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

enum Types { kReal, kCodes, kFloat, kInt };
bool type_ok(at::ScalarType t, Types want) {
  switch (want) {
    case kReal: return t == at::kBFloat16 || t == at::kFloat;
    case kCodes: return t == at::kFloat8_e4m3fn || t == at::kByte;
    case kFloat: return t == at::kFloat;
    default: return t == at::kInt;
  }
}
const char* type_names(Types want) {
  return want == kReal ? "bfloat16 or float32" : want == kCodes ? "float8_e4m3fn or uint8" : want == kFloat ? "float32" : "int32";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad("%s must be a CUDA tensor", name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) bad("%s must be a CUDA tensor", name);
  if (t.requires_grad() && at::GradMode::is_enabled()) bad("%s requires grad: this operator has no backward", name);
  if (t._fw_grad(/*level=*/0).defined()) bad("%s carries a forward-mode tangent: this operator has no derivative", name);
  return t;
}

// A given tensor has been written: a graph that saved it refuses its old values
// as after any operation in place.
void written(PyObject* o) {
  if (o == Py_None || o == Py_False) return;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// Row stride of a 2-D tensor with unit column stride; rows, cols < 0: any.
int64_t matrix(const at::Tensor& t, const char* name, Types types, const at::Tensor* like, int64_t rows = -1, int64_t cols = -1) {
  if (like != nullptr && t.device() != like->device())
    bad("%s is on %s, expected %s", name, t.device().str().c_str(), like->device().str().c_str());
  if (!type_ok(t.scalar_type(), types)) bad("%s is %s, expected %s", name, c10::toString(t.scalar_type()), type_names(types));
  if (t.dim() != 2 || (rows >= 0 && t.size(0) != rows) || (cols >= 0 && t.size(1) != cols))
    bad("%s has shape %s, expected [%s, %s]", name, shape_of(t).c_str(), rows < 0 ? "rows" : std::to_string(rows).c_str(),
        cols < 0 ? "columns" : std::to_string(cols).c_str());
  if (t.size(1) > 1 && t.stride(1) != 1)
    bad("%s must have contiguous rows (column stride 1, got %lld)", name, (long long)t.stride(1));
  if (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX) bad("%s has more than 2^31 - 1 rows or columns", name);
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

const at::Tensor* bf16_vector(PyObject* o, const char* name, const at::Tensor& like, int64_t n) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.device() != like.device() || t.scalar_type() != at::kBFloat16 || t.dim() != 1 || t.size(0) != n ||
      (n > 1 && t.stride(0) != 1))
    bad("%s must be a contiguous bfloat16 tensor of %lld values on %s", name, (long long)n, like.device().str().c_str());
  return &t;
}

fm_dtype dtype_of(const at::Tensor& t) { return t.scalar_type() == at::kFloat ? FM_F32 : FM_BF16; }
int64_t groups(int64_t cols) { return (cols + 127) / 128; }
at::Tensor empty(at::IntArrayRef size, const at::Tensor& like, at::ScalarType type) {
  return at::detail::empty_cuda(size, type, like.device(), std::nullopt);
}

// An output matrix: the one given, or a new one.
struct Out {
  at::Tensor t;
  int64_t ld;
};
Out out_matrix(PyObject* o, const char* name, Types types, at::ScalarType type, const at::Tensor& like, int64_t rows, int64_t cols) {
  if (o == Py_None) return Out{empty({rows, cols}, like, type), cols};
  const at::Tensor& t = tensor(o, name);
  const int64_t ld = matrix(t, name, types, &like, rows, cols);
  return Out{t, ld};
}

// The tensors' device, and the stream the call is given (an integer handle; None:
// the device's current one), are current while it allocates and launches, so
// that new outputs belong to the stream that writes them.
struct Scope {
  c10::cuda::CUDAGuard device;
  std::optional<c10::cuda::CUDAStreamGuard> stream;
  Scope(const at::Tensor& like, PyObject* handle) : device(like.device()) {
    if (handle == Py_None) return;
    void* st = PyLong_AsVoidPtr(handle);
    if (st == nullptr && PyErr_Occurred()) throw python_error();
    stream.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(st), like.device().index()));
  }
};

template <typename F>
void run(const char* call, const at::Tensor& like, F f) {
  const fm_status s = f(static_cast<void*>(c10::cuda::getCurrentCUDAStream(like.device().index()).stream()));
  if (s != FM_OK) throw Failed{call, (int)s};
}

int as_int(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  if (v < INT32_MIN || v > INT32_MAX) bad("%ld does not fit 32 bits", v);
  return (int)v;
}
double as_double(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
void* ptr(const at::Tensor& t) { return t.data_ptr(); }
void* ptr(const at::Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }

PyObject* give(const at::Tensor& t) { return THPVariable_Wrap(t); }
PyObject* give_or(PyObject* given, const at::Tensor& t) {
  if (given == Py_None) return give(t);
  Py_INCREF(given);
  return given;
}
PyObject* pack(std::initializer_list<PyObject*> items) {
  PyObject* r = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  for (PyObject* o : items) PyTuple_SET_ITEM(r, i++, o);
  return r;
}

void set_failed(const Failed& f) {
  PyObject* m = PyImport_ImportModule("vla_flow_matching_denoise_b200.binding");
  PyObject* cls = m != nullptr ? PyObject_GetAttrString(m, "FmError") : nullptr;
  if (cls != nullptr) {
    PyObject* e = PyObject_CallFunction(cls, "sis", f.call, f.status, fm_last_error(nullptr));
    if (e != nullptr) PyErr_SetObject(cls, e);
    Py_XDECREF(e);
  }
  Py_XDECREF(cls);
  Py_XDECREF(m);
}

#define ENTRY(n)                                                                    \
  HANDLE_TH_ERRORS                                                                  \
  if (nargs != (n)) {                                                               \
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");                  \
    return nullptr;                                                                 \
  }                                                                                 \
  try {
#define LEAVE                                      \
  }                                                \
  catch (const Bad& e) {                           \
    PyErr_SetString(PyExc_ValueError, e.what());   \
    return nullptr;                                \
  }                                                \
  catch (const Failed& f) {                        \
    set_failed(f);                                 \
    return nullptr;                                \
  }                                                \
  END_HANDLE_TH_ERRORS

// (x, gain, residual, eps, gain_offset, h_out, codes, scales, stream) -> (h, codes, scales)
PyObject* add_rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ENTRY(9)
  const at::Tensor& x = tensor(a[0], "x");
  const Scope scope(x, a[8]);
  const int64_t ldx = matrix(x, "x", kReal, nullptr), rows = x.size(0), d = x.size(1);
  const at::Tensor* gain = bf16_vector(a[1], "gain", x, d);
  const at::Tensor* res = a[2] == Py_None ? nullptr : &tensor(a[2], "residual");
  const int64_t ldr = res != nullptr ? matrix(*res, "residual", kReal, &x, rows, d) : 0;
  at::Tensor h;
  int64_t ldh = 0;
  if (a[5] != Py_None || res != nullptr) {
    Out o = out_matrix(a[5], "h_out", kReal, res != nullptr ? res->scalar_type() : x.scalar_type(), x, rows, d);
    h = o.t;
    ldh = o.ld;
    if (res != nullptr && h.scalar_type() != res->scalar_type()) bad("h_out is not of the residual's type");
  }
  const fm_dtype ht = h.defined() ? dtype_of(h) : dtype_of(x);
  Out c = out_matrix(a[6], "codes", kCodes, at::kFloat8_e4m3fn, x, rows, d);
  Out s = out_matrix(a[7], "scales", kFloat, at::kFloat, x, rows, groups(d));
  const float eps = (float)as_double(a[3]), off = (float)as_double(a[4]);
  run("fm_add_rmsnorm_e4m3", x, [&](void* st) {
    return fm_add_rmsnorm_e4m3(ptr(x), dtype_of(x), ldx, ptr(res), ht, ldr, (const uint16_t*)ptr(gain), off, eps, (int)rows,
                               (int)d, h.defined() ? ptr(h) : nullptr, ldh, (uint8_t*)ptr(c.t), c.ld, (float*)ptr(s.t), s.ld, st);
  });
  for (int i = 5; i < 8; ++i) written(a[i]);
  PyObject* ho;
  if (a[5] == Py_None && h.defined()) {
    ho = give(h);
  } else {
    ho = a[5] != Py_None ? a[5] : a[0];
    Py_INCREF(ho);
  }
  return pack({ho, give_or(a[6], c.t), give_or(a[7], s.t)});
  LEAVE
}

// (x, act, codes, scales, stream) -> (codes, scales)
PyObject* gated(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ENTRY(5)
  const at::Tensor& x = tensor(a[0], "x");
  const Scope scope(x, a[4]);
  const int64_t ldx = matrix(x, "x", kReal, nullptr), rows = x.size(0);
  const int act = as_int(a[1]);
  int64_t f = x.size(1);
  if (act != FM_ACT_NONE) {
    if (f % 2 != 0) bad("x has %lld columns: gate and up need an even number", (long long)f);
    f /= 2;
  }
  Out c = out_matrix(a[2], "codes", kCodes, at::kFloat8_e4m3fn, x, rows, f);
  Out s = out_matrix(a[3], "scales", kFloat, at::kFloat, x, rows, groups(f));
  run("fm_gated_e4m3", x, [&](void* st) {
    return fm_gated_e4m3(ptr(x), dtype_of(x), ldx, (fm_act)act, (int)rows, (int)f, (uint8_t*)ptr(c.t), c.ld, (float*)ptr(s.t),
                         s.ld, st);
  });
  written(a[2]);
  written(a[3]);
  return pack({give_or(a[2], c.t), give_or(a[3], s.t)});
  LEAVE
}

// (w, stream) -> (codes, scales)
PyObject* quantize_weight(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ENTRY(2)
  const at::Tensor& w = tensor(a[0], "w");
  if (w.scalar_type() != at::kBFloat16) bad("w is %s, expected bfloat16", c10::toString(w.scalar_type()));
  const Scope scope(w, a[1]);
  const int64_t ldw = matrix(w, "w", kReal, nullptr), n = w.size(0), k = w.size(1);
  at::Tensor c = empty({n, k}, w, at::kFloat8_e4m3fn), s = empty({groups(n), groups(k)}, w, at::kFloat);
  run("fm_quantize_weight_e4m3_b128", w, [&](void* st) {
    return fm_quantize_weight_e4m3_b128((const uint16_t*)ptr(w), ldw, (int)n, (int)k, (uint8_t*)ptr(c), k, (float*)ptr(s),
                                        groups(k), st);
  });
  return pack({give(c), give(s)});
  LEAVE
}

// (a, sa, w, sw, bias, out, f32, stream) -> out
PyObject* gemm(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ENTRY(8)
  const at::Tensor& x = tensor(a[0], "a");
  const Scope scope(x, a[7]);
  const int64_t lda = matrix(x, "a", kCodes, nullptr), m = x.size(0), k = x.size(1), g = groups(k);
  const at::Tensor& w = tensor(a[2], "w");
  const int64_t ldw = matrix(w, "w", kCodes, &x, -1, k), n = w.size(0);
  const at::Tensor& sa = tensor(a[1], "sa");
  const int64_t ldsa = matrix(sa, "sa", kFloat, &x, m, g);
  const at::Tensor& sw = tensor(a[3], "sw");
  const int64_t ldsw = matrix(sw, "sw", kFloat, &x, groups(n), g);
  const at::Tensor* bias = bf16_vector(a[4], "bias", x, n);
  Out o = out_matrix(a[5], "out", kReal, a[6] == Py_True ? at::kFloat : at::kBFloat16, x, m, n);
  run("fm_gemm_e4m3_b128", x, [&](void* st) {
    return fm_gemm_e4m3_b128((const uint8_t*)ptr(x), lda, (const float*)ptr(sa), ldsa, (const uint8_t*)ptr(w), ldw,
                             (const float*)ptr(sw), ldsw, (const uint16_t*)ptr(bias), (int)m, (int)n, (int)k, ptr(o.t),
                             dtype_of(o.t), o.ld, st);
  });
  written(a[5]);
  return give_or(a[5], o.t);
  LEAVE
}

// A [rows, heads, hd] output: a new one (None), none (False) or the one given.
struct Heads {
  at::Tensor t;
  int64_t ld = 0;
};
Heads heads_out(PyObject* o, const char* name, const at::Tensor& x, int64_t rows, int64_t heads, int64_t hd) {
  if (o == Py_False) return Heads{};
  if (o == Py_None) return Heads{empty({rows, heads, hd}, x, x.scalar_type()), heads * hd};
  const at::Tensor& t = tensor(o, name);
  if (t.device() != x.device() || t.scalar_type() != x.scalar_type() || t.dim() != 3 || t.size(0) != rows ||
      t.size(1) != heads || t.size(2) != hd)
    bad("%s must be a %s tensor [%lld, %lld, %lld] on %s", name, c10::toString(x.scalar_type()), (long long)rows,
        (long long)heads, (long long)hd, x.device().str().c_str());
  if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != hd)) bad("%s must have contiguous heads in each row", name);
  return Heads{t, rows > 1 ? t.stride(0) : heads * hd};
}

// A contiguous 1-D buffer of `size`-byte elements of struct format `code`.
struct View {
  Py_buffer b;
  View(PyObject* o, char code, Py_ssize_t size) {
    const int flags = PyBUF_ND | PyBUF_FORMAT | PyBUF_C_CONTIGUOUS;
    if (PyObject_GetBuffer(o, &b, flags) != 0) throw python_error();
    if (b.ndim != 1 || b.itemsize != size || b.format == nullptr || b.format[0] != code || b.format[1] != 0) {
      PyBuffer_Release(&b);
      bad("pairs must be (uint8 [n], float64 [n]) contiguous arrays (see rope_pairs)");
    }
  }
  View(const View&) = delete;
  ~View() { PyBuffer_Release(&b); }
  Py_ssize_t size() const { return b.shape[0]; }
};

// (x, positions, axis, freq, n_q, n_kv, head_dim, q_out, k_out, v_out, stream) -> (q, k, v)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ENTRY(11)
  const at::Tensor& x = tensor(a[0], "x");
  const Scope scope(x, a[10]);
  const int64_t ldx = matrix(x, "x", kReal, nullptr), rows = x.size(0);
  const int n_q = as_int(a[4]), n_kv = as_int(a[5]), hd = as_int(a[6]);
  if (n_q < 0 || n_kv < 0 || hd < 1 || n_q > 1024 || n_kv > 1024 || hd > 256)
    bad("n_q %d / n_kv %d / head_dim %d out of range (0 .. 1024 heads of 2 .. 256)", n_q, n_kv, hd);
  const bool with_v = a[9] != Py_False;
  const int64_t want = (int64_t)(n_q + (with_v ? 2 : 1) * n_kv) * hd;
  if (x.size(1) < want || (with_v && x.size(1) != want)) bad("x has %lld columns, expected %lld", (long long)x.size(1), (long long)want);
  const at::Tensor& pos = tensor(a[1], "positions");
  int64_t ldp, axes;
  if (pos.dim() == 1) {
    if (pos.scalar_type() != at::kInt || pos.device() != x.device() || pos.size(0) != rows || (rows > 1 && pos.stride(0) != 1))
      bad("positions must be a contiguous int32 tensor of %lld values on %s", (long long)rows, x.device().str().c_str());
    ldp = rows;
    axes = 1;
  } else {
    ldp = matrix(pos, "positions", kInt, &x, -1, rows);
    axes = pos.size(0);
  }
  Heads q = heads_out(a[7], "q_out", x, rows, n_q, hd), k = heads_out(a[8], "k_out", x, rows, n_kv, hd),
        v = heads_out(a[9], "v_out", x, rows, n_kv, hd);
  const View axis(a[2], 'B', 1), freq(a[3], 'd', 8);
  if (axis.size() != freq.size() || axis.size() > 256) bad("pairs: %lld axes and %lld frequencies", (long long)axis.size(), (long long)freq.size());
  auto at_ = [](const Heads& h) { return h.t.defined() ? ptr(h.t) : nullptr; };
  run("fm_rope_axes", x, [&](void* st) {
    return fm_rope_axes(ptr(x), dtype_of(x), ldx, (int)rows, n_q, n_kv, hd, (const int32_t*)ptr(pos), ldp, (int)axes, (const uint8_t*)axis.b.buf,
                        (const double*)freq.b.buf, (int)axis.size(), at_(q), q.ld, at_(k), k.ld, at_(v), v.ld, st);
  });
  for (int i = 7; i < 10; ++i) written(a[i]);
  auto back = [](PyObject* o, const Heads& h) {
    if (o == Py_False) o = Py_None;
    else if (o == Py_None) return give(h.t);
    Py_INCREF(o);
    return o;
  };
  return pack({back(a[7], q), back(a[8], k), back(a[9], v)});
  LEAVE
}

#define METHOD(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {METHOD(add_rmsnorm), METHOD(gated), METHOD(quantize_weight), METHOD(gemm), METHOD(rope),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// The Python and torch this was built with; the build looks for it in the file.
#ifndef FM_OPS_BUILT_FOR
#define FM_OPS_BUILT_FOR "fm_ops"
#endif
PyMODINIT_FUNC PyInit__ops(void) {
  PyObject* m = PyModule_Create(&kModule);
  if (m != nullptr && PyModule_AddStringConstant(m, "built_for", FM_OPS_BUILT_FOR) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
