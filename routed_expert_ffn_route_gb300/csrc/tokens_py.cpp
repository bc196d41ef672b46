// tokens_py.cpp -- the token operators' entry points for Python.
//
// The package's other functions go through ctypes.  A call of a token operator has up to six
// tensors and twenty arguments; reading the tensors from Python and converting the arguments with
// ctypes took 5 us, twice the launch, and at decode sizes that is most of the call (7.3 us for a
// norm of one row, 2.3 this way).  These functions read the tensors through torch's C++ headers,
// check them, and call the C entry point with the operands' device current, on that device's
// current stream or a given one, with the interpreter's lock released.  They return its status;
// wrong shapes and strides raise ValueError, wrong types TypeError.  They are private: tokens.py
// documents them.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/grad_mode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <exception>
#include <initializer_list>
#include <string>
#include <vector>

#include "../../include/moe.h"

namespace {

struct Raised {};  // a Python exception is set

[[noreturn]] void raise(PyObject *type, const std::string &text) {
  PyErr_SetString(type, text.c_str());
  throw Raised{};
}

const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

int row_type(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return MOE_DT_F32;
    case at::kBFloat16: return MOE_DT_BF16;
    case at::kHalf: return MOE_DT_F16;
    case at::kFloat8_e4m3fn: return MOE_DT_E4M3;
    default:
      raise(PyExc_TypeError, "rows must be float32, bfloat16, float16 or float8_e4m3fn, got " +
                                 std::string(c10::toString(t)));
  }
}

std::string text(std::initializer_list<int64_t> shape) {
  std::string s = "[";
  for (int64_t v : shape) s += (s.size() > 1 ? ", " : "") + std::to_string(v);
  return s + "]";
}

// a 32-bit size of the C interface
int size32(int64_t v, const char *name) {
  if (v > 2147483647 || v < -2147483647 - 1)
    raise(PyExc_ValueError, std::string(name) + " is out of range: " + std::to_string(v));
  return (int)v;
}

// the interpreter's lock, released for a scope
struct Unlocked {
  PyThreadState *state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// an attribute of a stream object as a Python integer; null where there is none and it may be so
PyObject *attribute(PyObject *o, PyObject *name, bool needed) {
  PyObject *v = PyObject_GetAttr(o, name);
  if (v) return v;
  if (needed || !PyErr_ExceptionMatches(PyExc_AttributeError)) throw Raised{};
  PyErr_Clear();
  return nullptr;
}

// the handle of a torch.cuda.Stream, which must be one of device `dev`
void *handle(PyObject *stream, int dev) {
  static PyObject *device_index = PyUnicode_InternFromString("device_index");
  static PyObject *cuda_stream = PyUnicode_InternFromString("cuda_stream");
  if (PyObject *d = attribute(stream, device_index, false)) {
    const long on = PyLong_AsLong(d);
    Py_DECREF(d);
    if (on == -1 && PyErr_Occurred()) throw Raised{};
    if (on != dev)
      raise(PyExc_ValueError, "the stream is on device " + std::to_string(on) +
                                  ", the operands are on device " + std::to_string(dev));
  }
  PyObject *h = attribute(stream, cuda_stream, true);
  void *s = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (PyErr_Occurred()) throw Raised{};
  return s;
}

// Runs body(stream) with device `dev`, the operands', current.  A stream's handle does not say
// where a kernel runs: every device's default stream has the handle 0, and launches, SM counts and
// kernel attributes go by the calling thread's device.  RT: the CUDA runtime, or its stand-in.
template <typename RT, typename F>
long on_device(int dev, PyObject *stream, F body) {
  if (dev < 0) raise(PyExc_ValueError, "operands must be on a CUDA device");
  void *st = stream == Py_None ? RT::current(dev) : handle(stream, dev);
  const typename RT::Guard guard((c10::DeviceIndex)dev);
  const Unlocked unlocked;
  return body(st);
}

struct Cuda {
  struct Guard {  // one look at the current device where it is the right one
    c10::cuda::OptionalCUDAGuard g;
    explicit Guard(c10::DeviceIndex dev) {
      if (c10::cuda::current_device() != dev) g.set_index(dev);
    }
  };
  static void *current(int dev) {
    return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
  }
};

// What a call would do to the runtime, in order, without a GPU (for the tests).
struct Told {
  static std::vector<std::string> &steps() {
    static thread_local std::vector<std::string> s;
    return s;
  }
  struct Guard {
    explicit Guard(c10::DeviceIndex d) { steps().push_back("set " + std::to_string(d)); }
    ~Guard() { steps().push_back("restore"); }
  };
  static void *current(int dev) {
    steps().push_back("current stream of " + std::to_string(dev));
    return nullptr;  // a default stream
  }
};

// The operands of one call: all on one CUDA device.
struct Call {
  int dev;
  c10::SmallVector<const at::Tensor *, 4> written;
  explicit Call(const at::Tensor &first) : dev(first.is_cuda() ? first.get_device() : -1) {}

  void check(const at::Tensor &t, const char *name, at::ScalarType type,
             std::initializer_list<int64_t> shape) const {
    if (!t.sizes().equals(c10::IntArrayRef(shape.begin(), shape.size()))) {
      std::string got = "[";
      for (int64_t v : t.sizes()) got += (got.size() > 1 ? ", " : "") + std::to_string(v);
      raise(PyExc_ValueError,
            std::string(name) + " must have shape " + text(shape) + ", got " + got + "]");
    }
    if (t.scalar_type() != type)
      raise(PyExc_TypeError, std::string(name) + " must be " + c10::toString(type) + ", got " +
                                 c10::toString(t.scalar_type()));
    if ((t.is_cuda() ? t.get_device() : -1) != dev)
      raise(PyExc_ValueError, std::string(name) + " is on another device than the first operand");
  }
  // rows that may lie apart: the address, and the distance between rows
  void *rows(PyObject *o, const char *name, at::ScalarType type, int64_t n, int64_t width,
             long &ld) const {
    const at::Tensor &t = tensor(o, name);
    check(t, name, type, {n, width});
    ld = (long)t.stride(0);
    if (width > 1 && t.stride(1) != 1)
      raise(PyExc_ValueError, std::string(name) + "'s last dimension must be contiguous");
    if (ld < width) {
      if (n > 1) raise(PyExc_ValueError, std::string(name) + "'s rows overlap");
      ld = (long)width;
    }
    return t.data_ptr();
  }
  void *rows_or_null(PyObject *o, const char *name, at::ScalarType type, int64_t n, int64_t width,
                     long &ld) const {
    ld = 0;
    return o == Py_None ? nullptr : rows(o, name, type, n, width, ld);
  }
  void *flat(PyObject *o, const char *name, at::ScalarType type,
             std::initializer_list<int64_t> shape) const {
    const at::Tensor &t = tensor(o, name);
    check(t, name, type, shape);
    if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
    return t.data_ptr();
  }
  void *flat_or_null(PyObject *o, const char *name, at::ScalarType type,
                     std::initializer_list<int64_t> shape) const {
    return o == Py_None ? nullptr : flat(o, name, type, shape);
  }
  // The same for a tensor that the call writes.  Autograd does not see the call: a tensor that is
  // part of a graph may not be written while graphs are recorded, and the others' version counters
  // move on, so that a backward pass finds out when a tensor that it saved has been overwritten.
  void writes(PyObject *o, const char *name) {
    const at::Tensor &t = tensor(o, name);
    if (t.requires_grad() && at::GradMode::is_enabled())
      raise(PyExc_ValueError, std::string(name) + " requires a gradient, and autograd does not "
                              "record the call: write it under torch.no_grad()");
    written.push_back(&t);
  }
  void *out_rows(PyObject *o, const char *name, at::ScalarType type, int64_t n, int64_t width,
                 long &ld) {
    writes(o, name);
    return rows(o, name, type, n, width, ld);
  }
  void *out_flat(PyObject *o, const char *name, at::ScalarType type,
                 std::initializer_list<int64_t> shape) {
    writes(o, name);
    return flat(o, name, type, shape);
  }
  // body(stream) on the operands' device
  template <typename F>
  long launch(PyObject *stream, F body) const {
    const long status = on_device<Cuda>(dev, stream, body);
    if (status == MOE_OK)
      for (const at::Tensor *t : written)
        if (!t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
    return status;
  }
};

int64_t dim(const at::Tensor &t, const char *name, int dims, int i) {
  if (t.dim() != dims)
    raise(PyExc_ValueError, std::string(name) + " must have " + std::to_string(dims) +
                                " dimensions, got " + std::to_string(t.dim()));
  return t.size(i);
}

long number(PyObject *o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
int number32(PyObject *o, const char *name) { return size32(number(o), name); }

// Runs a function that returns a status; C++ exceptions become Python's.
template <typename F>
PyObject *run(Py_ssize_t n, Py_ssize_t want, F body) {
  try {
    if (n != want) raise(PyExc_TypeError, "wrong number of arguments");
    return PyLong_FromLong(body());
  } catch (const Raised &) {
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}
// x, q, scale, add, weight, resid, eps, group, normalize, stream
PyObject *rmsnorm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run(n, 10, [&]() {
    const at::Tensor &x = tensor(a[0], "x");
    Call c(x);
    const int64_t T = dim(x, "x", 2, 0), H = x.size(1);
    const at::ScalarType dt = x.scalar_type();
    const int group = number32(a[7], "group"), normalize = PyObject_IsTrue(a[8]);
    const float eps = (float)PyFloat_AsDouble(a[6]);
    if (PyErr_Occurred()) throw Raised{};
    long ldx, ldq, lda, ldr;
    const void *px = c.rows(a[0], "x", dt, T, H, ldx);
    uint8_t *pq = (uint8_t *)c.out_rows(a[1], "q", at::kFloat8_e4m3fn, T, H, ldq);
    float *ps = (float *)c.out_flat(a[2], "scale", at::kFloat,
                                    {T, group > 0 ? (H + group - 1) / group : 1});
    const void *pa = c.rows_or_null(a[3], "add", dt, T, H, lda);
    const void *pw = c.flat_or_null(a[4], "weight", dt, {H});
    ldr = 0;
    void *pr = a[5] == Py_None ? nullptr : c.out_rows(a[5], "resid", dt, T, H, ldr);
    const int rt = row_type(dt);
    const int t32 = size32(T, "x"), h32 = size32(H, "x");
    return c.launch(a[9], [&](void *st) {
      return moe_rmsnorm_e4m3(t32, h32, px, ldx, (moe_dtype)rt, pa, lda, pw, eps, normalize,
                              group, pr, ldr, pq, ldq, ps, st);
    });
  });
}

// ids, n_experts, offsets, perm, slot_pos, stream
PyObject *sort(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run(n, 6, [&]() {
    const at::Tensor &ids = tensor(a[0], "ids");
    Call c(ids);
    const int64_t T = dim(ids, "ids", 2, 0), k = ids.size(1), E = number(a[1]);
    const int32_t *pi = (const int32_t *)c.flat(a[0], "ids", at::kInt, {T, k});
    int32_t *po = (int32_t *)c.out_flat(a[2], "offsets", at::kInt, {E + 1});
    int32_t *pp = (int32_t *)c.out_flat(a[3], "perm", at::kInt, {T * k});
    int32_t *ps = (int32_t *)c.out_flat(a[4], "slot_pos", at::kInt, {T, k});
    const int t32 = size32(T, "ids"), k32 = size32(k, "ids"), e32 = size32(E, "n_experts");
    return c.launch(a[5], [&](void *st) {
      return moe_sort_tokens(t32, k32, e32, pi, po, pp, ps, st);
    });
  });
}

// x, slot_pos, offsets, xs, scale, scale_s, stream
PyObject *dispatch(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run(n, 7, [&]() {
    const at::Tensor &x = tensor(a[0], "x");
    Call c(x);
    const int64_t T = dim(x, "x", 2, 0), H = x.size(1);
    const int64_t k = dim(tensor(a[1], "slot_pos"), "slot_pos", 2, 1);
    const int64_t E1 = dim(tensor(a[2], "offsets"), "offsets", 1, 0);
    const at::ScalarType dt = x.scalar_type();
    long ldx, ldsc = 0;
    const void *px = c.rows(a[0], "x", dt, T, H, ldx);
    const int32_t *pp = (const int32_t *)c.flat(a[1], "slot_pos", at::kInt, {T, k});
    const int32_t *po = (const int32_t *)c.flat(a[2], "offsets", at::kInt, {E1});
    void *pxs = c.out_flat(a[3], "xs", dt, {T * k, H});
    int64_t S = 0;
    const float *psc = nullptr;
    float *pss = nullptr;
    if (a[4] != Py_None) {
      S = dim(tensor(a[4], "scale"), "scale", 2, 1);
      psc = (const float *)c.rows(a[4], "scale", at::kFloat, T, S, ldsc);
      if (a[5] == Py_None) raise(PyExc_ValueError, "scale_s is needed with scale");
      pss = (float *)c.out_flat(a[5], "scale_s", at::kFloat, {T * k, S});
    }
    const int rt = row_type(dt), t32 = size32(T, "x"), k32 = size32(k, "slot_pos");
    const int h32 = size32(H, "x"), s32 = size32(S, "scale"), e32 = size32(E1 - 1, "offsets");
    return c.launch(a[6], [&](void *st) {
      return moe_dispatch_rows(t32, k32, e32, h32, (moe_dtype)rt, px, ldx, pp, po, pxs, s32, psc,
                               ldsc, pss, st);
    });
  });
}

// y, slot_pos, out, w, add, stream
PyObject *combine(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run(n, 6, [&]() {
    const at::Tensor &y = tensor(a[0], "y"), &pos = tensor(a[1], "slot_pos");
    const at::Tensor &out = tensor(a[2], "out");
    Call c(y);
    const int64_t T = dim(pos, "slot_pos", 2, 0), k = pos.size(1), H = dim(out, "out", 2, 1);
    const at::ScalarType yt = y.scalar_type(), ot = out.scalar_type();
    long ldo, lda;
    const void *py = c.flat(a[0], "y", yt, {T * k, H});
    const int32_t *pp = (const int32_t *)c.flat(a[1], "slot_pos", at::kInt, {T, k});
    void *po = c.out_rows(a[2], "out", ot, T, H, ldo);
    const float *pw = (const float *)c.flat_or_null(a[3], "w", at::kFloat, {T, k});
    const void *pa = c.rows_or_null(a[4], "add", ot, T, H, lda);
    const int ry = row_type(yt), ro = row_type(ot), t32 = size32(T, "slot_pos");
    const int k32 = size32(k, "slot_pos"), h32 = size32(H, "out");
    return c.launch(a[5], [&](void *st) {
      return moe_combine_rows(t32, k32, h32, py, (moe_dtype)ry, pp, pw, pa, lda, po, ldo,
                              (moe_dtype)ro, st);
    });
  });
}

// dout, y, slot_pos, offsets, w, dy, dw, stream
PyObject *combine_grad(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run(n, 8, [&]() {
    const at::Tensor &dout = tensor(a[0], "dout"), &pos = tensor(a[2], "slot_pos");
    Call c(dout);
    const int64_t T = dim(pos, "slot_pos", 2, 0), k = pos.size(1), H = dim(dout, "dout", 2, 1);
    const int64_t E1 = dim(tensor(a[3], "offsets"), "offsets", 1, 0);
    const at::ScalarType dt = dout.scalar_type();
    long ldd;
    const void *pd = c.rows(a[0], "dout", dt, T, H, ldd);
    const void *py = c.flat(a[1], "y", dt, {T * k, H});
    const int32_t *pp = (const int32_t *)c.flat(a[2], "slot_pos", at::kInt, {T, k});
    const int32_t *po = (const int32_t *)c.flat(a[3], "offsets", at::kInt, {E1});
    const float *pw = (const float *)c.flat_or_null(a[4], "w", at::kFloat, {T, k});
    void *pdy = c.out_flat(a[5], "dy", dt, {T * k, H});
    float *pdw = (float *)c.out_flat(a[6], "dw", at::kFloat, {T, k});
    const int rt = row_type(dt), t32 = size32(T, "slot_pos"), k32 = size32(k, "slot_pos");
    const int h32 = size32(H, "dout"), e32 = size32(E1 - 1, "offsets");
    return c.launch(a[7], [&](void *st) {
      return moe_combine_rows_grad(t32, k32, e32, h32, (moe_dtype)rt, pd, ldd, py, pp, po, pw,
                                   pdy, pdw, st);
    });
  });
}

// dxs, slot_pos, dx, stream
PyObject *dispatch_grad(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run(n, 4, [&]() {
    const at::Tensor &dxs = tensor(a[0], "dxs"), &pos = tensor(a[1], "slot_pos");
    const at::Tensor &dx = tensor(a[2], "dx");
    Call c(dxs);
    const int64_t T = dim(pos, "slot_pos", 2, 0), k = pos.size(1), H = dim(dx, "dx", 2, 1);
    const at::ScalarType dt = dxs.scalar_type(), xt = dx.scalar_type();
    long ldx;
    const void *pd = c.flat(a[0], "dxs", dt, {T * k, H});
    const int32_t *pp = (const int32_t *)c.flat(a[1], "slot_pos", at::kInt, {T, k});
    void *px = c.out_rows(a[2], "dx", xt, T, H, ldx);
    const int rd = row_type(dt), rx = row_type(xt), t32 = size32(T, "slot_pos");
    const int k32 = size32(k, "slot_pos"), h32 = size32(H, "dx");
    return c.launch(a[3], [&](void *st) {
      return moe_dispatch_rows_grad(t32, k32, h32, (moe_dtype)rd, pd, pp, px, ldx, (moe_dtype)rx,
                                    st);
    });
  });
}

// x, w, out, x_scale, w_scale, bias, act, residual, offsets, status, stream
PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return run(n, 11, [&]() {
    const at::Tensor &x = tensor(a[0], "x"), &out = tensor(a[2], "out");
    Call c(x);
    const int64_t R = dim(x, "x", 2, 0), K = x.size(1), N = dim(out, "out", 2, 1);
    const at::ScalarType dt = x.scalar_type(), ot = out.scalar_type();
    const int act = number32(a[6], "act");
    const int64_t rows = act == MOE_ACT_SWIGLU ? 2 * N : N;
    const bool dense = a[8] == Py_None;
    int64_t E = 0;
    const int32_t *po = nullptr;
    if (!dense) {
      E = dim(tensor(a[8], "offsets"), "offsets", 1, 0) - 1;
      if (E < 1) raise(PyExc_ValueError, "offsets must hold E + 1 values");
      po = (const int32_t *)c.flat(a[8], "offsets", at::kInt, {E + 1});
    }
    long ldx, ldo, ldr;
    const void *px = c.rows(a[0], "x", dt, R, K, ldx);
    const void *pw = dense ? c.flat(a[1], "w", dt, {rows, K}) : c.flat(a[1], "w", dt, {E, rows, K});
    void *pout = c.out_rows(a[2], "out", ot, R, N, ldo);
    const float *pxs = nullptr;
    if (a[3] != Py_None)
      pxs = (const float *)(tensor(a[3], "x_scale").dim() == 1
                                ? c.flat(a[3], "x_scale", at::kFloat, {R})
                                : c.flat(a[3], "x_scale", at::kFloat, {R, 1}));
    auto per_row = [&](PyObject *o, const char *name) {
      return (const float *)(dense ? c.flat_or_null(o, name, at::kFloat, {rows})
                                   : c.flat_or_null(o, name, at::kFloat, {E, rows}));
    };
    const float *pws = per_row(a[4], "w_scale"), *pb = per_row(a[5], "bias");
    const void *pr = c.rows_or_null(a[7], "residual", ot, R, N, ldr);
    int32_t *pst = nullptr;
    if (a[9] != Py_None) pst = (int32_t *)c.out_flat(a[9], "status", at::kInt, {1});
    const int rt = row_type(dt), ro = row_type(ot), r32 = size32(R, "x"), n32 = size32(N, "out");
    const int k32 = size32(K, "x"), e32 = size32(E, "offsets");
    return c.launch(a[10], [&](void *st) {
      return moe_linear(r32, n32, k32, e32, px, ldx, (moe_dtype)rt, pxs, pw, pws, pb,
                        (moe_act)act, pr, ldr, po, pout, ldo, (moe_dtype)ro, pst, st);
    });
  });
}

// dev, stream -> what a call with operands on device `dev` does
PyObject *trace(PyObject *, PyObject *const *a, Py_ssize_t n) {
  Told::steps().clear();
  PyObject *r = run(n, 2, [&]() {
    return on_device<Told>(number32(a[0], "dev"), a[1], [](void *st) {
      Told::steps().push_back("call on " + std::to_string((uintptr_t)st));
      return 0;
    });
  });
  if (!r) return nullptr;
  Py_DECREF(r);
  PyObject *out = PyList_New(0);
  for (const std::string &t : Told::steps()) {
    PyObject *v = out ? PyUnicode_FromString(t.c_str()) : nullptr;
    if (!v || PyList_Append(out, v) < 0) Py_CLEAR(out);
    Py_XDECREF(v);
  }
  return out;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(rmsnorm),      METHOD(sort),          METHOD(dispatch),
                         METHOD(combine),      METHOD(combine_grad),  METHOD(dispatch_grad),
                         METHOD(linear),       METHOD(trace),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tokens_native", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tokens_native(void) {
  PyObject *m = PyModule_Create(&module);
  if (m) PyModule_AddStringConstant(m, "torch_version", TOKENS_TORCH);
  return m;
}
