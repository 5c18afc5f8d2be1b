// Native marshalling of the feed-forward operators for torch tensors: the
// checks, output allocations and argument structures of layers.py without the
// interpreter, for calls whose time is the host's (a few tokens).  Every
// function returns None for anything it does not take (another type, layout,
// device or device context, a tensor subclass), and the caller goes on in
// Python, which takes it or says what is wrong; an integer is the status of a
// call the library refused.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mt_layers.h"

namespace {

using at::ScalarType;

// The library's entry points (use_library).
mt_status (*g_rms_norm)(const mt_rms_norm_args*, cudaStream_t);
mt_status (*g_rms_norm_backward)(const mt_rms_norm_backward_args*, cudaStream_t);
mt_status (*g_linear)(const mt_linear_args*, cudaStream_t);
mt_status (*g_linear_backward)(const mt_linear_backward_args*, cudaStream_t);

int code_of(ScalarType t) {
  switch (t) {
    case ScalarType::Half: return MT_DTYPE_F16;
    case ScalarType::BFloat16: return MT_DTYPE_BF16;
    case ScalarType::Float: return MT_DTYPE_F32;
    case ScalarType::Float8_e4m3fn: return MT_DTYPE_E4M3;
    default: return 0;
  }
}
bool is_half(ScalarType t) { return t == ScalarType::Half || t == ScalarType::BFloat16; }

// An operand: a plain strided tensor, or (where allowed) None.
struct Operand {
  const at::Tensor* t = nullptr;
  bool read(PyObject* o, bool optional) {
    if (o == Py_None) return optional;
    if (!THPVariable_CheckExact(o)) return false;
    t = &THPVariable_Unpack(o);
    return t->layout() == at::kStrided;
  }
};

struct Matrix {
  void* p = nullptr;
  int64_t ld = 0;
  bool read(const at::Tensor& t, int64_t rows, int64_t cols, ScalarType type, c10::Device device) {
    if (t.scalar_type() != type || t.device() != device || t.dim() != 2 || t.size(0) != rows ||
        t.size(1) != cols || (t.stride(1) != 1 && cols > 1) || (rows > 1 && t.stride(0) < 1))
      return false;
    p = t.data_ptr();
    ld = rows <= 1 ? (cols > 0 ? cols : 1) : t.stride(0);
    return true;
  }
};

// A contiguous vector of n values of `type` or of `other`.
bool vector(const at::Tensor& t, int64_t n, ScalarType type, ScalarType other, c10::Device device) {
  return (t.scalar_type() == type || t.scalar_type() == other) && t.device() == device &&
         t.dim() == 1 && t.size(0) == n && (n <= 1 || t.stride(0) == 1);
}

at::Tensor make(at::IntArrayRef size, ScalarType type, const at::Tensor& like) {
  return at::empty(size, like.options().dtype(type).requires_grad(false));
}

// The operand the others follow: 2-D, on the current CUDA device.
bool lead(const at::Tensor& t) {
  return t.is_cuda() && t.dim() == 2 && t.device().index() == c10::cuda::current_device();
}

cudaStream_t stream_of(const at::Tensor& t) {
  return c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
}

bool flag(PyObject* o) { return o == Py_True; }

// Leaves the interpreter to other threads for a scope: allocations and launches
// may wait (for the device, a full queue, a host callback written in Python).
// The operands stay alive through the caller's references.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(state); }
};

PyObject* none() { Py_RETURN_NONE; }
PyObject* refused(mt_status st) { return PyLong_FromLong(st); }

template <class... T>
PyObject* tuple(T&&... t) {
  PyObject* items[] = {t...};
  constexpr Py_ssize_t n = sizeof...(T);
  PyObject* r = PyTuple_New(n);
  for (Py_ssize_t i = 0; i < n; ++i) PyTuple_SET_ITEM(r, i, items[i]);
  return r;
}
PyObject* wrap(const at::Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}

// Runs f, turning a C++ exception into the Python one that torch raises for
// it (torch.OutOfMemoryError for an allocation that fails).
template <class F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
}

// rms_norm(x, weight, residual, eps, out_dtype)
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Operand x, w, r;
    if (n != 5 || !x.read(a[0], false) || !w.read(a[1], true) || !r.read(a[2], true) ||
        !PyFloat_Check(a[3]) || !lead(*x.t))
      return none();
    const ScalarType type = x.t->scalar_type();
    ScalarType out = type;
    if (a[4] != Py_None) {
      if (!THPDtype_Check(a[4])) return none();
      out = reinterpret_cast<THPDtype*>(a[4])->scalar_type;
    }
    const bool e4m3 = out == ScalarType::Float8_e4m3fn;
    if ((!is_half(type) && type != ScalarType::Float) || (out != type && !e4m3)) return none();
    const c10::Device dev = x.t->device();
    mt_rms_norm_args g{};
    g.rows = x.t->size(0);
    g.d = x.t->size(1);
    Matrix m;
    if (!m.read(*x.t, g.rows, g.d, type, dev)) return none();
    g.x = m.p;
    g.ldx = m.ld;
    if (w.t) {
      if (!vector(*w.t, g.d, type, ScalarType::Float, dev)) return none();
      g.weight = w.t->data_ptr();
      g.weight_dtype = code_of(w.t->scalar_type());
    }
    if (r.t) {
      if (!m.read(*r.t, g.rows, g.d, type, dev)) return none();
      g.residual = m.p;
      g.ldr = m.ld;
    }
    g.eps = static_cast<float>(PyFloat_AS_DOUBLE(a[3]));
    g.dtype = code_of(type);
    g.out_dtype = code_of(out);
    at::Tensor h, y, rstd, scale;
    mt_status st;
    {
      Unlocked unlocked;
      if (r.t) {
        h = make({g.rows, g.d}, type, *x.t);
        g.h = h.data_ptr();
        g.ldh = g.d > 0 ? g.d : 1;
      }
      y = make({g.rows, g.d}, out, *x.t);
      g.y = y.data_ptr();
      g.ldy = g.d > 0 ? g.d : 1;
      rstd = make({g.rows}, ScalarType::Float, *x.t);
      g.rstd = static_cast<float*>(rstd.data_ptr());
      if (e4m3) {
        scale = make({g.rows}, ScalarType::Float, *x.t);
        g.scale = static_cast<float*>(scale.data_ptr());
      }
      st = g_rms_norm(&g, stream_of(*x.t));
    }
    if (st != MT_OK) return refused(st);
    PyObject* hp = a[0];
    if (r.t) hp = wrap(h);
    else Py_INCREF(hp);
    return e4m3 ? tuple(wrap(y), wrap(scale), hp, wrap(rstd)) : tuple(wrap(y), hp, wrap(rstd));
  });
}

// rms_norm_backward(dy, h, weight, rstd, dh, need_weight)
PyObject* rms_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Operand dy, h, w, rstd, dh;
    if (n != 6 || !dy.read(a[0], false) || !h.read(a[1], false) || !w.read(a[2], true) ||
        !rstd.read(a[3], false) || !dh.read(a[4], true) || !lead(*dy.t))
      return none();
    const ScalarType type = dy.t->scalar_type();
    if (!is_half(type) && type != ScalarType::Float) return none();
    const c10::Device dev = dy.t->device();
    mt_rms_norm_backward_args g{};
    g.rows = dy.t->size(0);
    g.d = dy.t->size(1);
    Matrix m;
    if (!m.read(*dy.t, g.rows, g.d, type, dev)) return none();
    g.dy = m.p;
    g.lddy = m.ld;
    if (!m.read(*h.t, g.rows, g.d, type, dev)) return none();
    g.h = m.p;
    g.ldh = m.ld;
    if (w.t) {
      if (!vector(*w.t, g.d, type, ScalarType::Float, dev)) return none();
      g.weight = w.t->data_ptr();
      g.weight_dtype = code_of(w.t->scalar_type());
    }
    if (!vector(*rstd.t, g.rows, ScalarType::Float, ScalarType::Float, dev)) return none();
    g.rstd = static_cast<const float*>(rstd.t->data_ptr());
    if (dh.t) {
      if (!m.read(*dh.t, g.rows, g.d, type, dev)) return none();
      g.dh = m.p;
      g.lddh = m.ld;
    }
    g.dtype = code_of(type);
    const bool need_weight = flag(a[5]);
    at::Tensor dx, dw;
    mt_status st;
    {
      Unlocked unlocked;
      dx = make({g.rows, g.d}, type, *dy.t);
      g.dx = dx.data_ptr();
      g.lddx = g.d > 0 ? g.d : 1;
      if (need_weight) {
        dw = make({g.d}, ScalarType::Float, *dy.t);
        g.dweight = static_cast<float*>(dw.data_ptr());
      }
      st = g_rms_norm_backward(&g, stream_of(*dy.t));
    }
    if (st != MT_OK) return refused(st);
    return tuple(wrap(dx), wrap(dw));
  });
}

// linear(a, b, bias, activation code, residual, trans_b, scale_a, scale_b,
//        out_dtype, preact)
PyObject* linear(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Operand a, b, bias, res, sa, sb;
    if (n != 10 || !a.read(o[0], false) || !b.read(o[1], false) || !bias.read(o[2], true) ||
        !PyLong_Check(o[3]) || !res.read(o[4], true) || !sa.read(o[6], true) ||
        !sb.read(o[7], true) || !lead(*a.t) || b.t->dim() != 2)
      return none();
    const ScalarType type = a.t->scalar_type();
    const bool e4m3 = type == ScalarType::Float8_e4m3fn, trans = flag(o[5]);
    if (!is_half(type) && !e4m3) return none();
    ScalarType out = e4m3 ? ScalarType::BFloat16 : type;
    if (o[8] != Py_None) {
      if (!THPDtype_Check(o[8])) return none();
      out = reinterpret_cast<THPDtype*>(o[8])->scalar_type;
    }
    if (out != ScalarType::Float && (e4m3 ? !is_half(out) : out != type)) return none();
    if (e4m3 ? !trans || !sa.t || !sb.t : sa.t || sb.t) return none();
    const c10::Device dev = a.t->device();
    mt_linear_args g{};
    g.M = a.t->size(0);
    g.K = a.t->size(1);
    g.N = b.t->size(trans ? 0 : 1);
    Matrix m;
    if (!m.read(*a.t, g.M, g.K, type, dev)) return none();
    g.A = m.p;
    g.lda = m.ld;
    if (!m.read(*b.t, trans ? g.N : g.K, trans ? g.K : g.N, type, dev)) return none();
    g.B = m.p;
    g.ldb = m.ld;
    const ScalarType f32 = ScalarType::Float;
    if (bias.t) {
      if (!vector(*bias.t, g.N, f32, f32, dev)) return none();
      g.bias = static_cast<const float*>(bias.t->data_ptr());
    }
    if (e4m3) {
      if (!vector(*sa.t, g.M, f32, f32, dev) || !vector(*sb.t, g.N, f32, f32, dev)) return none();
      g.scale_a = static_cast<const float*>(sa.t->data_ptr());
      g.scale_b = static_cast<const float*>(sb.t->data_ptr());
    }
    if (res.t) {
      if (!m.read(*res.t, g.M, g.N, out, dev)) return none();
      g.residual = m.p;
      g.ldr = m.ld;
    }
    const bool preact = flag(o[9]);
    g.trans_b = trans;
    g.dtype = code_of(type);
    g.out_dtype = code_of(out);
    g.activation = static_cast<int32_t>(PyLong_AsLong(o[3]));
    at::Tensor y, z;
    mt_status st;
    {
      Unlocked unlocked;
      y = make({g.M, g.N}, out, *a.t);
      g.Y = y.data_ptr();
      g.ldy = g.ldz = g.N > 0 ? g.N : 1;
      if (preact) {
        z = make({g.M, g.N}, out, *a.t);
        g.Z = z.data_ptr();
      }
      st = g_linear(&g, stream_of(*a.t));
    }
    if (st != MT_OK) return refused(st);
    return preact ? tuple(wrap(y), wrap(z)) : wrap(y);
  });
}

// linear_backward(dy, a, b, z, activation code, trans_b, need_a, need_b,
//                 need_bias, db_dtype)
PyObject* linear_backward(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Operand dy, a, b, z;
    if (n != 10 || !dy.read(o[0], false) || !a.read(o[1], false) || !b.read(o[2], false) ||
        !z.read(o[3], true) || !PyLong_Check(o[4]) || !lead(*dy.t) || a.t->dim() != 2)
      return none();
    const ScalarType type = dy.t->scalar_type();
    if (!is_half(type)) return none();
    ScalarType db_type = type;
    if (o[9] != Py_None) {
      if (!THPDtype_Check(o[9])) return none();
      db_type = reinterpret_cast<THPDtype*>(o[9])->scalar_type;
    }
    if (db_type != type && db_type != ScalarType::Float) return none();
    const c10::Device dev = dy.t->device();
    const bool trans = flag(o[5]);
    mt_linear_backward_args g{};
    g.M = dy.t->size(0);
    g.N = dy.t->size(1);
    g.K = a.t->size(1);
    g.activation = static_cast<int32_t>(PyLong_AsLong(o[4]));
    const int64_t rows = trans ? g.N : g.K, cols = trans ? g.K : g.N;
    Matrix m;
    if (!m.read(*dy.t, g.M, g.N, type, dev)) return none();
    g.dY = m.p;
    g.lddy = m.ld;
    if (!m.read(*a.t, g.M, g.K, type, dev)) return none();
    g.A = m.p;
    g.lda = m.ld;
    if (!m.read(*b.t, rows, cols, type, dev)) return none();
    g.B = m.p;
    g.ldb = m.ld;
    if (g.activation != MT_ACT_NONE) {
      if (!z.t || !m.read(*z.t, g.M, g.N, type, dev)) return none();
      g.Z = m.p;
      g.ldz = m.ld;
    }
    g.trans_b = trans;
    g.dtype = code_of(type);
    g.db_dtype = code_of(db_type);
    const bool need_a = flag(o[6]), need_b = flag(o[7]), need_bias = flag(o[8]);
    at::Tensor da, db, dbias;
    mt_status st;
    {
      Unlocked unlocked;
      if (need_a) {
        da = make({g.M, g.K}, type, *dy.t);
        g.dA = da.data_ptr();
        g.ldda = g.K > 0 ? g.K : 1;
      }
      if (need_b) {
        db = make({rows, cols}, db_type, *dy.t);
        g.dB = db.data_ptr();
        g.lddb = cols > 0 ? cols : 1;
      }
      if (need_bias) {
        dbias = make({g.N}, ScalarType::Float, *dy.t);
        g.dbias = static_cast<float*>(dbias.data_ptr());
      }
      st = g_linear_backward(&g, stream_of(*dy.t));
    }
    if (st != MT_OK) return refused(st);
    return tuple(wrap(da), wrap(db), wrap(dbias));
  });
}

// use_library(mt_rms_norm, mt_rms_norm_backward, mt_linear,
//             mt_linear_backward): the entry points' addresses.
PyObject* use_library(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "use_library takes four addresses");
    return nullptr;
  }
  void* p[4];
  for (int i = 0; i < 4; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_rms_norm = reinterpret_cast<decltype(g_rms_norm)>(p[0]);
  g_rms_norm_backward = reinterpret_cast<decltype(g_rms_norm_backward)>(p[1]);
  g_linear = reinterpret_cast<decltype(g_linear)>(p[2]);
  g_linear_backward = reinterpret_cast<decltype(g_linear_backward)>(p[3]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return PyMethodDef{name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F)),
                     METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<rms_norm>("rms_norm"),
                           method<rms_norm_backward>("rms_norm_backward"),
                           method<linear>("linear"),
                           method<linear_backward>("linear_backward"),
                           method<use_library>("use_library"),
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "mt_torch_binding", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit_mt_torch_binding(void) { return PyModule_Create(&g_module); }
