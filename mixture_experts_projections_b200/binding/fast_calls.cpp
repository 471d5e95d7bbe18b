// The hot calls of the binding (rom.py) with their tensors checked in C++: types,
// shapes, layout and device in 0.35 us of a call with nine tensors, so that a call of
// a few microseconds of GPU work is not bound by its own checks (the norm of one row:
// 7.7 us of host time per call checked in Python, 2.3 with these, on an idle host).
//
// Every function here takes the arguments of the rom.py function of its name
// without the stream, returns the library's status, or None when anything is not
// as the call expects it; rom.py then goes through its own checks, which name
// the argument. So these accept nothing that those refuse. They run on the
// current stream of the device of the first tensor.
//
// The library's entry points come in as addresses (bind), so this file links
// against torch only.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <initializer_list>

#include "../../include/rom.h"

namespace {

decltype(&rom_add_rmsnorm) p_add_rmsnorm;
decltype(&rom_add_rmsnorm_bwd) p_add_rmsnorm_bwd;
decltype(&rom_quant_rows) p_quant_rows;
decltype(&rom_expert_proj_q8) p_expert_proj_q8;
decltype(&rom_expert_proj_w4) p_expert_proj_w4;

constexpr auto kBf16 = at::ScalarType::BFloat16;
constexpr auto kF32 = at::ScalarType::Float;
constexpr auto kI32 = at::ScalarType::Int;
constexpr auto kU8 = at::ScalarType::Byte;
constexpr auto kE4m3 = at::ScalarType::Float8_e4m3fn;

// The tensor behind an argument, or nullptr.
const at::Tensor* tensor(PyObject* o) {
  return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}

// Collects the checks of one call; `ok` turns false at the first that fails.
struct Args {
  bool ok = true;
  int dev = -1;

  // First tensor: its device is the call's.
  const at::Tensor* first(PyObject* o, int dims) {
    const at::Tensor* t = tensor(o);
    if (!t || !t->is_cuda() || t->dim() != dims) {
      ok = false;
      return nullptr;
    }
    dev = t->get_device();
    return t;
  }
  void* ptr(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape) {
    const at::Tensor* t = ok ? tensor(o) : nullptr;
    if (!t || t->scalar_type() != type || !t->is_cuda() || t->get_device() != dev ||
        t->sizes() != at::IntArrayRef(shape) || !t->is_contiguous()) {
      ok = false;
      return nullptr;
    }
    return t->data_ptr();
  }
  void* opt(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape) {
    return o == Py_None ? nullptr : ptr(o, type, shape);
  }
  int64_t integer(PyObject* o) {
    const long long v = PyLong_Check(o) ? PyLong_AsLongLong(o) : -1;
    if (!PyLong_Check(o) || v < 0 || v > INT32_MAX) ok = false;
    PyErr_Clear();
    return v;
  }
};

int dtype_code(at::ScalarType t) { return t == kBf16 ? ROM_BF16 : t == kF32 ? ROM_F32 : -1; }
bool fits(int64_t v) { return v <= INT32_MAX; }

// Lets other Python threads run: a launch blocks while the stream's queue is full,
// and what is in the queue may be a host function that needs the lock.
struct WithoutLock {
  PyThreadState* state = PyEval_SaveThread();
  ~WithoutLock() { PyEval_RestoreThread(state); }
};

template <typename F>
PyObject* run(const Args& a, F&& f) {
  if (!a.ok) Py_RETURN_NONE;
  int status;
  {
    WithoutLock unlocked;
    if (c10::cuda::current_device() == a.dev) {
      status = f(c10::cuda::getCurrentCUDAStream(a.dev).stream());
    } else {
      c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(a.dev));
      status = f(c10::cuda::getCurrentCUDAStream(a.dev).stream());
    }
  }
  return PyLong_FromLong(status);
}

// x, residual, weight, eps, res_out, y, y8, y_scale, rstd
PyObject* add_rmsnorm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  Args a;
  const at::Tensor* x = n == 9 && p_add_rmsnorm ? a.first(v[0], 2) : nullptr;
  if (!x) Py_RETURN_NONE;
  const int64_t T = x->size(0), D = x->size(1);
  const at::ScalarType xt = x->scalar_type();
  const at::Tensor* r = tensor(v[1] != Py_None ? v[1] : v[4]);
  const at::ScalarType rt = r ? r->scalar_type() : kF32;
  if (dtype_code(xt) < 0 || dtype_code(rt) < 0 || !PyFloat_Check(v[3]) || !fits(D))
    Py_RETURN_NONE;
  const float eps = static_cast<float>(PyFloat_AS_DOUBLE(v[3]));
  void* px = a.ptr(v[0], xt, {T, D});
  void* pr = a.opt(v[1], rt, {T, D});
  void* pw = a.ptr(v[2], kF32, {D});
  void* po = a.opt(v[4], rt, {T, D});
  void* py = a.opt(v[5], xt, {T, D});
  void* p8 = a.opt(v[6], kE4m3, {T, D});
  void* ps = a.opt(v[7], kF32, {T});
  void* pq = a.opt(v[8], kF32, {T});
  return run(a, [&](cudaStream_t s) {
    return p_add_rmsnorm(px, dtype_code(xt), pr, dtype_code(rt), T, static_cast<int>(D),
                         static_cast<float*>(pw), eps, po, py, p8, static_cast<float*>(ps),
                         static_cast<float*>(pq), s);
  });
}

// dy, dres_out, res_out, weight, rstd, dx, dres, dw, ws
PyObject* add_rmsnorm_bwd(PyObject*, PyObject* const* v, Py_ssize_t n) {
  Args a;
  const at::Tensor* dy = n == 9 && p_add_rmsnorm_bwd ? a.first(v[0], 2) : nullptr;
  const at::Tensor* r = dy ? tensor(v[2]) : nullptr;
  if (!r) Py_RETURN_NONE;
  const int64_t T = dy->size(0), D = dy->size(1);
  const at::ScalarType xt = dy->scalar_type(), rt = r->scalar_type();
  if (dtype_code(xt) < 0 || dtype_code(rt) < 0 || !fits(D)) Py_RETURN_NONE;
  void* pdy = a.ptr(v[0], xt, {T, D});
  void* pdr = a.opt(v[1], rt, {T, D});
  void* pro = a.ptr(v[2], rt, {T, D});
  void* pw = a.ptr(v[3], kF32, {D});
  void* prs = a.ptr(v[4], kF32, {T});
  void* pdx = a.opt(v[5], xt, {T, D});
  void* pds = a.opt(v[6], rt, {T, D});
  void* pdw = a.opt(v[7], kF32, {D});
  void* ws = nullptr;
  size_t ws_bytes = 0;
  if (v[8] != Py_None) {
    const at::Tensor* w = tensor(v[8]);
    if (!w || !w->is_cuda() || w->get_device() != a.dev || !w->is_contiguous()) Py_RETURN_NONE;
    ws = w->data_ptr();
    ws_bytes = w->nbytes();
  }
  return run(a, [&](cudaStream_t s) {
    return p_add_rmsnorm_bwd(pdy, dtype_code(xt), pdr, pro, dtype_code(rt), T,
                             static_cast<int>(D), static_cast<float*>(pw),
                             static_cast<float*>(prs), pdx, pds, static_cast<float*>(pdw), ws,
                             ws_bytes, s);
  });
}

// x, q, scale
PyObject* quant_rows(PyObject*, PyObject* const* v, Py_ssize_t n) {
  Args a;
  const at::Tensor* x = n == 3 && p_quant_rows ? a.first(v[0], 2) : nullptr;
  if (!x || dtype_code(x->scalar_type()) < 0 || !fits(x->size(1))) Py_RETURN_NONE;
  const int64_t rows = x->size(0), K = x->size(1);
  void* px = a.ptr(v[0], x->scalar_type(), {rows, K});
  void* pq = a.ptr(v[1], kE4m3, {rows, K});
  void* ps = a.ptr(v[2], kF32, {rows});
  return run(a, [&](cudaStream_t s) {
    return p_quant_rows(px, dtype_code(x->scalar_type()), rows, static_cast<int>(K), pq,
                        static_cast<float*>(ps), s);
  });
}

// proj, a_sorted, a_scale, w0, w0_scale, w1, w1_scale, k, offsets, sorted_slot, topk_w, out
PyObject* expert_proj_q8(PyObject*, PyObject* const* v, Py_ssize_t n) {
  Args a;
  const at::Tensor* rows = n == 12 && p_expert_proj_q8 ? a.first(v[1], 2) : nullptr;
  const at::Tensor* w = rows ? tensor(v[3]) : nullptr;
  if (!w || w->dim() != 3) Py_RETURN_NONE;
  const int64_t R = rows->size(0), K = rows->size(1), E = w->size(0), N = w->size(1);
  const int64_t proj = a.integer(v[0]), k = a.integer(v[7]);
  const bool gate = proj == ROM_PROJ_CONV_GATE || proj == ROM_PROJ_CONV_GATE_SLOTS;
  if (!a.ok || k < 1 || R % k != 0 || !fits(K) || !fits(N) || !fits(E)) Py_RETURN_NONE;
  void* pa = a.ptr(v[1], kE4m3, {R, K});
  void* ps = a.ptr(v[2], kF32, {R});
  void* w0 = a.ptr(v[3], kE4m3, {E, N, K});
  void* s0 = a.ptr(v[4], kF32, {E, N});
  void* w1 = gate ? a.ptr(v[5], kE4m3, {E, N, K}) : nullptr;
  void* s1 = gate ? a.ptr(v[6], kF32, {E, N}) : nullptr;
  void* off = a.opt(v[8], kI32, {E + 1});
  void* slot = nullptr;
  if (v[9] != Py_None) {
    const at::Tensor* t = tensor(v[9]);
    if (!t || t->dim() != 1 || t->size(0) < R) Py_RETURN_NONE;
    slot = a.ptr(v[9], kI32, {t->size(0)});
  }
  void* r = a.opt(v[10], kF32, {R / k, k});
  void* out;
  if (k == 1 && (proj == ROM_PROJ_OUT || proj == ROM_PROJ_INPROJ || proj == ROM_PROJ_CONV_GATE))
    out = a.ptr(v[11], kBf16, {R, N});
  else if (gate)
    out = a.ptr(v[11], kF32, {2, R, N});
  else
    out = a.ptr(v[11], kF32, {R, N});
  return run(a, [&](cudaStream_t s) {
    return p_expert_proj_q8(static_cast<int>(proj), pa, static_cast<float*>(ps), R,
                            static_cast<int>(K), w0, static_cast<float*>(s0), w1,
                            static_cast<float*>(s1), static_cast<int>(N), static_cast<int>(E),
                            static_cast<int>(k), static_cast<int32_t*>(off),
                            static_cast<int32_t*>(slot), static_cast<float*>(r), out, s);
  });
}

// proj, x, q0, s0, q1, s1, N, k, topk_idx, topk_w, out
PyObject* expert_proj_w4(PyObject*, PyObject* const* v, Py_ssize_t n) {
  Args a;
  const at::Tensor* x = n == 11 && p_expert_proj_w4 ? a.first(v[1], 2) : nullptr;
  const at::Tensor* q = x ? tensor(v[2]) : nullptr;
  const at::Tensor* sc = x ? tensor(v[3]) : nullptr;
  if (!q || !sc || q->dim() != 7 || sc->dim() != 5) Py_RETURN_NONE;
  const int64_t T = x->size(0), K = x->size(1), E = q->size(0), nt = q->size(1), kb = q->size(2);
  const int64_t groups = sc->size(4);
  const int64_t proj = a.integer(v[0]), N = a.integer(v[6]), k = a.integer(v[7]);
  const bool gate = proj == ROM_PROJ_CONV_GATE_SLOTS;
  if (!a.ok || k < 1 || nt != (N + 15) / 16 || kb != (K + 127) / 128 || !fits(K) || !fits(E) ||
      (groups != 1 && groups != 2 && groups != 4) || gate != (v[4] != Py_None) ||
      gate != (v[5] != Py_None))
    Py_RETURN_NONE;
  void* px = a.ptr(v[1], kBf16, {T, K});
  void* q0 = a.ptr(v[2], kU8, {E, nt, kb, 2, 8, 4, 16});
  void* s0 = a.ptr(v[3], kBf16, {E, nt, kb, 16, groups});
  void* q1 = a.opt(v[4], kU8, {E, nt, kb, 2, 8, 4, 16});
  void* s1 = a.opt(v[5], kBf16, {E, nt, kb, 16, groups});
  void* idx = a.ptr(v[8], kI32, {T, k});
  void* r = a.opt(v[9], kF32, {T, k});
  void* out;
  if (gate)
    out = a.ptr(v[10], kF32, {2, T * k, N});
  else if (k == 1 && proj != ROM_PROJ_SLOTS)
    out = a.ptr(v[10], kBf16, {T, N});
  else
    out = a.ptr(v[10], kF32, {T * k, N});
  return run(a, [&](cudaStream_t s) {
    return p_expert_proj_w4(static_cast<int>(proj), px, T, static_cast<int>(K), q0, s0, q1, s1,
                            static_cast<int>(N), static_cast<int>(E), static_cast<int>(k),
                            static_cast<int>(128 / groups), static_cast<int32_t*>(idx),
                            static_cast<float*>(r), out, s);
  });
}

// bind(addresses of rom_add_rmsnorm, rom_add_rmsnorm_bwd, rom_quant_rows,
// rom_expert_proj_q8, rom_expert_proj_w4)
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long f[5];
  if (!PyArg_ParseTuple(args, "KKKKK", f, f + 1, f + 2, f + 3, f + 4)) return nullptr;
  p_add_rmsnorm = reinterpret_cast<decltype(p_add_rmsnorm)>(f[0]);
  p_add_rmsnorm_bwd = reinterpret_cast<decltype(p_add_rmsnorm_bwd)>(f[1]);
  p_quant_rows = reinterpret_cast<decltype(p_quant_rows)>(f[2]);
  p_expert_proj_q8 = reinterpret_cast<decltype(p_expert_proj_q8)>(f[3]);
  p_expert_proj_w4 = reinterpret_cast<decltype(p_expert_proj_w4)>(f[4]);
  Py_RETURN_NONE;
}

// A C++ exception (a CUDA error that torch reports, an allocation) becomes a
// Python one instead of ending the process.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* safe(PyObject* self, PyObject* const* v, Py_ssize_t n) {
  try {
    return F(self, v, n);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

#define FAST(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(safe<name>)), METH_FASTCALL, \
   nullptr}

PyMethodDef methods[] = {FAST(add_rmsnorm),
                         FAST(add_rmsnorm_bwd),
                         FAST(quant_rows),
                         FAST(expert_proj_q8),
                         FAST(expert_proj_w4),
                         {"bind", bind, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__fast_calls() {
  PyObject* m = PyModule_Create(&module);
  // what the loader compares with the torch that runs
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
