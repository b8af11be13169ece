// marshal.cpp -- the Python binding's argument checks for the layer's short
// calls, in C++: tensors to pointers, strides and sizes, then the C ABI.
//
// These calls take a few microseconds on the device.  Looking at a dozen
// tensors from Python (type, device, shape, strides, address: about 0.1 us
// each on the GPU's host, and the bytecode around them) took up to 30 us a
// call; here it takes one.  The functions take their arguments by position
// (binding.py documents them and gives them their names and defaults), raise
// ValueError or TypeError for tensors that do not fit, and return the C ABI's
// status.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <stdarg.h>
#include <stdint.h>
#include <torch/csrc/autograd/python_variable.h>

#include "seqattn.h"

namespace {

bool refuse(const char* fmt, ...) __attribute__((format(printf, 1, 2)));
bool refuse(const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(PyExc_ValueError, fmt, ap);
  va_end(ap);
  return false;
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kLong: return "torch.int64";
    case at::kByte: return "torch.uint8";
    default: return c10::toString(t);
  }
}

const at::Tensor* tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor, not %s", name, Py_TYPE(o)->tp_name);
    return nullptr;
  }
  return &THPVariable_Unpack(o);
}

// A CUDA tensor of `type` on device `dev`.
bool fits(const at::Tensor& t, const char* name, at::ScalarType type, int dev) {
  if (!t.is_cuda() || t.scalar_type() != type) return refuse("%s must be a CUDA tensor of %s", name, type_name(type));
  if (t.get_device() != dev)
    return refuse("%s is on cuda:%d, the current device is cuda:%d", name, static_cast<int>(t.get_device()), dev);
  return true;
}

// The current device, for a call whose first tensor is `t`.
bool device_for(const at::Tensor& t, const char* name, at::ScalarType type, int* dev) {
  if (!t.is_cuda()) return refuse("%s must be a CUDA tensor of %s", name, type_name(type));
  *dev = c10::cuda::current_device();
  return true;
}

bool stream_of(PyObject* o, int dev, seqattn_stream_t* out) {
  if (o == Py_None) {
    *out = reinterpret_cast<seqattn_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
    return true;
  }
  PyObject* raw = PyObject_GetAttrString(o, "cuda_stream");
  if (raw == nullptr) return false;
  *out = reinterpret_cast<seqattn_stream_t>(PyLong_AsVoidPtr(raw));
  Py_DECREF(raw);
  return PyErr_Occurred() == nullptr;
}

// A tensor seen as a matrix of its last dimension: address, rows, row stride;
// the leading dimensions must lie at one uniform row stride.
struct Matrix {
  void* ptr = nullptr;
  int64_t rows = 0, ld = 0;
};

bool matrix(PyObject* o, const char* name, int64_t cols, int64_t rows, int dev, Matrix* m) {
  const at::Tensor* tp = tensor(o, name);
  if (tp == nullptr) return false;
  const at::Tensor& t = *tp;
  if (!fits(t, name, at::kBFloat16, dev)) return false;
  const int64_t dims = t.dim();
  if (dims < 2) return refuse("%s must have at least two dimensions", name);
  const int64_t c = t.size(dims - 1);
  int64_t r = 1, ld = -1;
  for (int64_t i = dims - 2; i >= 0; --i) {
    const int64_t size = t.size(i);
    if (size == 1) continue;
    if (ld < 0) ld = t.stride(i);
    else if (t.stride(i) != r * ld && size * r > 0) return refuse("the rows of %s must lie at one uniform stride", name);
    r *= size;
  }
  if (t.stride(dims - 1) != 1 && c > 1) return refuse("the last dimension of %s must be contiguous", name);
  if (c != cols)
    return refuse("%s has %lld columns, expected %lld", name, static_cast<long long>(c), static_cast<long long>(cols));
  if (rows >= 0 && r != rows)
    return refuse("%s has %lld rows, expected %lld", name, static_cast<long long>(r), static_cast<long long>(rows));
  m->ptr = t.data_ptr();
  m->rows = r;
  m->ld = r > 1 ? ld : c;
  return true;
}

// The same for an operand that may be None.
bool matrix_or_none(PyObject* o, const char* name, int64_t cols, int64_t rows, int dev, Matrix* m) {
  return o == Py_None || matrix(o, name, cols, rows, dev, m);
}

// A contiguous tensor of the given sizes.
bool dense(PyObject* o, const char* name, at::IntArrayRef sizes, at::ScalarType type, int dev, void** ptr) {
  const at::Tensor* t = tensor(o, name);
  if (t == nullptr || !fits(*t, name, type, dev)) return false;
  if (t->sizes() != sizes || !t->is_contiguous()) {
    if (sizes.size() == 1)
      return refuse("%s must be a contiguous vector of %lld elements", name, static_cast<long long>(sizes[0]));
    PyObject* shape = PyTuple_New(static_cast<Py_ssize_t>(sizes.size()));
    if (shape == nullptr) return false;
    for (size_t i = 0; i < sizes.size(); ++i)
      PyTuple_SET_ITEM(shape, static_cast<Py_ssize_t>(i), PyLong_FromLongLong(sizes[i]));
    PyErr_Format(PyExc_ValueError, "%s must be a contiguous tensor of shape %S", name, shape);
    Py_DECREF(shape);
    return false;
  }
  *ptr = t->data_ptr();
  return true;
}

bool weight(PyObject* o, int dev, int64_t* k, int64_t* n, void** ptr) {
  const at::Tensor* t = tensor(o, "w");
  if (t == nullptr || !fits(*t, "w", at::kBFloat16, dev)) return false;
  if (t->dim() != 2 || !t->is_contiguous()) return refuse("w must be a contiguous [k, n] matrix");
  *k = t->size(0);
  *n = t->size(1);
  *ptr = t->data_ptr();
  return true;
}

// [B, c, H, d] with dense heads and rows (b, r) at one uniform stride.
bool head_rows(PyObject* o, const char* name, int64_t B, int64_t c, int64_t H, int64_t d, at::ScalarType type, int dev,
               Matrix* m) {
  const at::Tensor* tp = tensor(o, name);
  if (tp == nullptr || !fits(*tp, name, type, dev)) return false;
  const at::Tensor& t = *tp;
  if (t.dim() != 4 || t.size(0) != B || t.size(1) != c || t.size(2) != H || t.size(3) != d)
    return refuse("%s must have shape (%lld, %lld, %lld, %lld)", name, static_cast<long long>(B),
                  static_cast<long long>(c), static_cast<long long>(H), static_cast<long long>(d));
  if (t.stride(3) != 1 || (t.stride(2) != d && H > 1)) return refuse("the heads of %s must be dense", name);
  if (c > 1 && B > 1 && t.stride(0) != c * t.stride(1))
    return refuse("the rows of %s must lie at one uniform stride", name);
  m->ptr = t.data_ptr();
  m->ld = c > 1 ? t.stride(1) : B > 1 && c == 1 ? t.stride(0) : H * d;
  return true;
}

// One call of the C ABI without the interpreter's lock.
template <typename F>
PyObject* status_of(F&& call) {
  seqattn_status s;
  Py_BEGIN_ALLOW_THREADS;
  s = call();
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(s);
}

bool arguments(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", got, want);
  return false;
}

bool small(int64_t v, const char* name) {
  return v <= INT32_MAX || refuse("%s = %lld exceeds 2^31 - 1", name, static_cast<long long>(v));
}

// ---- (x, w, y, bias, act, residual, z, stream)
PyObject* linear_fwd(PyObject* const* a, Py_ssize_t n_args) {
  if (!arguments(n_args, 8)) return nullptr;
  const at::Tensor* w = tensor(a[1], "w");
  int dev = 0;
  int64_t k = 0, n = 0;
  void *wp = nullptr, *bias = nullptr;
  if (w == nullptr || !device_for(*w, "w", at::kBFloat16, &dev) || !weight(a[1], dev, &k, &n, &wp)) return nullptr;
  Matrix x, y, r, z;
  if (!matrix(a[0], "x", k, -1, dev, &x) || !matrix(a[2], "y", n, x.rows, dev, &y)) return nullptr;
  if (a[3] != Py_None && !dense(a[3], "bias", {n}, at::kBFloat16, dev, &bias)) return nullptr;
  const long act = PyLong_AsLong(a[4]);
  if (act == -1 && PyErr_Occurred()) return nullptr;
  if (!matrix_or_none(a[5], "residual", n, x.rows, dev, &r) || !matrix_or_none(a[6], "z", n, x.rows, dev, &z))
    return nullptr;
  seqattn_stream_t st;
  if (!small(k, "k") || !small(n, "n") || !stream_of(a[7], dev, &st)) return nullptr;
  return status_of([&] {
    return seqattn_linear_fwd(x.rows, static_cast<int32_t>(k), static_cast<int32_t>(n), x.ptr, x.ld, wp, bias,
                              static_cast<int32_t>(act), r.ptr, r.ld, z.ptr, z.ld, y.ptr, y.ld, st);
  });
}

// ---- (g, w, dx, act, z, residual, stream)
PyObject* linear_dgrad(PyObject* const* a, Py_ssize_t n_args) {
  if (!arguments(n_args, 7)) return nullptr;
  const at::Tensor* w = tensor(a[1], "w");
  int dev = 0;
  int64_t k = 0, n = 0;
  void* wp = nullptr;
  if (w == nullptr || !device_for(*w, "w", at::kBFloat16, &dev) || !weight(a[1], dev, &k, &n, &wp)) return nullptr;
  Matrix g, dx, r, z;
  if (!matrix(a[0], "g", n, -1, dev, &g) || !matrix(a[2], "dx", k, g.rows, dev, &dx)) return nullptr;
  const long act = PyLong_AsLong(a[3]);
  if (act == -1 && PyErr_Occurred()) return nullptr;
  if (act != 0) {
    if (a[4] == Py_None) {
      refuse("z is needed when act is given");
      return nullptr;
    }
    if (!matrix(a[4], "z", k, g.rows, dev, &z)) return nullptr;
  }
  if (!matrix_or_none(a[5], "residual", k, g.rows, dev, &r)) return nullptr;
  seqattn_stream_t st;
  if (!small(k, "k") || !small(n, "n") || !stream_of(a[6], dev, &st)) return nullptr;
  return status_of([&] {
    return seqattn_linear_dgrad(g.rows, static_cast<int32_t>(k), static_cast<int32_t>(n), g.ptr, g.ld, wp,
                                static_cast<int32_t>(act), z.ptr, z.ld, r.ptr, r.ld, dx.ptr, dx.ld, st);
  });
}

// ---- (x, g, dw, dbias, stream)
PyObject* linear_wgrad(PyObject* const* a, Py_ssize_t n_args) {
  if (!arguments(n_args, 5)) return nullptr;
  const at::Tensor *xt = tensor(a[0], "x"), *gt = tensor(a[1], "g");
  int dev = 0;
  if (xt == nullptr || gt == nullptr || !device_for(*xt, "x", at::kBFloat16, &dev)) return nullptr;
  if (xt->dim() < 2 || gt->dim() < 2) {
    refuse("x and g must have at least two dimensions");
    return nullptr;
  }
  const int64_t k = xt->size(-1), n = gt->size(-1);
  Matrix x, g;
  void *dw = nullptr, *dbias = nullptr;
  if (!matrix(a[0], "x", k, -1, dev, &x) || !matrix(a[1], "g", n, x.rows, dev, &g) ||
      !dense(a[2], "dw", {k, n}, at::kFloat, dev, &dw))
    return nullptr;
  if (a[3] != Py_None && !dense(a[3], "dbias", {n}, at::kFloat, dev, &dbias)) return nullptr;
  seqattn_stream_t st;
  if (!small(k, "k") || !small(n, "n") || !stream_of(a[4], dev, &st)) return nullptr;
  return status_of([&] {
    return seqattn_linear_wgrad(x.rows, static_cast<int32_t>(k), static_cast<int32_t>(n), x.ptr, x.ld, g.ptr, g.ld,
                                static_cast<float*>(dw), static_cast<float*>(dbias), st);
  });
}

// What the forward and backward of the head norm share: sizes from the chunk's
// queries (q or dq) and the caches (k_cache or dk_accum), gammas, plan and
// positions.
struct RopeCall {
  seqattn_problem pb{};
  int64_t B = 0, c = 0, Hq = 0, Hkv = 0, d = 0, T = 0, q_start = 0;
  int dev = 0;
  at::ScalarType type = at::kBFloat16;
  float eps = 0;
  void *gamma_q = nullptr, *gamma_k = nullptr, *positions = nullptr;
  seqattn_rope_plan plan{};
  const seqattn_rope_plan* plan_ptr = nullptr;

  bool sizes(const at::Tensor& q, const char* q_name, const at::Tensor& cache, const char* cache_name,
             at::ScalarType element) {
    type = element;
    if (type != at::kBFloat16 && type != at::kFloat) {
      PyErr_Format(PyExc_TypeError, "unsupported element type %s", type_name(type));
      return false;
    }
    if (q.dim() != 4) return refuse("%s must have shape [B, c, Hq, d]", q_name);
    if (cache.dim() != 4 || cache.size(0) != q.size(0) || cache.size(3) != q.size(3))
      return refuse("%s does not go with %s: batch or head_dim differ", cache_name, q_name);
    B = q.size(0), c = q.size(1), Hq = q.size(2), d = q.size(3);
    T = cache.size(1), Hkv = cache.size(2);
    if (!small(B, "batch") || !small(Hq, "heads") || !small(Hkv, "heads") || !small(d, "head_dim")) return false;
    pb.batch = static_cast<int32_t>(B);
    pb.num_q_heads = static_cast<int32_t>(Hq);
    pb.num_kv_heads = static_cast<int32_t>(Hkv);
    pb.head_dim = static_cast<int32_t>(d);
    pb.seq_capacity = T;
    pb.dtype = type == at::kBFloat16 ? SEQATTN_BF16 : SEQATTN_FP32;
    return true;
  }

  bool rest(PyObject* start, PyObject* gq, PyObject* gk, PyObject* e, PyObject* plan_o, PyObject* pos) {
    q_start = PyLong_AsLongLong(start);
    if (q_start == -1 && PyErr_Occurred()) return false;
    if ((gq == Py_None) != (gk == Py_None)) return refuse("gamma_q and gamma_k must both be given or both be None");
    if (gq != Py_None && (!dense(gq, "gamma_q", {d}, type, dev, &gamma_q) || !dense(gk, "gamma_k", {d}, type, dev, &gamma_k)))
      return false;
    const double v = PyFloat_AsDouble(e);
    if (v == -1.0 && PyErr_Occurred()) return false;
    eps = static_cast<float>(v);
    int64_t axes = 1;
    if (plan_o != Py_None) {
      Py_buffer buf;
      if (PyObject_GetBuffer(plan_o, &buf, PyBUF_SIMPLE) != 0) return false;
      const bool whole = buf.len == static_cast<Py_ssize_t>(sizeof(plan));
      if (whole) memcpy(&plan, buf.buf, sizeof(plan));
      PyBuffer_Release(&buf);
      if (!whole) return refuse("plan must be a RopePlan");
      plan_ptr = &plan;
      axes = plan.axes;
    }
    if (pos != Py_None) {
      const at::Tensor* t = tensor(pos, "positions");
      if (t == nullptr) return false;
      if (t->dim() == 2 && axes == 1) return dense(pos, "positions", {B, c}, at::kLong, dev, &positions);
      return dense(pos, "positions", {axes, B, c}, at::kLong, dev, &positions);
    }
    return true;
  }
};

// ---- (q_in, k_in, v_in, q, k_cache, v_cache, q_start, gamma_q, gamma_k, eps, plan, positions, stream)
PyObject* norm_rope_fwd(PyObject* const* a, Py_ssize_t n_args) {
  if (!arguments(n_args, 13)) return nullptr;
  const at::Tensor *q = tensor(a[3], "q"), *cache = tensor(a[4], "k_cache");
  RopeCall rc;
  if (q == nullptr || cache == nullptr || !device_for(*q, "q", q->scalar_type(), &rc.dev) ||
      !rc.sizes(*q, "q", *cache, "k_cache", q->scalar_type()))
    return nullptr;
  if ((a[2] == Py_None) != (a[5] == Py_None)) {
    refuse("v_in and v_cache must both be given or both be None");
    return nullptr;
  }
  Matrix xq, xk, xv;
  void *qo = nullptr, *ko = nullptr, *vo = nullptr;
  const bool values = a[2] != Py_None;
  if (!head_rows(a[0], "q_in", rc.B, rc.c, rc.Hq, rc.d, rc.type, rc.dev, &xq) ||
      !head_rows(a[1], "k_in", rc.B, rc.c, rc.Hkv, rc.d, rc.type, rc.dev, &xk) ||
      (values && !head_rows(a[2], "v_in", rc.B, rc.c, rc.Hkv, rc.d, rc.type, rc.dev, &xv)) ||
      !dense(a[3], "q", {rc.B, rc.c, rc.Hq, rc.d}, rc.type, rc.dev, &qo) ||
      !dense(a[4], "k_cache", {rc.B, rc.T, rc.Hkv, rc.d}, rc.type, rc.dev, &ko) ||
      (values && !dense(a[5], "v_cache", {rc.B, rc.T, rc.Hkv, rc.d}, rc.type, rc.dev, &vo)) ||
      !rc.rest(a[6], a[7], a[8], a[9], a[10], a[11]))
    return nullptr;
  seqattn_stream_t st;
  if (!stream_of(a[12], rc.dev, &st)) return nullptr;
  return status_of([&] {
    return seqattn_qk_norm_rope_fwd(&rc.pb, rc.q_start, rc.c, xq.ptr, xq.ld, xk.ptr, xk.ld, xv.ptr, xv.ld, rc.gamma_q,
                                    rc.gamma_k, rc.eps, rc.plan_ptr, static_cast<const int64_t*>(rc.positions), qo, ko,
                                    vo, st);
  });
}

// ---- (q_in, k_in, dq, dk_accum, dv_accum, dq_in, dk_in, dv_in, q_start, gamma_q, gamma_k, dgamma_q, dgamma_k, eps,
//       plan, positions, workspace, stream)
PyObject* norm_rope_bwd(PyObject* const* a, Py_ssize_t n_args) {
  if (!arguments(n_args, 18)) return nullptr;
  const at::Tensor *dq = tensor(a[2], "dq"), *cache = tensor(a[3], "dk_accum"), *out = tensor(a[5], "dq_in");
  RopeCall rc;
  if (dq == nullptr || cache == nullptr || out == nullptr || !device_for(*dq, "dq", at::kFloat, &rc.dev) ||
      !rc.sizes(*dq, "dq", *cache, "dk_accum", out->scalar_type()))
    return nullptr;
  if ((a[4] == Py_None) != (a[7] == Py_None)) {
    refuse("dv_accum and dv_in must both be given or both be None");
    return nullptr;
  }
  const bool values = a[4] != Py_None;
  Matrix oq, ok, ov, xq, xk;
  void *gq = nullptr, *gk = nullptr, *gv = nullptr, *dgq = nullptr, *dgk = nullptr, *ws = nullptr;
  if (!head_rows(a[5], "dq_in", rc.B, rc.c, rc.Hq, rc.d, rc.type, rc.dev, &oq) ||
      !head_rows(a[6], "dk_in", rc.B, rc.c, rc.Hkv, rc.d, rc.type, rc.dev, &ok) ||
      (values && !head_rows(a[7], "dv_in", rc.B, rc.c, rc.Hkv, rc.d, rc.type, rc.dev, &ov)) ||
      !dense(a[2], "dq", {rc.B, rc.c, rc.Hq, rc.d}, at::kFloat, rc.dev, &gq) ||
      !dense(a[3], "dk_accum", {rc.B, rc.T, rc.Hkv, rc.d}, at::kFloat, rc.dev, &gk) ||
      (values && !dense(a[4], "dv_accum", {rc.B, rc.T, rc.Hkv, rc.d}, at::kFloat, rc.dev, &gv)) ||
      !rc.rest(a[8], a[9], a[10], a[13], a[14], a[15]))
    return nullptr;
  at::Tensor temp;
  size_t ws_bytes = 0;
  if (rc.gamma_q != nullptr) {
    if (a[11] == Py_None || a[12] == Py_None) {
      refuse("dgamma_q and dgamma_k are needed with a norm");
      return nullptr;
    }
    if (!head_rows(a[0], "q_in", rc.B, rc.c, rc.Hq, rc.d, rc.type, rc.dev, &xq) ||
        !head_rows(a[1], "k_in", rc.B, rc.c, rc.Hkv, rc.d, rc.type, rc.dev, &xk) ||
        !dense(a[11], "dgamma_q", {rc.d}, at::kFloat, rc.dev, &dgq) ||
        !dense(a[12], "dgamma_k", {rc.d}, at::kFloat, rc.dev, &dgk))
      return nullptr;
    if (a[16] == Py_None) {
      // on the current stream, which binding.py has made the call's own
      ws_bytes = seqattn_qk_norm_rope_bwd_workspace_size(&rc.pb);
      temp = at::empty({static_cast<int64_t>(ws_bytes)}, dq->options().dtype(at::kByte));
      ws = temp.data_ptr();
    } else {
      const at::Tensor* w = tensor(a[16], "workspace");
      if (w == nullptr || !fits(*w, "workspace", at::kByte, rc.dev)) return nullptr;
      if (!w->is_contiguous()) {
        refuse("workspace must be contiguous");
        return nullptr;
      }
      ws = w->data_ptr();
      ws_bytes = static_cast<size_t>(w->numel());
    }
  }
  seqattn_stream_t st;
  if (!stream_of(a[17], rc.dev, &st)) return nullptr;
  return status_of([&] {
    return seqattn_qk_norm_rope_bwd(&rc.pb, rc.q_start, rc.c, xq.ptr, xq.ld, xk.ptr, xk.ld, rc.gamma_q, rc.gamma_k,
                                    rc.eps, rc.plan_ptr, static_cast<const int64_t*>(rc.positions),
                                    static_cast<const float*>(gq), static_cast<const float*>(gk),
                                    static_cast<const float*>(gv), oq.ptr, oq.ld, ok.ptr, ok.ld, ov.ptr, ov.ld,
                                    static_cast<float*>(dgq), static_cast<float*>(dgk), ws, ws_bytes, st);
  });
}

// C++ exceptions (PyTorch's, an allocation that fails) become Python's.
template <PyObject* (*kCall)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    return kCall(a, n);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

template <PyObject* (*kCall)(PyObject* const*, Py_ssize_t)>
PyCFunction entry() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<kCall>));
}

PyMethodDef methods[] = {
    {"linear_fwd", entry<linear_fwd>(), METH_FASTCALL, nullptr},
    {"linear_dgrad", entry<linear_dgrad>(), METH_FASTCALL, nullptr},
    {"linear_wgrad", entry<linear_wgrad>(), METH_FASTCALL, nullptr},
    {"norm_rope_fwd", entry<norm_rope_fwd>(), METH_FASTCALL, nullptr},
    {"norm_rope_bwd", entry<norm_rope_bwd>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
