// The prompt side's calls as a Python extension: the tensors' checks and the C
// call in one step.
//
// These calls take microseconds on the GPU, and through ctypes their
// marshalling took longer (a rotation of 512 tokens: 8.5 us a call, 3.7 here).  A
// function returns the C call's status, or -1 when anything is not as the call
// needs it; the binding then goes its own way, which names the reason.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "medusa.h"

namespace {

decltype(&medusa_rope) g_rope;
decltype(&medusa_rope_append) g_append;
decltype(&medusa_chunk_attention) g_attention;
decltype(&medusa_sample_tokens) g_sample;

// Raised (and caught below) where the binding has to take over.
struct Odd {};

void need(bool ok) {
  if (!ok) throw Odd{};
}

const at::Tensor& tensor(PyObject* o) {
  need(THPVariable_Check(o));
  return THPVariable_Unpack(o);
}

medusa_dtype_t dtype(const at::Tensor& t) {
  need(t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kFloat);
  return t.scalar_type() == at::kBFloat16 ? MEDUSA_BF16 : MEDUSA_F32;
}

// the device of the call: the current one, where `t` has to be
int device_of(const at::Tensor& t) {
  need(t.is_cuda());
  const int dev = c10::cuda::current_device();
  need(t.get_device() == dev);
  return dev;
}

void on(const at::Tensor& t, int dev) { need(t.is_cuda() && t.get_device() == dev); }

// [T, H, dh] with dense heads and elements
struct Rows {
  void* p = nullptr;
  long long stride = 0;
};

Rows rows(PyObject* o, at::ScalarType dt, int64_t T, int64_t H, int64_t dh, int dev) {
  const at::Tensor& t = tensor(o);
  on(t, dev);
  need(t.scalar_type() == dt && t.dim() == 3 && t.size(0) == T && t.size(1) == H &&
       t.size(2) == dh);
  const auto st = t.strides();
  need((dh <= 1 || st[2] == 1) && (H <= 1 || st[1] == dh));
  return {t.data_ptr(), T > 1 ? st[0] : (long long)(H * dh)};
}

void* vec(PyObject* o, at::ScalarType dt, int64_t n, int dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o);
  on(t, dev);
  need(t.scalar_type() == dt && t.numel() == n && t.is_contiguous());
  return t.data_ptr();
}

void* address(PyObject* o) {
  if (o == Py_None) return nullptr;
  void* p = PyLong_AsVoidPtr(o);
  need(!PyErr_Occurred());
  return p;
}

// a token or element count that an int holds
int count(int64_t n) {
  need(n <= 0x7fffffff);
  return static_cast<int>(n);
}

// The C call itself runs without the interpreter's lock, as through ctypes: a
// launch waits where the stream's queue is full, and other threads go on.
template <typename F>
int unlocked(F&& call) {
  PyThreadState* state = PyEval_SaveThread();
  const int st = static_cast<int>(call());
  PyEval_RestoreThread(state);
  return st;
}

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(dev).stream(); }

template <typename F>
PyObject* run(F&& call) {
  int st = -1;
  try {
    st = call();
  } catch (const Odd&) {
    PyErr_Clear();
  } catch (const std::exception&) {
    PyErr_Clear();
  }
  return PyLong_FromLong(st);
}

// (functions' addresses)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) return PyErr_Format(PyExc_TypeError, "bind: four addresses");
  void* p[4];
  for (int i = 0; i < 4; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_rope = reinterpret_cast<decltype(g_rope)>(p[0]);
  g_append = reinterpret_cast<decltype(g_append)>(p[1]);
  g_attention = reinterpret_cast<decltype(g_attention)>(p[2]);
  g_sample = reinterpret_cast<decltype(g_sample)>(p[3]);
  Py_RETURN_NONE;
}

// (rope struct, turns, q, k, positions, q_out, k_out, inverse)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run([&] {
    need(n == 8 && g_rope != nullptr);
    const at::Tensor& q = tensor(a[2]);
    const int dev = device_of(q);
    const medusa_dtype_t dt = dtype(q);
    need(q.dim() == 3);
    const int64_t T = q.size(0), Hq = q.size(1), dh = q.size(2);
    const Rows qr = rows(a[2], q.scalar_type(), T, Hq, dh, dev);
    const Rows qo = rows(a[5], q.scalar_type(), T, Hq, dh, dev);
    Rows kr, ko;
    int64_t Hkv = 0;
    if (a[3] != Py_None) {
      const at::Tensor& k = tensor(a[3]);
      need(k.dim() == 3);
      Hkv = k.size(1);
      kr = rows(a[3], q.scalar_type(), T, Hkv, dh, dev);
      ko = rows(a[6], q.scalar_type(), T, Hkv, dh, dev);
    }
    need(a[4] != Py_None);
    const auto* pos = static_cast<const int32_t*>(vec(a[4], at::kInt, T, dev));
    on(tensor(a[1]), dev);
    const int inverse = PyObject_IsTrue(a[7]);
    need(inverse >= 0);
    const auto* r = static_cast<const medusa_rope_t*>(address(a[0]));
    const int t = count(T), hq = count(Hq), hkv = count(Hkv), d = count(dh);
    void* const stream = stream_of(dev);
    return unlocked([&] {
      return g_rope(r, qr.p, qr.stride, kr.p, kr.stride, dt, pos, t, hq, hkv, d, inverse, qo.p,
                    qo.stride, ko.p, ko.stride, stream);
    });
  });
}

// (rope struct, turns, q, k, v, cu_q, kv_len, q_out, cache struct, its K, B, positions, status)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run([&] {
    need(n == 13 && g_append != nullptr);
    const at::Tensor& k = tensor(a[3]);
    const at::Tensor& K = tensor(a[9]);
    const int dev = device_of(K);
    const medusa_dtype_t dt = dtype(K);
    const at::ScalarType type = K.scalar_type();
    need(k.dim() == 3);
    const int64_t T = k.size(0), Hkv = K.size(1), dh = K.size(3), B = PyLong_AsLongLong(a[10]);
    const Rows kr = rows(a[3], type, T, Hkv, dh, dev), vr = rows(a[4], type, T, Hkv, dh, dev);
    Rows qr, qo;
    int64_t Hq = 0;
    if (a[2] != Py_None) {
      const at::Tensor& q = tensor(a[2]);
      need(q.dim() == 3);
      Hq = q.size(1);
      qr = rows(a[2], type, T, Hq, dh, dev);
      qo = rows(a[7], type, T, Hq, dh, dev);
    }
    if (a[0] != Py_None) on(tensor(a[1]), dev);
    const auto* r = static_cast<const medusa_rope_t*>(address(a[0]));
    const auto* pages = static_cast<const medusa_pages_t*>(address(a[8]));
    const auto* pos = static_cast<const int32_t*>(vec(a[11], at::kInt, T, dev));
    const auto* cu = static_cast<const int32_t*>(vec(a[5], at::kInt, B + 1, dev));
    const auto* kv = static_cast<const int32_t*>(vec(a[6], at::kInt, B, dev));
    auto* status = static_cast<int32_t*>(vec(a[12], at::kInt, 1, dev));
    const int nb = count(B), t = count(T), hq = count(Hq), hkv = count(Hkv), d = count(dh);
    void* const stream = stream_of(dev);
    return unlocked([&] {
      return g_append(r, qr.p, qr.stride, kr.p, kr.stride, vr.p, vr.stride, dt, pos, cu, kv, nb, t,
                      hq, hkv, d, qo.p, qo.stride, pages, status, stream);
    });
  });
}

// (q, cache struct, its K, cu_q, kv_len, out, B, scale, ws, status)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run([&] {
    need(n == 10 && g_attention != nullptr);
    const at::Tensor& q = tensor(a[0]);
    const at::Tensor& K = tensor(a[2]);
    const int dev = device_of(K);
    const medusa_dtype_t dt = dtype(K);
    need(q.dim() == 3);
    const int64_t T = q.size(0), Hq = q.size(1), dh = K.size(3), B = PyLong_AsLongLong(a[6]);
    const Rows qr = rows(a[0], K.scalar_type(), T, Hq, dh, dev);
    const Rows out = rows(a[5], K.scalar_type(), T, Hq, dh, dev);
    need(out.stride == (long long)(Hq * dh));
    const double scale = PyFloat_AsDouble(a[7]);
    need(!PyErr_Occurred());
    const int64_t bytes = tensor(a[8]).numel();
    void* ws = vec(a[8], at::kByte, bytes, dev);
    const auto* pages = static_cast<const medusa_pages_t*>(address(a[1]));
    const auto* cu = static_cast<const int32_t*>(vec(a[3], at::kInt, B + 1, dev));
    const auto* kv = static_cast<const int32_t*>(vec(a[4], at::kInt, B, dev));
    auto* status = static_cast<int32_t*>(vec(a[9], at::kInt, 1, dev));
    const int nb = count(B), t = count(T), hq = count(Hq), hkv = count(K.size(1)), d = count(dh);
    void* const stream = stream_of(dev);
    return unlocked([&] {
      return g_attention(qr.p, qr.stride, pages, dt, cu, kv, nb, t, hq, hkv, d,
                         static_cast<float>(scale), out.p, ws, static_cast<size_t>(bytes), status,
                         stream);
    });
  });
}

// (logits, u, tokens, temperature, top_k, top_p, min_p, row_idx, kept, status)
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run([&] {
    need(n == 10 && g_sample != nullptr);
    const at::Tensor& z = tensor(a[0]);
    const int dev = device_of(z);
    const medusa_dtype_t dt = dtype(z);
    need(z.dim() == 2 && (z.size(1) <= 1 || z.stride(1) == 1));
    const int64_t rows = z.size(0), V = z.size(1), R = tensor(a[1]).numel();
    need(a[2] != Py_None);
    auto f32 = [&](int i) { return static_cast<const float*>(vec(a[i], at::kFloat, R, dev)); };
    auto i32 = [&](int i) { return static_cast<int32_t*>(vec(a[i], at::kInt, R, dev)); };
    const float *u = f32(1), *temperature = f32(3), *top_p = f32(5), *min_p = f32(6);
    const int32_t *row_idx = i32(7), *top_k = i32(4);
    int32_t *tokens = i32(2), *kept = i32(8);
    auto* status = static_cast<int32_t*>(vec(a[9], at::kInt, 1, dev));
    const int n_rows = count(rows), r = count(R), v = count(V);
    const void* logits = z.data_ptr();
    const long long stride = rows > 1 ? z.stride(0) : V;
    void* const stream = stream_of(dev);
    return unlocked([&] {
      return g_sample(logits, dt, stride, n_rows, row_idx, r, v, u, temperature, top_k, top_p,
                      min_p, tokens, kept, status, stream);
    });
  });
}

template <typename F>
PyCFunction fast(F* f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"rope", fast(rope), METH_FASTCALL, nullptr},
                         {"append", fast(append), METH_FASTCALL, nullptr},
                         {"attention", fast(attention), METH_FASTCALL, nullptr},
                         {"sample", fast(sample), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
