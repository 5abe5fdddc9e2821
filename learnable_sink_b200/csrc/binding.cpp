// The binding's short way for the paged calls.  They serve single tokens, where a
// kernel takes 3 to 9 us and the host's time shows: reading five tensors' metadata
// from Python takes about 4 us and a ctypes call with 18 arguments 1.6 us, here both
// take well under one.
//
// Each function checks the metadata that the Python path checks and makes the C ABI
// call; it returns the ABI's code, or -1 without having launched anything if some
// check fails or an argument is of a kind it does not handle.  The Python path then
// says what is wrong, or makes the call itself.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include "../../include/sinkattn.h"

namespace {

using Append = decltype(&sinkattn_paged_append);
using Decode = decltype(&sinkattn_paged_decode);
Append g_append[2];  // 16-bit, 8-bit cache
Decode g_decode[2];

constexpr int kDeclined = -1;

// An optional tensor argument; false if it is something else.
bool tensor(PyObject* o, const at::Tensor** t) {
  if (o == Py_None) {
    *t = nullptr;
    return true;
  }
  if (!THPVariable_Check(o)) return false;
  *t = &THPVariable_Unpack(o);
  return true;
}
bool plain(const at::Tensor& t, at::ScalarType type, int dev, std::initializer_list<int64_t> shape) {
  return t.is_cuda() && t.get_device() == dev && t.scalar_type() == type && t.is_contiguous() &&
         t.sizes() == at::IntArrayRef(shape);
}
// A packed [T, H, D] input whose tokens may be strided.
bool tokens(const at::Tensor& t, at::ScalarType type, int dev, int64_t T, int64_t H, int64_t D,
            long long* stride) {
  if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || t.dim() != 3 ||
      t.size(0) != T || t.size(1) != H || t.size(2) != D)
    return false;
  *stride = T <= 1 ? H * D : t.stride(0);
  return t.stride(2) == 1 && (H == 1 || t.stride(1) == D) && *stride >= H * D && *stride % 8 == 0 &&
         reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0;
}

struct Cache {
  const sinkattn_paged_cache* c;
  int coded, dev;  // 8-bit cache; device
  at::ScalarType type;  // of the pages (16-bit cache)
};
// The first four arguments: the descriptor's address, whether the call is the 8-bit
// one, the pages' kind (0 bf16, 1 f16, 2 codes) and the device.
bool cache_args(PyObject* const* a, Cache* c) {
  c->c = reinterpret_cast<const sinkattn_paged_cache*>(PyLong_AsVoidPtr(a[0]));
  c->coded = (int)PyLong_AsLong(a[1]);
  const long kind = PyLong_AsLong(a[2]);
  c->dev = (int)PyLong_AsLong(a[3]);
  c->type = kind == 0 ? at::kBFloat16 : at::kHalf;
  return c->c && (kind == 2) == (c->coded != 0);
}
int dtype_code(at::ScalarType t) {
  return t == at::kBFloat16 ? SINKATTN_BF16 : t == at::kHalf ? SINKATTN_FP16 : -1;
}
template <class T>
T* data(const at::Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}
sinkattn_stream_t stream_of(int dev) {
  return reinterpret_cast<sinkattn_stream_t>(
      c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
}

// Other Python threads run while a launch waits for room in a stream's queue (what
// the stream waits for may be theirs to do), as they do in a ctypes call.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// (descriptor, coded, kind, device, k, v, cu_new, rope, interleaved, q, q_out, k_out)
int append(PyObject* const* a) {
  Cache c;
  const at::Tensor *k, *v, *cu, *rope, *q, *q_out, *k_out;
  if (!cache_args(a, &c) || !tensor(a[4], &k) || !tensor(a[5], &v) || !tensor(a[6], &cu) ||
      !tensor(a[7], &rope) || !tensor(a[9], &q) || !tensor(a[10], &q_out) || !tensor(a[11], &k_out))
    return kDeclined;
  const int interleaved = PyObject_IsTrue(a[8]);
  if (!k || !v || k->dim() != 3 || !q != !q_out || interleaved < 0) return kDeclined;
  const at::ScalarType type = k->scalar_type();
  const int dt = dtype_code(type);
  if (dt < 0 || (!c.coded && type != c.type)) return kDeclined;
  const int64_t T = k->size(0), D = c.c->D, Hkv = c.c->Hkv, B = c.c->B;
  long long ks = 0, vs = 0, qs = 0;
  int64_t Hq = 0;
  if (!tokens(*k, type, c.dev, T, Hkv, D, &ks) || !tokens(*v, type, c.dev, T, Hkv, D, &vs))
    return kDeclined;
  if (q) {
    if (q->dim() != 3) return kDeclined;
    Hq = q->size(1);
    if (!tokens(*q, type, c.dev, T, Hq, D, &qs) || !plain(*q_out, type, c.dev, {T, Hq, D}))
      return kDeclined;
  }
  if (k_out && !plain(*k_out, type, c.dev, {T, Hkv, D})) return kDeclined;
  if (cu ? !plain(*cu, at::kInt, c.dev, {B + 1}) : T != B) return kDeclined;
  int rot = 0, n_pos = 0;
  if (rope) {
    if (rope->dim() != 2 || !plain(*rope, at::kFloat, c.dev, {rope->size(0), rope->size(1)}))
      return kDeclined;
    if (rope->size(0) < 1 || rope->size(0) > INT_MAX || rope->size(1) % 16 != 0 ||
        rope->size(1) < 16 || rope->size(1) > D)
      return kDeclined;
    n_pos = (int)rope->size(0);
    rot = (int)rope->size(1);
  }
  if (T > INT_MAX || Hq > INT_MAX || c10::cuda::current_device() != c.dev) return kDeclined;
  const sinkattn_stream_t stream = stream_of(c.dev);
  const Unlocked unlocked;
  return g_append[c.coded](static_cast<sinkattn_dtype>(dt), (int)T, (int)Hq, c.c, data<void>(k), ks,
                           data<void>(v), vs, data<void>(q), qs, data<int32_t>(cu),
                           data<float>(rope), rot, n_pos, interleaved, data<void>(q_out),
                           data<void>(k_out), stream);
}

// (descriptor, coded, kind, device, q, sink, n_sink, window, scale, workspace, out, lse, sink_s)
int decode(PyObject* const* a) {
  Cache c;
  const at::Tensor *q, *sink, *ws, *out, *lse, *sink_s;
  if (!cache_args(a, &c) || !tensor(a[4], &q) || !tensor(a[5], &sink) || !tensor(a[9], &ws) ||
      !tensor(a[10], &out) || !tensor(a[11], &lse) || !tensor(a[12], &sink_s))
    return kDeclined;
  if (!q || !ws || !out || !lse || !sink_s || q->dim() != 3) return kDeclined;
  const at::ScalarType type = q->scalar_type();
  const int dt = dtype_code(type);
  const int64_t B = c.c->B, Hq = q->size(1), D = c.c->D;
  if (dt < 0 || (!c.coded && type != c.type) || !plain(*q, type, c.dev, {B, Hq, D}) ||
      !plain(*out, type, c.dev, {B, Hq, D}) || !plain(*lse, at::kFloat, c.dev, {B, Hq}) ||
      !plain(*sink_s, at::kFloat, c.dev, {B, Hq}) ||
      (sink && !plain(*sink, at::kFloat, c.dev, {Hq})) || !ws->is_cuda() ||
      ws->get_device() != c.dev || !ws->is_contiguous())
    return kDeclined;
  if (!PyLong_CheckExact(a[6]) || !PyLong_CheckExact(a[7])) return kDeclined;
  int over[2];
  const long long n_sink = PyLong_AsLongLongAndOverflow(a[6], &over[0]);
  const long long window = PyLong_AsLongLongAndOverflow(a[7], &over[1]);
  if (over[0] || over[1] || n_sink < 0 || n_sink > INT_MAX || window < 0 || window > INT_MAX)
    return kDeclined;
  double scale = 1.0 / std::sqrt((double)D);
  if (a[8] != Py_None) {
    if (!PyFloat_Check(a[8])) return kDeclined;
    scale = PyFloat_AsDouble(a[8]);
  }
  if (Hq > INT_MAX || c10::cuda::current_device() != c.dev) return kDeclined;
  const sinkattn_stream_t stream = stream_of(c.dev);
  const Unlocked unlocked;
  return g_decode[c.coded](static_cast<sinkattn_dtype>(dt), (int)Hq, (float)scale, data<void>(q), c.c,
                           (int)n_sink, (int)window, data<float>(sink), data<void>(out),
                           data<float>(lse), data<float>(sink_s), data<void>(ws), ws->nbytes(), stream);
}

// No C++ exception passes into the interpreter: what throws is declined (nothing
// throws behind the ABI call).
template <int (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  int rc = kDeclined;
  try {
    rc = F(args);
  } catch (...) {
    rc = kDeclined;
  }
  if (PyErr_Occurred()) {
    PyErr_Clear();
    rc = kDeclined;
  }
  return PyLong_FromLong(rc);
}

// The entry points of the loaded library, by address.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "four addresses");
    return nullptr;
  }
  for (int i = 0; i < 2; ++i) {
    g_append[i] = reinterpret_cast<Append>(PyLong_AsVoidPtr(args[i]));
    g_decode[i] = reinterpret_cast<Decode>(PyLong_AsVoidPtr(args[2 + i]));
  }
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"paged_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<append, 12>)),
     METH_FASTCALL, nullptr},
    {"paged_decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<decode, 13>)),
     METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&kModule);
  // the torch whose tensors this file can read
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
