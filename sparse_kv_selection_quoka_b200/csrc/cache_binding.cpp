// Python binding of the paged cache's calls (module _cache_binding).
//
// A decode step's kernels take a few microseconds each: here a call's tensors
// are checked, its outputs and workspace allocated and the C ABI entered in
// about as little host time as the launches themselves need. Nothing is
// computed; the entry points of libquoka.so are handed over by address (bind).
//
// Every function takes its arguments by position, first the address of the
// cache's quoka_cache and its CUDA device (-1: none), and returns its outputs,
// or a quoka_status when the library refused.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <stdexcept>
#include <string>

#include "quoka.h"

namespace {

using at::Tensor;
using Shape4 = std::array<int64_t, 4>;

struct WrongType : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct WrongValue : std::runtime_error {
  using std::runtime_error::runtime_error;
};

decltype(&quoka_cache_append) g_append;
decltype(&quoka_cache_select) g_select;
decltype(&quoka_cache_select_padded) g_select_padded;
decltype(&quoka_cache_gather) g_gather;
decltype(&quoka_cache_attn) g_attn;
decltype(&quoka_select_workspace_size) g_select_ws;
decltype(&quoka_cache_attn_workspace_size) g_attn_ws;

// A tensor argument; null for None.
const Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw WrongType(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const Tensor& required(PyObject* o, const char* name) {
  const Tensor* t = tensor(o, name);
  if (t == nullptr) throw WrongType(std::string(name) + " must be a tensor, not None");
  return *t;
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw std::runtime_error("");
  return v;
}
int small(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) throw WrongValue(std::string(name) + " is out of range");
  return (int)v;
}

std::string text(c10::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

[[noreturn]] void wrong(const char* name, const Tensor& t, c10::IntArrayRef shape, const char* how) {
  throw WrongValue(std::string(name) + " must be " + how + text(shape) + " on the cache's device, not " + text(t.sizes()) +
                   " on " + t.device().str());
}
[[noreturn]] void wrong_type(const char* name, const Tensor& t, const char* want) {
  throw WrongType(std::string(name) + " must be " + want + ", not " + std::string(c10::toString(t.scalar_type())));
}

// The cache and what every tensor of a call has to match.
struct Call {
  const quoka_cache& c;
  int dev;

  Call(PyObject* handle, PyObject* device)
      : c(*reinterpret_cast<const quoka_cache*>(PyLong_AsVoidPtr(handle))), dev((int)integer(device)) {}

  // Rows (b, heads, rows, d) of float32 or bfloat16, any strides; -1: free.
  quoka_tensor rows(const Tensor& t, const char* name, int64_t heads, int64_t n, int dtype = -1) const {
    const auto st = t.scalar_type();
    const int code = st == at::kFloat ? QUOKA_F32 : st == at::kBFloat16 ? QUOKA_BF16 : -1;
    if (code < 0 || (dtype >= 0 && code != dtype))
      wrong_type(name, t, dtype < 0 ? "float32 or bfloat16" : dtype == QUOKA_F32 ? "float32" : "bfloat16");
    if (t.dim() != 4 || t.size(0) != c.b || (heads >= 0 && t.size(1) != heads) || (n >= 0 && t.size(2) != n) ||
        t.size(3) != c.d || t.get_device() != dev)
      wrong(name, t, {c.b, heads, n, c.d}, "");
    quoka_tensor v;
    v.data = t.data_ptr();
    v.dtype = (quoka_dtype)code;
    for (int i = 0; i < 4; ++i) {
      v.shape[i] = t.size(i);
      v.stride[i] = t.stride(i);
    }
    return v;
  }

  // A contiguous tensor of this type and shape: its address.
  void* plain(const Tensor& t, const char* name, at::ScalarType type, c10::IntArrayRef shape) const {
    if (t.scalar_type() != type) wrong_type(name, t, c10::toString(type));
    if (t.sizes() != shape || !t.is_contiguous() || t.get_device() != dev) wrong(name, t, shape, "contiguous of shape ");
    return t.data_ptr();
  }

  // The workspace given, or none.
  void* workspace(const Tensor* ws, size_t* bytes) const {
    *bytes = 0;
    if (ws == nullptr) return nullptr;
    if (!ws->is_contiguous() || ws->get_device() != dev)
      throw WrongValue("ws must be contiguous on the cache's device");
    *bytes = ws->nbytes();
    return ws->data_ptr();
  }

  void on_gpu() const {
    if (dev < 0) throw WrongValue("the cache must be on a CUDA device");
  }
  // An output (made without the dispatcher, which takes longer than the rest).
  Tensor make(at::ScalarType type, c10::IntArrayRef shape, bool zero = false) const {
    const c10::Device d(at::kCUDA, (c10::DeviceIndex)dev);
    if (zero) return at::zeros(shape, at::TensorOptions().dtype(type).device(d));
    return Tensor(at::detail::empty_cuda(shape, type, d, std::nullopt));
  }
  // A workspace of the current stream for this call (the device guard is set).
  static c10::DataPtr scratch(size_t bytes) { return c10::cuda::CUDACachingAllocator::get()->allocate(bytes); }
  void* stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
};

// The object given for an output, or one for the tensor made.
PyObject* out(PyObject* given, const Tensor& made) {
  if (made.defined()) return THPVariable_Wrap(made);
  Py_INCREF(given);
  return given;
}

template <typename F>
PyObject* guarded(const char* name, Py_ssize_t have, Py_ssize_t want, F&& f) {
  if (have != want) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments", name, want);
    return nullptr;
  }
  try {
    return f();
  } catch (const WrongType& e) {
    PyErr_SetString(PyExc_TypeError, e.what());
  } catch (const WrongValue& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (...) {  // (torch's own types: torch.OutOfMemoryError when there is no room for an output or a workspace)
    if (!PyErr_Occurred()) torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// handle, device, K, V, Q, cos, sin, neighbours, new_len, Kr, Qr, want_Kr, ws -> (Kr, Qr)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("append", n, 13, [&]() -> PyObject* {
    const Call call(a[0], a[1]);
    const auto& c = call.c;
    const Tensor &K = required(a[2], "K"), &V = required(a[3], "V");
    const Tensor *Q = tensor(a[4], "Q"), *cos = tensor(a[5], "cos"), *sin = tensor(a[6], "sin");
    const Tensor *fresh = tensor(a[8], "new_len"), *Kr = tensor(a[9], "Kr"), *Qr = tensor(a[10], "Qr");
    const quoka_tensor kv = call.rows(K, "K", c.nkv, -1);
    const int64_t BCP = kv.shape[2];
    const quoka_tensor vv = call.rows(V, "V", c.nkv, BCP, kv.dtype);
    const auto type = K.scalar_type();
    quoka_tensor qv;
    if (Q != nullptr) qv = call.rows(*Q, "Q", -1, BCP, kv.dtype);
    if (Q == nullptr && Qr != nullptr) throw WrongValue("Qr without Q");
    if ((cos == nullptr) != (sin == nullptr)) throw WrongValue("cos and sin go together");
    const float *cp = nullptr, *sp = nullptr;
    int64_t npos = 0, half = 0;
    if (cos != nullptr) {
      if (cos->dim() != 2) throw WrongValue("cos and sin must be (npos, rot / 2)");
      npos = cos->size(0);
      half = cos->size(1);
      if (half > c.d) throw WrongValue("cos and sin must be (npos, rot / 2), rot at most d");
      cp = (const float*)call.plain(*cos, "cos", at::kFloat, {npos, half});
      sp = (const float*)call.plain(*sin, "sin", at::kFloat, {npos, half});
    }
    const int32_t* np = fresh ? (const int32_t*)call.plain(*fresh, "new_len", at::kInt, {c.b}) : nullptr;
    void* krp = Kr ? call.plain(*Kr, "Kr", type, K.sizes()) : nullptr;
    void* qrp = Qr ? call.plain(*Qr, "Qr", type, Q->sizes()) : nullptr;
    size_t wn;
    void* wp = call.workspace(tensor(a[12], "ws"), &wn);
    call.on_gpu();
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)call.dev);
    // Rows that are left out are zeros in what is made here, and stay as they are in
    // what was given: the kernel's option acts on both.
    const bool given = Kr != nullptr || Qr != nullptr;
    Tensor made_k, made_q;
    if (Kr == nullptr && a[11] == Py_True) {
      made_k = call.make(type, K.sizes(), given);
      krp = made_k.data_ptr();
    }
    if (Qr == nullptr && Q != nullptr) {
      made_q = call.make(type, Q->sizes(), given);
      qrp = made_q.data_ptr();
    }
    const uint32_t flags = (a[7] == Py_True ? QUOKA_ROTATE_NEIGHBOURS : 0u) | (given ? 0u : QUOKA_ZERO_REST);
    const quoka_status st =
        g_append(&c, &kv, &vv, Q ? &qv : nullptr, cp, sp, npos, (int)(2 * half),
                 flags, np, krp, qrp, wp, wn, call.stream());
    if (st != QUOKA_OK) return PyLong_FromLong(st);
    return Py_BuildValue("(NN)", out(a[9], made_k), out(a[10], made_q));
  });
}

// handle, device, Q, max_len, NQ, BSA, kv_idx, kv_count, q_idx, s_agg, want_q_idx, want_s_agg, ws, new_len
// -> (kv_idx, kv_count, q_idx, s_agg)
PyObject* select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("select", n, 14, [&]() -> PyObject* {
    const Call call(a[0], a[1]);
    const auto& c = call.c;
    const Tensor& Q = required(a[2], "Q");
    const quoka_tensor qv = call.rows(Q, "Q", -1, -1);
    const int64_t nq = qv.shape[1], BCP = qv.shape[2];
    const int max_len = small(a[3], "max_len"), NQ = small(a[4], "NQ"), BSA = small(a[5], "BSA");
    const int64_t m = std::max(0, std::min(BSA, max_len));
    const Tensor *idx = tensor(a[6], "kv_idx"), *cnt = tensor(a[7], "kv_count"), *qi = tensor(a[8], "q_idx"),
                 *sa = tensor(a[9], "s_agg");
    void* ip = idx ? call.plain(*idx, "kv_idx", at::kInt, {c.b, c.nkv, m}) : nullptr;
    void* np = cnt ? call.plain(*cnt, "kv_count", at::kInt, {c.b, c.nkv}) : nullptr;
    void* qp = qi ? call.plain(*qi, "q_idx", at::kInt, {c.b, nq, NQ}) : nullptr;
    void* sp = sa ? call.plain(*sa, "s_agg", at::kFloat, {c.b, c.nkv, max_len}) : nullptr;
    size_t wn;
    void* wp = call.workspace(tensor(a[12], "ws"), &wn);
    const Tensor* fresh = tensor(a[13], "new_len");
    const int32_t* live = fresh ? (const int32_t*)call.plain(*fresh, "new_len", at::kInt, {c.b}) : nullptr;
    call.on_gpu();
    if (max_len < 0 || NQ < 1) return PyLong_FromLong(QUOKA_ERR_INVALID_ARG);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)call.dev);
    Tensor made_i, made_n, made_q, made_s;
    c10::DataPtr made_w;
    if (idx == nullptr) ip = (made_i = call.make(at::kInt, {c.b, c.nkv, m})).data_ptr();
    if (cnt == nullptr) np = (made_n = call.make(at::kInt, {c.b, c.nkv})).data_ptr();
    if (qi == nullptr && a[10] == Py_True) qp = (made_q = call.make(at::kInt, {c.b, nq, NQ})).data_ptr();
    if (sa == nullptr && a[11] == Py_True) sp = (made_s = call.make(at::kFloat, {c.b, c.nkv, max_len})).data_ptr();
    if (wp == nullptr) {
      wn = std::max<size_t>(256, g_select_ws(c.b, (int)nq, c.nkv, c.d, max_len, (int)BCP, NQ, std::max(0, BSA), qv.dtype));
      wp = (made_w = Call::scratch(wn)).get();
    }
    int32_t* ix = m ? (int32_t*)ip : nullptr;
    float* sx = max_len ? (float*)sp : nullptr;
    const quoka_status st =
        live ? g_select_padded(&qv, live, &c, max_len, NQ, BSA, ix, (int32_t*)np, (int32_t*)qp, sx, wp, wn, call.stream())
             : g_select(&qv, &c, max_len, NQ, BSA, ix, (int32_t*)np, (int32_t*)qp, sx, wp, wn, call.stream());
    if (st != QUOKA_OK) return PyLong_FromLong(st);
    return Py_BuildValue("(NNNN)", out(a[6], made_i), out(a[7], made_n), out(a[8], made_q), out(a[9], made_s));
  });
}

// An index list (b, nkv, N) with counts, or none: N, and addresses (not null for an empty list).
struct List {
  int n;
  const int32_t *idx = nullptr, *cnt = nullptr;
  List(const Call& call, int max_len, PyObject* i, PyObject* k) : n(max_len) {
    const Tensor *ti = tensor(i, "kv_idx"), *tk = tensor(k, "kv_count");
    if ((ti == nullptr) != (tk == nullptr)) throw WrongValue("kv_idx and kv_count go together");
    if (ti == nullptr) return;
    if (ti->dim() != 3 || ti->size(2) > INT32_MAX) throw WrongValue("kv_idx must be (b, nkv, N)");
    n = (int)ti->size(2);
    idx = (const int32_t*)call.plain(*ti, "kv_idx", at::kInt, {call.c.b, call.c.nkv, n});
    cnt = (const int32_t*)call.plain(*tk, "kv_count", at::kInt, {call.c.b, call.c.nkv});
    if (n == 0) idx = cnt;
  }
};

// handle, device, max_len, kv_idx, kv_count, float32?, Ksel, Vsel, ws -> (Ksel, Vsel)
PyObject* gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("gather", n, 9, [&]() -> PyObject* {
    const Call call(a[0], a[1]);
    const auto& c = call.c;
    const int max_len = small(a[2], "max_len");
    const List list(call, max_len, a[3], a[4]);
    const bool f32 = a[5] == Py_True;
    const auto type = f32 ? at::kFloat : at::kBFloat16;
    const Shape4 shape = {c.b, c.nkv, list.n, c.d};
    const Tensor *K = tensor(a[6], "Ksel"), *V = tensor(a[7], "Vsel");
    void* kp = K ? call.plain(*K, "Ksel", type, shape) : nullptr;
    void* vp = V ? call.plain(*V, "Vsel", type, shape) : nullptr;
    size_t wn;
    void* wp = call.workspace(tensor(a[8], "ws"), &wn);
    call.on_gpu();
    if (list.n < 0) return PyLong_FromLong(QUOKA_ERR_INVALID_ARG);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)call.dev);
    Tensor made_k, made_v;
    if (K == nullptr) kp = (made_k = call.make(type, shape)).data_ptr();
    if (V == nullptr) vp = (made_v = call.make(type, shape)).data_ptr();
    const quoka_status st = g_gather(&c, max_len, list.idx, list.cnt, list.n, f32 ? QUOKA_F32 : QUOKA_BF16,
                                     list.n ? kp : nullptr, list.n ? vp : nullptr, wp, wn, call.stream());
    if (st != QUOKA_OK) return PyLong_FromLong(st);
    return Py_BuildValue("(NN)", out(a[6], made_k), out(a[7], made_v));
  });
}

// handle, device, Q, max_len, kv_idx, kv_count, Kc, Vc, scale, O, lse, want_lse, ws -> (O, lse)
PyObject* attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("attn", n, 13, [&]() -> PyObject* {
    const Call call(a[0], a[1]);
    const auto& c = call.c;
    const Tensor& Q = required(a[2], "Q");
    const quoka_tensor qv = call.rows(Q, "Q", -1, -1);
    const int64_t nq = qv.shape[1], BCP = qv.shape[2];
    const int max_len = small(a[3], "max_len");
    const List list(call, max_len, a[4], a[5]);
    const Tensor *Kc = tensor(a[6], "Kc"), *Vc = tensor(a[7], "Vc"), *O = tensor(a[9], "O"), *lse = tensor(a[10], "lse");
    if ((Kc == nullptr) != (Vc == nullptr)) throw WrongValue("Kc and Vc go together");
    quoka_tensor kcv, vcv;
    if (Kc != nullptr) {
      kcv = call.rows(*Kc, "Kc", c.nkv, BCP, qv.dtype);
      vcv = call.rows(*Vc, "Vc", c.nkv, BCP, qv.dtype);
    }
    const double scale = PyFloat_AsDouble(a[8]);
    if (scale == -1.0 && PyErr_Occurred()) throw std::runtime_error("");
    void* op = O ? call.plain(*O, "O", Q.scalar_type(), Q.sizes()) : nullptr;
    void* lp = lse ? call.plain(*lse, "lse", at::kFloat, {c.b, nq, BCP}) : nullptr;
    size_t wn;
    void* wp = call.workspace(tensor(a[12], "ws"), &wn);
    call.on_gpu();
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)call.dev);
    Tensor made_o, made_l;
    c10::DataPtr made_w;
    if (O == nullptr) op = (made_o = call.make(Q.scalar_type(), Q.sizes())).data_ptr();
    if (lse == nullptr && a[11] == Py_True) lp = (made_l = call.make(at::kFloat, {c.b, nq, BCP})).data_ptr();
    if (wp == nullptr) {
      wn = std::max<size_t>(256, g_attn_ws(c.b, (int)nq, c.nkv, c.d, (int)BCP, list.n, qv.dtype));
      wp = (made_w = Call::scratch(wn)).get();
    }
    const quoka_status st = g_attn(&qv, &c, max_len, list.idx, list.cnt, list.n, Kc ? &kcv : nullptr, Kc ? &vcv : nullptr,
                                   (float)scale, op, (float*)lp, wp, wn, call.stream());
    if (st != QUOKA_OK) return PyLong_FromLong(st);
    return Py_BuildValue("(NN)", out(a[9], made_o), out(a[10], made_l));
  });
}

// The addresses of the entry points.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("bind", n, 7, [&]() -> PyObject* {
    g_append = reinterpret_cast<decltype(g_append)>(PyLong_AsVoidPtr(a[0]));
    g_select = reinterpret_cast<decltype(g_select)>(PyLong_AsVoidPtr(a[1]));
    g_select_padded = reinterpret_cast<decltype(g_select_padded)>(PyLong_AsVoidPtr(a[2]));
    g_gather = reinterpret_cast<decltype(g_gather)>(PyLong_AsVoidPtr(a[3]));
    g_attn = reinterpret_cast<decltype(g_attn)>(PyLong_AsVoidPtr(a[4]));
    g_select_ws = reinterpret_cast<decltype(g_select_ws)>(PyLong_AsVoidPtr(a[5]));
    g_attn_ws = reinterpret_cast<decltype(g_attn_ws)>(PyLong_AsVoidPtr(a[6]));
    Py_RETURN_NONE;
  });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"bind", FAST(bind), nullptr},     {"append", FAST(append), nullptr},
                         {"select", FAST(select), nullptr}, {"gather", FAST(gather), nullptr},
                         {"attn", FAST(attn), nullptr},     {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_cache_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cache_binding() { return PyModule_Create(&module); }
