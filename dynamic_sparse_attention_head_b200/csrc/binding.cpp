// Argument checks and marshalling of the calls around the layer (serving.py), in C++: a decode step makes
// them once per layer and token, and through ctypes the checks of ten tensors cost more than the
// launch (a slot map 10.6 us of host time, against 3.5 here and the 4 us of its kernel).  Each function checks
// its tensors, takes the device's current stream (or the one given), makes the device current, and
// returns the library's status; what is wrong with an argument is raised as TypeError or ValueError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <stdexcept>

#include "../../include/msa.h"

namespace {

struct Bad : std::runtime_error {
  PyObject* type;
  Bad(PyObject* t, const std::string& m) : std::runtime_error(m), type(t) {}
};

[[noreturn]] void refuse(const char* name, const at::Tensor& t, const std::string& want) {
  std::ostringstream s;
  s << name << ": " << want << " is wanted, got " << t.sizes() << " " << t.dtype().name() << " with strides " << t.strides()
    << " on " << t.device();
  throw Bad(PyExc_ValueError, s.str());
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Bad(PyExc_TypeError, std::string(name) + ": a tensor is wanted, got " + Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

std::string on(int dev) { return " on cuda:" + std::to_string(dev); }

bool there(const at::Tensor& t, at::ScalarType type, int64_t dim, int dev) {
  return t.scalar_type() == type && t.dim() == dim && t.is_cuda() && t.get_device() == dev && t.layout() == at::kStrided;
}

// a contiguous vector of n entries (n < 0: any number)
const at::Tensor& vec(PyObject* o, const char* name, at::ScalarType type, int dev, int64_t n = -1) {
  const at::Tensor& t = tensor(o, name);
  if (!there(t, type, 1, dev) || !t.is_contiguous() || (n >= 0 && t.numel() != n)) {
    std::ostringstream s;
    s << "a contiguous " << type << " vector";
    if (n >= 0) s << " of " << n;
    refuse(name, t, s.str() + on(dev));
  }
  return t;
}

// [heads, tokens, 128] bf16 with contiguous rows (-1: any number)
const at::Tensor& rows(PyObject* o, const char* name, int64_t heads, int64_t tokens, int dev) {
  const at::Tensor& t = tensor(o, name);
  if (!there(t, at::kBFloat16, 3, dev) || t.size(2) != 128 || (t.stride(2) != 1 && t.numel()) ||
      (heads >= 0 && t.size(0) != heads) || (tokens >= 0 && t.size(1) != tokens)) {
    std::ostringstream s;
    s << "a bf16 [" << (heads < 0 ? "H" : std::to_string(heads)) << ", " << (tokens < 0 ? "T" : std::to_string(tokens))
      << ", 128] tensor with contiguous rows";
    refuse(name, t, s.str() + on(dev));
  }
  return t;
}

// The same, written to: rows that share elements (an expanded tensor) would be written over one another.
const at::Tensor& rows_out(PyObject* o, const char* name, int64_t heads, int64_t tokens, int dev) {
  const at::Tensor& t = rows(o, name, heads, tokens, dev);
  for (int axis = 0; axis < 2; ++axis)
    if (t.size(axis) > 1 && t.stride(axis) < 128 && t.numel()) refuse(name, t, "a tensor whose rows do not overlap" + on(dev));
  return t;
}

// A tensor's stride along an axis.  That of an axis of one says nothing (a tensor that came through DLPack has 1 there).
int64_t step(const at::Tensor& t, int64_t axis) { return t.size(axis) > 1 ? t.stride(axis) : 0; }

// block table [B, blocks] with contiguous rows
const at::Tensor& table(PyObject* o, int64_t B, int dev, int64_t& stride) {
  const at::Tensor& t = tensor(o, "block_table");
  if (!there(t, at::kInt, 2, dev) || t.size(0) != B || (t.size(1) > 1 && t.stride(1) != 1) ||
      (B > 1 && t.stride(0) < t.size(1)) || t.size(1) > INT32_MAX)
    refuse("block_table", t, "an int32 [" + std::to_string(B) + ", blocks] tensor with contiguous rows" + on(dev));
  stride = std::max(t.stride(0), t.size(1));
  return t;
}

int whole(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Bad(PyExc_TypeError, std::string(name) + ": a whole number is wanted");
  }
  if (v < INT32_MIN || v > INT32_MAX) throw Bad(PyExc_ValueError, std::string(name) + " does not fit 32 bits");
  return (int)v;
}

double number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Bad(PyExc_TypeError, std::string(name) + ": a number is wanted");
  }
  return v;
}

void* address(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) {
    PyErr_Clear();
    throw Bad(PyExc_TypeError, "an address is wanted");
  }
  return p;
}

void* stream_of(PyObject* o, int dev) {
  return o == Py_None ? static_cast<void*>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream()) : address(o);
}

template <class T>
T* ptr(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

struct Cache {  // the first two arguments of every call on a cache: its description and its device
  const msa_kv4_cache* c;
  int dev;
  c10::cuda::CUDAGuard guard;
  Cache(PyObject* const* a)
      : c(static_cast<const msa_kv4_cache*>(address(a[0]))), dev(whole(a[1], "device")), guard((c10::DeviceIndex)dev) {}
};

template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  try {
    if (n != want) throw Bad(PyExc_TypeError, "wrong number of arguments");
    return PyLong_FromLong((long)f());
  } catch (const Bad& e) {
    PyErr_SetString(e.type, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// Python's other threads run while the library is in the call: a status call waits for the stream, and a launch for room
// in the queue.  The arguments live on in the caller's frame; every one is taken apart before.
struct Unlocked {
  PyThreadState* const state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// Q, K, Qo, Ko, positions, rope (address), axes, wq, wk, eps, stream
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    const at::Tensor& first = tensor(a[0], "Q");
    if (!first.is_cuda()) refuse("Q", first, "a CUDA tensor");
    const int dev = first.get_device();
    const at::Tensor &Q = rows(a[0], "Q", -1, -1, dev), &K = rows(a[1], "K", -1, Q.size(1), dev);
    const int64_t T = Q.size(1), axes = whole(a[6], "axes");
    const at::Tensor &Qo = rows_out(a[2], "Qo", Q.size(0), T, dev), &Ko = rows_out(a[3], "Ko", K.size(0), T, dev);
    const msa_rope rope = *static_cast<const msa_rope*>(address(a[5]));
    const int32_t* positions = nullptr;  // a norm alone has none
    int64_t pos_stride = T;
    if (rope.dim || a[4] != Py_None) {
      const at::Tensor& pos = tensor(a[4], "positions");
      if (!there(pos, at::kInt, pos.dim() == 2 ? 2 : 1, dev) || pos.size(-1) != T || (pos.dim() == 2 ? pos.size(0) : 1) != axes ||
          (T > 1 && pos.stride(-1) != 1))
        refuse("positions", pos, "int32 [" + std::to_string(axes) + ", " + std::to_string(T) + "] with contiguous rows" + on(dev));
      positions = ptr<const int32_t>(pos);
      if (pos.dim() == 2) pos_stride = pos.stride(0);
    }
    const void* wq = a[7] == Py_None ? nullptr : vec(a[7], "wq", at::kBFloat16, dev, 128).data_ptr();
    const void* wk = a[8] == Py_None ? nullptr : vec(a[8], "wk", at::kBFloat16, dev, 128).data_ptr();
    if (Q.size(0) > INT32_MAX || K.size(0) > INT32_MAX) throw Bad(PyExc_ValueError, "too many heads");
    msa_strides in{}, out{};
    in.q_head = step(Q, 0), in.q_row = step(Q, 1), in.k_head = step(K, 0), in.k_row = step(K, 1);
    out.q_head = step(Qo, 0), out.q_row = step(Qo, 1), out.k_head = step(Ko, 0), out.k_row = step(Ko, 1);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    const float eps = (float)number(a[9], "eps");
    void* const st = stream_of(a[10], dev);
    const Unlocked u;
    return msa_qk_norm_rope(Q.data_ptr(), K.data_ptr(), &in, Qo.data_ptr(), Ko.data_ptr(), &out, T, (int32_t)Q.size(0),
                            (int32_t)K.size(0), wq, wk, eps, &rope, positions, pos_stride, st);
  });
}

// cache, device, kv_lens, new_lens, block_table, free_pages, n_free, slots, positions, cu_new, kv_lens_out, n_free_out, stream
PyObject* slots(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    const Cache k(a);
    const at::Tensor& kv = vec(a[2], "kv_lens", at::kInt, k.dev);
    const int64_t B = kv.numel();
    const at::Tensor& fresh = vec(a[3], "new_lens", at::kInt, k.dev, B);
    int64_t stride;
    const at::Tensor& tab = table(a[4], B, k.dev, stride);
    const at::Tensor &free = vec(a[5], "free_pages", at::kInt, k.dev, k.c->n_pages), &nf = vec(a[6], "n_free", at::kInt, k.dev, 1);
    const at::Tensor& sl = vec(a[7], "slots", at::kLong, k.dev);
    const at::Tensor &pos = vec(a[8], "positions", at::kInt, k.dev, sl.numel()), &cu = vec(a[9], "cu_new", at::kInt, k.dev, B + 1);
    const at::Tensor& kv_out = a[10] == Py_None ? kv : vec(a[10], "kv_lens_out", at::kInt, k.dev, B);
    const at::Tensor& nf_out = a[11] == Py_None ? nf : vec(a[11], "n_free_out", at::kInt, k.dev, 1);
    if (B > INT32_MAX) throw Bad(PyExc_ValueError, "too many requests");
    void* const st = stream_of(a[12], k.dev);
    const Unlocked u;
    return msa_kv4_slots(k.c, ptr<int32_t>(kv), ptr<int32_t>(fresh), (int32_t)B, ptr<int32_t>(tab), stride, (int32_t)tab.size(1),
                         ptr<int32_t>(free), ptr<int32_t>(nf), ptr<int32_t>(kv_out), ptr<int32_t>(nf_out), ptr<int32_t>(cu),
                         ptr<int64_t>(sl), ptr<int32_t>(pos), sl.numel(), st);
  });
}

// cache, device, ids, kv_lens, block_table, free_pages, n_free, stream
PyObject* release(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    const Cache k(a);
    const at::Tensor &ids = vec(a[2], "ids", at::kInt, k.dev), &kv = vec(a[3], "kv_lens", at::kInt, k.dev);
    int64_t stride;
    const at::Tensor& tab = table(a[4], kv.numel(), k.dev, stride);
    const at::Tensor &free = vec(a[5], "free_pages", at::kInt, k.dev, k.c->n_pages), &nf = vec(a[6], "n_free", at::kInt, k.dev, 1);
    if (kv.numel() > INT32_MAX || ids.numel() > INT32_MAX) throw Bad(PyExc_ValueError, "too many requests");
    void* const st = stream_of(a[7], k.dev);
    const Unlocked u;
    return msa_kv4_release(k.c, ptr<int32_t>(ids), (int32_t)ids.numel(), ptr<int32_t>(kv), (int32_t)kv.numel(), ptr<int32_t>(tab),
                           stride, (int32_t)tab.size(1), ptr<int32_t>(free), ptr<int32_t>(nf), st);
  });
}

// cache, device, K, V, slots, stream
template <bool WRITE>
PyObject* rows_at(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    const Cache k(a);
    const at::Tensor& sl = vec(a[4], "slots", at::kLong, k.dev);
    constexpr auto rows_of = WRITE ? rows : rows_out;  // an append reads K and V
    const at::Tensor &K = rows_of(a[2], "K", k.c->Hkv, sl.numel(), k.dev), &V = rows_of(a[3], "V", k.c->Hkv, sl.numel(), k.dev);
    msa_strides s{};
    s.k_head = step(K, 0), s.k_row = step(K, 1), s.v_head = step(V, 0), s.v_row = step(V, 1);
    void* const st = stream_of(a[5], k.dev);
    const Unlocked u;
    return WRITE ? msa_kv4_append(k.c, K.data_ptr(), V.data_ptr(), &s, ptr<int64_t>(sl), sl.numel(), st)
                 : msa_kv4_read(k.c, K.data_ptr(), V.data_ptr(), &s, ptr<int64_t>(sl), sl.numel(), st);
  });
}

// cache, device, Q, O, block_table, kv_lens, cu_q, max_q, scale, ws, lse, stream
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    const Cache k(a);
    const at::Tensor& Q = rows(a[2], "Q", -1, -1, k.dev);
    const at::Tensor& O = rows_out(a[3], "O", Q.size(0), Q.size(1), k.dev);
    const at::Tensor& kv = vec(a[5], "kv_lens", at::kInt, k.dev);
    const int64_t B = kv.numel();
    int64_t stride;
    const at::Tensor& tab = table(a[4], B, k.dev, stride);
    const at::Tensor& cu = vec(a[6], "cu_q", at::kInt, k.dev, B + 1);
    const at::Tensor& ws = vec(a[9], "ws", at::kByte, k.dev);
    float* lse = nullptr;
    if (a[10] != Py_None) {
      const at::Tensor& t = tensor(a[10], "lse");
      if (!there(t, at::kFloat, 2, k.dev) || t.size(0) != Q.size(0) || t.size(1) != Q.size(1) || !t.is_contiguous())
        refuse("lse", t, "a contiguous float32 [" + std::to_string(Q.size(0)) + ", " + std::to_string(Q.size(1)) + "] tensor" + on(k.dev));
      lse = ptr<float>(t);
    }
    if (B > INT32_MAX || Q.size(0) > INT32_MAX || Q.size(1) > INT32_MAX) throw Bad(PyExc_ValueError, "too many rows");
    msa_strides s{};
    s.q_head = step(Q, 0), s.q_row = step(Q, 1), s.o_head = step(O, 0), s.o_row = step(O, 1);
    const float scale = (float)number(a[8], "scale");
    const int max_q = whole(a[7], "max_q");
    void* const st = stream_of(a[11], k.dev);
    const Unlocked u;
    return msa_kv4_attend(k.c, Q.data_ptr(), O.data_ptr(), &s, (int32_t)Q.size(1), (int32_t)Q.size(0), scale,
                          ptr<int32_t>(tab), stride, (int32_t)tab.size(1), ptr<int32_t>(kv), ptr<int32_t>(cu), (int32_t)B,
                          max_q, lse, ws.data_ptr(), (size_t)ws.numel(), st);
  });
}

// cache, device, stream
PyObject* status(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&] {
    const Cache k(a);
    void* const st = stream_of(a[2], k.dev);
    const Unlocked u;
    return msa_kv4_status(k.c, st);
  });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f))
PyMethodDef methods[] = {{"norm_rope", FAST(norm_rope), METH_FASTCALL, nullptr},
                         {"slots", FAST(slots), METH_FASTCALL, nullptr},
                         {"release", FAST(release), METH_FASTCALL, nullptr},
                         {"append", FAST(rows_at<true>), METH_FASTCALL, nullptr},
                         {"read", FAST(rows_at<false>), METH_FASTCALL, nullptr},
                         {"attend", FAST(attend), METH_FASTCALL, nullptr},
                         {"status", FAST(status), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
