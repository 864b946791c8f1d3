// pkv_torch.cpp -- the Python side of the 4-bit, norm and table calls: checks of the tensors'
// types, devices and shapes, outputs allocated by torch, the current stream, one C call. A decode
// step makes several of these calls of a few microseconds each, and the same written with ctypes
// and Tensor attributes took longer than the kernels: norm of 64 tokens 15.8 us a call (2.0 of
// them on the GPU), now 5.7; two table calls with four outputs 26.4 (8.8), now 11.3; append and
// widening of 64 tokens 14.3 (3.4), now 4.9.
//
// The library itself is reached through the addresses of its entry points, handed over by bind(),
// so that this file needs no second copy of it and a variant can be bound instead.
#define PY_SSIZE_T_CLEAN
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>

#include "../../include/pkv.h"

namespace {

struct {
  decltype(&pkv_kv_append_int4) kv_append_int4;
  decltype(&pkv_widen_blocks_int4) widen_blocks_int4;
  decltype(&pkv_paged_attn_decode_int4) decode_int4;
  decltype(&pkv_paged_attn_decode_append_int4) decode_append_int4;
  decltype(&pkv_qk_norm_rope) qk_norm_rope;
  decltype(&pkv_extend_tables) extend_tables;
  decltype(&pkv_truncate_tables) truncate_tables;
} lib;
constexpr int kEntryPoints = 7;
PyObject* error_class = nullptr;   // pkv.PkvError(entry point, status)

constexpr auto kF16 = at::kHalf;
constexpr auto kF32 = at::kFloat;
constexpr auto kU8 = at::kByte;
constexpr auto kI32 = at::kInt;
constexpr auto kI64 = at::kLong;
constexpr int kRow = 80;

PyObject* fail(const char* fn, int status) {
  PyObject* e = PyObject_CallFunction(error_class, "si", fn, status);
  if (e) {
    PyErr_SetObject(error_class, e);
    Py_DECREF(e);
  }
  return nullptr;
}

struct Raised {};   // a Python error is set

// One call's arguments, in the order of the Python signature (the last is the stream or None).
struct Args {
  const char* fn;
  PyObject* const* a;
  int dev;
  bool ok = true;   // every tensor so far is one, of the type wanted, here and contiguous

  const at::Tensor& any(int i) {
    static const at::Tensor none;
    if (!THPVariable_Check(a[i])) {
      ok = false;
      return none;
    }
    return THPVariable_Unpack(a[i]);
  }
  const at::Tensor& strided(int i, at::ScalarType type) {
    const at::Tensor& t = any(i);
    ok = ok && t.is_cuda() && t.scalar_type() == type && t.get_device() == dev;
    return t;
  }
  const at::Tensor& tensor(int i, at::ScalarType type) {
    const at::Tensor& t = strided(i, type);
    ok = ok && t.is_contiguous();
    return t;
  }
  int64_t whole(int i) {
    const int64_t v = PyLong_AsLongLong(a[i]);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    if (v < INT32_MIN || v > INT32_MAX) ok = false;
    return v;
  }
  float number(int i) {
    const double v = PyFloat_AsDouble(a[i]);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return static_cast<float>(v);
  }
  pkv_stream_t stream(int i) {
    if (a[i] == Py_None) return c10::cuda::getCurrentCUDAStream(dev).stream();
    PyObject* handle = PyObject_GetAttrString(a[i], "cuda_stream");
    if (!handle) throw Raised();
    void* s = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (PyErr_Occurred()) throw Raised();
    return s;
  }
};

// The library is called without Python's lock: a launch waits where the GPU's queue is full, and
// other threads go on meanwhile.
template <class F>
int unlocked(F&& call) {
  struct Lock {
    PyThreadState* const state = PyEval_SaveThread();
    ~Lock() { PyEval_RestoreThread(state); }
  } lock;
  return call();
}

// Outputs of a call with the stream argument i, allocated on the stream that it runs on: memory freed
// on another one may still be in use there.
struct Outputs {
  c10::cuda::OptionalCUDAStreamGuard guard;
  Outputs(const Args& A, int i, pkv_stream_t s) {
    if (A.a[i] == Py_None) return;
    // (the legacy default stream has two handles)
    const auto handle = static_cast<cudaStream_t>(s);
    guard.reset_stream(handle == cudaStreamLegacy ? c10::cuda::getDefaultCUDAStream(A.dev)
                                                  : c10::cuda::getStreamFromExternal(handle, A.dev));
  }
};

bool fits(int64_t v) { return v <= INT32_MAX; }

bool same(const at::Tensor& x, const at::Tensor& y) { return x.sizes() == y.sizes(); }

bool shaped(const at::Tensor& t, std::initializer_list<int64_t> s) {
  return t.sizes() == at::IntArrayRef(s.begin(), s.size());
}

template <class T = void>
T* ptr(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

PyObject* none() { Py_RETURN_NONE; }

PyObject* kv_append_int4(Args& A) {   // k, v, slots, k_cache, v_cache, stream
  const at::Tensor &k = A.tensor(0, kF16), &v = A.tensor(1, kF16), &slots = A.tensor(2, kI64),
                   &kc = A.tensor(3, kU8), &vc = A.tensor(4, kU8);
  if (!A.ok || kc.dim() != 4) return fail(A.fn, PKV_EINVAL);
  const int64_t nb = kc.size(0), hkv = kc.size(1), bs = kc.size(2), n = slots.numel();
  if (kc.size(3) != kRow || !same(vc, kc) || !shaped(k, {n, hkv, 128}) || !same(v, k) ||
      !fits(nb) || !fits(hkv) || !fits(bs) || !fits(n))
    return fail(A.fn, PKV_EINVAL);
  const pkv_stream_t s = A.stream(5);
  const int st = unlocked([&] {
    return lib.kv_append_int4(ptr(k), ptr(v), ptr<int64_t>(slots), n, ptr(kc), ptr(vc), nb, hkv, 128,
                              bs, s);
  });
  return st ? fail(A.fn, st) : none();
}

PyObject* widen_blocks_int4(Args& A) {   // k_cache, v_cache, src, dst, k_out, v_out, stream
  const at::Tensor &kc = A.tensor(0, kU8), &vc = A.tensor(1, kU8), &src = A.tensor(2, kI32),
                   &dst = A.tensor(3, kI32), &ko = A.tensor(4, kF16), &vo = A.tensor(5, kF16);
  if (!A.ok || kc.dim() != 4 || ko.dim() != 4) return fail(A.fn, PKV_EINVAL);
  const int64_t nb = kc.size(0), hkv = kc.size(1), bs = kc.size(2), n = src.numel(),
                nbo = ko.size(0);
  if (kc.size(3) != kRow || !same(vc, kc) || dst.numel() != n || !shaped(ko, {nbo, hkv, bs, 128}) ||
      !same(vo, ko) || !fits(nb) || !fits(nbo) || !fits(hkv) || !fits(bs) || !fits(n))
    return fail(A.fn, PKV_EINVAL);
  const pkv_stream_t s = A.stream(6);
  const int st = unlocked([&] {
    return lib.widen_blocks_int4(ptr(kc), ptr(vc), ptr<int32_t>(src), ptr<int32_t>(dst), n, nb,
                                 ptr(ko), ptr(vo), nbo, hkv, 128, bs, s);
  });
  return st ? fail(A.fn, st) : none();
}

// out, q, [k_new, v_new,] k_cache, v_cache, block_tables, context_lens, scale, workspace, stream
template <bool APPEND>
PyObject* decode(Args& A) {
  constexpr int at0 = APPEND ? 4 : 2;
  const at::Tensor &out = A.tensor(0, kF16), &q = A.tensor(1, kF16), &kc = A.tensor(at0, kU8),
                   &vc = A.tensor(at0 + 1, kU8), &bt = A.tensor(at0 + 2, kI32),
                   &cl = A.tensor(at0 + 3, kI32), &ws = A.any(at0 + 5);
  const at::Tensor &kn = APPEND ? A.tensor(2, kF16) : q, &vn = APPEND ? A.tensor(3, kF16) : q;
  if (!A.ok || !ws.is_cuda() || ws.get_device() != A.dev || !ws.is_contiguous() || q.dim() != 4 ||
      kc.dim() != 4 || bt.dim() != 2)
    return fail(A.fn, PKV_EINVAL);
  const int64_t B = q.size(0), q_len = q.size(1), hq = q.size(2), d = q.size(3);
  const int64_t nb = kc.size(0), hkv = kc.size(1), bs = kc.size(2), width = bt.size(1);
  if (kc.size(3) != kRow || !same(vc, kc) || !same(out, q) || bt.size(0) != B ||
      cl.numel() != B || !fits(B) || !fits(q_len) || !fits(hq) || !fits(d) || !fits(nb) ||
      !fits(hkv) || !fits(bs) || !fits(width))
    return fail(A.fn, PKV_EINVAL);
  if (APPEND && (!shaped(kn, {B * q_len, hkv, 128}) || !same(vn, kn)))
    return fail(A.fn, PKV_EINVAL);
  const float scale = A.number(at0 + 4);
  const pkv_stream_t s = A.stream(at0 + 6);
  const int32_t *btp = ptr<int32_t>(bt), *clp = ptr<int32_t>(cl);
  const int st = unlocked([&] {
    return APPEND ? lib.decode_append_int4(ptr(out), ptr(q), ptr(kn), ptr(vn), ptr(kc), ptr(vc), nb,
                                           btp, width, clp, B, q_len, hq, hkv, d, bs, scale,
                                           ptr(ws), ws.nbytes(), s)
                  : lib.decode_int4(ptr(out), ptr(q), ptr(kc), ptr(vc), nb, btp, width, clp, B,
                                    q_len, hq, hkv, d, bs, scale, ptr(ws), ws.nbytes(), s);
  });
  if (st) return fail(A.fn, st);
  Py_INCREF(A.a[0]);
  return A.a[0];
}

// q, k, q_weight, k_weight, eps, positions, cos_sin, q_out, k_out, stream
PyObject* qk_norm_rope(Args& A) {
  const at::Tensor &q = A.strided(0, kF16), &k = A.strided(1, kF16), &qw = A.tensor(2, kF16),
                   &kw = A.tensor(3, kF16), &pos = A.tensor(5, kI64), &cs = A.tensor(6, kF32);
  if (!A.ok || q.dim() != 3 || k.dim() != 3 || cs.dim() != 3) return fail(A.fn, PKV_EINVAL);
  const int64_t T = q.size(0), hq = q.size(1), hkv = k.size(1), n_index = cs.size(0);
  if (q.size(2) != 128 || !shaped(k, {T, hkv, 128}) || pos.numel() != T || q.stride(2) != 1 ||
      k.stride(2) != 1 || (q.stride(1) != 128 && hq != 1) || (k.stride(1) != 128 && hkv != 1) ||
      qw.numel() != 128 || kw.numel() != 128 || !shaped(cs, {n_index, 64, 2}) || !fits(T) ||
      !fits(hq) || !fits(hkv) || !fits(n_index))
    return fail(A.fn, PKV_EINVAL);
  // the stride of a single token means nothing
  const int64_t qs = T <= 1 ? hq * 128 : q.stride(0), ks = T <= 1 ? hkv * 128 : k.stride(0);
  at::Tensor qo, ko;
  if (A.a[7] != Py_None) {
    qo = A.tensor(7, kF16);
    if (!A.ok || !same(qo, q)) return fail(A.fn, PKV_EINVAL);
  }
  if (A.a[8] != Py_None) {
    ko = A.tensor(8, kF16);
    if (!A.ok || !same(ko, k)) return fail(A.fn, PKV_EINVAL);
  }
  const float eps = A.number(4);
  const pkv_stream_t s = A.stream(9);
  const int st = unlocked([&] {
    const Outputs on(A, 9, s);
    if (!qo.defined()) qo = at::empty({T, hq, 128}, q.options());
    if (!ko.defined()) ko = at::empty({T, hkv, 128}, q.options());
    return lib.qk_norm_rope(ptr(qo), ptr(ko), ptr(q), ptr(k), qs, ks, ptr(qw), ptr(kw), eps,
                            ptr<int64_t>(pos), ptr<float>(cs), n_index, T, hq, hkv, 128, s);
  });
  if (st) return fail(A.fn, st);
  PyObject* r = PyTuple_New(2);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(qo)));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(ko)));
  return r;
}

// block_tables, context_lens, new_lens, block_size, free_blocks, free_count, max_tokens, out, stream
PyObject* extend_tables(Args& A) {
  const at::Tensor &bt = A.tensor(0, kI32), &cl = A.tensor(1, kI32), &nl = A.tensor(2, kI32),
                   &fb = A.tensor(4, kI32), &fc = A.tensor(5, kI32);
  const int64_t bs = A.whole(3), n = A.whole(6);
  if (!A.ok || bt.dim() != 2 || n < 0) return fail(A.fn, PKV_EINVAL);
  const int64_t B = bt.size(0), width = bt.size(1), nb = fb.numel();
  if (cl.numel() != B || nl.numel() != B || fc.numel() != 1 || !fits(B) || !fits(width) ||
      !fits(nb))
    return fail(A.fn, PKV_EINVAL);
  const pkv_stream_t s = A.stream(8);
  at::Tensor slots, seqs, pos, cu;
  const bool given = A.a[7] != Py_None;
  if (given) {
    if (!PyTuple_Check(A.a[7]) || PyTuple_GET_SIZE(A.a[7]) != 4) return fail(A.fn, PKV_EINVAL);
    Args O{A.fn, &PyTuple_GET_ITEM(A.a[7], 0), A.dev};
    slots = O.tensor(0, kI64);
    seqs = O.tensor(1, kI32);
    pos = O.tensor(2, kI64);
    cu = O.tensor(3, kI32);
    if (!O.ok || slots.numel() != n || seqs.numel() != n || pos.numel() != n ||
        cu.numel() != B + 1)
      return fail(A.fn, PKV_EINVAL);
  }
  const int st = unlocked([&] {
    if (!given) {
      const Outputs on(A, 8, s);
      const auto wide = bt.options().dtype(kI64), narrow = bt.options();
      slots = at::empty({n}, wide);
      seqs = at::empty({n}, narrow);
      pos = at::empty({n}, wide);
      cu = at::empty({B + 1}, narrow);
    }
    return lib.extend_tables(ptr<int32_t>(bt), ptr<int32_t>(cl), ptr<int32_t>(nl), B, width, bs,
                             ptr<int32_t>(fb), ptr<int32_t>(fc), nb, ptr<int64_t>(slots),
                             ptr<int32_t>(seqs), ptr<int64_t>(pos), ptr<int32_t>(cu), n, s);
  });
  if (st) return fail(A.fn, st);
  if (given) {
    Py_INCREF(A.a[7]);
    return A.a[7];
  }
  PyObject* r = PyTuple_New(4);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(slots)));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(seqs)));
  PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(std::move(pos)));
  PyTuple_SET_ITEM(r, 3, THPVariable_Wrap(std::move(cu)));
  return r;
}

// block_tables, context_lens, keep_lens, block_size, free_blocks, free_count, stream
PyObject* truncate_tables(Args& A) {
  const at::Tensor &bt = A.tensor(0, kI32), &cl = A.tensor(1, kI32), &kl = A.tensor(2, kI32),
                   &fb = A.tensor(4, kI32), &fc = A.tensor(5, kI32);
  const int64_t bs = A.whole(3);
  if (!A.ok || bt.dim() != 2) return fail(A.fn, PKV_EINVAL);
  const int64_t B = bt.size(0), width = bt.size(1), nb = fb.numel();
  if (cl.numel() != B || kl.numel() != B || fc.numel() != 1 || !fits(B) || !fits(width) ||
      !fits(nb))
    return fail(A.fn, PKV_EINVAL);
  const pkv_stream_t s = A.stream(6);
  const int st = unlocked([&] {
    return lib.truncate_tables(ptr<int32_t>(bt), ptr<int32_t>(cl), ptr<int32_t>(kl), B, width, bs,
                               ptr<int32_t>(fb), ptr<int32_t>(fc), nb, s);
  });
  return st ? fail(A.fn, st) : none();
}

// C++ exceptions (no CUDA device, no memory for an output) become the Python ones torch raises.
template <PyObject* (*F)(Args&), Py_ssize_t N>
PyObject* entry(const char* fn, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!error_class) {
    PyErr_SetString(PyExc_RuntimeError, "the library is not bound");
    return nullptr;
  }
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments", fn, N);
    return nullptr;
  }
  try {
    Args A{fn, args, static_cast<int>(c10::cuda::current_device())};
    return F(A);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

#define PKV_ENTRY(name, function, n)                                               \
  PyObject* py_##name(PyObject*, PyObject* const* args, Py_ssize_t nargs) {        \
    return entry<&function, n>("pkv_" #name, args, nargs);                         \
  }
PKV_ENTRY(kv_append_int4, kv_append_int4, 6)
PKV_ENTRY(widen_blocks_int4, widen_blocks_int4, 7)
PKV_ENTRY(paged_attn_decode_int4, decode<false>, 9)
PKV_ENTRY(paged_attn_decode_append_int4, decode<true>, 11)
PKV_ENTRY(qk_norm_rope, qk_norm_rope, 10)
PKV_ENTRY(extend_tables, extend_tables, 9)
PKV_ENTRY(truncate_tables, truncate_tables, 7)

// bind(error class, addresses of the entry points in the order of `lib`)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 1 + kEntryPoints) {
    PyErr_SetString(PyExc_TypeError, "bind: wrong number of entry points");
    return nullptr;
  }
  void* f[kEntryPoints];
  for (int i = 0; i < kEntryPoints; ++i) {
    f[i] = PyLong_AsVoidPtr(args[1 + i]);
    if (!f[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: no address");
      return nullptr;
    }
  }
  static_assert(sizeof(lib) == sizeof(f), "one address for each");
  memcpy(&lib, f, sizeof(f));
  Py_INCREF(args[0]);
  Py_XSETREF(error_class, args[0]);
  Py_RETURN_NONE;
}

#define PKV_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&py_##name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    PKV_METHOD(kv_append_int4),
    PKV_METHOD(widen_blocks_int4),
    PKV_METHOD(paged_attn_decode_int4),
    PKV_METHOD(paged_attn_decode_append_int4),
    PKV_METHOD(qk_norm_rope),
    PKV_METHOD(extend_tables),
    PKV_METHOD(truncate_tables),
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&bind)), METH_FASTCALL,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pkv_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pkv_torch() { return PyModule_Create(&module); }
