// binding.cpp -- the Python side of the serving step's entry points: checks
// and marshals torch tensors and calls the C ABI (addresses given by bind(),
// so that it uses the library mmq.py loaded).  In C++ because a decode step
// calls these every few microseconds: the same checks in Python took two to
// four times the launch.  Everything of the computation is in libmmq.so.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <optional>

#include "mmq.h"

namespace {

decltype(&mmq_page_tables) g_page_tables;
decltype(&mmq_kv_write) g_kv_write;
decltype(&mmq_paged_attention) g_paged_attention;
decltype(&mmq_verify_draft) g_verify_draft;

struct PyFail {};  // a Python error is set
[[noreturn]] void fail(PyObject *type, const char *form, ...) {
  char text[512];
  va_list va;
  va_start(va, form);
  vsnprintf(text, sizeof(text), form, va);
  va_end(va);
  PyErr_SetString(type, text);
  throw PyFail{};
}

const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a CUDA tensor", name);
  const at::Tensor &t = THPVariable_Unpack(o);
  if (!t.is_cuda()) fail(PyExc_TypeError, "%s must be a CUDA tensor", name);
  return t;
}
// The first tensor gives the call's device, which has to be the current one.
const at::Tensor &first(PyObject *o, const char *name, int &dev) {
  const at::Tensor &t = tensor(o, name);
  dev = static_cast<int>(t.get_device());
  const int now = c10::cuda::current_device();
  if (dev != now) fail(PyExc_ValueError, "%s is on device %d, the current device is %d", name, dev, now);
  return t;
}
const at::Tensor &on(PyObject *o, const char *name, int dev) {
  const at::Tensor &t = tensor(o, name);
  if (t.get_device() != dev) fail(PyExc_TypeError, "%s must be a tensor on CUDA device %d", name, dev);
  return t;
}
// A contiguous tensor of this type and shape.
const at::Tensor &plain(PyObject *o, const char *name, int dev, at::ScalarType type, std::initializer_list<int64_t> shape) {
  const at::Tensor &t = on(o, name, dev);
  if (t.scalar_type() != type || t.sizes() != at::IntArrayRef(shape.begin(), shape.size())) {
    char want[64] = "";
    int at = 0;
    for (int64_t n : shape) at += snprintf(want + at, sizeof(want) - at, "%s%lld", at ? ", " : "", static_cast<long long>(n));
    fail(PyExc_ValueError, "%s must be %s of shape (%s)", name, c10::toString(type), want);
  }
  if (!t.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", name);
  return t;
}
template <class T>
T *ptr(const at::Tensor &t) { return static_cast<T *>(t.data_ptr()); }

int type_of(at::ScalarType t) {
  return t == at::kHalf ? MMQ_DT_F16 : t == at::kFloat ? MMQ_DT_F32 : t == at::kBFloat16 ? MMQ_DT_BF16 : 0;
}

// A 3-D tensor with contiguous rows; its two outer strides (0 for a dimension
// of one element, whose stride says nothing).
struct Rows {
  void *p;
  int64_t s0, s1;
};
Rows rows3(const at::Tensor &t, const char *name) {
  if (t.dim() != 3) fail(PyExc_ValueError, "%s must have 3 dimensions", name);
  if (t.stride(2) != 1 && t.size(2) > 1) fail(PyExc_ValueError, "the last dimension of %s must be contiguous", name);
  return {t.data_ptr(), t.size(0) > 1 ? t.stride(0) : 0, t.size(1) > 1 ? t.stride(1) : 0};
}

struct Table {
  int32_t *p;
  int64_t width, stride;
};
Table page_table(PyObject *o, int64_t nreq, int dev) {
  const at::Tensor &t = on(o, "block_table", dev);
  if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != nreq)
    fail(PyExc_ValueError, "block_table must be int32 of shape (%lld, width)", static_cast<long long>(nreq));
  const int64_t width = t.size(1);
  if (t.stride(1) != 1 && width > 1) fail(PyExc_ValueError, "the rows of block_table must be contiguous");
  return {ptr<int32_t>(t), width, nreq > 1 ? t.stride(0) : std::max(t.stride(0), width)};
}

mmq_paged_cache paged_cache(PyObject *ko, PyObject *vo, int dev) {
  const at::Tensor &k = on(ko, "k_cache", dev), &v = on(vo, "v_cache", dev);
  if (k.dim() != 4 || k.sizes() != v.sizes())
    fail(PyExc_ValueError, "k_cache and v_cache must be (pages, page_size, heads, head_dim), both the same");
  const int type = type_of(k.scalar_type());
  if (k.scalar_type() != v.scalar_type() || (type != MMQ_DT_F16 && type != MMQ_DT_BF16))
    fail(PyExc_ValueError, "k_cache and v_cache must both be float16 or bfloat16");
  if (k.stride(3) != 1 || v.stride(3) != 1) fail(PyExc_ValueError, "the last dimension of the cache must be contiguous");
  if (k.size(1) > INT32_MAX || k.size(2) > INT32_MAX || k.size(3) > INT32_MAX) fail(PyExc_ValueError, "the cache is too large");
  mmq_paged_cache c;
  auto stride = [](const at::Tensor &t, int i) { return t.size(i) > 1 ? t.stride(i) : 0; };
  c.k = k.data_ptr(), c.v = v.data_ptr();
  c.k_page = stride(k, 0), c.k_token = stride(k, 1), c.k_head = stride(k, 2);
  c.v_page = stride(v, 0), c.v_token = stride(v, 1), c.v_head = stride(v, 2);
  c.pages = k.size(0), c.page_size = static_cast<int32_t>(k.size(1)), c.heads = static_cast<int32_t>(k.size(2));
  c.head_dim = static_cast<int32_t>(k.size(3)), c.type = type;
  return c;
}

// The stream of the call (None: torch's current one); tensors allocated while
// it is held belong to it.
struct CallStream {
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  mmq_stream_t handle;
  CallStream(PyObject *o, int dev) {
    if (o == Py_None) {
      handle = reinterpret_cast<mmq_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
      return;
    }
    PyObject *of = PyObject_GetAttrString(o, "cuda_stream"), *n = of;
    if (!n) {
      PyErr_Clear();
      n = o;
    }
    const unsigned long long raw = PyLong_AsUnsignedLongLong(n);
    Py_XDECREF(of);
    if (PyErr_Occurred()) throw PyFail{};
    handle = reinterpret_cast<mmq_stream_t>(raw);
    const auto index = static_cast<c10::DeviceIndex>(dev);
    guard.emplace(raw ? c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(raw), index)
                      : c10::cuda::getDefaultCUDAStream(index));
  }
};

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, int dev) {
  return at::detail::empty_cuda(shape, type, c10::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt);
}

int64_t number(PyObject *o, const char *name) {
  const long long n = PyLong_AsLongLong(o);
  if (n == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    fail(PyExc_TypeError, "%s must be an integer", name);
  }
  return n;
}
int32_t small(PyObject *o, const char *name) {
  const int64_t n = number(o, name);
  if (n < INT32_MIN || n > INT32_MAX) fail(PyExc_ValueError, "%s is out of range", name);
  return static_cast<int32_t>(n);
}

// Runs f with Python's and C++'s errors as Python errors.
template <class F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, F &&f) {
  try {
    if (got != want) fail(PyExc_TypeError, "%zd arguments wanted, %zd given", want, got);
    return f();
  } catch (const PyFail &) {
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject * {
    void *p[4];
    for (int i = 0; i < 4; ++i) {
      p[i] = PyLong_AsVoidPtr(a[i]);
      if (PyErr_Occurred()) throw PyFail{};
    }
    g_page_tables = reinterpret_cast<decltype(g_page_tables)>(p[0]);
    g_kv_write = reinterpret_cast<decltype(g_kv_write)>(p[1]);
    g_paged_attention = reinterpret_cast<decltype(g_paged_attention)>(p[2]);
    g_verify_draft = reinterpret_cast<decltype(g_verify_draft)>(p[3]);
    Py_RETURN_NONE;
  });
}

// (cached, new, n_blocks, table, free, page_size, max_tokens, out or None, stream) -> status, or (status, out)
PyObject *page_tables(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject * {
    int dev;
    const at::Tensor &cached = first(a[0], "cached_lens", dev);
    if (cached.dim() != 1) fail(PyExc_ValueError, "cached_lens must have 1 dimension");
    const int64_t nreq = cached.size(0), room = number(a[6], "max_tokens");
    if (room < 0) fail(PyExc_ValueError, "max_tokens is negative");
    plain(a[0], "cached_lens", dev, at::kInt, {nreq});
    const at::Tensor &fresh = plain(a[1], "new_lens", dev, at::kInt, {nreq}), &held = plain(a[2], "n_blocks", dev, at::kInt, {nreq});
    const Table table = page_table(a[3], nreq, dev);
    const at::Tensor &pages = on(a[4], "free_pages", dev);
    if (pages.dim() != 1) fail(PyExc_ValueError, "free_pages must have 1 dimension");
    plain(a[4], "free_pages", dev, at::kInt, {pages.size(0)});
    const int32_t page = small(a[5], "page_size");
    const CallStream s(a[8], dev);
    at::Tensor out[6];
    if (a[7] == Py_None) {
      out[0] = empty({nreq + 1}, at::kInt, dev), out[1] = empty({nreq}, at::kInt, dev), out[2] = empty({nreq}, at::kInt, dev);
      out[3] = empty({room}, at::kLong, dev), out[4] = empty({room}, at::kInt, dev), out[5] = empty({2}, at::kInt, dev);
    } else {
      if (!PyTuple_Check(a[7]) || PyTuple_GET_SIZE(a[7]) != 6) fail(PyExc_TypeError, "out must be a tuple of six tensors");
      auto item = [&](int i) { return PyTuple_GET_ITEM(a[7], i); };
      out[0] = plain(item(0), "out.q_start", dev, at::kInt, {nreq + 1}), out[1] = plain(item(1), "out.seq_lens", dev, at::kInt, {nreq});
      out[2] = plain(item(2), "out.n_blocks", dev, at::kInt, {nreq}), out[3] = plain(item(3), "out.slots", dev, at::kLong, {room});
      out[4] = plain(item(4), "out.positions", dev, at::kInt, {room}), out[5] = plain(item(5), "out.taken", dev, at::kInt, {2});
    }
    const int rc = g_page_tables(ptr<int32_t>(cached), ptr<int32_t>(fresh), ptr<int32_t>(held), nreq, table.p, table.width, table.stride,
                                 ptr<int32_t>(pages), pages.size(0), page, room, ptr<int32_t>(out[0]), ptr<int32_t>(out[1]),
                                 ptr<int32_t>(out[2]), ptr<int64_t>(out[3]), ptr<int32_t>(out[4]), ptr<int32_t>(out[5]), s.handle);
    if (a[7] != Py_None) return PyLong_FromLong(rc);
    return Py_BuildValue("(i(NNNNNN))", rc, THPVariable_Wrap(out[0]), THPVariable_Wrap(out[1]), THPVariable_Wrap(out[2]),
                         THPVariable_Wrap(out[3]), THPVariable_Wrap(out[4]), THPVariable_Wrap(out[5]));
  });
}

// (k, v, k_cache, v_cache, slots, stream) -> status
PyObject *kv_write(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject * {
    int dev;
    const at::Tensor &k = first(a[0], "k", dev), &v = on(a[1], "v", dev);
    const mmq_paged_cache c = paged_cache(a[2], a[3], dev);
    const Rows kr = rows3(k, "k"), vr = rows3(v, "v");
    const int type = type_of(k.scalar_type());
    if (k.sizes() != v.sizes() || k.scalar_type() != v.scalar_type() || !type || k.size(1) != c.heads || k.size(2) != c.head_dim)
      fail(PyExc_ValueError, "k and v must be (tokens, %d, %d), both float32, float16 or bfloat16", c.heads, c.head_dim);
    const at::Tensor &slots = plain(a[4], "slots", dev, at::kLong, {k.size(0)});
    const CallStream s(a[5], dev);
    return PyLong_FromLong(g_kv_write(&c, kr.p, kr.s0, kr.s1, vr.p, vr.s0, vr.s1, type, ptr<int64_t>(slots), k.size(0), s.handle));
  });
}

// (q, k_cache, v_cache, table, seq_lens, q_start, scale or None, causal, window, out or None, lse: tensor, bool or None,
//  out_dtype or None, stream) -> (status, out, lse or None)
PyObject *paged_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject * {
    int dev;
    const at::Tensor &q = first(a[0], "q", dev);
    const mmq_paged_cache c = paged_cache(a[1], a[2], dev);
    const Rows qr = rows3(q, "q");
    const int64_t ntok = q.size(0), hq = q.size(1);
    // (a cache without heads is the library's to refuse)
    if (type_of(q.scalar_type()) != c.type || q.size(2) != c.head_dim || hq < 1 || hq > INT32_MAX || (c.heads && hq % c.heads))
      fail(PyExc_ValueError, "q must be (tokens, a multiple of %d, %d) of the cache's type", c.heads, c.head_dim);
    mmq_attention t;
    t.scale = a[6] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(c.head_dim)))
                              : static_cast<float>(PyFloat_AsDouble(a[6]));
    if (PyErr_Occurred()) throw PyFail{};
    t.causal = PyObject_IsTrue(a[7]);
    if (t.causal < 0) throw PyFail{};
    t.window = small(a[8], "window");
    const at::Tensor &lens = on(a[4], "seq_lens", dev);
    if (lens.dim() != 1) fail(PyExc_ValueError, "seq_lens must have 1 dimension");
    t.nreq = lens.size(0), t.ntok = ntok, t.q_heads = static_cast<int32_t>(hq);
    t.seq_lens = ptr<int32_t>(plain(a[4], "seq_lens", dev, at::kInt, {t.nreq}));
    t.q_start = ptr<int32_t>(plain(a[5], "q_start", dev, at::kInt, {t.nreq + 1}));
    const Table table = page_table(a[3], t.nreq, dev);
    if (table.width > INT32_MAX) fail(PyExc_ValueError, "block_table is too wide");
    t.table = table.p, t.table_width = static_cast<int32_t>(table.width), t.table_stride = table.stride;
    std::optional<at::ScalarType> want;
    if (a[11] != Py_None) {
      if (!THPDtype_Check(a[11])) fail(PyExc_TypeError, "out_dtype must be a torch.dtype");
      want = reinterpret_cast<THPDtype *>(a[11])->scalar_type;
    }
    const CallStream s(a[12], dev);
    at::Tensor out, lse;
    if (a[9] == Py_None) {
      out = empty({ntok, hq, c.head_dim}, want.value_or(q.scalar_type()), dev);
    } else {
      out = on(a[9], "out", dev);
      if (out.sizes() != q.sizes() || (want && out.scalar_type() != *want)) fail(PyExc_ValueError, "out must have q's shape (and out_dtype)");
    }
    if (a[10] == Py_True) lse = empty({ntok, hq}, at::kFloat, dev);
    else if (a[10] != Py_None && a[10] != Py_False) lse = plain(a[10], "lse", dev, at::kFloat, {ntok, hq});
    const Rows o = rows3(out, "out");
    t.q = qr.p, t.q_token = qr.s0, t.q_head = qr.s1;
    t.out = o.p, t.out_token = o.s0, t.out_head = o.s1, t.out_type = type_of(out.scalar_type());
    t.lse = lse.defined() ? ptr<float>(lse) : nullptr;
    const int rc = g_paged_attention(&c, &t, s.handle);
    PyObject *l = Py_None;
    if (lse.defined()) l = THPVariable_Wrap(lse);
    else Py_INCREF(l);
    return Py_BuildValue("(iNN)", rc, THPVariable_Wrap(out), l);
  });
}

// (target, draft or None, tokens, n_draft or None, u, noise, stream) -> (status, tokens, accepted)
PyObject *verify_draft(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject * {
    int dev;
    const at::Tensor &target = first(a[0], "target_probs", dev);
    const Rows tr = rows3(target, "target_probs");
    mmq_verification t;
    t.nreq = target.size(0), t.vocab = target.size(2);
    const int64_t k = target.size(1) - 1;
    if (k < 0 || k >= INT32_MAX) fail(PyExc_ValueError, "target_probs must have a row for each drafted token and one more");
    t.k = static_cast<int32_t>(k), t.type = type_of(target.scalar_type());
    t.target = tr.p, t.target_req = tr.s0, t.target_row = tr.s1;
    t.draft = nullptr, t.draft_req = t.draft_row = 0;
    if (a[1] != Py_None) {
      const at::Tensor &draft = on(a[1], "draft_probs", dev);
      const Rows dr = rows3(draft, "draft_probs");
      if (draft.scalar_type() != target.scalar_type() || draft.size(0) != t.nreq || draft.size(1) != k || draft.size(2) != t.vocab)
        fail(PyExc_ValueError, "draft_probs must be of target_probs' type and shape (%lld, %lld, %lld)", static_cast<long long>(t.nreq),
             static_cast<long long>(k), static_cast<long long>(t.vocab));
      t.draft = dr.p, t.draft_req = dr.s0, t.draft_row = dr.s1;
    }
    t.tokens = ptr<int32_t>(plain(a[2], "draft_tokens", dev, at::kInt, {t.nreq, k})), t.tokens_stride = k;
    t.n_draft = a[3] == Py_None ? nullptr : ptr<int32_t>(plain(a[3], "n_draft", dev, at::kInt, {t.nreq}));
    t.u = ptr<float>(plain(a[4], "u", dev, at::kFloat, {t.nreq, k})), t.u_stride = k;
    t.noise = ptr<float>(plain(a[5], "noise", dev, at::kFloat, {t.nreq, t.vocab})), t.noise_stride = t.vocab;
    const CallStream s(a[6], dev);
    const at::Tensor out = empty({t.nreq, k + 1}, at::kInt, dev), accepted = empty({t.nreq}, at::kInt, dev);
    t.out = ptr<int32_t>(out), t.accepted = ptr<int32_t>(accepted);
    const int rc = g_verify_draft(&t, s.handle);
    return Py_BuildValue("(iNN)", rc, THPVariable_Wrap(out), THPVariable_Wrap(accepted));
  });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef g_methods[] = {{"bind", FAST(bind), nullptr},
                           {"page_tables", FAST(page_tables), nullptr},
                           {"kv_write", FAST(kv_write), nullptr},
                           {"paged_attention", FAST(paged_attention), nullptr},
                           {"verify_draft", FAST(verify_draft), nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&g_module); }
