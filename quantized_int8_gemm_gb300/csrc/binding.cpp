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
decltype(&mmq_page_fork) g_page_fork;
decltype(&mmq_page_compact) g_page_compact;
decltype(&mmq_page_copy) g_page_copy;
decltype(&mmq_token_probs) g_token_probs;
decltype(&mmq_lora_plan_words) g_lora_plan_words;
decltype(&mmq_lora_plan) g_lora_plan;
decltype(&mmq_lora) g_lora;

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
Table page_table(PyObject *o, int64_t nreq, int dev, const char *name = "block_table") {
  const at::Tensor &t = on(o, name, dev);
  if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != nreq)
    fail(PyExc_ValueError, "%s must be int32 of shape (%lld, width)", name, static_cast<long long>(nreq));
  const int64_t width = t.size(1);
  if (t.stride(1) != 1 && width > 1) fail(PyExc_ValueError, "the rows of %s must be contiguous", name);
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

template <class F>
void take(F &f, PyObject *address) {
  void *p = PyLong_AsVoidPtr(address);
  if (PyErr_Occurred()) throw PyFail{};
  f = reinterpret_cast<F>(p);
}
// The addresses of the C ABI's functions, in the order below.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject * {
    take(g_page_tables, a[0]), take(g_kv_write, a[1]), take(g_paged_attention, a[2]), take(g_verify_draft, a[3]);
    take(g_page_fork, a[4]), take(g_page_compact, a[5]), take(g_page_copy, a[6]), take(g_token_probs, a[7]);
    take(g_lora_plan_words, a[8]), take(g_lora_plan, a[9]), take(g_lora, a[10]);
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

// The members of out, a tuple of n tensors.
PyObject *item(PyObject *out, int n, int i) {
  if (!PyTuple_Check(out) || PyTuple_GET_SIZE(out) != n) fail(PyExc_TypeError, "out must be a tuple of %d tensors", n);
  return PyTuple_GET_ITEM(out, i);
}
// A vector of the call, or NULL for None.
template <class T>
const T *maybe(PyObject *o, const char *name, int dev, at::ScalarType type, std::initializer_list<int64_t> shape) {
  return o == Py_None ? nullptr : ptr<T>(plain(o, name, dev, type, shape));
}
int64_t length_of(PyObject *o, const char *name, int dev) {
  const at::Tensor &t = on(o, name, dev);
  if (t.dim() != 1) fail(PyExc_ValueError, "%s must have 1 dimension", name);
  return t.size(0);
}

// (table, n_blocks, parents, lens, page_size, n_pages, out or None, stream) -> status, or (status, out)
PyObject *page_fork(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject * {
    int dev;
    first(a[0], "block_table", dev);
    const int64_t nold = length_of(a[1], "n_blocks", dev), nnew = length_of(a[2], "parents", dev);
    const Table table = page_table(a[0], nold, dev);
    mmq_fork t;
    t.held = ptr<int32_t>(plain(a[1], "n_blocks", dev, at::kInt, {nold})), t.parents = ptr<int32_t>(plain(a[2], "parents", dev, at::kInt, {nnew}));
    t.lens = ptr<int32_t>(plain(a[3], "lens", dev, at::kInt, {nnew}));
    t.page_size = small(a[4], "page_size"), t.npages = number(a[5], "n_pages");
    if (t.npages < 0) fail(PyExc_ValueError, "n_pages is negative");
    const CallStream s(a[7], dev);
    at::Tensor out[6];
    if (a[6] == Py_None) {
      if (t.npages > INT32_MAX) fail(PyExc_ValueError, "n_pages is out of range");
      out[0] = empty({nnew, table.width}, at::kInt, dev), out[1] = empty({nnew}, at::kInt, dev), out[2] = empty({nnew, 2}, at::kInt, dev);
      out[3] = empty({nnew}, at::kInt, dev), out[4] = empty({t.npages}, at::kInt, dev), out[5] = empty({2}, at::kInt, dev);
    } else {
      out[0] = on(item(a[6], 6, 0), "out.block_table", dev), out[1] = plain(item(a[6], 6, 1), "out.n_blocks", dev, at::kInt, {nnew});
      out[2] = plain(item(a[6], 6, 2), "out.pairs", dev, at::kInt, {nnew, 2}), out[3] = plain(item(a[6], 6, 3), "out.tokens", dev, at::kInt, {nnew});
      out[4] = plain(item(a[6], 6, 4), "out.free_pages", dev, at::kInt, {t.npages}), out[5] = plain(item(a[6], 6, 5), "out.counts", dev, at::kInt, {2});
    }
    const Table fresh = a[6] == Py_None ? Table{ptr<int32_t>(out[0]), table.width, table.width} : page_table(item(a[6], 6, 0), nnew, dev, "out.block_table");
    if (fresh.width != table.width) fail(PyExc_ValueError, "out.block_table must be as wide as block_table");
    t.table = table.p, t.table_width = table.width, t.table_stride = table.stride, t.nold = nold, t.nnew = nnew;
    t.new_table = fresh.p, t.new_stride = fresh.stride, t.held_out = ptr<int32_t>(out[1]), t.pairs = ptr<int32_t>(out[2]);
    t.tokens = ptr<int32_t>(out[3]), t.free_pages = ptr<int32_t>(out[4]), t.counts = ptr<int32_t>(out[5]);
    const int rc = g_page_fork(&t, s.handle);
    if (a[6] != Py_None) return PyLong_FromLong(rc);
    return Py_BuildValue("(i(NNNNNN))", rc, THPVariable_Wrap(out[0]), THPVariable_Wrap(out[1]), THPVariable_Wrap(out[2]),
                         THPVariable_Wrap(out[3]), THPVariable_Wrap(out[4]), THPVariable_Wrap(out[5]));
  });
}

// (table, n_blocks, n_pages, out or None, stream) -> status, or (status, out)
PyObject *page_compact(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject * {
    int dev;
    first(a[0], "block_table", dev);
    const int64_t nreq = length_of(a[1], "n_blocks", dev), npages = number(a[2], "n_pages");
    const Table table = page_table(a[0], nreq, dev);
    const at::Tensor &held = plain(a[1], "n_blocks", dev, at::kInt, {nreq});
    if (npages < 0 || npages > INT32_MAX) fail(PyExc_ValueError, "n_pages is out of range");
    const CallStream s(a[4], dev);
    at::Tensor out[3];
    if (a[3] == Py_None) {
      out[0] = empty({nreq, table.width}, at::kInt, dev), out[1] = empty({npages / 2, 2}, at::kInt, dev), out[2] = empty({2}, at::kInt, dev);
    } else {
      out[0] = on(item(a[3], 3, 0), "out.block_table", dev), out[1] = plain(item(a[3], 3, 1), "out.pairs", dev, at::kInt, {npages / 2, 2});
      out[2] = plain(item(a[3], 3, 2), "out.counts", dev, at::kInt, {2});
    }
    const Table fresh = a[3] == Py_None ? Table{ptr<int32_t>(out[0]), table.width, table.width} : page_table(item(a[3], 3, 0), nreq, dev, "out.block_table");
    if (fresh.width != table.width) fail(PyExc_ValueError, "out.block_table must be as wide as block_table");
    const int rc = g_page_compact(table.p, ptr<int32_t>(held), nreq, table.width, table.stride, npages, fresh.p, fresh.stride,
                                  ptr<int32_t>(out[1]), ptr<int32_t>(out[2]), s.handle);
    if (a[3] != Py_None) return PyLong_FromLong(rc);
    return Py_BuildValue("(i(NNN))", rc, THPVariable_Wrap(out[0]), THPVariable_Wrap(out[1]), THPVariable_Wrap(out[2]));
  });
}

// (k_cache, v_cache, pairs, tokens or None, stream) -> status
PyObject *page_copy(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject * {
    int dev;
    first(a[0], "k_cache", dev);
    const mmq_paged_cache c = paged_cache(a[0], a[1], dev);
    const at::Tensor &pairs = on(a[2], "pairs", dev);
    const int64_t npairs = pairs.dim() ? pairs.size(0) : 0;
    plain(a[2], "pairs", dev, at::kInt, {npairs, 2});
    const int32_t *tokens = maybe<int32_t>(a[3], "tokens", dev, at::kInt, {npairs});
    const CallStream s(a[4], dev);
    return PyLong_FromLong(g_page_copy(&c, ptr<int32_t>(pairs), tokens, npairs, s.handle));
  });
}

// (logits, temperature, tokens, token_lens, prompt_lens, draft_tokens, n_draft, repetition, frequency, presence,
//  bias: (start, ids, values), mask, mask_rows, probs: tensor or bool, adjusted: tensor or bool, stream; None where there is none)
//  -> (status, probs or None, adjusted or None)
PyObject *token_probs(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> PyObject * {
    int dev;
    const at::Tensor &logits = first(a[0], "logits", dev);
    const Rows lr = rows3(logits, "logits");
    mmq_token_rules t = {};
    t.nreq = logits.size(0), t.vocab = logits.size(2), t.type = type_of(logits.scalar_type());
    const int64_t rows = logits.size(1);
    if (rows < 1 || rows > INT32_MAX) fail(PyExc_ValueError, "logits must have a row for each drafted token and one more");
    if (!t.type) fail(PyExc_ValueError, "logits must be float32, float16 or bfloat16");
    t.rows = static_cast<int32_t>(rows), t.logits = lr.p, t.logits_req = lr.s0, t.logits_row = lr.s1;
    t.temperature = maybe<float>(a[1], "temperature", dev, at::kFloat, {t.nreq});
    if (a[2] != Py_None) {
      const at::Tensor &tokens = on(a[2], "tokens", dev);
      if (tokens.scalar_type() != at::kInt || tokens.dim() != 2 || tokens.size(0) != t.nreq || (tokens.size(1) > 1 && tokens.stride(1) != 1))
        fail(PyExc_ValueError, "tokens must be int32 of shape (%lld, width), its rows contiguous", static_cast<long long>(t.nreq));
      t.tokens = ptr<int32_t>(tokens), t.tokens_width = tokens.size(1), t.tokens_stride = t.nreq > 1 ? tokens.stride(0) : 0;
    } else if (a[3] != Py_None || a[4] != Py_None) {
      fail(PyExc_ValueError, "token_lens and prompt_lens belong to tokens");
    }
    t.token_lens = maybe<int32_t>(a[3], "token_lens", dev, at::kInt, {t.nreq});
    t.prompt_lens = maybe<int32_t>(a[4], "prompt_lens", dev, at::kInt, {t.nreq});
    if (a[5] != Py_None) t.draft = ptr<int32_t>(plain(a[5], "draft_tokens", dev, at::kInt, {t.nreq, rows - 1})), t.draft_stride = rows - 1;
    t.n_draft = maybe<int32_t>(a[6], "n_draft", dev, at::kInt, {t.nreq});
    t.repetition = maybe<float>(a[7], "repetition", dev, at::kFloat, {t.nreq});
    t.frequency = maybe<float>(a[8], "frequency", dev, at::kFloat, {t.nreq});
    t.presence = maybe<float>(a[9], "presence", dev, at::kFloat, {t.nreq});
    if (a[10] != Py_None) {
      if (!PyTuple_Check(a[10]) || PyTuple_GET_SIZE(a[10]) != 3) fail(PyExc_TypeError, "bias must be a tuple (start, ids, values)");
      t.nbias = length_of(PyTuple_GET_ITEM(a[10], 1), "bias ids", dev);
      t.bias_start = ptr<int32_t>(plain(PyTuple_GET_ITEM(a[10], 0), "bias start", dev, at::kInt, {t.nreq + 1}));
      t.bias_ids = ptr<int32_t>(plain(PyTuple_GET_ITEM(a[10], 1), "bias ids", dev, at::kInt, {t.nbias}));
      t.bias_values = ptr<float>(plain(PyTuple_GET_ITEM(a[10], 2), "bias values", dev, at::kFloat, {t.nbias}));
    }
    if (a[11] != Py_None) {
      const at::Tensor &mask = on(a[11], "mask", dev);
      const int64_t words = (t.vocab + 31) / 32;
      if (mask.scalar_type() != at::kInt || mask.dim() != 2 || mask.size(1) != words || (words > 1 && mask.stride(1) != 1))
        fail(PyExc_ValueError, "mask must be int32 of shape (masks, %lld), its rows contiguous", static_cast<long long>(words));
      t.mask = ptr<int32_t>(mask), t.nmasks = mask.size(0), t.mask_stride = t.nmasks > 1 ? mask.stride(0) : words;
      if (t.nmasks == 0) t.mask = nullptr;
      t.mask_rows = maybe<int32_t>(a[12], "mask_rows", dev, at::kInt, {t.nreq, rows});
      if (!t.mask_rows && t.nmasks != t.nreq * rows) fail(PyExc_ValueError, "without mask_rows mask must have a row for each of logits'");
    } else if (a[12] != Py_None) {
      fail(PyExc_ValueError, "mask_rows belongs to mask");
    }
    const CallStream s(a[15], dev);
    at::Tensor out[2];
    void **p[2] = {&t.probs, &t.adjusted};
    int64_t *req[2] = {&t.probs_req, &t.adjusted_req}, *row[2] = {&t.probs_row, &t.adjusted_row};
    int32_t *type[2] = {&t.probs_type, &t.adjusted_type};
    const char *name[2] = {"probs", "adjusted"};
    for (int i = 0; i < 2; ++i) {
      PyObject *o = a[13 + i];
      if (o == Py_None || o == Py_False) continue;
      out[i] = o == Py_True ? empty({t.nreq, rows, t.vocab}, at::kFloat, dev) : on(o, name[i], dev);
      if (out[i].sizes() != logits.sizes() || !type_of(out[i].scalar_type())) fail(PyExc_ValueError, "%s must be float32, float16 or bfloat16 of logits' shape", name[i]);
      const Rows r = rows3(out[i], name[i]);
      *p[i] = r.p, *req[i] = r.s0, *row[i] = r.s1, *type[i] = type_of(out[i].scalar_type());
    }
    if (!out[0].defined() && !out[1].defined()) fail(PyExc_ValueError, "neither probs nor adjusted is wanted");
    const int rc = g_token_probs(&t, s.handle);
    auto wrap = [](const at::Tensor &o) {
      if (o.defined()) return THPVariable_Wrap(o);
      Py_INCREF(Py_None);
      return Py_None;
    };
    return Py_BuildValue("(iNN)", rc, wrap(out[0]), wrap(out[1]));
  });
}

// (adapters, q_start, max_tokens, n_adapters, out or None, stream) -> (status, words)
PyObject *lora_plan(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject * {
    int dev;
    const at::Tensor &adapters = first(a[0], "adapters", dev);
    const int64_t nreq = length_of(a[0], "adapters", dev), ntok = number(a[2], "max_tokens"), many = number(a[3], "n_adapters");
    plain(a[0], "adapters", dev, at::kInt, {nreq});
    const at::Tensor &start = plain(a[1], "q_start", dev, at::kInt, {nreq + 1});
    const int64_t words = g_lora_plan_words(ntok, nreq, many);
    const CallStream s(a[5], dev);
    const at::Tensor out = a[4] == Py_None ? empty({std::max<int64_t>(words, 0)}, at::kInt, dev) : plain(a[4], "out", dev, at::kInt, {words});
    const int rc = g_lora_plan(ptr<int32_t>(adapters), ptr<int32_t>(start), nreq, ntok, many, ptr<int32_t>(out), s.handle);
    return Py_BuildValue("(iN)", rc, THPVariable_Wrap(out));
  });
}

struct Matrix {
  void *p;
  int64_t row;
};
Matrix rows2(const at::Tensor &t, const char *name, int64_t rows) {
  if (t.dim() != 2 || t.size(0) != rows) fail(PyExc_ValueError, "%s must have 2 dimensions, the first the plan's %lld tokens", name, static_cast<long long>(rows));
  if (t.size(1) > 1 && t.stride(1) != 1) fail(PyExc_ValueError, "the rows of %s must be contiguous", name);
  return {t.data_ptr(), t.size(0) > 1 ? t.stride(0) : 0};
}

// (x, y, a, b, plan words, tokens, requests, adapters, scales or None, ranks or None, out or None, stream) -> (status, out)
PyObject *lora(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject * {
    int dev;
    const at::Tensor &x = first(a[0], "x", dev), &y = on(a[1], "y", dev), &down = on(a[2], "a", dev), &up = on(a[3], "b", dev);
    mmq_lora_args t = {};
    t.ntok = number(a[5], "plan.tokens"), t.nreq = number(a[6], "plan.requests"), t.nadapters = number(a[7], "plan.adapters");
    const int64_t words = g_lora_plan_words(t.ntok, t.nreq, t.nadapters);
    t.plan = ptr<int32_t>(plain(a[4], "plan.words", dev, at::kInt, {words}));
    const Matrix xr = rows2(x, "x", t.ntok), yr = rows2(y, "y", t.ntok);
    t.id = x.size(1), t.od = y.size(1), t.x_type = type_of(x.scalar_type()), t.type = type_of(down.scalar_type());
    if (!t.x_type) fail(PyExc_ValueError, "x must be float32, float16 or bfloat16");
    if (y.scalar_type() != at::kFloat) fail(PyExc_ValueError, "y must be float32");
    if (down.scalar_type() != up.scalar_type() || (t.type != MMQ_DT_F16 && t.type != MMQ_DT_BF16)) fail(PyExc_ValueError, "a and b must both be float16 or bfloat16");
    if (down.dim() != 3) fail(PyExc_ValueError, "a must have 3 dimensions");
    const int64_t rank = down.size(1);
    if (rank > INT32_MAX) fail(PyExc_ValueError, "the rank is out of range");
    t.a = ptr<void>(plain(a[2], "a", dev, down.scalar_type(), {t.nadapters, rank, t.id}));
    t.b = ptr<void>(plain(a[3], "b", dev, down.scalar_type(), {t.nadapters, t.od, rank}));
    t.rank = static_cast<int32_t>(rank);
    t.scales = maybe<float>(a[8], "scales", dev, at::kFloat, {t.nadapters});
    t.ranks = maybe<int32_t>(a[9], "ranks", dev, at::kInt, {t.nadapters});
    const CallStream s(a[11], dev);
    const at::Tensor out = a[10] == Py_None ? empty({t.ntok, t.od}, at::kFloat, dev) : on(a[10], "out", dev);
    if (out.scalar_type() != at::kFloat || out.sizes() != y.sizes()) fail(PyExc_ValueError, "out must be float32 of y's shape");
    const Matrix to = rows2(out, "out", t.ntok);
    t.x = xr.p, t.x_row = xr.row, t.y = static_cast<const float *>(yr.p), t.y_row = yr.row, t.out = static_cast<float *>(to.p), t.out_row = to.row;
    const int rc = g_lora(&t, s.handle);
    return Py_BuildValue("(iN)", rc, THPVariable_Wrap(out));
  });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef g_methods[] = {{"bind", FAST(bind), nullptr},
                           {"page_tables", FAST(page_tables), nullptr},
                           {"kv_write", FAST(kv_write), nullptr},
                           {"paged_attention", FAST(paged_attention), nullptr},
                           {"verify_draft", FAST(verify_draft), nullptr},
                           {"page_fork", FAST(page_fork), nullptr},
                           {"page_compact", FAST(page_compact), nullptr},
                           {"page_copy", FAST(page_copy), nullptr},
                           {"token_probs", FAST(token_probs), nullptr},
                           {"lora_plan", FAST(lora_plan), nullptr},
                           {"lora", FAST(lora), nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&g_module); }
