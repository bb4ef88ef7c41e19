// binding.cpp -- the quick way from Python to the C entry points of the operators between
// a QKV projection and its attention output.
//
// A call of those runs for a few microseconds, and the checks and conversions of their
// twenty-odd arguments took four to five times that in the interpreter.  Each function here
// makes the same checks as its wrapper in __init__.py for the usual call (plain CUDA
// tensors on the current device and stream), allocates what was not given, and calls the C
// ABI.  It returns the wrapper's result, an int for a status other than ATTN_OK, or None
// for everything it does not know, which the wrapper then handles, errors included.
#include <Python.h>

#include <ATen/EmptyTensor.h>
#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <c10/core/Allocator.h>
#include <c10/core/TensorImpl.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <exception>
#include <initializer_list>
#include <optional>

#include "gbattn.h"

namespace {

// Entry points by address (this module is not linked against the library), and torch's
// functions for the current device and a device's current stream.
struct Entry {
  decltype(&::qkv_norm_rope) rope;
  decltype(&::qkv_norm_rope_bwd) rope_bwd;
  decltype(&::qkv_norm_rope_bwd_workspace_size) rope_bwd_ws;
  decltype(&::paged_qkv_append) append;
  decltype(&::paged_kv4_append) append4;
  decltype(&::paged_kv4_gather) gather;
  decltype(&::paged_kv4_attn_decode) decode;
  decltype(&::paged_kv4_attn_decode_workspace_size) decode_ws;
  decltype(&::paged_kv4_attn_prefill) prefill;
  decltype(&::paged_kv4_attn_prefill_workspace_size) prefill_ws;
} g_entry;
// Those of the operators for trees of drafted tokens.
struct TreeEntry {
  decltype(&::paged_attn_tree) attend;
  decltype(&::paged_attn_tree_workspace_size) attend_ws;
  decltype(&::draft_verify) verify;
  decltype(&::paged_kv_keep) keep;
} g_tree;
PyObject *g_get_device = nullptr, *g_get_stream = nullptr;

constexpr int64_t kMaxSize = 0x7fffffff;  // the C ABI's sizes are ints

// What a plain CUDA tensor is made of.  Others (those that a function transform wraps or
// batches, zeros without memory, values kept negated) have no memory, or hold something
// else in it.
const c10::DispatchKeySet kPlain({c10::DispatchKey::CUDA, c10::DispatchKey::AutogradCUDA,
                                  c10::DispatchKey::ADInplaceOrView, c10::DispatchKey::AutocastCUDA});

// The arguments of one call; `ok` falls when something is not the usual.
struct Call {
  PyObject* const* args;
  bool differentiable = false;  // whether a gradient might be expected of the call
  bool ok = true;
  int dev = -1;
  void* stream = nullptr;

  // Argument i as a tensor, nullptr for None.
  const at::Tensor* tensor(int i) {
    PyObject* o = args[i];
    if (o == Py_None) return nullptr;
    if (!THPVariable_CheckExact(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || t.layout() != at::kStrided || !t.is_cuda() || !t.has_storage() ||
        !kPlain.has_all(t.key_set())) {
      ok = false;
      return nullptr;
    }
    // (the wrapper refuses what the outputs would silently be cut off from)
    if (differentiable && ((t.requires_grad() && at::GradMode::is_enabled()) || t._fw_grad(0).defined())) {
      ok = false;
      return nullptr;
    }
    return &t;
  }
  // The same, of a type, contiguous, on the call's device, with the given sizes (-1: any).
  const at::Tensor* dense(int i, at::ScalarType type, std::initializer_list<int64_t> sizes) {
    const at::Tensor* t = tensor(i);
    if (!t) return nullptr;
    if (t->scalar_type() != type || !t->is_contiguous() || t->get_device() != dev ||
        t->dim() != static_cast<int64_t>(sizes.size())) {
      ok = false;
      return nullptr;
    }
    int d = 0;
    for (int64_t n : sizes) {
      if (n >= 0 && t->size(d) != n) ok = false;
      if (t->size(d) > kMaxSize && t->dim() > 1) ok = false;
      ++d;
    }
    return t;
  }
  // A [B, T, H, D] bf16 operand: any strides but contiguous channels.
  const at::Tensor* rows(int i) {
    const at::Tensor* t = tensor(i);
    if (!t) return nullptr;
    if (t->scalar_type() != at::kBFloat16 || t->dim() != 4 ||
        (t->stride(3) != 1 && t->size(3) != 1) || (dev >= 0 && t->get_device() != dev)) {
      ok = false;
      return nullptr;
    }
    for (int d = 0; d < 4; ++d)
      if (t->size(d) > kMaxSize) ok = false;
    return t;
  }
  // An argument that has to be there.
  const at::Tensor* need(const at::Tensor* t) {
    if (!t) ok = false;
    return t;
  }
  // Takes the device of t, which has to be the current one, and its current stream.
  bool on(const at::Tensor& t) {
    dev = t.get_device();
    PyObject* d = PyObject_CallNoArgs(g_get_device);
    if (!d) return fail();
    const long now = PyLong_AsLong(d);
    if (now != dev) {
      Py_DECREF(d);
      return fail();
    }
    PyObject* s = PyObject_CallOneArg(g_get_stream, d);
    Py_DECREF(d);
    if (!s) return fail();
    stream = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    return !PyErr_Occurred() || fail();
  }
  bool fail() {
    PyErr_Clear();
    ok = false;
    return false;
  }
  // Plain numbers.
  double real(int i) {
    if (!PyFloat_CheckExact(args[i])) ok = false;
    return ok ? PyFloat_AS_DOUBLE(args[i]) : 0.0;
  }
  int integer(int i) {
    int overflow = 0;
    const long v = PyLong_CheckExact(args[i]) ? PyLong_AsLongAndOverflow(args[i], &overflow) : -1;
    if (overflow || v < 0 || v > 0x7fffffffl) ok = false;
    return static_cast<int>(v);
  }
  int truth(int i) {
    if (!PyBool_Check(args[i])) ok = false;
    return args[i] == Py_True;
  }
};

void* ptr(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

struct Strides {
  int64_t s[3] = {0, 0, 0};
  explicit Strides(const at::Tensor* t) {
    for (int i = 0; t && i < 3; ++i) s[i] = t->size(i) > 1 ? t->stride(i) : 0;
  }
};

bool same_sizes(const at::Tensor& t, int64_t a, int64_t b, int64_t c, int64_t d) {
  return t.size(0) == a && t.size(1) == b && t.size(2) == c && t.size(3) == d;
}

// What is returned for a tensor argument that was given (the object itself), or that this
// call made.
PyObject* result(PyObject* given, const at::Tensor& made) {
  if (given != Py_None) {
    Py_INCREF(given);
    return given;
  }
  if (!made.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(made);
}

// A tuple of new references; a null one is an error that is set.
PyObject* pack(std::initializer_list<PyObject*> items) {
  PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
  bool whole = t != nullptr;
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    whole = whole && o;
    if (t)
      PyTuple_SET_ITEM(t, i++, o);
    else
      Py_XDECREF(o);
  }
  if (whole) return t;
  Py_XDECREF(t);
  return nullptr;
}

// Calls an entry point without the interpreter's lock: a launch waits when the GPU's queue
// is full, and what it waits for may need another thread.  The arguments, which may throw,
// are made before the lock is given up, and it is taken back however the call ends.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(state); }
};

template <typename... P, typename... A>
int released(int (*entry)(P...), A... args) {
  const Unlocked unlocked;
  return entry(static_cast<P>(args)...);
}

// Device memory comes from torch's allocator for the current device, without the
// dispatcher's way there.
c10::Allocator* allocator() { return c10::GetAllocator(at::kCUDA); }

at::Tensor make(at::IntArrayRef sizes, at::ScalarType type) {
  return at::detail::empty_generic(sizes, allocator(), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                   type, std::nullopt);
}

// Heads h0 .. h0 + n - 1 of a fused [B, T, H, D] buffer.
at::Tensor heads_of(const at::Tensor& fused, int64_t h0, int64_t n) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      c10::TensorImpl::VIEW, c10::Storage(fused.storage()), fused.key_set(), fused.dtype());
  const int64_t sizes[4] = {fused.size(0), fused.size(1), n, fused.size(3)};
  t.unsafeGetTensorImpl()->set_storage_offset(h0 * fused.size(3));
  t.unsafeGetTensorImpl()->set_sizes_and_strides(sizes, fused.strides());
  return t;
}

// Memory of a call's own, given back to the allocator (which reuses it in stream order) when
// the call returns.
c10::DataPtr scratch(size_t bytes) { return allocator()->allocate(bytes); }

// The norm and rotation operands from argument i on: cos_sin, q_weight, k_weight, eps,
// interleaved, positions.
struct Rope {
  const at::Tensor *cs, *qw, *kw, *pos;
  float eps;
  int interleaved, rot = 0, max_pos = 0;
  Rope(Call& c, int i, int64_t B, int64_t T, int64_t D) {
    cs = c.dense(i, at::kFloat, {-1, -1});
    qw = c.dense(i + 1, at::kBFloat16, {D});
    kw = c.dense(i + 2, at::kBFloat16, {D});
    eps = static_cast<float>(c.real(i + 3));
    interleaved = c.truth(i + 4);
    pos = c.dense(i + 5, at::kInt, {B, T});
    if (cs) {
      if (cs->size(0) == 0 || cs->size(0) > 0x7fffffff || cs->size(1) == 0 || cs->size(1) > D) {
        c.ok = false;
        return;
      }
      max_pos = static_cast<int>(cs->size(0));
      rot = static_cast<int>(cs->size(1));
    }
  }
};

// Every entry: arguments in, result out.  A body returns nullptr for a call that it leaves
// to the wrapper, or with a Python error after the call was made; what C++ throws before
// (an allocation that fails) is left to the wrapper, which meets it again.
template <typename F>
PyObject* guarded(PyObject* const* args, Py_ssize_t n, Py_ssize_t expected, F body) {
  if (n != expected) Py_RETURN_NONE;
  try {
    Call c{args};
    PyObject* r = body(c);
    if (r || PyErr_Occurred()) return r;
  } catch (const std::exception&) {
    PyErr_Clear();
  }
  Py_RETURN_NONE;
}

// q, k, v, cos_sin, q_weight, k_weight, eps, interleaved, positions, q_out, k_out, v_out
PyObject* rope(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 12, [&](Call& c) -> PyObject* {
    c.differentiable = true;
    const at::Tensor *q = c.rows(0), *k = c.rows(1), *v = c.rows(2);
    const at::Tensor* some = q ? q : (k ? k : v);
    if (!c.ok || !some || !c.on(*some)) return nullptr;
    const int64_t B = some->size(0), T = some->size(1), D = some->size(3);
    const at::Tensor* kv = k ? k : v;
    const int64_t Hq = q ? q->size(2) : 0, Hkv = kv ? kv->size(2) : 0;
    for (const at::Tensor* t : {q, k, v})
      if (t && (!same_sizes(*t, B, T, t == q ? Hq : Hkv, D) || t->get_device() != c.dev))
        return nullptr;
    const Rope r(c, 3, B, T, D);
    const at::Tensor* out[3] = {c.dense(9, at::kBFloat16, {B, Hq, T, D}),
                                c.dense(10, at::kBFloat16, {B, Hkv, T, D}),
                                c.dense(11, at::kBFloat16, {B, Hkv, T, D})};
    const at::Tensor* in[3] = {q, k, v};
    if (!c.ok) return nullptr;
    at::Tensor made[3];
    for (int i = 0; i < 3; ++i) {
      if (!in[i] && out[i]) return nullptr;
      if (in[i] && !out[i]) {
        made[i] = make({B, i == 0 ? Hq : Hkv, T, D}, at::kBFloat16);
        out[i] = &made[i];
      }
    }
    const Strides sq(q), sk(k), sv(v);
    const int st = released(g_entry.rope, ptr(q), ptr(k), ptr(v), sq.s, sk.s, sv.s, ptr(r.qw),
                            ptr(r.kw), ptr(r.cs), ptr(r.pos), B, T, Hq, Hkv, D, r.rot, r.max_pos,
                            r.interleaved, r.eps, ptr(out[0]), ptr(out[1]), ptr(out[2]), c.stream);
    if (st != ATTN_OK) return PyLong_FromLong(st);
    return pack({result(args[9], made[0]), result(args[10], made[1]), result(args[11], made[2])});
  });
}

// dq_out, dk_out, dv_out, q, k, cos_sin, q_weight, k_weight, eps, interleaved, positions
// (gradient buffers and workspace made here)
PyObject* rope_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 11, [&](Call& c) -> PyObject* {
    c.differentiable = true;
    const at::Tensor* g[3] = {c.tensor(0), c.tensor(1), c.tensor(2)};
    const at::Tensor* some = g[0] ? g[0] : (g[1] ? g[1] : g[2]);
    if (!c.ok || !some || some->dim() != 4 || !c.on(*some)) return nullptr;
    const int64_t B = some->size(0), T = some->size(2), D = some->size(3);
    const at::Tensor* kv = g[1] ? g[1] : g[2];
    if (kv && kv->dim() != 4) return nullptr;
    const int64_t Hq = g[0] ? g[0]->size(1) : 0, Hkv = kv ? kv->size(1) : 0;
    c.dense(0, at::kBFloat16, {B, Hq, T, D});
    c.dense(1, at::kBFloat16, {B, Hkv, T, D});
    c.dense(2, at::kBFloat16, {B, Hkv, T, D});
    const Rope r(c, 5, B, T, D);
    const at::Tensor *q = r.qw ? c.need(c.rows(3)) : nullptr, *k = r.kw ? c.need(c.rows(4)) : nullptr;
    if (!c.ok || (q && !same_sizes(*q, B, T, Hq, D)) || (k && !same_sizes(*k, B, T, Hkv, D)))
      return nullptr;
    const int64_t nq = g[0] ? Hq : 0, nk = g[1] ? Hkv : 0, nv = g[2] ? Hkv : 0;
    if (B == 0 || T == 0 || nq + nk + nv == 0) return nullptr;
    const at::Tensor fused = make({B, T, nq + nk + nv, D}, at::kBFloat16);
    at::Tensor d[3], dw[2];
    if (nq) d[0] = heads_of(fused, 0, nq);
    if (nk) d[1] = heads_of(fused, nq, nk);
    if (nv) d[2] = heads_of(fused, nq + nk, nv);
    if (r.qw) dw[0] = make({D}, at::kFloat);
    if (r.kw) dw[1] = make({D}, at::kFloat);
    size_t bytes = 0;
    c10::DataPtr ws;
    if (r.qw || r.kw) {
      bytes = g_entry.rope_bwd_ws(B, T, D);
      ws = scratch(bytes);
    }
    const at::Tensor* dp[3];
    for (int i = 0; i < 3; ++i) dp[i] = d[i].defined() ? &d[i] : nullptr;
    const Strides sq(q), sk(k), s0(dp[0]), s1(dp[1]), s2(dp[2]);
    const int st = released(
        g_entry.rope_bwd, ptr(g[0]), ptr(g[1]), ptr(g[2]), ptr(q), ptr(k), sq.s, sk.s, ptr(r.qw),
        ptr(r.kw), ptr(r.cs), ptr(r.pos), B, T, Hq, Hkv, D, r.rot, r.max_pos, r.interleaved, r.eps,
        ptr(dp[0]), ptr(dp[1]), ptr(dp[2]), s0.s, s1.s, s2.s, ptr(r.qw ? &dw[0] : nullptr),
        ptr(r.kw ? &dw[1] : nullptr), ws.get(), bytes, c.stream);
    if (st != ATTN_OK) return PyLong_FromLong(st);
    return pack({result(Py_None, d[0]), result(Py_None, d[1]), result(Py_None, d[2]),
                 result(Py_None, dw[0]), result(Py_None, dw[1])});
  });
}

// q, k, v, k_pool, v_pool (four: the 4-bit pool and None), block_table, seq_lens, cos_sin,
// q_weight, k_weight, eps, interleaved, positions, q_out, new_seq_lens
PyObject* append_to(PyObject* const* args, Py_ssize_t n, bool four) {
  return guarded(args, n, 15, [&](Call& c) -> PyObject* {
    const at::Tensor *q = c.rows(0), *k = c.need(c.rows(1)), *v = c.need(c.rows(2));
    if (!c.ok || !c.on(*k)) return nullptr;
    const int64_t S = k->size(0), Tn = k->size(1), Hkv = k->size(2), D = k->size(3);
    if (!same_sizes(*v, S, Tn, Hkv, D) || v->get_device() != c.dev) return nullptr;
    const int64_t Hq = q ? q->size(2) : 0;
    if (q && (!same_sizes(*q, S, Tn, Hq, D) || q->get_device() != c.dev)) return nullptr;
    if (four != (args[4] == Py_None)) return nullptr;
    const at::Tensor *kp, *vp = nullptr;
    if (four) {
      kp = c.need(c.dense(3, at::kByte, {-1, Hkv, 18 * D}));
    } else {
      kp = c.need(c.dense(3, at::kBFloat16, {-1, Hkv, -1, D}));
      if (!c.ok) return nullptr;
      vp = c.need(c.dense(4, at::kBFloat16, {kp->size(0), Hkv, kp->size(2), D}));
    }
    const at::Tensor* bt = c.need(c.dense(5, at::kInt, {S, -1}));
    const at::Tensor* sl = c.need(c.dense(6, at::kInt, {S}));
    const Rope r(c, 7, S, Tn, D);
    const at::Tensor* qo = c.dense(13, at::kBFloat16, {S, Hq, Tn, D});
    const at::Tensor* nsl = c.dense(14, at::kInt, {S});
    if (!c.ok || (qo && !q)) return nullptr;
    at::Tensor made;
    if (q && !qo) {
      made = make({S, Hq, Tn, D}, at::kBFloat16);
      qo = &made;
    }
    const Strides sq(q), sk(k), sv(v);
    const int st =
        four ? released(g_entry.append4, ptr(q), ptr(k), ptr(v), sq.s, sk.s, sv.s, ptr(r.qw),
                        ptr(r.kw), ptr(r.cs), ptr(r.pos), ptr(kp), ptr(bt), ptr(sl), ptr(nsl), 16,
                        S, Tn, Hq, Hkv, D, bt->size(1), kp->size(0), r.rot, r.max_pos,
                        r.interleaved, r.eps, ptr(qo), c.stream)
             : released(g_entry.append, ptr(q), ptr(k), ptr(v), sq.s, sk.s, sv.s, ptr(r.qw),
                        ptr(r.kw), ptr(r.cs), ptr(r.pos), ptr(kp), ptr(vp), ptr(bt), ptr(sl),
                        ptr(nsl), kp->size(2), S, Tn, Hq, Hkv, D, bt->size(1), kp->size(0), r.rot,
                        r.max_pos, r.interleaved, r.eps, ptr(qo), c.stream);
    if (st != ATTN_OK) return PyLong_FromLong(st);
    PyObject* after_obj = args[14];
    Py_INCREF(after_obj);
    return pack({result(args[13], made), after_obj});
  });
}

PyObject* append(PyObject*, PyObject* const* args, Py_ssize_t n) { return append_to(args, n, false); }
PyObject* append4(PyObject*, PyObject* const* args, Py_ssize_t n) { return append_to(args, n, true); }

// kv_pool, block_table, seq_lens, max_seq_len, k_out, v_out (both given)
PyObject* gather(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 6, [&](Call& c) -> PyObject* {
    const at::Tensor* pool = c.need(c.tensor(0));
    if (!c.ok || pool->dim() != 3 || pool->size(2) % 18 != 0 || !c.on(*pool)) return nullptr;
    c.dense(0, at::kByte, {-1, -1, -1});
    const int64_t Hkv = pool->size(1), D = pool->size(2) / 18;
    const at::Tensor* sl = c.need(c.dense(2, at::kInt, {-1}));
    if (!c.ok) return nullptr;
    const int64_t S = sl->size(0);
    const at::Tensor* bt = c.need(c.dense(1, at::kInt, {S, -1}));
    const int len = c.integer(3);
    const at::Tensor* ko = c.need(c.dense(4, at::kBFloat16, {S, Hkv, len, D}));
    const at::Tensor* vo = c.need(c.dense(5, at::kBFloat16, {S, Hkv, len, D}));
    if (!c.ok) return nullptr;
    const int st = released(g_entry.gather, ptr(pool), ptr(bt), ptr(sl), 16, S, Hkv, D,
                            bt->size(1), pool->size(0), len, ptr(ko), ptr(vo), c.stream);
    if (st != ATTN_OK) return PyLong_FromLong(st);
    return pack({result(args[4], at::Tensor()), result(args[5], at::Tensor())});
  });
}

// q, kv_pool, block_table, lengths, length bound, scale (None: 1 / sqrt(D)), out, lse,
// workspace, return_lse; causal (prefill only)
PyObject* attend(PyObject* const* args, Py_ssize_t n, bool prefill) {
  return guarded(args, n, prefill ? 11 : 10, [&](Call& c) -> PyObject* {
    const at::Tensor* q = c.need(c.tensor(0));
    if (!c.ok || q->dim() != (prefill ? 4 : 3) || !c.on(*q)) return nullptr;
    const int64_t S = q->size(0), Hq = q->size(1), Tq = prefill ? q->size(2) : 1;
    const int64_t D = q->size(q->dim() - 1);
    if (prefill)
      c.dense(0, at::kBFloat16, {S, Hq, Tq, D});
    else
      c.dense(0, at::kBFloat16, {S, Hq, D});
    const at::Tensor* pool = c.need(c.dense(1, at::kByte, {-1, -1, 18 * D}));
    const at::Tensor* bt = c.need(c.dense(2, at::kInt, {S, -1}));
    const at::Tensor* sl = c.need(c.dense(3, at::kInt, {S}));
    const int len = c.integer(4);
    const float scale = args[5] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)))
                                           : static_cast<float>(c.real(5));
    const at::Tensor* out = prefill ? c.dense(6, at::kBFloat16, {S, Hq, Tq, D})
                                    : c.dense(6, at::kBFloat16, {S, Hq, D});
    const at::Tensor* lse =
        prefill ? c.dense(7, at::kFloat, {S, Hq, Tq}) : c.dense(7, at::kFloat, {S, Hq});
    const at::Tensor* ws = c.dense(8, at::kByte, {-1});
    const int want_lse = c.truth(9);
    const int causal = prefill ? c.truth(10) : 0;
    if (!c.ok) return nullptr;
    const int64_t Hkv = pool->size(1);
    at::Tensor made_out, made_lse;
    c10::DataPtr own_ws;
    size_t bytes = ws ? static_cast<size_t>(ws->numel()) : 0;
    void* work = ptr(ws);
    if (!ws) {
      bytes = prefill ? g_entry.prefill_ws(S, Hq, Hkv, Tq, D, len) : g_entry.decode_ws(S, Hq, Hkv, D, len);
      if (bytes) {
        own_ws = scratch(bytes);
        work = own_ws.get();
      }
    }
    if (!out) {
      made_out = make(q->sizes(), at::kBFloat16);
      out = &made_out;
    }
    if (!lse && want_lse) {
      made_lse = make(q->sizes().slice(0, q->dim() - 1), at::kFloat);
      lse = &made_lse;
    }
    const int st =
        prefill ? released(g_entry.prefill, ptr(q), ptr(pool), ptr(bt), ptr(sl), 16, S, Hq, Hkv, Tq,
                           D, bt->size(1), pool->size(0), len, causal, scale, ptr(out), ptr(lse),
                           work, bytes, c.stream)
                : released(g_entry.decode, ptr(q), ptr(pool), ptr(bt), ptr(sl), 16, S, Hq, Hkv, D,
                           bt->size(1), pool->size(0), len, scale, ptr(out), ptr(lse), work, bytes,
                           c.stream);
    if (st != ATTN_OK) return PyLong_FromLong(st);
    return pack({result(args[6], made_out), result(args[7], made_lse)});
  });
}

PyObject* decode(PyObject*, PyObject* const* args, Py_ssize_t n) { return attend(args, n, false); }
PyObject* prefill(PyObject*, PyObject* const* args, Py_ssize_t n) { return attend(args, n, true); }

// q, k_pool, v_pool, block_table, seq_lens, parents, length bound, tree_lens, scale (None: 1 /
// sqrt(D)), out, lse, workspace, return_lse
PyObject* tree(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 13, [&](Call& c) -> PyObject* {
    const at::Tensor* q = c.need(c.tensor(0));
    if (!c.ok || q->dim() != 4 || !c.on(*q)) return nullptr;
    const int64_t S = q->size(0), Hq = q->size(1), Tn = q->size(2), D = q->size(3);
    c.dense(0, at::kBFloat16, {S, Hq, Tn, D});
    const at::Tensor* kp = c.need(c.dense(1, at::kBFloat16, {-1, -1, -1, D}));
    if (!c.ok) return nullptr;
    const at::Tensor* vp =
        c.need(c.dense(2, at::kBFloat16, {kp->size(0), kp->size(1), kp->size(2), D}));
    const at::Tensor* bt = c.need(c.dense(3, at::kInt, {S, -1}));
    const at::Tensor* sl = c.need(c.dense(4, at::kInt, {S}));
    const at::Tensor* pa = c.need(c.dense(5, at::kInt, {S, Tn}));
    const int len = c.integer(6);
    const at::Tensor* tl = c.dense(7, at::kInt, {S});
    const float scale = args[8] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)))
                                           : static_cast<float>(c.real(8));
    const at::Tensor* out = c.dense(9, at::kBFloat16, {S, Hq, Tn, D});
    const at::Tensor* lse = c.dense(10, at::kFloat, {S, Hq, Tn});
    const at::Tensor* ws = c.dense(11, at::kByte, {-1});
    const int want_lse = c.truth(12);
    if (!c.ok) return nullptr;
    const int64_t Hkv = kp->size(1);
    at::Tensor made_out, made_lse;
    c10::DataPtr own_ws;
    size_t bytes = ws ? static_cast<size_t>(ws->numel()) : 0;
    void* work = ptr(ws);
    if (!ws) {
      bytes = g_tree.attend_ws(S, Tn, Hq, Hkv, D, len);
      if (bytes) {
        own_ws = scratch(bytes);
        work = own_ws.get();
      }
    }
    if (!out) {
      made_out = make(q->sizes(), at::kBFloat16);
      out = &made_out;
    }
    if (!lse && want_lse) {
      made_lse = make(q->sizes().slice(0, 3), at::kFloat);
      lse = &made_lse;
    }
    const int st = released(g_tree.attend, ptr(q), ptr(kp), ptr(vp), ptr(bt), ptr(sl), ptr(pa),
                            ptr(tl), kp->size(2), S, Tn, Hq, Hkv, D, bt->size(1), kp->size(0), len,
                            scale, ptr(out), ptr(lse), work, bytes, c.stream);
    if (st != ATTN_OK) return PyLong_FromLong(st);
    return pack({result(args[9], made_out), result(args[10], made_lse)});
  });
}

// target_probs, draft_probs, tokens, parents, uniforms, tree_lens, tokens_out, path, counts
PyObject* verify(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 9, [&](Call& c) -> PyObject* {
    const at::Tensor *p = c.need(c.tensor(0)), *q = c.tensor(1);
    if (!c.ok || p->dim() != 3 || !c.on(*p)) return nullptr;
    const at::ScalarType type = p->scalar_type();
    if (type != at::kFloat && type != at::kBFloat16) return nullptr;
    const int64_t S = p->size(0), Tn = p->size(1), V = p->size(2);
    for (const at::Tensor* t : {p, q})
      if (t && (t->scalar_type() != type || t->dim() != 3 || t->size(0) != S || t->size(1) != Tn ||
                t->size(2) != V || (t->stride(2) != 1 && V > 1) || t->get_device() != c.dev))
        return nullptr;
    if (S > kMaxSize || Tn > kMaxSize || V > kMaxSize) return nullptr;
    const at::Tensor* in[3] = {c.need(c.dense(2, at::kInt, {S, Tn})),
                               c.need(c.dense(3, at::kInt, {S, Tn})),
                               c.need(c.dense(4, at::kFloat, {S, Tn}))};
    const at::Tensor* tl = c.dense(5, at::kInt, {S});
    const at::Tensor* out[3] = {c.dense(6, at::kInt, {S, Tn}), c.dense(7, at::kInt, {S, Tn}),
                                c.dense(8, at::kInt, {S})};
    if (!c.ok) return nullptr;
    at::Tensor made[3];
    for (int i = 0; i < 3; ++i) {
      if (out[i]) continue;
      made[i] = i < 2 ? make({S, Tn}, at::kInt) : make({S}, at::kInt);
      out[i] = &made[i];
    }
    int64_t strides[2][2] = {};
    for (int i = 0; i < 2; ++i) {
      strides[0][i] = p->size(i) > 1 ? p->stride(i) : 0;
      if (q) strides[1][i] = q->size(i) > 1 ? q->stride(i) : 0;
    }
    const int st = released(g_tree.verify, ptr(p), ptr(q), strides[0], strides[1],
                            type == at::kBFloat16 ? 1 : 0, ptr(in[0]), ptr(in[1]), ptr(in[2]), ptr(tl),
                            S, Tn, V, ptr(out[0]), ptr(out[1]), ptr(out[2]), c.stream);
    if (st != ATTN_OK) return PyLong_FromLong(st);
    return pack({result(args[6], made[0]), result(args[7], made[1]), result(args[8], made[2])});
  });
}

// k_pool, v_pool (one layer's, or all layers' in one tensor), block_table, seq_lens, path,
// counts, new_seq_lens
PyObject* keep(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 7, [&](Call& c) -> PyObject* {
    if (!THPVariable_CheckExact(args[0]) || !THPVariable_CheckExact(args[1])) return nullptr;
    const at::Tensor *kp = c.tensor(0), *vp = c.tensor(1), *sl = c.need(c.tensor(3));
    if (!c.ok || sl->dim() != 1 || !c.on(*sl)) return nullptr;
    const int64_t dims = kp->dim(), S = sl->size(0);
    if ((dims != 4 && dims != 5) || kp->sizes() != vp->sizes()) return nullptr;
    for (const at::Tensor* t : {kp, vp})
      if (t->scalar_type() != at::kBFloat16 || !t->is_contiguous() || t->get_device() != c.dev)
        return nullptr;
    const int64_t layers = dims == 5 ? kp->size(0) : 1, *size = kp->sizes().data() + (dims - 4);
    constexpr int64_t kLayers = 256;
    if (layers < 1 || layers > kLayers || size[0] > kMaxSize || size[1] > kMaxSize) return nullptr;
    c.dense(3, at::kInt, {S});
    const at::Tensor* bt = c.need(c.dense(2, at::kInt, {S, -1}));
    const at::Tensor* path = c.need(c.dense(4, at::kInt, {S, -1}));
    const at::Tensor* counts = c.need(c.dense(5, at::kInt, {S}));
    const at::Tensor* after = c.dense(6, at::kInt, {S});
    if (!c.ok) return nullptr;
    void* pools[2][kLayers];
    const int64_t step = size[0] * size[1] * size[2] * size[3] * 2;
    for (int64_t i = 0; i < layers; ++i) {
      pools[0][i] = static_cast<char*>(ptr(kp)) + i * step;
      pools[1][i] = static_cast<char*>(ptr(vp)) + i * step;
    }
    const int st = released(g_tree.keep, pools[0], pools[1], layers, ptr(bt), ptr(sl), ptr(path),
                            ptr(counts), ptr(after), size[2], S, path->size(1), size[1], size[3],
                            bt->size(1), size[0], c.stream);
    if (st != ATTN_OK) return PyLong_FromLong(st);
    // (in a tuple, as a result may be None)
    return pack({result(args[6], at::Tensor())});
  });
}

// setup(torch's version, get_device, get_stream, addresses of the entry points in the order
// of Entry)
PyObject* setup(PyObject*, PyObject* const* args, Py_ssize_t n) {
  constexpr Py_ssize_t kEntries = sizeof(Entry) / sizeof(void*);
  if (n != 3 + kEntries || !PyUnicode_Check(args[0])) {
    PyErr_SetString(PyExc_TypeError, "setup takes a version, two functions and the entry points");
    return nullptr;
  }
  if (PyUnicode_CompareWithASCIIString(args[0], BUILT_FOR_TORCH) != 0) {
    PyErr_SetString(PyExc_ImportError, "built against torch " BUILT_FOR_TORCH);
    return nullptr;
  }
  void* address[kEntries];
  for (Py_ssize_t i = 0; i < kEntries; ++i) {
    address[i] = PyLong_AsVoidPtr(args[3 + i]);
    if (!address[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an entry point is missing");
      return nullptr;
    }
  }
  static_assert(sizeof(Entry) == kEntries * sizeof(void*), "Entry holds addresses only");
  memcpy(&g_entry, address, sizeof g_entry);
  Py_INCREF(args[1]);
  Py_INCREF(args[2]);
  g_get_device = args[1];
  g_get_stream = args[2];
  Py_RETURN_NONE;
}

// setup_tree(addresses of the entry points in the order of TreeEntry), after setup.
PyObject* setup_tree(PyObject*, PyObject* const* args, Py_ssize_t n) {
  constexpr Py_ssize_t kEntries = sizeof(TreeEntry) / sizeof(void*);
  if (n != kEntries) {
    PyErr_SetString(PyExc_TypeError, "setup_tree takes the entry points");
    return nullptr;
  }
  void* address[kEntries];
  for (Py_ssize_t i = 0; i < kEntries; ++i) {
    address[i] = PyLong_AsVoidPtr(args[i]);
    if (!address[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an entry point is missing");
      return nullptr;
    }
  }
  memcpy(&g_tree, address, sizeof g_tree);
  Py_RETURN_NONE;
}

#define ENTRY(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {ENTRY(setup),   ENTRY(rope),   ENTRY(rope_bwd),
                           ENTRY(append),  ENTRY(append4), ENTRY(gather),
                           ENTRY(decode),  ENTRY(prefill), ENTRY(setup_tree),
                           ENTRY(tree),    ENTRY(verify),  ENTRY(keep),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&g_module); }
