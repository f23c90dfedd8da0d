// The serving-cache calls of the Python package without the interpreter's share:
// argument checks, output tensors and one call into librf.so each.
//
// A decode step of a small batch takes the GPU 7 us; the same marshalling in
// Python (ctypes, four tensor checks, two torch allocations) takes the host 16 us.
// Nothing is computed here.  A function returns None when anything about its
// arguments is not as it has to be (the Python wrapper then goes its own checked
// way, which says what), the library's status as an int when that is not RF_OK,
// and the outputs as a tuple otherwise.
//
// Built beside librf.so against the installed torch; the package works without it.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <stdexcept>

#include "rf.h"

namespace {

// A CUDA tensor (no subclass) on `dev`, contiguous, of a type and sizes.
bool is(const at::Tensor& t, int dev, at::ScalarType type, at::IntArrayRef sizes) {
  return t.is_cuda() && t.get_device() == dev && t.scalar_type() == type && t.is_contiguous() &&
         t.sizes() == sizes;
}

const at::Tensor* tensor(PyObject* o) {
  return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr;
}

// A tensor or None: *t is null for None.
bool optional_tensor(PyObject* o, const at::Tensor** t) {
  *t = nullptr;
  if (o == Py_None) return true;
  *t = tensor(o);
  return *t != nullptr;
}

// The address of an optional tensor: null for none, and only then.
template <typename T>
const T* optional_address(const at::Tensor* t) {
  if (!t) return nullptr;
  const void* p = t->const_data_ptr();
  if (!p && t->numel() > 0) throw std::runtime_error("a tensor without memory");
  return static_cast<const T*>(p);
}

int type_code(at::ScalarType t) {
  return t == at::kBFloat16 ? RF_BF16 : t == at::kHalf ? RF_F16 : t == at::kFloat ? RF_F32 : -1;
}

// A Python int as a C int; counts too large for one become the largest.
bool count(PyObject* o, int* n) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &over);
  if (over > 0 || v > 0x7fffffffLL)
    *n = 0x7fffffff;
  else if (over < 0 || v < -1)
    *n = -1;
  else
    *n = (int)v;
  return true;
}

bool pointer(PyObject* o, void** p) {
  if (!PyLong_CheckExact(o)) return false;
  *p = PyLong_AsVoidPtr(o);
  return !PyErr_Occurred();
}

// The scale, 1 / sqrt(D) for None.
bool scale_of(PyObject* o, int D, float* scale) {
  if (o == Py_None)
    *scale = (float)(1.0 / std::sqrt((double)D));
  else if (PyFloat_CheckExact(o))
    *scale = (float)PyFloat_AS_DOUBLE(o);
  else
    return false;
  return true;
}

struct Cache {
  const at::Tensor *q, *k, *v, *lens;
  int dev, B, H, Hkv, cap, D, type;
  const int32_t* lens_ptr() const { return optional_address<int32_t>(lens); }
};

// q [B, H, D], k and v [B, Hkv, cap, D], lens [B] int32 or None, on the current device.
bool read_cache(PyObject* const* a, Cache* c) {
  c->q = tensor(a[0]);
  c->k = tensor(a[1]);
  c->v = tensor(a[2]);
  if (!c->q || !c->k || !c->v || !optional_tensor(a[3], &c->lens)) return false;
  if (!c->q->is_cuda() || c->q->dim() != 3 || c->k->dim() != 4) return false;
  for (const at::Tensor* t : {c->q, c->k})
    for (const int64_t n : t->sizes())
      if (n > 0x7fffffffLL) return false;
  const at::ScalarType type = c->q->scalar_type();
  c->dev = (int)c->q->get_device();
  c->B = (int)c->q->size(0);
  c->H = (int)c->q->size(1);
  c->D = (int)c->q->size(2);
  c->Hkv = (int)c->k->size(1);
  c->cap = (int)c->k->size(2);
  c->type = type_code(type);
  return c->type >= 0 && c->q->is_contiguous() &&
         is(*c->k, c->dev, type, {c->B, c->Hkv, c->cap, c->D}) &&
         is(*c->v, c->dev, type, c->k->sizes()) &&
         (!c->lens || is(*c->lens, c->dev, at::kInt, {c->B})) &&
         c10::cuda::current_device() == c->dev;
}

// A workspace's (device, B, H, Hkv, D) and four addresses.
struct Work {
  void *m, *l, *acc, *counters;
};
bool read_work(PyObject* sizes, PyObject* addresses, const Cache& c, Work* w) {
  if (!PyTuple_Check(sizes) || PyTuple_GET_SIZE(sizes) != 5 || !PyTuple_Check(addresses) ||
      PyTuple_GET_SIZE(addresses) != 4)
    return false;
  const int want[5] = {c.dev, c.B, c.H, c.Hkv, c.D};
  for (int i = 0; i < 5; ++i) {
    int n;
    if (!count(PyTuple_GET_ITEM(sizes, i), &n) || n != want[i]) return false;
  }
  void** p[4] = {&w->m, &w->l, &w->acc, &w->counters};
  for (int i = 0; i < 4; ++i)
    if (!pointer(PyTuple_GET_ITEM(addresses, i), p[i])) return false;
  return true;
}

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

at::Tensor like(const at::Tensor& t, at::IntArrayRef sizes, at::ScalarType type) {
  return at::empty(sizes, t.options().dtype(type));
}

// Elements at .. at + n - 1 of a 1-D tensor as one of their own, over the same memory.
at::Tensor part(const at::Tensor& all, int64_t at, int64_t n) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(at);
  t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
  return t;
}

template <typename... T>
PyObject* pack(T&&... t) {
  PyObject* items[] = {THPVariable_Wrap(std::forward<T>(t))...};
  PyObject* r = PyTuple_New(sizeof...(T));
  bool ok = r != nullptr;
  for (PyObject* o : items) ok = ok && o != nullptr;
  if (!ok) {
    Py_XDECREF(r);
    for (PyObject* o : items) Py_XDECREF(o);
    return nullptr;
  }
  Py_ssize_t i = 0;
  for (PyObject* o : items) PyTuple_SET_ITEM(r, i++, o);
  return r;
}

// Without the GIL while it lives.  An exception on its way out takes the GIL back
// (a tensor without memory, or a wrapper of one, throws when asked for its address).
class Released {
 public:
  Released() : state_(PyEval_SaveThread()) {}
  ~Released() { PyEval_RestoreThread(state_); }
  Released(const Released&) = delete;
  Released& operator=(const Released&) = delete;

 private:
  PyThreadState* state_;
};

// Runs `call` without the GIL; its status if that is not RF_OK, else null.
template <typename F>
PyObject* failed(F call) {
  int status;
  {
    Released released;
    status = call();
  }
  return status == RF_OK ? nullptr : PyLong_FromLong(status);
}

// No C++ exception leaves a function: an allocation that fails, say, becomes the
// Python error that the checked way would meet again.
template <typename F>
PyObject* guarded(F body) {
  try {
    at::AutoDispatchBelowADInplaceOrView below;
    return body();
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

// (function, q, k, v, lens, window, sinks, scale, S, sizes, addresses)
PyObject* decode_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Cache c;
    Work w;
    void* fn;
    int window, sinks, S;
    float scale;
    if (n != 11 || !pointer(a[0], &fn) || !read_cache(a + 1, &c) || !count(a[5], &window) ||
        !count(a[6], &sinks) || !scale_of(a[7], c.D, &scale) || !count(a[8], &S) ||
        !read_work(a[9], a[10], c, &w))
      Py_RETURN_NONE;
    at::Tensor out = like(*c.q, c.q->sizes(), c.q->scalar_type());
    at::Tensor lse = like(*c.q, {c.B, c.H}, at::kFloat);
    if (PyObject* e = failed([&] {
          return reinterpret_cast<decltype(&rf_attn_decode_window)>(fn)(
              c.q->const_data_ptr(), c.k->const_data_ptr(), c.v->const_data_ptr(), c.lens_ptr(), c.B,
              c.H, c.Hkv, c.cap, c.D, window, sinks, S, scale, c.type, static_cast<float*>(w.m),
              static_cast<float*>(w.l), static_cast<float*>(w.acc), static_cast<int*>(w.counters),
              out.mutable_data_ptr(), c.type, static_cast<float*>(lse.mutable_data_ptr()),
              stream_of(c.dev));
        }))
      return e;
    return pack(std::move(out), std::move(lse));
  });
}

// (function, q, kp, vp, k, v, lens, scale, prefix_S, S, sizes, addresses)
PyObject* decode_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Cache c;
    Work w;
    void* fn;
    int Sp, S;
    float scale;
    if (n != 12 || !pointer(a[0], &fn)) Py_RETURN_NONE;
    PyObject* cache[4] = {a[1], a[4], a[5], a[6]};
    const at::Tensor *kp = tensor(a[2]), *vp = tensor(a[3]);
    if (!kp || !vp || kp->dim() != 3 || !read_cache(cache, &c) || !scale_of(a[7], c.D, &scale) ||
        !count(a[8], &Sp) || !count(a[9], &S) || !read_work(a[10], a[11], c, &w))
      Py_RETURN_NONE;
    const int64_t prefix = kp->size(1);
    if (prefix > 0x7fffffffLL || !is(*kp, c.dev, c.q->scalar_type(), {c.Hkv, prefix, c.D}) ||
        !is(*vp, c.dev, c.q->scalar_type(), kp->sizes()))
      Py_RETURN_NONE;
    at::Tensor out = like(*c.q, c.q->sizes(), c.q->scalar_type());
    at::Tensor lse = like(*c.q, {c.B, c.H}, at::kFloat);
    if (PyObject* e = failed([&] {
          return reinterpret_cast<decltype(&rf_attn_decode_shared)>(fn)(
              c.q->const_data_ptr(), kp->const_data_ptr(), vp->const_data_ptr(), (int)prefix,
              c.k->const_data_ptr(), c.v->const_data_ptr(), c.lens_ptr(), c.B, c.H, c.Hkv, c.cap,
              c.D, Sp, S, scale, c.type, static_cast<float*>(w.m), static_cast<float*>(w.l),
              static_cast<float*>(w.acc), static_cast<int*>(w.counters), out.mutable_data_ptr(),
              c.type, static_cast<float*>(lse.mutable_data_ptr()), stream_of(c.dev));
        }))
      return e;
    return pack(std::move(out), std::move(lse));
  });
}

// (function, q, k, v, lens, weight, scale, S, sizes, addresses, scores)
PyObject* decode_weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Cache c;
    Work w;
    void* fn;
    int S;
    float scale;
    const at::Tensor *weight, *scores;
    if (n != 11 || !pointer(a[0], &fn) || !read_cache(a + 1, &c) || !optional_tensor(a[5], &weight) ||
        !scale_of(a[6], c.D, &scale) || !count(a[7], &S) || !read_work(a[8], a[9], c, &w) ||
        !(scores = tensor(a[10])) || !is(*scores, c.dev, at::kFloat, {c.B, c.H, c.cap}) ||
        (weight && !is(*weight, c.dev, at::kFloat, {c.B, c.Hkv, c.cap})))
      Py_RETURN_NONE;
    at::Tensor out = like(*c.q, c.q->sizes(), c.q->scalar_type());
    at::Tensor lse = like(*c.q, {c.B, c.H}, at::kFloat);
    at::Tensor total = like(*c.q, {c.B, c.Hkv, c.cap}, at::kFloat);
    if (PyObject* e = failed([&] {
          return reinterpret_cast<decltype(&rf_attn_decode_weights)>(fn)(
              c.q->const_data_ptr(), c.k->const_data_ptr(), c.v->const_data_ptr(), c.lens_ptr(), c.B,
              c.H, c.Hkv, c.cap, c.D, S, scale, c.type, static_cast<float*>(w.m),
              static_cast<float*>(w.l), static_cast<float*>(w.acc), static_cast<int*>(w.counters),
              static_cast<float*>(scores->mutable_data_ptr()), out.mutable_data_ptr(), c.type,
              static_cast<float*>(lse.mutable_data_ptr()),
              optional_address<float>(weight),
              static_cast<float*>(total.mutable_data_ptr()), stream_of(c.dev));
        }))
      return e;
    return pack(std::move(out), std::move(lse), std::move(total));
  });
}

// (function, q, k, v, window, sinks, scale)
PyObject* prefill_window(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    void* fn;
    int window, sinks;
    float scale;
    if (n != 7 || !pointer(a[0], &fn)) Py_RETURN_NONE;
    const at::Tensor *q = tensor(a[1]), *k = tensor(a[2]), *v = tensor(a[3]);
    if (!q || !k || !v || !q->is_cuda() || q->dim() != 4 || k->dim() != 4) Py_RETURN_NONE;
    for (const at::Tensor* t : {q, k})
      for (const int64_t s : t->sizes())
        if (s > 0x7fffffffLL) Py_RETURN_NONE;
    const at::ScalarType type = q->scalar_type();
    const int dev = (int)q->get_device(), code = type_code(type);
    const int64_t B = q->size(0), H = q->size(1), N = q->size(2), D = q->size(3);
    const int64_t Hkv = k->size(1), L = k->size(2);
    if (code < 0 || !q->is_contiguous() || !is(*k, dev, type, {B, Hkv, L, D}) ||
        !is(*v, dev, type, k->sizes()) || c10::cuda::current_device() != dev ||
        !count(a[4], &window) || !count(a[5], &sinks) || !scale_of(a[6], (int)D, &scale))
      Py_RETURN_NONE;
    at::Tensor out = like(*q, q->sizes(), type);
    at::Tensor lse = like(*q, {B, H, N}, at::kFloat);
    if (PyObject* e = failed([&] {
          return reinterpret_cast<decltype(&rf_attn_prefill_window)>(fn)(
              q->const_data_ptr(), k->const_data_ptr(), v->const_data_ptr(), (int)B, (int)H, (int)Hkv,
              (int)N, (int)L, (int)D, window, sinks, scale, code, out.mutable_data_ptr(),
              static_cast<float*>(lse.mutable_data_ptr()), stream_of(dev));
        }))
      return e;
    return pack(std::move(out), std::move(lse));
  });
}

// (function, k, v, weight, lens, keep, sinks, recent, k_out, v_out, weight_out);
// gives lens_out and kept
PyObject* cache_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    void* fn;
    int keep, sinks, recent;
    const at::Tensor *v, *lens, *v_out;
    if (n != 11 || !pointer(a[0], &fn)) Py_RETURN_NONE;
    const at::Tensor *k = tensor(a[1]), *weight = tensor(a[3]), *k_out = tensor(a[8]),
                     *weight_out = tensor(a[10]);
    if (!k || !weight || !k_out || !weight_out || !optional_tensor(a[2], &v) ||
        !optional_tensor(a[4], &lens) || !optional_tensor(a[9], &v_out) || !count(a[5], &keep) ||
        !count(a[6], &sinks) || !count(a[7], &recent) || !k->is_cuda() || k->dim() != 4 ||
        k_out->dim() != 4 || keep < 1)
      Py_RETURN_NONE;
    for (const at::Tensor* t : {k, k_out})
      for (const int64_t s : t->sizes())
        if (s > 0x7fffffffLL) Py_RETURN_NONE;
    const at::ScalarType type = k->scalar_type();
    const int dev = (int)k->get_device(), code = type_code(type);
    const int64_t B = k->size(0), Hkv = k->size(1), cap = k->size(2), D = k->size(3);
    const int64_t cap_out = k_out->size(2);
    if (code < 0 || !k->is_contiguous() || !is(*k_out, dev, type, {B, Hkv, cap_out, D}) ||
        (v && !is(*v, dev, type, k->sizes())) || (v_out && !is(*v_out, dev, type, k_out->sizes())) ||
        !is(*weight, dev, at::kFloat, {B, Hkv, cap}) ||
        !is(*weight_out, dev, at::kFloat, {B, Hkv, cap_out}) ||
        (lens && !is(*lens, dev, at::kInt, {B})) || c10::cuda::current_device() != dev)
      Py_RETURN_NONE;
    at::Tensor lens_out = like(*k, {B}, at::kInt);
    at::Tensor kept = like(*k, {B, Hkv, keep}, at::kInt);
    if (PyObject* e = failed([&] {
          return reinterpret_cast<decltype(&rf_cache_evict)>(fn)(
              k->const_data_ptr(), optional_address<void>(v),
              static_cast<const float*>(weight->const_data_ptr()),
              optional_address<int32_t>(lens), (int)B, (int)Hkv,
              (int)cap, (int)D, code, keep, sinks, recent, (int)cap_out, k_out->mutable_data_ptr(),
              v_out ? v_out->mutable_data_ptr() : nullptr,
              static_cast<float*>(weight_out->mutable_data_ptr()),
              static_cast<int32_t*>(lens_out.mutable_data_ptr()),
              static_cast<int32_t*>(kept.mutable_data_ptr()), stream_of(dev));
        }))
      return e;
    return pack(std::move(lens_out), std::move(kept));
  });
}

// (function, lens, news, table, stack, n_free, page, tokens); gives starts, positions, slots,
// lens_out and n_free_out
PyObject* page_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    void* fn;
    int page, tokens;
    if (n != 8 || !pointer(a[0], &fn) || !count(a[6], &page) || !count(a[7], &tokens)) Py_RETURN_NONE;
    const at::Tensor *lens = tensor(a[1]), *news = tensor(a[2]), *table = tensor(a[3]), *stack = tensor(a[4]),
                     *n_free = tensor(a[5]);
    if (!lens || !news || !table || !stack || !n_free || !lens->is_cuda() || table->dim() != 2 ||
        stack->dim() != 1 || tokens < 1)
      Py_RETURN_NONE;
    const int64_t B = table->size(0), width = table->size(1), pages = stack->size(0);
    const int dev = (int)lens->get_device();
    if (B > 0x7fffffffLL || width > 0x7fffffffLL || pages > 0x7fffffffLL || !is(*lens, dev, at::kInt, {B}) ||
        !is(*news, dev, at::kInt, {B}) || !is(*table, dev, at::kInt, {B, width}) ||
        !is(*stack, dev, at::kInt, {pages}) || !is(*n_free, dev, at::kInt, {1}) ||
        c10::cuda::current_device() != dev)
      Py_RETURN_NONE;
    // one allocation, each output from 256 bytes on (a call takes the host 5.2 us; of five, 9.4)
    const auto up = [](int64_t x) { return (x + 63) / 64 * 64; };
    const int64_t at1 = up(tokens), at2 = at1 + up(tokens), at3 = at2 + up(B + 1), at4 = at3 + up(B);
    const at::Tensor all = like(*lens, {at4 + 1}, at::kInt);
    at::Tensor positions = part(all, 0, tokens), slots = part(all, at1, tokens), starts = part(all, at2, B + 1);
    at::Tensor lens_out = part(all, at3, B), n_free_out = part(all, at4, 1);
    const auto in = [](const at::Tensor& t) { return static_cast<const int32_t*>(t.const_data_ptr()); };
    const auto out = [](const at::Tensor& t) { return static_cast<int32_t*>(t.mutable_data_ptr()); };
    if (PyObject* e = failed([&] {
          return reinterpret_cast<decltype(&rf_page_tables)>(fn)(
              in(*lens), in(*news), (int)B, out(*table), (int)width, out(*stack), (int)pages, in(*n_free),
              page, tokens, out(starts), out(positions), out(slots), out(lens_out), out(n_free_out),
              stream_of(dev));
        }))
      return e;
    return pack(std::move(starts), std::move(positions), std::move(slots), std::move(lens_out),
                std::move(n_free_out));
  });
}

// q, k or v [T, heads, D] with dense heads, and the elements from a token's row to the next.
bool token_rows(const at::Tensor& t, int dev, at::ScalarType type, at::IntArrayRef sizes, long long* step) {
  if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || t.sizes() != sizes ||
      (sizes[2] > 1 && t.stride(2) != 1) || (sizes[1] > 1 && t.stride(1) != sizes[2]))
    return false;
  *step = sizes[0] > 1 ? t.stride(0) : sizes[1] * sizes[2];
  return true;
}

// (function, q, k, positions, freq, q_weight, k_weight, axis, interleaved, eps, v, slots, kp, vp);
// gives q, and k without a cache
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    void* fn;
    if (n != 14 || !pointer(a[0], &fn) || !PyBool_Check(a[8]) || !PyFloat_CheckExact(a[9])) Py_RETURN_NONE;
    const at::Tensor *q = tensor(a[1]), *k = tensor(a[2]), *positions = tensor(a[3]), *freq = tensor(a[4]);
    const at::Tensor *qw, *kw, *axis, *v, *slots, *kp, *vp;
    if (!q || !k || !positions || !freq || !optional_tensor(a[5], &qw) || !optional_tensor(a[6], &kw) ||
        !optional_tensor(a[7], &axis) || !optional_tensor(a[10], &v) || !optional_tensor(a[11], &slots) ||
        !optional_tensor(a[12], &kp) || !optional_tensor(a[13], &vp) || !q->is_cuda() || q->dim() != 3 ||
        k->dim() != 3 || positions->dim() != 2 || freq->dim() != 1)
      Py_RETURN_NONE;
    if ((v != nullptr) != (slots != nullptr) || (v != nullptr) != (kp != nullptr) ||
        (v != nullptr) != (vp != nullptr) || (kp && kp->dim() != 4))
      Py_RETURN_NONE;
    for (const at::Tensor* t : {q, k, positions, freq, kp})
      if (t)
        for (const int64_t s : t->sizes())
          if (s > 0x3fffffffLL) Py_RETURN_NONE;
    const at::ScalarType type = q->scalar_type();
    const int dev = (int)q->get_device(), code = type_code(type);
    const int64_t T = q->size(0), H = q->size(1), D = q->size(2), Hkv = k->size(1), half = freq->size(0);
    const int64_t axes = positions->size(0), pages = kp ? kp->size(0) : 0, page = kp ? kp->size(2) : 0;
    long long q_step, k_step, v_step = 0;
    const at::Tensor* w = qw ? qw : kw;
    const at::ScalarType w_type = w ? w->scalar_type() : type;
    if (code < 0 || (w_type != type && w_type != at::kFloat) || !token_rows(*q, dev, type, {T, H, D}, &q_step) ||
        !token_rows(*k, dev, type, {T, Hkv, D}, &k_step) || !is(*positions, dev, at::kInt, {axes, T}) ||
        !is(*freq, dev, at::kFloat, {half}) || (qw && !is(*qw, dev, w_type, {D})) ||
        (kw && !is(*kw, dev, w_type, {D})) || (axis && !is(*axis, dev, at::kInt, {half})) ||
        (v && !token_rows(*v, dev, type, {T, Hkv, D}, &v_step)) || (slots && !is(*slots, dev, at::kInt, {T})) ||
        (kp && !is(*kp, dev, type, {pages, Hkv, page, D})) || (vp && !is(*vp, dev, type, kp->sizes())) ||
        c10::cuda::current_device() != dev)
      Py_RETURN_NONE;
    at::Tensor q_out = like(*q, {T, H, D}, type), k_out;
    if (!kp) k_out = like(*k, {T, Hkv, D}, type);
    if (PyObject* e = failed([&] {
          return reinterpret_cast<decltype(&rf_qk_norm_rope)>(fn)(
              q->const_data_ptr(), q_step, k->const_data_ptr(), k_step, optional_address<void>(v), v_step,
              (int)T, (int)H, (int)Hkv, (int)D, optional_address<void>(qw), optional_address<void>(kw),
              type_code(w_type), (float)PyFloat_AS_DOUBLE(a[9]),
              static_cast<const int32_t*>(positions->const_data_ptr()), (int)axes,
              static_cast<const float*>(freq->const_data_ptr()), optional_address<int32_t>(axis),
              (int)(2 * half), a[8] == Py_True, code, optional_address<int32_t>(slots), (int)pages, (int)page,
              q_out.mutable_data_ptr(), kp ? kp->mutable_data_ptr() : k_out.mutable_data_ptr(),
              vp ? vp->mutable_data_ptr() : nullptr, stream_of(dev));
        }))
      return e;
    return kp ? pack(std::move(q_out)) : pack(std::move(q_out), std::move(k_out));
  });
}

// (function, q, kp, vp, table, plan, sizes, max_new, max_len, window, sinks, scale); sizes: (device,
// B, T, H, Hkv)
PyObject* attn_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    void* fn;
    int max_new, max_len, window, sinks;
    float scale;
    if (n != 12 || !pointer(a[0], &fn)) Py_RETURN_NONE;
    const at::Tensor *q = tensor(a[1]), *kp = tensor(a[2]), *vp = tensor(a[3]), *table = tensor(a[4]),
                     *plan = tensor(a[5]);
    if (!q || !kp || !vp || !table || !plan || !q->is_cuda() || q->dim() != 3 || kp->dim() != 4 ||
        table->dim() != 2 || plan->dim() != 1 || !PyTuple_Check(a[6]) || PyTuple_GET_SIZE(a[6]) != 5 ||
        !count(a[7], &max_new) || !count(a[8], &max_len) || !count(a[9], &window) || !count(a[10], &sinks))
      Py_RETURN_NONE;
    for (const at::Tensor* t : {q, kp, table})
      for (const int64_t s : t->sizes())
        if (s > 0x7fffffffLL) Py_RETURN_NONE;
    const at::ScalarType type = q->scalar_type();
    const int dev = (int)q->get_device(), code = type_code(type);
    const int64_t T = q->size(0), H = q->size(1), D = q->size(2), pages = kp->size(0), Hkv = kp->size(1);
    const int64_t page = kp->size(2), B = table->size(0), width = table->size(1);
    const int64_t want[5] = {dev, B, T, H, Hkv};
    for (int i = 0; i < 5; ++i) {
      int x;
      if (!count(PyTuple_GET_ITEM(a[6], i), &x) || x != want[i]) Py_RETURN_NONE;
    }
    if (code < 0 || !scale_of(a[11], (int)D, &scale) || !q->is_contiguous() ||
        !is(*kp, dev, type, {pages, Hkv, page, D}) || !is(*vp, dev, type, kp->sizes()) ||
        !is(*table, dev, at::kInt, {B, width}) || !is(*plan, dev, at::kByte, plan->sizes()) ||
        c10::cuda::current_device() != dev)
      Py_RETURN_NONE;
    at::Tensor out = like(*q, q->sizes(), type), lse = like(*q, {T, H}, at::kFloat);
    if (PyObject* e = failed([&] {
          return reinterpret_cast<decltype(&rf_attn_paged)>(fn)(
              q->const_data_ptr(), kp->const_data_ptr(), vp->const_data_ptr(), (int)pages, (int)page,
              static_cast<const int32_t*>(table->const_data_ptr()), (int)width, plan->mutable_data_ptr(),
              (size_t)plan->numel(), (int)B, (int)T, (int)H, (int)Hkv, (int)D, max_new, max_len, window, sinks,
              scale, code, out.mutable_data_ptr(), static_cast<float*>(lse.mutable_data_ptr()),
              stream_of(dev));
        }))
      return e;
    return pack(std::move(out), std::move(lse));
  });
}

PyMethodDef methods[] = {
    {"page_tables", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(page_tables)), METH_FASTCALL,
     nullptr},
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(qk_norm_rope)), METH_FASTCALL,
     nullptr},
    {"attn_paged", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(attn_paged)), METH_FASTCALL, nullptr},
    {"decode_window", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(decode_window)),
     METH_FASTCALL, nullptr},
    {"decode_shared", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(decode_shared)),
     METH_FASTCALL, nullptr},
    {"decode_weights", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(decode_weights)),
     METH_FASTCALL, nullptr},
    {"prefill_window", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(prefill_window)),
     METH_FASTCALL, nullptr},
    {"cache_evict", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(cache_evict)),
     METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rf_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rf_calls() { return PyModule_Create(&module); }
