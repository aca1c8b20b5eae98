// Argument marshalling of the serving calls (norm and rotation, window
// attention, the 4-bit cache) without the interpreter: a decoding step makes
// several of them per layer, and reading a tensor's attributes, allocating the
// outputs and building the C structures in Python took most of a call (norm
// and rotation of 64 tokens: 15 us a call in Python, 7 us here, of which 3 us
// on the GPU; the cache's paging 16 and 6 us).
//
// Each function takes the Python call's arguments, and
//   - returns None, having done nothing, when an argument is not plainly what
//     the call takes: the Python code then checks them one by one and says
//     what is wrong;
//   - otherwise allocates the outputs that were not given, calls the C entry
//     point on the current stream and returns the outputs, or the status when
//     it is not RBS_OK.  What is returned is made before the call, so that
//     nothing fails after it and no call is made twice.
// The entry points' addresses come from the loaded librbs (bind()).
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "rbs.h"

namespace {

decltype(&rope_qk_norm) p_rope_qk_norm;
decltype(&swa_prefill) p_swa_prefill;
decltype(&kv4_extend) p_kv4_extend;
decltype(&kv4_append) p_kv4_append;
decltype(&kv4_load) p_kv4_load;
decltype(&kv4_attend) p_kv4_attend;
decltype(&rbs_kv4_attend_workspace_bytes) p_kv4_attend_workspace_bytes;

// Other Python threads run while an allocation or a launch may block.
struct NoGil {
  PyThreadState* state = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(state); }
};

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// A [B, L, H, D] bf16 tensor on `dev` with a contiguous last dimension.
bool bf16(const at::Tensor* x, int dev, rbs_bf16_tensor* t) {
  if (x == nullptr || !x->is_cuda() || x->get_device() != dev || x->scalar_type() != at::kBFloat16 || x->dim() != 4 ||
      x->stride(3) != 1)
    return false;
  *t = {x->data_ptr(), x->size(0), x->size(1), x->size(2), x->size(3), x->stride(0), x->stride(1), x->stride(2)};
  return true;
}

// A contiguous int32 tensor of the given shape on `dev`.
bool ints(const at::Tensor* x, int dev, at::IntArrayRef shape) {
  return x != nullptr && x->is_cuda() && x->get_device() == dev && x->scalar_type() == at::kInt && x->is_contiguous() &&
         x->sizes() == shape;
}

// An int32 [rows, width] table with contiguous rows on `dev`.
bool table(const at::Tensor* x, int dev, int64_t rows, int64_t* stride) {
  if (x == nullptr || !x->is_cuda() || x->get_device() != dev || x->scalar_type() != at::kInt || x->dim() != 2 ||
      x->size(0) != rows || (x->stride(1) != 1 && x->size(1) > 1))
    return false;
  *stride = rows > 1 ? x->stride(0) : std::max(x->stride(0), x->size(1));
  return true;
}

// 128 bf16 norm weights on `dev`, or None.
bool weights(PyObject* o, int dev, int64_t n, const void** p) {
  *p = nullptr;
  if (o == Py_None) return true;
  const at::Tensor* x = tensor(o);
  if (x == nullptr || !x->is_cuda() || x->get_device() != dev || x->scalar_type() != at::kBFloat16 || x->dim() != 1 ||
      x->size(0) != n || !x->is_contiguous())
    return false;
  *p = x->data_ptr();
  return true;
}

bool whole(PyObject* o, int64_t* v) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  *v = PyLong_AsLongLongAndOverflow(o, &over);
  return over == 0;
}
// A whole number that an int32 argument holds.
bool whole32(PyObject* o, int64_t* v) { return whole(o, v) && *v >= INT32_MIN && *v <= INT32_MAX; }

bool flag(PyObject* o, bool* v) {
  *v = o == Py_True;
  return *v || o == Py_False;
}

bool real(PyObject* o, float* v) {
  if (PyFloat_CheckExact(o)) *v = static_cast<float>(PyFloat_AS_DOUBLE(o));
  else if (int64_t i; whole(o, &i)) *v = static_cast<float>(i);
  else return false;
  return true;
}

// The softmax scale, or the default for None.
bool scale_of(PyObject* o, int64_t head_dim, float* v) {
  *v = static_cast<float>(1.0 / std::sqrt(static_cast<double>(head_dim)));
  return o == Py_None || real(o, v);
}

// The cache's structure from its buffer, page size and scales.
bool cache(PyObject* const* a, int dev, rbs_kv4_cache* c) {
  const at::Tensor* x = tensor(a[0]);
  int64_t page;
  if (x == nullptr || !x->is_cuda() || x->get_device() != dev || x->scalar_type() != at::kByte || !x->is_contiguous() ||
      x->dim() != 3 || !whole32(a[1], &page) || page < 16 || x->size(2) != page / 16 * 2304 || x->size(1) > INT32_MAX ||
      !real(a[2], &c->k_scale) || !real(a[3], &c->v_scale))
    return false;
  c->data = x->data_ptr();
  c->num_pages = x->size(0);
  c->kv_heads = static_cast<int32_t>(x->size(1));
  c->page_size = static_cast<int32_t>(page);
  return true;
}

rbs_stream_t stream(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, int dev) {
  NoGil g;
  return at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt);
}

// An output: the given tensor, or one of `like`'s layout (a plain layout is
// allocated directly, past the dispatcher's 2 us).
bool output(PyObject* o, const at::Tensor& like, at::Tensor* hold, const at::Tensor** x) {
  if (o == Py_None) {
    if (like.is_contiguous()) {
      *hold = empty(like.sizes(), at::kBFloat16, like.get_device());
    } else {
      NoGil g;
      *hold = at::empty_like(like);
    }
    *x = hold;
    return true;
  }
  *x = tensor(o);
  return *x != nullptr;
}
PyObject* give(PyObject* o, const at::Tensor& made) {
  if (o != Py_None) return Py_NewRef(o);
  return THPVariable_Wrap(made);
}
PyObject* tuple(std::initializer_list<PyObject*> items) {
  PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
  Py_ssize_t i = 0;
  bool whole = t != nullptr;
  for (PyObject* x : items) {
    whole = whole && x != nullptr;
    if (t != nullptr) PyTuple_SET_ITEM(t, i++, x);
    else Py_XDECREF(x);
  }
  if (whole) return t;
  Py_XDECREF(t);
  return nullptr;
}
template <class F>
PyObject* done(F call, PyObject* outputs) {
  if (outputs == nullptr) return nullptr;
  rbs_status st;
  {
    NoGil g;
    st = call();
  }
  if (st == RBS_OK) return outputs;
  Py_DECREF(outputs);
  return PyLong_FromLong(st);
}

// A failed allocation, of Python's or torch's, ends here, before the call:
// the Python code meets the same condition and raises it in the usual form.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    PyObject* r = F(a, n);
    if (r != nullptr) return r;
  } catch (const std::exception&) {
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

// (Q, K, q_weight, k_weight, pos, theta, eps, rope_style, q_out, k_out)
PyObject* fast_rope(PyObject* const* a, Py_ssize_t n) {
  const int dev = c10::cuda::current_device();
  rbs_bf16_tensor q, k, qo, ko;
  const at::Tensor *Q = n == 10 ? tensor(a[0]) : nullptr, *K = Q ? tensor(a[1]) : nullptr, *pos = K ? tensor(a[4]) : nullptr;
  const void *wq, *wk;
  float theta, eps;
  int64_t style;
  if (pos == nullptr || !bf16(Q, dev, &q) || !bf16(K, dev, &k) || !weights(a[2], dev, q.head_dim, &wq) ||
      !weights(a[3], dev, q.head_dim, &wk) || !real(a[5], &theta) || !real(a[6], &eps) || !whole32(a[7], &style))
    return nullptr;
  const bool shared = pos->dim() == 1;
  if (shared ? !ints(pos, dev, {q.seqlen}) : !ints(pos, dev, {q.batch, q.seqlen})) return nullptr;
  at::Tensor hq, hk;
  const at::Tensor *xq, *xk;
  if (!output(a[8], *Q, &hq, &xq) || !output(a[9], *K, &hk, &xk) || !bf16(xq, dev, &qo) || !bf16(xk, dev, &ko)) return nullptr;
  PyObject* r = tuple({give(a[8], hq), give(a[9], hk)});
  return done([&] { return p_rope_qk_norm(&q, &qo, &k, &ko, wq, wk, eps, static_cast<const int32_t*>(pos->data_ptr()),
                             shared ? 0 : q.seqlen, theta, static_cast<int32_t>(style), stream(dev)); },
              r);
}

// (Q, K, V, window, sinks, q_offset, softmax_scale, out, return_lse)
PyObject* fast_swa(PyObject* const* a, Py_ssize_t n) {
  const int dev = c10::cuda::current_device();
  rbs_bf16_tensor q, k, v, o;
  int64_t window, sinks, off;
  float scale;
  bool with_lse;
  const at::Tensor* Q = n == 9 ? tensor(a[0]) : nullptr;
  if (!bf16(Q, dev, &q) || !bf16(tensor(a[1]), dev, &k) || !bf16(tensor(a[2]), dev, &v) || !whole32(a[3], &window) ||
      !whole32(a[4], &sinks) || !whole(a[5], &off) || !scale_of(a[6], q.head_dim, &scale) || !flag(a[8], &with_lse))
    return nullptr;
  at::Tensor ho, lse;
  const at::Tensor* xo;
  if (!output(a[7], *Q, &ho, &xo) || !bf16(xo, dev, &o)) return nullptr;
  if (with_lse) lse = empty({q.batch, q.heads, q.seqlen}, at::kFloat, dev);
  PyObject* r = with_lse ? tuple({give(a[7], ho), THPVariable_Wrap(lse)}) : give(a[7], ho);
  return done([&] { return p_swa_prefill(&q, &k, &v, static_cast<int32_t>(window), static_cast<int32_t>(sinks), off, scale, &o,
                            with_lse ? static_cast<float*>(lse.data_ptr()) : nullptr, stream(dev)); },
              r);
}

// (block_table, old_lens, new_lens, free_pages, free_head, max_new, page_size, slots, pos, free_head_out)
PyObject* fast_extend(PyObject* const* a, Py_ssize_t n) {
  const int dev = c10::cuda::current_device();
  const at::Tensor* t = n == 10 ? tensor(a[0]) : nullptr;
  int64_t stride, max_new, page;
  if (t == nullptr || t->dim() != 2) return nullptr;
  const int64_t B = t->size(0);
  const at::Tensor *old_lens = tensor(a[1]), *new_lens = tensor(a[2]), *free = tensor(a[3]), *head = tensor(a[4]);
  if (!table(t, dev, B, &stride) || !ints(old_lens, dev, {B}) || !ints(new_lens, dev, {B}) || free == nullptr || free->dim() != 1 ||
      !ints(free, dev, {free->size(0)}) || !ints(head, dev, {1}) || !whole32(a[5], &max_new) || max_new < 0 ||
      !whole32(a[6], &page) || B > INT32_MAX || t->size(1) > INT32_MAX)
    return nullptr;
  at::Tensor made[3];
  const at::Tensor* x[3];
  for (int i = 0; i < 3; ++i) {
    const int64_t shape[2] = {B, max_new}, one[1] = {1};
    const at::IntArrayRef want = i < 2 ? at::IntArrayRef(shape, 2) : at::IntArrayRef(one, 1);
    if (a[7 + i] == Py_None) made[i] = empty(want, at::kInt, dev);
    x[i] = a[7 + i] == Py_None ? &made[i] : tensor(a[7 + i]);
    if (!ints(x[i], dev, want)) return nullptr;
  }
  auto p = [](const at::Tensor* y) { return static_cast<int32_t*>(y->data_ptr()); };
  PyObject* r = tuple({give(a[7], made[0]), give(a[8], made[1]), give(a[9], made[2])});
  return done([&] { return p_kv4_extend(p(t), stride, static_cast<int32_t>(B), static_cast<int32_t>(t->size(1)), p(old_lens), p(new_lens),
                           p(free), free->size(0), p(head), static_cast<int32_t>(page), static_cast<int32_t>(max_new), p(x[0]),
                           p(x[1]), p(x[2]), stream(dev)); },
              r);
}

// (data, page_size, k_scale, v_scale, K, V, slots)
PyObject* fast_append(PyObject* const* a, Py_ssize_t n) {
  const int dev = c10::cuda::current_device();
  rbs_kv4_cache c;
  rbs_bf16_tensor k, v;
  if (n != 7 || !cache(a, dev, &c) || !bf16(tensor(a[4]), dev, &k) || !bf16(tensor(a[5]), dev, &v)) return nullptr;
  const at::Tensor* slots = tensor(a[6]);
  if (!ints(slots, dev, {k.batch, k.seqlen})) return nullptr;
  PyObject* r = PyLong_FromLong(RBS_OK);
  return done([&] { return p_kv4_append(&c, &k, &v, static_cast<const int32_t*>(slots->data_ptr()), stream(dev)); }, r);
}

// (data, page_size, k_scale, v_scale, slots, k_out, v_out)
PyObject* fast_load(PyObject* const* a, Py_ssize_t n) {
  const int dev = c10::cuda::current_device();
  rbs_kv4_cache c;
  rbs_bf16_tensor k, v;
  const at::Tensor* slots = n == 7 ? tensor(a[4]) : nullptr;
  if (slots == nullptr || slots->dim() != 2 || !cache(a, dev, &c)) return nullptr;
  at::Tensor made[2];
  const at::Tensor* x[2];
  for (int i = 0; i < 2; ++i) {
    if (a[5 + i] == Py_None) made[i] = empty({slots->size(0), slots->size(1), c.kv_heads, RBS_HEAD_DIM}, at::kBFloat16, dev);
    x[i] = a[5 + i] == Py_None ? &made[i] : tensor(a[5 + i]);
  }
  if (!bf16(x[0], dev, &k) || !bf16(x[1], dev, &v) || !ints(slots, dev, {k.batch, k.seqlen})) return nullptr;
  PyObject* r = tuple({give(a[5], made[0]), give(a[6], made[1])});
  return done([&] { return p_kv4_load(&c, static_cast<const int32_t*>(slots->data_ptr()), &k, &v, stream(dev)); }, r);
}

// (data, page_size, k_scale, v_scale, Q, block_table, lens, starts, window, sinks, softmax_scale, out, return_lse, workspace)
PyObject* fast_attend(PyObject* const* a, Py_ssize_t n) {
  const int dev = c10::cuda::current_device();
  rbs_kv4_cache c;
  rbs_bf16_tensor q, o;
  int64_t stride, window, sinks;
  float scale;
  bool with_lse;
  const at::Tensor* Q = n == 14 ? tensor(a[4]) : nullptr;
  if (!bf16(Q, dev, &q) || !cache(a, dev, &c)) return nullptr;
  const at::Tensor *t = tensor(a[5]), *lens = tensor(a[6]), *starts = a[7] == Py_None ? nullptr : tensor(a[7]);
  if (!table(t, dev, q.batch, &stride) || t->size(1) > INT32_MAX || !ints(lens, dev, {q.batch}) ||
      (a[7] != Py_None && !ints(starts, dev, {q.batch})) || !whole32(a[8], &window) || !whole32(a[9], &sinks) ||
      !scale_of(a[10], q.head_dim, &scale) || !flag(a[12], &with_lse))
    return nullptr;
  at::Tensor ho, lse, hw;
  const at::Tensor *xo, *ws;
  if (!output(a[11], *Q, &ho, &xo) || !bf16(xo, dev, &o)) return nullptr;
  if (with_lse) lse = empty({q.batch, q.heads, q.seqlen}, at::kFloat, dev);
  if (a[13] == Py_None)
    hw = empty({static_cast<int64_t>(p_kv4_attend_workspace_bytes(q.seqlen, q.heads, c.kv_heads))}, at::kByte, dev);
  ws = a[13] == Py_None ? &hw : tensor(a[13]);
  if (ws == nullptr || !ws->is_cuda() || ws->get_device() != dev || ws->scalar_type() != at::kByte || !ws->is_contiguous())
    return nullptr;
  PyObject* r = with_lse ? tuple({give(a[11], ho), THPVariable_Wrap(lse)}) : give(a[11], ho);
  return done([&] { return p_kv4_attend(&q, &c, static_cast<const int32_t*>(t->data_ptr()), stride, static_cast<int32_t>(t->size(1)),
                           static_cast<const int32_t*>(lens->data_ptr()),
                           starts == nullptr ? nullptr : static_cast<const int32_t*>(starts->data_ptr()),
                           static_cast<int32_t>(window), static_cast<int32_t>(sinks), scale, ws->data_ptr(),
                           static_cast<size_t>(ws->numel()), &o, with_lse ? static_cast<float*>(lse.data_ptr()) : nullptr,
                           stream(dev)); },
              r);
}

// bind(addresses of the entry points, in the order of the pointers above)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "bind takes seven addresses");
    return nullptr;
  }
  void* p[7];
  for (int i = 0; i < 7; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: null address");
      return nullptr;
    }
  }
  p_rope_qk_norm = reinterpret_cast<decltype(p_rope_qk_norm)>(p[0]);
  p_swa_prefill = reinterpret_cast<decltype(p_swa_prefill)>(p[1]);
  p_kv4_extend = reinterpret_cast<decltype(p_kv4_extend)>(p[2]);
  p_kv4_append = reinterpret_cast<decltype(p_kv4_append)>(p[3]);
  p_kv4_load = reinterpret_cast<decltype(p_kv4_load)>(p[4]);
  p_kv4_attend = reinterpret_cast<decltype(p_kv4_attend)>(p[5]);
  p_kv4_attend_workspace_bytes = reinterpret_cast<decltype(p_kv4_attend_workspace_bytes)>(p[6]);
  Py_RETURN_NONE;
}

#define RBS_FAST(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<f>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    RBS_FAST("rope_qk_norm", fast_rope),
    RBS_FAST("swa_prefill", fast_swa),
    RBS_FAST("kv4_extend", fast_extend),
    RBS_FAST("kv4_append", fast_append),
    RBS_FAST("kv4_load", fast_load),
    RBS_FAST("kv4_attend", fast_attend),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", "Marshalling of the serving calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&module); }
