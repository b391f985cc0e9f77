// Python binding of the paged-cache operators: checks of torch tensors and the
// call of the C entry point, in one C++ function per operator.
//
// Argument marshalling only; the operators are the library's, whose entry
// points paged.py hands over as addresses (init), so that this module and the
// ctypes binding share one loaded library. A serving step makes these calls
// back to back, and for small batches the host's part of a call is what it
// takes: the same checks in Python took 8 to 13 us a call, here about 1
// (decode append of 64 tokens, whole call: 15.9 us there).
//
// Every function takes its arguments in order, raises ValueError for tensors
// that do not fit, and returns its outputs, or the library's error code as an
// int where the call was refused.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <sstream>
#include <stdexcept>
#include <string>

#include "../../include/attn.h"

// The torch, C++ ABI and Python that this build is for (build.py).
#ifndef ETA_BINDING_KEY
#error "build.py compiles this file"
#endif

namespace {

struct BadArgument : std::runtime_error {
  using std::runtime_error::runtime_error;
};

template <typename... A>
[[noreturn]] void refuse(const A&... what) {
  std::ostringstream s;
  (s << ... << what);
  throw BadArgument(s.str());
}

// The library's entry points (bf16, fp16).
struct Entry {
  decltype(&attn_paged) paged[2];
  decltype(&attn_rope) rope[2];
  decltype(&attn_rope_append) append[2];
  decltype(&attn_pages_update) update;
  decltype(&attn_pages_compact) compact;
} lib = {};

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(name, " must be a tensor");
  return THPVariable_Unpack(o);
}

int integer(PyObject* o, const char* name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(name, " must be a whole number");
  }
  if (v < INT32_MIN || v > INT32_MAX) refuse(name, " is out of range");
  return static_cast<int>(v);
}

float number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(name, " must be a number");
  }
  return static_cast<float>(v);
}

bool truth(PyObject* o) { return PyObject_IsTrue(o) == 1; }

// 0: bf16, 1: fp16.
int half_type(const at::Tensor& t, const char* name) {
  const auto s = t.scalar_type();
  if (s == at::kBFloat16) return 0;
  if (s == at::kHalf) return 1;
  refuse(name, " must be bf16 or fp16");
}

int on_cuda(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(name, " must be a CUDA tensor");
  return t.get_device();
}

// A contiguous int32 tensor on device `dev` with the given sizes.
int32_t* int32_of(const at::Tensor& t, const char* name, int dev, at::IntArrayRef sizes) {
  if (t.scalar_type() != at::kInt || t.get_device() != dev || !t.sizes().equals(sizes) ||
      !t.is_contiguous())
    refuse(name, " must be a contiguous int32 tensor ", sizes, " on cuda:", dev);
  return t.data_ptr<int32_t>();
}

struct Cache {
  attn_pages c;
  int type, dev, B;
  int layers;  // 0: one layer's pool, without the dimension
  long long layer_stride;
  const at::Tensor *k, *v, *table;
};

// Pools [num_pages, Hkv, page_size, d], or with layers in front, in any strides
// with d innermost; table [B, width].
Cache cache_of(PyObject* kp, PyObject* vp, PyObject* tp) {
  Cache r;
  const at::Tensor &k = tensor(kp, "kpages"), &v = tensor(vp, "vpages"), &t = tensor(tp, "table");
  r.type = half_type(k, "kpages");
  r.dev = on_cuda(k, "kpages");
  if (v.scalar_type() != k.scalar_type() || v.get_device() != r.dev ||
      !v.sizes().equals(k.sizes()) || !v.strides().equals(k.strides()))
    refuse("vpages must have kpages' type, device, shape and strides");
  const int64_t* n = k.sizes().data();
  const int64_t* s = k.strides().data();
  const int64_t dims = k.dim();
  r.layers = 0;
  r.layer_stride = 0;
  if (dims == 5) {
    if (n[0] < 1 || n[0] > INT32_MAX) refuse("kpages must have at least one layer");
    r.layers = static_cast<int>(n[0]);
    r.layer_stride = n[0] > 1 ? s[0] : 0;
    ++n, ++s;
  }
  if ((dims != 4 && dims != 5) || (s[3] != 1 && n[3] != 1))
    refuse("kpages must be [num_pages, Hkv, page_size, d] (or with layers in front), d innermost");
  for (int i = 0; i < 4; ++i)
    if (n[i] > INT32_MAX) refuse("kpages is too large");
  if (t.scalar_type() != at::kInt || t.dim() != 2 || t.get_device() != r.dev || !t.is_contiguous() ||
      t.size(0) > INT32_MAX || t.size(1) > INT32_MAX)
    refuse("table must be a contiguous int32 tensor [B, width] on cuda:", r.dev);
  r.c.k = k.data_ptr();
  r.c.v = v.data_ptr();
  r.c.table = t.data_ptr<int32_t>();
  r.c.num_pages = static_cast<int>(n[0]);
  r.c.Hkv = static_cast<int>(n[1]);
  r.c.page_size = static_cast<int>(n[2]);
  r.c.d = static_cast<int>(n[3]);
  r.c.table_width = static_cast<int>(t.size(1));
  // A dimension of one element has no stride that matters: give it the packed one.
  r.c.token_stride = n[2] > 1 ? s[2] : n[3];
  r.c.head_stride = n[1] > 1 ? s[1] : n[2] * n[3];
  r.c.page_stride = n[0] > 1 ? s[0] : std::max<int64_t>(n[1] * n[2] * n[3], 8);
  r.B = static_cast<int>(t.size(0));
  r.k = &k;
  r.v = &v;
  r.table = &t;
  return r;
}

Cache one_layer(PyObject* kp, PyObject* vp, PyObject* tp) {
  Cache r = cache_of(kp, vp, tp);
  if (r.layers) refuse("kpages must be one layer's pool [num_pages, Hkv, page_size, d]");
  return r;
}

// Token stride of a packed tensor [tokens, heads, d] whose rows may be parts of wider ones.
long long packed(const at::Tensor& t, const char* name, const Cache& c, int64_t heads) {
  if (t.scalar_type() != c.k->scalar_type() || t.dim() != 3 || t.get_device() != c.dev)
    refuse(name, " must be a 3-D ", c.k->scalar_type(), " tensor [tokens, heads, d] on cuda:", c.dev);
  const int64_t *n = t.sizes().data(), *s = t.strides().data();
  if (n[2] != c.c.d || (heads >= 0 && n[1] != heads) || n[0] > INT32_MAX || n[1] > INT32_MAX)
    refuse(name, " must be [tokens, ", heads >= 0 ? "Hkv" : "heads", ", d] of the cache's sizes");
  if ((s[2] != 1 && n[2] > 1) || (s[1] != n[2] && n[1] > 1))
    refuse("the heads of a token of ", name, " must be contiguous");
  return n[0] > 1 ? s[0] : n[1] * n[2];
}

int rotated(const at::Tensor& turns, int dev, int64_t d) {
  if (turns.scalar_type() != at::kDouble || turns.dim() != 1 || turns.get_device() != dev ||
      !turns.is_contiguous())
    refuse("turns must be a contiguous float64 tensor [rot / 2] on cuda:", dev);
  if (2 * turns.size(0) > d) refuse("turns must have at most d / 2 entries");
  return static_cast<int>(2 * turns.size(0));
}

// The device made current, and the stream: None is the current one. A given
// stream is made current too, so that outputs allocated here come from its own
// memory: a block of the current stream's may have been freed there while work
// queued on that stream still uses it, which the given one does not wait for.
struct Place {
  c10::cuda::OptionalCUDAGuard guard;
  c10::cuda::CUDAStream before;
  c10::cuda::OptionalCUDAStreamGuard on;
  attn_stream_t stream;
  bool given;
  Place(int dev, PyObject* s)
      : guard(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev))),
        before(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev))),
        given(s != Py_None) {
    stream = reinterpret_cast<attn_stream_t>(before.stream());
    if (!given) return;
    const unsigned long long handle = PyLong_AsUnsignedLongLong(s);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      refuse("stream must be a stream or its handle");
    }
    stream = reinterpret_cast<attn_stream_t>(handle);
    on.reset_stream(c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(handle),
                                                     static_cast<c10::DeviceIndex>(dev)));
  }
  // A tensor allocated here for a caller on the stream that was current: its
  // memory is not handed out again before that stream's work with it is done.
  void allocated(const at::Tensor& t) const {
    if (given && t.defined()) t.record_stream(before.unwrap());
  }
};

template <typename F, typename... A>
int call(F f, A... args) {
  int code;
  Py_BEGIN_ALLOW_THREADS;
  code = f(args...);
  Py_END_ALLOW_THREADS;
  return code;
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

PyObject* give(std::initializer_list<PyObject*> out) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(out.size()));
  Py_ssize_t i = 0;
  for (PyObject* o : out) PyTuple_SET_ITEM(r, i++, o);
  return r;
}

PyObject* again(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// A tensor that the call writes in place: autograd's count of its versions moves
// on, so that a graph that saved it finds out. (Inference tensors have none.)
void written(const at::Tensor& t) {
  if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// An output: the one given (checked by the caller), or a new tensor.
struct Out {
  at::Tensor t;
  PyObject* given;  // borrowed, or NULL
  PyObject* result() const { return given ? again(given) : wrap(t); }
  void keep(const Place& place) const {
    if (given)
      written(t);
    else
      place.allocated(t);
  }
};

Out int32_out(PyObject* o, const char* name, const at::Tensor& like, int dev, at::IntArrayRef sizes) {
  if (o == Py_None) return {at::empty(sizes, like.options().dtype(at::kInt)), nullptr};
  int32_of(tensor(o, name), name, dev, sizes);
  return {tensor(o, name), o};
}

// (q, kpages, vpages, table, cu_q, kv_lens, max_q, window, scale, o, lse, want_lse, stream)
PyObject* paged(PyObject* const* a) {
  const Cache c = one_layer(a[1], a[2], a[3]);
  const at::Tensor& q = tensor(a[0], "q");
  const long long stride = packed(q, "q", c, -1);
  const int total = static_cast<int>(q.size(0)), Hq = static_cast<int>(q.size(1));
  const int32_t* cu = int32_of(tensor(a[4], "cu_q"), "cu_q", c.dev, {c.B + 1});
  const int32_t* lens = int32_of(tensor(a[5], "kv_lens"), "kv_lens", c.dev, {c.B});
  const int max_q = a[6] == Py_None ? total : integer(a[6], "max_q");
  const int window = integer(a[7], "window");
  const float scale = a[8] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(c.c.d)))
                                      : number(a[8], "scale");
  Place place(c.dev, a[12]);
  Out o{{}, nullptr}, lse{{}, nullptr};
  if (a[9] == Py_None) {
    o.t = at::empty(q.sizes(), q.options());
  } else {
    o.given = a[9];
    o.t = tensor(a[9], "o");
    if (o.t.scalar_type() != q.scalar_type() || o.t.get_device() != c.dev ||
        !o.t.sizes().equals(q.sizes()) || !o.t.is_contiguous())
      refuse("o must be a contiguous tensor of q's shape, type and device");
  }
  if (a[10] != Py_None) {
    lse.given = a[10];
    lse.t = tensor(a[10], "lse");
    if (lse.t.scalar_type() != at::kFloat || lse.t.get_device() != c.dev ||
        !lse.t.sizes().equals({total, Hq}) || !lse.t.is_contiguous())
      refuse("lse must be a contiguous float32 tensor [total, Hq] on q's device");
  } else if (truth(a[11])) {
    lse.t = at::empty({total, Hq}, q.options().dtype(at::kFloat));
  }
  float* lse_p = lse.t.defined() ? lse.t.data_ptr<float>() : nullptr;
  const int code = call(lib.paged[c.type], q.data_ptr(), stride, &c.c, cu, lens, o.t.data_ptr(), lse_p,
                        c.B, Hq, total, max_q, scale, window, place.stream);
  if (code != ATTN_OK) return PyLong_FromLong(code);
  o.keep(place);
  lse.keep(place);
  return give({o.result(), lse.t.defined() ? lse.result() : again(Py_None)});
}

// Batch, head and token strides of [B, H, N, d] (0 where a dimension has one element).
void strides3(const at::Tensor& t, long long* out) {
  const int64_t *n = t.sizes().data(), *s = t.strides().data();
  if (s[3] != 1 && n[3] > 1)
    refuse("the last dimension of q, k and the outputs must be contiguous");
  for (int i = 0; i < 3; ++i) out[i] = n[i] > 1 ? s[i] : 0;
}

Out like(PyObject* o, const at::Tensor& x) {
  if (o == Py_None) return {at::empty_like(x), nullptr};
  const at::Tensor& t = tensor(o, "an output");
  if (!t.sizes().equals(x.sizes()) || t.scalar_type() != x.scalar_type() ||
      t.get_device() != x.get_device())
    refuse("an output must have its input's shape, type and device");
  return {t, o};
}

// (q, k, pos, turns, amp, interleaved, q_out, k_out, backward, stream)
PyObject* rope(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q");
  const int type = half_type(q, "q"), dev = on_cuda(q, "q");
  if (q.dim() != 4) refuse("q must be a 4-D tensor [B, H, N, d]");
  const int64_t B = q.size(0), N = q.size(2), d = q.size(3);
  for (int i = 0; i < 4; ++i)
    if (q.size(i) > INT32_MAX) refuse("q is too large");
  const at::Tensor* k = nullptr;
  if (a[1] != Py_None) {
    k = &tensor(a[1], "k");
    if (k->dim() != 4 || k->scalar_type() != q.scalar_type() || k->get_device() != dev ||
        k->size(0) != B || k->size(2) != N || k->size(3) != d || k->size(1) > INT32_MAX)
      refuse("k must be [B, Hkv, N, d] of q's B, N, d, type and device");
  } else if (a[7] != Py_None) {
    refuse("k_out without k");
  }
  const at::Tensor& pos = tensor(a[2], "pos");
  const bool own = pos.dim() == 2;
  if (pos.scalar_type() != at::kInt || pos.get_device() != dev || !pos.is_contiguous() ||
      !(pos.sizes().equals({N}) || pos.sizes().equals({B, N})))
    refuse("pos must be a contiguous int32 tensor [N] or [B, N] on cuda:", dev);
  const at::Tensor& turns = tensor(a[3], "turns");
  const int rot = rotated(turns, dev, d);
  const float amp = number(a[4], "amp");
  Place place(dev, a[9]);
  Out qo = like(a[6], q), ko{{}, nullptr};
  long long s[12] = {};
  strides3(q, s);
  strides3(qo.t, s + 3);
  if (k) {
    ko = like(a[7], *k);
    strides3(*k, s + 6);
    strides3(ko.t, s + 9);
  }
  const int code =
      call(lib.rope[type], q.data_ptr(), qo.t.data_ptr(), k ? k->data_ptr() : nullptr,
           k ? ko.t.data_ptr() : nullptr, s, pos.data_ptr<int32_t>(), own ? N : 0LL,
           turns.data_ptr<double>(), static_cast<int>(B), static_cast<int>(q.size(1)),
           k ? static_cast<int>(k->size(1)) : 0, static_cast<int>(N), static_cast<int>(d), rot, amp,
           truth(a[5]) ? 1 : 0, truth(a[8]) ? 1 : 0, place.stream);
  if (code != ATTN_OK) return PyLong_FromLong(code);
  qo.keep(place);
  ko.keep(place);
  return give({qo.result(), k ? ko.result() : again(Py_None)});
}

// (q, k, v, kpages, vpages, table, cu_q, kv_lens, turns, amp, interleaved, pos, q_out, stream)
PyObject* append(PyObject* const* a) {
  const Cache c = one_layer(a[3], a[4], a[5]);
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
  const long long qs = packed(q, "q", c, -1), ks = packed(k, "k", c, c.c.Hkv),
                  vs = packed(v, "v", c, c.c.Hkv);
  const int total = static_cast<int>(q.size(0)), Hq = static_cast<int>(q.size(1));
  if (k.size(0) != total || v.size(0) != total) refuse("q, k and v must have the same tokens");
  const int32_t* cu = int32_of(tensor(a[6], "cu_q"), "cu_q", c.dev, {c.B + 1});
  const int32_t* lens = int32_of(tensor(a[7], "kv_lens"), "kv_lens", c.dev, {c.B});
  const at::Tensor& turns = tensor(a[8], "turns");
  const int rot = rotated(turns, c.dev, c.c.d);
  const float amp = number(a[9], "amp");
  const int32_t* pos =
      a[11] == Py_None ? nullptr : int32_of(tensor(a[11], "pos"), "pos", c.dev, {total});
  Place place(c.dev, a[13]);
  Out o{{}, nullptr};
  if (a[12] == Py_None) {
    o.t = at::empty(q.sizes(), q.options());
  } else {
    o.given = a[12];
    o.t = tensor(a[12], "q_out");
    if (!o.t.sizes().equals(q.sizes())) refuse("q_out must have q's shape");
  }
  const long long os = packed(o.t, "q_out", c, -1);
  const int code = call(lib.append[c.type], q.data_ptr(), qs, o.t.data_ptr(), os, k.data_ptr(), ks,
                        v.data_ptr(), vs, &c.c, cu, lens, pos, turns.data_ptr<double>(), c.B, Hq,
                        total, rot, amp, truth(a[10]) ? 1 : 0, place.stream);
  if (code != ATTN_OK) return PyLong_FromLong(code);
  written(*c.k);
  written(*c.v);
  o.keep(place);
  return o.result();
}

// (kpages, vpages, table, lens, refs, source, add, table_out, lens_out, refs_out, info, stream)
PyObject* update(PyObject* const* a) {
  const Cache c = cache_of(a[0], a[1], a[2]);
  const at::Tensor& lens = tensor(a[3], "lens");
  const int32_t* lens_p = int32_of(lens, "lens", c.dev, {c.B});
  const int32_t* refs_p = int32_of(tensor(a[4], "refs"), "refs", c.dev, {c.c.num_pages});
  const int32_t* source = int32_of(tensor(a[5], "source"), "source", c.dev, {c.B});
  const int32_t* add = int32_of(tensor(a[6], "add"), "add", c.dev, {c.B});
  Place place(c.dev, a[11]);
  const Out t = int32_out(a[7], "table_out", lens, c.dev, {c.B, c.c.table_width});
  const Out l = int32_out(a[8], "lens_out", lens, c.dev, {c.B});
  const Out r = int32_out(a[9], "refs_out", lens, c.dev, {c.c.num_pages});
  const Out info = int32_out(a[10], "info", lens, c.dev, {2});
  const int code = call(lib.update, &c.c, c.layers ? c.layers : 1, c.layer_stride, lens_p, refs_p,
                        source, add, t.t.data_ptr<int32_t>(), l.t.data_ptr<int32_t>(),
                        r.t.data_ptr<int32_t>(), info.t.data_ptr<int32_t>(), c.B, place.stream);
  if (code != ATTN_OK) return PyLong_FromLong(code);
  written(*c.k);
  written(*c.v);
  for (const Out* x : {&t, &l, &r, &info}) x->keep(place);
  return give({t.result(), l.result(), r.result(), info.result()});
}

// (kpages, vpages, table, lens, refs, table_out, refs_out, info, stream)
PyObject* compact(PyObject* const* a) {
  const Cache c = cache_of(a[0], a[1], a[2]);
  const at::Tensor& lens = tensor(a[3], "lens");
  const int32_t* lens_p = int32_of(lens, "lens", c.dev, {c.B});
  const int32_t* refs_p = int32_of(tensor(a[4], "refs"), "refs", c.dev, {c.c.num_pages});
  Place place(c.dev, a[8]);
  const Out t = int32_out(a[5], "table_out", lens, c.dev, {c.B, c.c.table_width});
  const Out r = int32_out(a[6], "refs_out", lens, c.dev, {c.c.num_pages});
  const Out info = int32_out(a[7], "info", lens, c.dev, {2});
  const int code = call(lib.compact, &c.c, c.layers ? c.layers : 1, c.layer_stride, lens_p, refs_p,
                        t.t.data_ptr<int32_t>(), r.t.data_ptr<int32_t>(),
                        info.t.data_ptr<int32_t>(), c.B, place.stream);
  if (code != ATTN_OK) return PyLong_FromLong(code);
  written(*c.k);
  written(*c.v);
  for (const Out* x : {&t, &r, &info}) x->keep(place);
  return give({t.result(), r.result(), info.result()});
}

// Runs F on the arguments; C++ exceptions become Python's.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const BadArgument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (paged, paged_f16, rope, rope_f16, append, append_f16, update, compact): addresses.
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "expected 8 addresses");
    return nullptr;
  }
  void* p[8];
  for (int i = 0; i < 8; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an entry point has no address");
      return nullptr;
    }
  }
  for (int i = 0; i < 2; ++i) {
    lib.paged[i] = reinterpret_cast<decltype(&attn_paged)>(p[i]);
    lib.rope[i] = reinterpret_cast<decltype(&attn_rope)>(p[2 + i]);
    lib.append[i] = reinterpret_cast<decltype(&attn_rope_append)>(p[4 + i]);
  }
  lib.update = reinterpret_cast<decltype(&attn_pages_update)>(p[6]);
  lib.compact = reinterpret_cast<decltype(&attn_pages_compact)>(p[7]);
  Py_RETURN_NONE;
}

#define ETA_METHOD(name, n) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<name, n>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    {"init", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&init)), METH_FASTCALL, nullptr},
    ETA_METHOD(paged, 13),
    ETA_METHOD(rope, 10),
    ETA_METHOD(append, 14),
    ETA_METHOD(update, 12),
    ETA_METHOD(compact, 9),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "built_for", ETA_BINDING_KEY) != 0) {
    Py_DECREF(m);
    m = nullptr;
  }
  return m;
}
