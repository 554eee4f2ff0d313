// Marshalling of the calls around a layer's products (norm, routing, rotary,
// cache, attention): the checks of the tensors, the outputs and the call into libhum, as one native call.
//
// A decode step makes these calls once per layer with little work in each, so
// the host side is what a small one costs: marshalled in Python a call took
// 9 to 10 us (two of them for the outputs, three to four for the launch),
// here half of that.  The public functions are those of the Python module,
// which documents them; nothing is computed here.
#include <hip/hip_runtime_api.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>

#include <cmath>

#include "hum.h"

namespace {

PyObject* g_hum_error = nullptr;   // HumError(status, message)
PyObject* g_raw_stream = nullptr;  // device number -> its current stream
PyObject* g_workspace = nullptr;   // (device number, bytes) -> scratch of a call
PyObject* g_workspaces = nullptr;  // {(device number, stream): Workspace}

// A Python exception, set and thrown.
template <typename... A>
[[noreturn]] void fail(const char* format, A... args) {
  PyErr_Format(PyExc_ValueError, format, args...);
  throw python_error();
}

const char* dtype_name(at::ScalarType t) {
  switch (t) {
    case at::kByte: return "torch.uint8";
    case at::kChar: return "torch.int8";
    case at::kShort: return "torch.int16";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kHalf: return "torch.float16";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kDouble: return "torch.float64";
    default: return c10::toString(t);
  }
}

// The tensor behind an argument; None is an error, or null where it may be.
const at::Tensor* maybe(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) fail("%s must be a tensor", name);
  return &THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o, const char* name, int dims, const char* what) {
  const at::Tensor* t = maybe(o, name);
  if (!t || t->dim() != dims) fail("%s must be a %d-D tensor %s", name, dims, what);
  return *t;
}

void want_dtype(const at::Tensor& t, const char* name, at::ScalarType dt) {
  if (t.scalar_type() != dt) fail("%s must be %s, got %s", name, dtype_name(dt), dtype_name(t.scalar_type()));
  if (t.is_neg()) fail("%s must hold its values (a negated view does not: resolve_neg())", name);
}

// A [rows, heads, dim] tensor of the given shape and type; rows and heads may
// be strided (a slice of a fused qkv product).
void want_rows(const at::Tensor& t, const char* name, at::ScalarType dt, int64_t n, int64_t h, int64_t d) {
  want_dtype(t, name, dt);
  if (t.dim() != 3 || t.size(0) != n || t.size(1) != h || t.size(2) != d)
    fail("%s must have shape (%lld, %lld, %lld)", name, (long long)n, (long long)h, (long long)d);
  if (d > 1 && t.stride(2) != 1) fail("%s's head elements must be contiguous", name);
}
void want_contiguous(const at::Tensor& t, const char* name) {
  if (!t.is_contiguous()) fail("%s must be contiguous", name);
}
// An output that the caller gives must not hold two of its elements at one address.
void want_spread(const at::Tensor& t, const char* name) {
  for (int64_t i = 0; i < t.dim(); ++i)
    if (t.size(i) > 1 && t.stride(i) == 0 && t.numel()) fail("%s must not be expanded (stride 0)", name);
}
// A contiguous 1-D tensor of n elements.
void want_vec(const at::Tensor* t, const char* name, at::ScalarType dt, int64_t n) {
  if (!t) fail("%s must be a tensor", name);
  want_dtype(*t, name, dt);
  if (t->dim() != 1 || t->size(0) != n) fail("%s must have shape (%lld,)", name, (long long)n);
  if (n > 1 && t->stride(0) != 1) fail("%s must be contiguous", name);
}
void want_cache(const at::Tensor* t) {
  if (!t || t->scalar_type() != at::kByte || !t->is_contiguous()) fail("cache must be a contiguous uint8 tensor");
}

// The number of the GPU that every tensor is on.
int device_of(const char* name, std::initializer_list<const at::Tensor*> ts) {
  const at::Device d = (*ts.begin())->device();
  for (const at::Tensor* t : ts)
    if (t && t->device() != d) fail("tensors on different devices: %s and %s", d.str().c_str(), t->device().str().c_str());
  if (!d.is_cuda()) fail("%s must be a device tensor", name);
  return d.index();
}

// A description: a ctypes structure of the C type's size.
template <typename T>
const T* desc_of(PyObject* o, Py_buffer* view) {
  if (PyObject_GetBuffer(o, view, PyBUF_SIMPLE) != 0) throw python_error();
  if (view->len != (Py_ssize_t)sizeof(T)) {
    PyBuffer_Release(view);
    fail("desc must be a KvDesc");
  }
  return static_cast<const T*>(view->buf);
}
struct KvDesc {
  Py_buffer view;
  const hum_kv_desc* d;
  explicit KvDesc(PyObject* o) : d(desc_of<hum_kv_desc>(o, &view)) {}
  ~KvDesc() { PyBuffer_Release(&view); }
  const hum_kv_desc* operator->() const { return d; }
};

[[noreturn]] void raise_status(int status) {
  PyObject* e = PyObject_CallFunction(g_hum_error, "is", status, hum_last_error());
  if (e) {
    PyErr_SetObject(g_hum_error, e);
    Py_DECREF(e);
  }
  throw python_error();
}

// Makes a GPU current, as every call needs, and the caller's again.
struct DeviceGuard {
  int before = -1, dev;
  explicit DeviceGuard(int d) : dev(d) {
    if (hipGetDevice(&before) != hipSuccess) before = d;
    if (before != dev) (void)hipSetDevice(dev);
  }
  ~DeviceGuard() {
    if (before != dev) (void)hipSetDevice(before);
  }
};

struct Ref {
  PyObject* o;
  explicit Ref(PyObject* p) : o(p) {
    if (!o) throw python_error();
  }
  ~Ref() { Py_DECREF(o); }
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
};

void* stream_of(int dev) {
  const Ref d(PyLong_FromLong(dev));
  const Ref s(PyObject_CallOneArg(g_raw_stream, d.o));
  return PyLong_AsVoidPtr(s.o);
}

long long whole(PyObject* o, const char* name) {
  const Ref i(PyNumber_Index(o));
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(i.o, &over);
  if (over) fail("%s is out of range", name);
  return v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}
void want_args(Py_ssize_t n, Py_ssize_t expected) {
  if (n != expected) fail("expected %zd arguments", expected);
}

PyObject* pair(const at::Tensor& a, PyObject* a_given, const at::Tensor* b, PyObject* b_given) {
  auto wrap = [](const at::Tensor* t, PyObject* given) -> PyObject* {
    if (given == Py_None && t) return THPVariable_Wrap(*t);
    Py_INCREF(given);
    return given;
  };
  const Ref x(wrap(&a, a_given)), y(wrap(b, b_given));
  return PyTuple_Pack(2, x.o, y.o);
}

// rotary(q, k, positions, inv_freq, layout, factor, inverse, q_out, k_out)
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want_args(n, 9);
  const char* heads = "[T, heads, head_dim]";
  const at::Tensor& q = tensor(a[0], "q", 3, heads);
  const at::Tensor* k = a[1] == Py_None ? nullptr : &tensor(a[1], "k", 3, heads);
  const at::ScalarType dt = q.scalar_type();
  if (dt != at::kBFloat16 && dt != at::kFloat) fail("q must be torch.bfloat16 or torch.float32, got %s", dtype_name(dt));
  const int64_t t = q.size(0), hq = q.size(1), d = q.size(2), hk = k ? k->size(1) : 0;
  want_rows(q, "q", dt, t, hq, d);
  if (k) want_rows(*k, "k", dt, t, hk, d);
  const at::Tensor* pos = maybe(a[2], "positions");
  want_vec(pos, "positions", at::kLong, t);
  const at::Tensor& freq = tensor(a[3], "inv_freq", 1, "of float64");
  const int64_t half = freq.size(0);
  want_vec(&freq, "inv_freq", at::kDouble, half);
  const at::Tensor *qo = maybe(a[7], "q_out"), *ko = maybe(a[8], "k_out");
  if (ko && !k) fail("k_out without k");
  if (qo) {
    want_rows(*qo, "q_out", dt, t, hq, d);
    want_spread(*qo, "q_out");
  }
  if (ko) {
    want_rows(*ko, "k_out", dt, t, hk, d);
    want_spread(*ko, "k_out");
  }
  const int dev = device_of("q", {&q, k, pos, &freq, qo, ko});
  hum_rotary_desc desc{};
  desc.dtype = dt == at::kFloat ? HUM_F32 : HUM_BF16;
  desc.layout = (int32_t)whole(a[4], "layout");
  desc.head_dim = (int32_t)(d < INT32_MAX ? d : INT32_MAX);
  desc.rotary_dim = (int32_t)(half < INT32_MAX / 2 ? 2 * half : INT32_MAX - 1);
  desc.num_q_heads = (int32_t)(hq < INT32_MAX ? hq : INT32_MAX);
  desc.num_kv_heads = (int32_t)(hk < INT32_MAX ? hk : INT32_MAX);
  desc.factor = (float)real(a[5]);
  desc.inverse = truth(a[6]);
  at::Tensor q_new, k_new;
  if (!qo) {
    q_new = at::empty({t, hq, d}, q.options());
    qo = &q_new;
  }
  if (k && !ko) {
    k_new = at::empty({t, hk, d}, k->options());
    ko = &k_new;
  }
  const DeviceGuard guard(dev);
  const hum_status st = hum_rotary(
      &desc, t, static_cast<const int64_t*>(pos->data_ptr()), static_cast<const double*>(freq.data_ptr()), q.data_ptr(),
      q.stride(0), q.stride(1), qo->data_ptr(), qo->stride(0), qo->stride(1), k ? k->data_ptr() : nullptr,
      k ? k->stride(0) : 0, k ? k->stride(1) : 0, k ? ko->data_ptr() : nullptr, k ? ko->stride(0) : 0,
      k ? ko->stride(1) : 0, stream_of(dev));
  if (st != HUM_OK) raise_status(st);
  return pair(*qo, a[7], ko, a[8]);
  END_HANDLE_TH_ERRORS
}

// kv_write(desc, cache, k, v, slots)
PyObject* kv_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want_args(n, 5);
  const KvDesc desc(a[0]);
  const at::Tensor* cache = maybe(a[1], "cache");
  want_cache(cache);
  const char* shape = "[T, num_kv_heads, head_dim]";
  const at::Tensor &k = tensor(a[2], "k", 3, shape), &v = tensor(a[3], "v", 3, shape);
  const int64_t t = k.size(0);
  want_rows(k, "k", at::kBFloat16, t, desc->num_kv_heads, desc->head_dim);
  want_rows(v, "v", at::kBFloat16, t, desc->num_kv_heads, desc->head_dim);
  const at::Tensor* slots = maybe(a[4], "slots");
  want_vec(slots, "slots", at::kLong, t);
  const int dev = device_of("cache", {cache, &k, &v, slots});
  const DeviceGuard guard(dev);
  const hum_status st = hum_kv_write(desc.d, cache->data_ptr(), (size_t)cache->numel(), t,
                                     static_cast<const int64_t*>(slots->data_ptr()), k.data_ptr(), k.stride(0),
                                     k.stride(1), v.data_ptr(), v.stride(0), v.stride(1), stream_of(dev));
  if (st != HUM_OK) raise_status(st);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// kv_read(desc, cache, slots, k_out, v_out)
PyObject* kv_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want_args(n, 5);
  const KvDesc desc(a[0]);
  const at::Tensor* cache = maybe(a[1], "cache");
  want_cache(cache);
  const at::Tensor& slots = tensor(a[2], "slots", 1, "of int64");
  const int64_t t = slots.size(0);
  want_vec(&slots, "slots", at::kLong, t);
  const at::Tensor* out[2] = {maybe(a[3], "k_out"), maybe(a[4], "v_out")};
  const char* names[2] = {"k_out", "v_out"};
  for (int i = 0; i < 2; ++i) {
    if (!out[i]) continue;
    want_rows(*out[i], names[i], at::kBFloat16, t, desc->num_kv_heads, desc->head_dim);
    want_contiguous(*out[i], names[i]);
  }
  const int dev = device_of("cache", {cache, &slots, out[0], out[1]});
  if (!hum_kv_cache_bytes(desc.d)) raise_status(HUM_ERR_UNSUPPORTED);
  at::Tensor fresh[2];
  for (int i = 0; i < 2; ++i) {
    if (out[i]) continue;
    fresh[i] = at::empty({t, desc->num_kv_heads, desc->head_dim}, cache->options().dtype(at::kBFloat16));
    out[i] = &fresh[i];
  }
  const DeviceGuard guard(dev);
  const hum_status st = hum_kv_read(desc.d, cache->data_ptr(), (size_t)cache->numel(), t,
                                    static_cast<const int64_t*>(slots.data_ptr()), out[0]->data_ptr(),
                                    out[1]->data_ptr(), stream_of(dev));
  if (st != HUM_OK) raise_status(st);
  return pair(*out[0], a[3], out[1], a[4]);
  END_HANDLE_TH_ERRORS
}

// Scratch of one call: the stream's own, if it is there and large enough and
// the stream is not being captured; otherwise what the Python side decides.
at::Tensor scratch(int dev, void* stream, size_t need) {
  hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
  if (hipStreamIsCapturing(static_cast<hipStream_t>(stream), &capture) == hipSuccess &&
      capture == hipStreamCaptureStatusNone) {
    const Ref key(Py_BuildValue("(iN)", dev, PyLong_FromVoidPtr(stream)));
    PyObject* ws = PyDict_GetItemWithError(g_workspaces, key.o);
    if (ws) {
      const Ref buf(PyObject_GetAttrString(ws, "buf"));
      if (THPVariable_Check(buf.o) && (size_t)THPVariable_Unpack(buf.o).numel() >= need)
        return THPVariable_Unpack(buf.o);
    } else if (PyErr_Occurred()) {
      throw python_error();
    }
  }
  const Ref t(PyObject_CallFunction(g_workspace, "iK", dev, (unsigned long long)need));
  return THPVariable_Unpack(t.o);
}

// kv_attention(desc, cache, q, block_table, seq_lens, scale, window, out, return_lse, workspace)
PyObject* kv_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want_args(n, 10);
  const KvDesc desc(a[0]);
  const at::Tensor* cache = maybe(a[1], "cache");
  want_cache(cache);
  const at::Tensor& q = tensor(a[2], "q", 3, "[B, num_q_heads, head_dim]");
  const int64_t b = q.size(0), hq = q.size(1), d = desc->head_dim;
  want_rows(q, "q", at::kBFloat16, b, hq, d);
  if (hq > INT32_MAX) fail("q has too many heads");
  const at::Tensor& table = tensor(a[3], "block_table", 2, "[B, max_pages]");
  const int64_t pages = table.size(1);
  if (table.size(0) != b) fail("block_table must have one row per sequence");
  want_dtype(table, "block_table", at::kInt);
  if (pages > 1 && table.stride(1) != 1) fail("block_table's rows must be contiguous");
  const at::Tensor* lens = maybe(a[4], "seq_lens");
  want_vec(lens, "seq_lens", at::kInt, b);
  const at::Tensor *out = maybe(a[7], "out"), *ws = maybe(a[9], "workspace");
  if (out) {
    want_rows(*out, "out", at::kBFloat16, b, hq, d);
    want_contiguous(*out, "out");
  }
  if (ws) {
    want_dtype(*ws, "workspace", at::kByte);
    want_contiguous(*ws, "workspace");
  }
  const int dev = device_of("cache", {cache, &q, &table, lens, out, ws});
  const size_t need = hum_kv_attention_workspace_bytes(desc.d, (int32_t)hq, b, pages);
  if (!need) raise_status(HUM_ERR_INVALID_ARG);
  const DeviceGuard guard(dev);
  void* stream = stream_of(dev);
  at::Tensor own, fresh, lse;
  if (!ws) {
    own = scratch(dev, stream, need);
    ws = &own;
  }
  if (!out) {
    fresh = at::empty({b, hq, d}, q.options());
    out = &fresh;
  }
  const double scale = a[5] == Py_None ? 1.0 / std::sqrt((double)d) : real(a[5]);
  const bool with_lse = truth(a[8]);
  if (with_lse) lse = at::empty({b, hq}, q.options().dtype(at::kFloat));
  const hum_status st = hum_kv_attention(
      desc.d, cache->data_ptr(), (size_t)cache->numel(), (int32_t)hq, b, q.data_ptr(), q.stride(0), q.stride(1),
      static_cast<const int32_t*>(table.data_ptr()), table.stride(0), pages,
      static_cast<const int32_t*>(lens->data_ptr()), whole(a[6], "window"), (float)scale, out->data_ptr(),
      with_lse ? static_cast<float*>(lse.data_ptr()) : nullptr, ws->data_ptr(), (size_t)ws->numel(), stream);
  if (st != HUM_OK) raise_status(st);
  if (with_lse) return pair(*out, a[7], &lse, Py_None);
  if (a[7] == Py_None) return THPVariable_Wrap(*out);
  Py_INCREF(a[7]);
  return a[7];
  END_HANDLE_TH_ERRORS
}

// A [rows, elements] tensor whose elements are contiguous; rows may be strided.
void want_matrix(const at::Tensor& t, const char* name, int64_t n, int64_t k) {
  if (t.is_neg()) fail("%s must hold its values (a negated view does not: resolve_neg())", name);
  if (t.dim() != 2 || t.size(0) != n || t.size(1) != k) fail("%s must have shape (%lld, %lld)", name, (long long)n, (long long)k);
  if (k > 1 && t.stride(1) != 1) fail("%s's rows must be contiguous", name);
}
void want_float(const at::Tensor& t, const char* name) {
  if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat)
    fail("%s must be torch.bfloat16 or torch.float32, got %s", name, dtype_name(t.scalar_type()));
}
int32_t hum_dtype_of(const at::Tensor& t) { return t.scalar_type() == at::kFloat ? HUM_F32 : HUM_BF16; }
int32_t whole32(PyObject* o, const char* name) {
  const long long v = whole(o, name);
  if (v < INT32_MIN || v > INT32_MAX) fail("%s is out of range", name);
  return (int32_t)v;
}
PyObject* given_or(const at::Tensor& t, PyObject* given) {
  if (given == Py_None) return THPVariable_Wrap(t);
  Py_INCREF(given);
  return given;
}

// rms_norm(x, weight, eps, residual, act_fmt, weight_offset, residual_out, out, with_bf16)
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want_args(n, 9);
  const at::Tensor& x = tensor(a[0], "x", 2, "[m, k]");
  const int64_t m = x.size(0), k = x.size(1);
  want_dtype(x, "x", at::kBFloat16);
  want_matrix(x, "x", m, k);
  const at::Tensor& w = tensor(a[1], "weight", 1, "[k]");
  want_float(w, "weight");
  want_vec(&w, "weight", w.scalar_type(), k);
  const at::Tensor *res = maybe(a[3], "residual"), *res_out = maybe(a[6], "residual_out"), *out = maybe(a[7], "out");
  if (res) {
    want_float(*res, "residual");
    want_matrix(*res, "residual", m, k);
  }
  if (res_out) {
    if (!res) fail("residual_out without residual");
    want_dtype(*res_out, "residual_out", res->scalar_type());
    want_matrix(*res_out, "residual_out", m, k);
    want_spread(*res_out, "residual_out");
  }
  if (PyUnicode_Check(a[4])) fail("act_fmt must be bf16, fp8_token, mxfp8, mxfp4 or fp8_group");
  const int32_t fmt = whole32(a[4], "act_fmt");
  if (fmt < HUM_ACT_BF16 || fmt > HUM_ACT_FP8_GROUP) fail("act_fmt must be bf16, fp8_token, mxfp8, mxfp4 or fp8_group");
  const bool quant = fmt != HUM_ACT_BF16, with_bf16 = truth(a[8]);
  if (out) {
    if (quant && !with_bf16) fail("out is of the bf16 result: give with_bf16 too");
    want_dtype(*out, "out", at::kBFloat16);
    want_matrix(*out, "out", m, k);
    want_spread(*out, "out");
  }
  const int dev = device_of("x", {&x, &w, res, res_out, out});
  const int64_t unit = fmt == HUM_ACT_FP8_TOKEN ? 8 : fmt == HUM_ACT_FP8_GROUP ? 128 : quant ? 32 : 1;
  if (k < 1 || k % unit) fail("x must have a multiple of %lld columns", (long long)unit);
  hum_norm_desc desc{};
  desc.act_fmt = fmt;
  desc.residual_dtype = res ? hum_dtype_of(*res) : HUM_BF16;
  desc.weight_dtype = hum_dtype_of(w);
  desc.eps = (float)real(a[2]);
  desc.weight_offset = (float)real(a[5]);
  at::Tensor q, scales, fresh, fresh_res;
  if (quant) {
    const auto bytes = x.options().dtype(at::kByte);
    const auto f32 = x.options().dtype(at::kFloat);
    q = at::empty({m, fmt == HUM_ACT_MXFP4 ? k / 2 : k}, bytes);
    scales = fmt == HUM_ACT_FP8_TOKEN ? at::empty({m}, f32) : fmt == HUM_ACT_FP8_GROUP ? at::empty({m, k / 128}, f32) : at::empty({m, k / 32}, bytes);
  }
  if (!out && (!quant || with_bf16)) {
    fresh = at::empty({m, k}, x.options());
    out = &fresh;
  }
  if (res && !res_out) {
    fresh_res = at::empty({m, k}, res->options());
    res_out = &fresh_res;
  }
  const DeviceGuard guard(dev);
  const hum_status st = hum_rms_norm(
      &desc, m, k, x.data_ptr(), x.stride(0), res ? res->data_ptr() : nullptr, res ? res->stride(0) : 0,
      res ? res_out->data_ptr() : nullptr, res ? res_out->stride(0) : 0, w.data_ptr(), out ? out->data_ptr() : nullptr,
      out ? out->stride(0) : 0, quant ? q.data_ptr() : nullptr, quant ? scales.data_ptr() : nullptr, stream_of(dev));
  if (st != HUM_OK) raise_status(st);
  PyObject* y;
  if (!quant) {
    y = given_or(*out, a[7]);
  } else {
    const Ref c(THPVariable_Wrap(q)), s(THPVariable_Wrap(scales));
    if (with_bf16) {
      const Ref b(given_or(*out, a[7]));
      y = PyTuple_Pack(3, c.o, s.o, b.o);
    } else {
      y = PyTuple_Pack(2, c.o, s.o);
    }
  }
  if (!res) return y;
  const Ref yr(y), rr(given_or(*res_out, a[6]));
  return PyTuple_Pack(2, yr.o, rr.o);
  END_HANDLE_TH_ERRORS
}

// moe_route(logits, topk, score, bias, num_groups, topk_groups, group_score, renormalize, scale, topk_ids, topk_weights)
PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want_args(n, 11);
  const at::Tensor& x = tensor(a[0], "logits", 2, "[T, E]");
  const int64_t t = x.size(0), e = x.size(1);
  want_float(x, "logits");
  want_matrix(x, "logits", t, e);
  hum_route_desc desc{};
  desc.logits_dtype = hum_dtype_of(x);
  desc.num_experts = (int32_t)(e < INT32_MAX ? e : INT32_MAX);
  desc.topk = whole32(a[1], "topk");
  desc.score = whole32(a[2], "score");
  desc.num_groups = whole32(a[4], "num_groups");
  desc.topk_groups = whole32(a[5], "topk_groups");
  desc.group_score = whole32(a[6], "group_score");
  desc.renormalize = truth(a[7]);
  desc.scale = (float)real(a[8]);
  if (desc.topk < 1 || desc.topk > e) fail("topk must be 1 .. the number of experts");
  const at::Tensor *bias = maybe(a[3], "bias"), *ids = maybe(a[9], "topk_ids"), *weights = maybe(a[10], "topk_weights");
  if (bias) want_vec(bias, "bias", at::kFloat, e);
  if (ids) {
    want_dtype(*ids, "topk_ids", at::kInt);
    want_matrix(*ids, "topk_ids", t, desc.topk);
    want_contiguous(*ids, "topk_ids");
  }
  if (weights) {
    want_dtype(*weights, "topk_weights", at::kFloat);
    want_matrix(*weights, "topk_weights", t, desc.topk);
    want_contiguous(*weights, "topk_weights");
  }
  const int dev = device_of("logits", {&x, bias, ids, weights});
  at::Tensor new_ids, new_weights;
  if (!ids) {
    new_ids = at::empty({t, desc.topk}, x.options().dtype(at::kInt));
    ids = &new_ids;
  }
  if (!weights) {
    new_weights = at::empty({t, desc.topk}, x.options().dtype(at::kFloat));
    weights = &new_weights;
  }
  const DeviceGuard guard(dev);
  const hum_status st = hum_moe_route(&desc, t, x.data_ptr(), x.stride(0), bias ? static_cast<const float*>(bias->data_ptr()) : nullptr,
                                      static_cast<int32_t*>(ids->data_ptr()), static_cast<float*>(weights->data_ptr()), stream_of(dev));
  if (st != HUM_OK) raise_status(st);
  return pair(*ids, a[9], weights, a[10]);
  END_HANDLE_TH_ERRORS
}

// rotary_kv_write(desc, cache, q, k, v, positions, inv_freq, slots, layout, factor, q_norm, k_norm, eps, weight_offset, q_out)
PyObject* rotary_kv_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want_args(n, 15);
  const KvDesc desc(a[0]);
  const at::Tensor* cache = maybe(a[1], "cache");
  want_cache(cache);
  const char* heads = "[T, heads, head_dim]";
  const at::Tensor* q = a[2] == Py_None ? nullptr : &tensor(a[2], "q", 3, heads);
  const at::Tensor &k = tensor(a[3], "k", 3, heads), &v = tensor(a[4], "v", 3, heads);
  const int64_t t = k.size(0), hq = q ? q->size(1) : 0, hk = desc->num_kv_heads, d = desc->head_dim;
  if (q) want_rows(*q, "q", at::kBFloat16, t, hq, d);
  want_rows(k, "k", at::kBFloat16, t, hk, d);
  want_rows(v, "v", at::kBFloat16, t, hk, d);
  const at::Tensor *pos = maybe(a[5], "positions"), *slots = maybe(a[7], "slots");
  want_vec(pos, "positions", at::kLong, t);
  want_vec(slots, "slots", at::kLong, t);
  const at::Tensor& freq = tensor(a[6], "inv_freq", 1, "of float64");
  const int64_t half = freq.size(0);
  want_vec(&freq, "inv_freq", at::kDouble, half);
  const at::Tensor *norm[2] = {maybe(a[10], "q_norm"), maybe(a[11], "k_norm")}, *qo = maybe(a[14], "q_out");
  const char* names[2] = {"q_norm", "k_norm"};
  for (int i = 0; i < 2; ++i) {
    if (!norm[i]) continue;
    want_float(*norm[i], names[i]);
    want_vec(norm[i], names[i], norm[i]->scalar_type(), d);
  }
  if (norm[0] && norm[1]) want_dtype(*norm[1], "k_norm", norm[0]->scalar_type());
  if (norm[0] && !q) fail("q_norm without q");
  if (qo) {
    if (!q) fail("q_out without q");
    want_rows(*qo, "q_out", at::kBFloat16, t, hq, d);
    want_spread(*qo, "q_out");
  }
  const int dev = device_of("cache", {cache, q, &k, &v, pos, slots, &freq, norm[0], norm[1], qo});
  hum_rotary_desc rot{};
  rot.dtype = HUM_BF16;
  rot.layout = whole32(a[8], "layout");
  rot.head_dim = (int32_t)d;
  rot.rotary_dim = (int32_t)(half < INT32_MAX / 2 ? 2 * half : INT32_MAX - 1);
  rot.num_q_heads = (int32_t)(hq < INT32_MAX ? hq : INT32_MAX);
  rot.num_kv_heads = (int32_t)hk;
  rot.factor = (float)real(a[9]);
  hum_head_norm hn{};
  const at::Tensor* any = norm[0] ? norm[0] : norm[1];
  if (any) {
    hn.q_weight = norm[0] ? norm[0]->data_ptr() : nullptr;
    hn.k_weight = norm[1] ? norm[1]->data_ptr() : nullptr;
    hn.weight_dtype = hum_dtype_of(*any);
    hn.eps = (float)real(a[12]);
    hn.weight_offset = (float)real(a[13]);
  }
  at::Tensor fresh;
  if (q && !qo) {
    fresh = at::empty({t, hq, d}, q->options());
    qo = &fresh;
  }
  const DeviceGuard guard(dev);
  const hum_status st = hum_rotary_kv_write(
      &rot, desc.d, any ? &hn : nullptr, cache->data_ptr(), (size_t)cache->numel(), t,
      static_cast<const int64_t*>(pos->data_ptr()), static_cast<const double*>(freq.data_ptr()),
      static_cast<const int64_t*>(slots->data_ptr()), q ? q->data_ptr() : nullptr, q ? q->stride(0) : 0,
      q ? q->stride(1) : 0, q ? qo->data_ptr() : nullptr, q ? qo->stride(0) : 0, q ? qo->stride(1) : 0, k.data_ptr(),
      k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1), stream_of(dev));
  if (st != HUM_OK) raise_status(st);
  if (!q) Py_RETURN_NONE;
  return given_or(*qo, a[14]);
  END_HANDLE_TH_ERRORS
}

// setup(HumError, raw stream function, workspace function, workspaces)
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  want_args(n, 4);
  PyObject** slots[4] = {&g_hum_error, &g_raw_stream, &g_workspace, &g_workspaces};
  for (int i = 0; i < 4; ++i) {
    Py_INCREF(a[i]);
    Py_XDECREF(*slots[i]);
    *slots[i] = a[i];
  }
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define HUM_METHOD(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {HUM_METHOD(rms_norm), HUM_METHOD(moe_route),    HUM_METHOD(rotary),
                           HUM_METHOD(kv_write), HUM_METHOD(kv_read),      HUM_METHOD(rotary_kv_write),
                           HUM_METHOD(setup),    HUM_METHOD(kv_attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", "Marshalling of the calls around a layer's products.", -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&g_module); }
