// The paged-cache calls on torch tensors: argument checks, outputs, workspace
// and stream, then the C entry points.  A single token's attention takes a few
// microseconds on the device, fewer than these checks take in Python.
//
// Functions take their arguments by position, exactly as kv_cache.py passes
// them; a C status other than MUSE_OK raises the package's MuseError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/fill.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>
#include <string>

#include "muse.h"

namespace {

PyObject* g_error = nullptr;  // MuseError(status, message)

struct Refusal {  // a Python exception to raise
  PyObject* type;
  std::string text;
};
[[noreturn]] void value_error(const std::string& s) { throw Refusal{PyExc_ValueError, s}; }
[[noreturn]] void type_error(const std::string& s) { throw Refusal{PyExc_TypeError, s}; }
struct Raised {};  // the Python error is set already

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
const at::Tensor* maybe(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }
long long integer(PyObject* o, const char* name, long long lo, long long hi) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  if (v < lo || v > hi) value_error(std::string(name) + " out of range");
  return v;
}
std::string shape_text(std::initializer_list<int64_t> s) {
  std::string t = "[";
  for (auto i = s.begin(); i != s.end(); ++i) t += (i == s.begin() ? "" : ", ") + std::to_string(*i);
  return t + "]";
}
bool has_shape(const at::Tensor& t, std::initializer_list<int64_t> s) { return t.sizes() == at::IntArrayRef(s); }

muse_dtype compute_dtype(at::ScalarType t) {
  if (t == at::kBFloat16) return MUSE_BF16;
  if (t == at::kFloat) return MUSE_F32;
  type_error("unsupported dtype (bf16 or fp32)");
}

void on(const at::Tensor* t, const char* name, c10::Device dev) {
  if (t && t->device() != dev)
    value_error(std::string(name) + " must be on " + dev.str() + ", the device of the cache");
}
// Where the call runs: the cache's device, and the caller's stream (None, or
// the (stream_id, device_index, device_type) of a torch stream) or the
// device's current one.
struct Place {
  c10::cuda::CUDAStream stream;
  bool other = false;  // not the current stream: the call's tensors are marked as used on it
  std::optional<c10::cuda::CUDAGuard> guard;

  Place(c10::Device dev, PyObject* s) : stream(c10::cuda::getCurrentCUDAStream(dev.index())) {
    if (s != Py_None) {
      if (!PyTuple_Check(s) || PyTuple_GET_SIZE(s) != 3) type_error("stream must be a torch.cuda.Stream");
      const auto given = c10::Stream::unpack3(integer(PyTuple_GET_ITEM(s, 0), "stream", INT64_MIN, INT64_MAX),
                                              (c10::DeviceIndex)integer(PyTuple_GET_ITEM(s, 1), "stream", 0, 127),
                                              (c10::DeviceType)integer(PyTuple_GET_ITEM(s, 2), "stream", 0, 127));
      if (given.device() != dev) value_error("stream must be one of " + dev.str());
      other = c10::cuda::CUDAStream(given) != stream;
      stream = c10::cuda::CUDAStream(given);
    }
    if (c10::cuda::current_device() != dev.index()) guard.emplace(dev);
  }
  void uses(const at::Tensor& t) const {
    if (other) t.record_stream(stream.unwrap());
  }
  // every tensor among a call's arguments: its owner may let go of it before
  // the other stream has read it
  void uses_arguments(PyObject* const* o, Py_ssize_t n) const {
    if (!other) return;
    for (Py_ssize_t i = 0; i < n; ++i)
      if (THPVariable_Check(o[i])) uses(THPVariable_Unpack(o[i]));
  }
};

struct CacheArgs {
  muse_cache ca{};
  muse_cache_index ix{};
  c10::Device dev;
};
const int32_t* index_array(const at::Tensor* t, const char* name, int64_t B) {
  if (!t) return nullptr;
  if (t->scalar_type() != at::kInt || !has_shape(*t, {B}) || !t->is_contiguous())
    value_error(std::string(name) + " must be contiguous int32 " + shape_text({B}));
  return t->const_data_ptr<int32_t>();
}
// Checked descriptors of a cache and of the batch's place in it.
CacheArgs cache_args(const at::Tensor& k, const at::Tensor& v, const at::Tensor* ks, const at::Tensor* vs,
                     const at::Tensor& table, const at::Tensor& kv_len, const at::Tensor* new_len, int64_t B,
                     int64_t Hkv, int64_t D) {
  if (!k.is_cuda()) value_error("tensors must be CUDA tensors");
  CacheArgs a{{}, {}, k.device()};
  on(&v, "v_cache", a.dev);
  on(ks, "k_scale", a.dev);
  on(vs, "v_scale", a.dev);
  on(&table, "table", a.dev);
  on(&kv_len, "kv_len", a.dev);
  on(new_len, "new_len", a.dev);
  switch (k.scalar_type()) {
    case at::kBFloat16: a.ca.dtype = MUSE_CACHE_BF16; break;
    case at::kFloat: a.ca.dtype = MUSE_CACHE_F32; break;
    case at::kFloat8_e4m3fn: a.ca.dtype = MUSE_CACHE_E4M3; break;
    case at::kChar: a.ca.dtype = MUSE_CACHE_I8; break;
    default: type_error("k_cache and v_cache must share a dtype: bf16, fp32, float8_e4m3fn or int8");
  }
  if (v.scalar_type() != k.scalar_type())
    type_error("k_cache and v_cache must share a dtype: bf16, fp32, float8_e4m3fn or int8");
  if (k.dim() != 4 || v.sizes() != k.sizes() || !k.is_contiguous() || !v.is_contiguous())
    value_error("k_cache and v_cache must be contiguous [pages, Hkv, page_size, D]");
  if (k.size(1) != Hkv || k.size(3) != D)
    value_error("the cache holds " + std::to_string(k.size(1)) + " heads of " + std::to_string(k.size(3)) +
                ", the call " + std::to_string(Hkv) + " of " + std::to_string(D));
  const bool scaled = a.ca.dtype == MUSE_CACHE_E4M3 || a.ca.dtype == MUSE_CACHE_I8;
  for (const auto& [name, s] : {std::pair{"k_scale", ks}, std::pair{"v_scale", vs}}) {
    if ((s != nullptr) != scaled) value_error(std::string(name) + " belongs to an 8-bit cache, and to no other");
    if (s && (s->scalar_type() != at::kFloat || s->sizes() != k.sizes().slice(0, 3) || !s->is_contiguous()))
      value_error(std::string(name) + " must be contiguous fp32 [pages, Hkv, page_size]");
  }
  if (table.scalar_type() != at::kInt || table.dim() != 2 || table.size(0) != B || !table.is_contiguous())
    value_error("table must be contiguous int32 [" + std::to_string(B) + ", wide]");
  if (k.size(0) > INT32_MAX || k.size(2) > INT32_MAX || table.size(1) > INT32_MAX)
    value_error("more pages, page rows or table columns than an int counts");
  a.ca.k = k.data_ptr();
  a.ca.v = v.data_ptr();
  a.ca.k_scale = ks ? ks->data_ptr<float>() : nullptr;
  a.ca.v_scale = vs ? vs->data_ptr<float>() : nullptr;
  a.ca.pages = (int)k.size(0);
  a.ca.page_size = (int)k.size(2);
  a.ix.table = table.const_data_ptr<int32_t>();
  a.ix.wide = (int)table.size(1);
  a.ix.kv_len = index_array(&kv_len, "kv_len", B);
  a.ix.new_len = index_array(new_len, "new_len", B);
  return a;
}

muse_shape shape(int64_t B, int64_t Hq, int64_t Hkv, int64_t N, int64_t D, muse_dtype dt) {
  for (int64_t x : {B, Hq, Hkv, N, D})
    if (x > INT32_MAX) value_error("a dimension is larger than an int counts");
  muse_shape s{};
  s.B = (int)B;
  s.Hq = (int)Hq;
  s.Hkv = (int)Hkv;
  s.N = (int)N;
  s.D = (int)D;
  s.dtype = dt;
  s.out_f32 = 0;
  return s;
}
// A tensor's strides, of a [B, H, n, D] view whose rows are contiguous (the
// stride of a dimension of one is never used: 0).
muse_strides strides(const at::Tensor& t, const char* name) {
  if (t.dim() != 4 || (t.stride(3) != 1 && t.size(3) > 1))
    value_error(std::string(name) + " must be [B, H, n, D] with a contiguous last dimension");
  auto s = [&](int d) { return t.size(d) == 1 ? 0 : t.stride(d); };
  return muse_strides{s(0), s(1), s(2)};
}
int32_t* error_word(const at::Tensor* t, c10::Device dev) {
  if (!t) return nullptr;
  if (t->scalar_type() != at::kInt || t->numel() != 1 || t->device() != dev)
    value_error("device_error must be one int32 on " + dev.str());
  return t->data_ptr<int32_t>();
}
void check(muse_status st) {
  if (st == MUSE_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", (int)st, muse_last_error());
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

// Runs a call's body; its exceptions become Python's.
template <typename F>
PyObject* guarded(const char* name, Py_ssize_t n, Py_ssize_t want, F&& body) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, not %zd", name, want, n);
    return nullptr;
  }
  try {
    return body();
  } catch (const Refusal& r) {
    PyErr_SetString(r.type, r.text.c_str());
  } catch (const Raised&) {
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// (k, v, k_cache, v_cache, table, kv_len, new_len, k_scale, v_scale, device_error, stream)
PyObject* cache_write(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded("cache_write", n, 11, [&]() -> PyObject* {
    const at::Tensor &k = tensor(o[0], "k"), &v = tensor(o[1], "v");
    if (k.dim() != 4 || k.sizes() != v.sizes() || k.scalar_type() != v.scalar_type())
      value_error("k and v must be [B, Hkv, n, D] of one shape and dtype");
    const at::Tensor& kc = tensor(o[2], "k_cache");
    const CacheArgs a = cache_args(kc, tensor(o[3], "v_cache"), maybe(o[7], "k_scale"), maybe(o[8], "v_scale"),
                                   tensor(o[4], "table"), tensor(o[5], "kv_len"), maybe(o[6], "new_len"), k.size(0),
                                   k.size(1), k.size(3));
    on(&k, "k", a.dev);
    on(&v, "v", a.dev);
    const muse_shape sh = shape(k.size(0), k.size(1), k.size(1), k.size(2), k.size(3), compute_dtype(k.scalar_type()));
    const muse_strides ks = strides(k, "k"), vs = strides(v, "v");
    int32_t* err = error_word(maybe(o[9], "device_error"), a.dev);
    const Place p(a.dev, o[10]);
    p.uses_arguments(o, n);
    check(muse_cache_write(k.data_ptr(), &ks, v.data_ptr(), &vs, &sh, &a.ca, &a.ix, err, p.stream.stream()));
    Py_RETURN_NONE;
  });
}

// (k_cache, v_cache, table, kv_len, N, start, k_scale, v_scale, bf16 output, out_k, out_v,
//  device_error, stream) -> (k, v)
PyObject* cache_read(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded("cache_read", n, 13, [&]() -> PyObject* {
    const at::Tensor &kc = tensor(o[0], "k_cache"), &table = tensor(o[2], "table");
    if (kc.dim() != 4 || table.dim() != 2)
      value_error("k_cache must be [pages, Hkv, page_size, D] and table [B, wide]");
    const int64_t B = table.size(0), H = kc.size(1), D = kc.size(3), N = integer(o[4], "N", 0, INT32_MAX);
    const CacheArgs a = cache_args(kc, tensor(o[1], "v_cache"), maybe(o[6], "k_scale"), maybe(o[7], "v_scale"), table,
                                   tensor(o[3], "kv_len"), nullptr, B, H, D);
    const at::Tensor* start = maybe(o[5], "start");
    on(start, "start", a.dev);
    const int32_t* sp = index_array(start, "start", B);
    const Place p(a.dev, o[12]);
    p.uses_arguments(o, n);
    at::Tensor k, v;
    if (o[9] == Py_None) {
      const auto opt = at::TensorOptions().device(a.dev).dtype(o[8] == Py_True ? at::kBFloat16 : at::kFloat);
      k = at::empty({B, H, N, D}, opt);
      v = at::empty({B, H, N, D}, opt);
      p.uses(k);
      p.uses(v);
    } else {
      k = tensor(o[9], "out");
      v = tensor(o[10], "out");
      for (const at::Tensor* t : {&k, &v})
        if (!has_shape(*t, {B, H, N, D}) || t->scalar_type() != k.scalar_type() || !t->is_contiguous())
          value_error("out must be two contiguous " + shape_text({B, H, N, D}) + " tensors of one dtype");
      on(&k, "out", a.dev);
      on(&v, "out", a.dev);
    }
    const muse_shape sh = shape(B, H, H, N, D, compute_dtype(k.scalar_type()));
    int32_t* err = error_word(maybe(o[11], "device_error"), a.dev);
    check(muse_cache_read(k.data_ptr(), v.data_ptr(), &sh, &a.ca, &a.ix, sp, err, p.stream.stream()));
    PyObject* pk = THPVariable_Wrap(std::move(k));
    PyObject* pv = pk ? THPVariable_Wrap(std::move(v)) : nullptr;
    PyObject* r = pv ? PyTuple_Pack(2, pk, pv) : nullptr;
    Py_XDECREF(pk);
    Py_XDECREF(pv);
    return r;
  });
}

// (q, k_cache, v_cache, table, kv_len, k_scale, v_scale) -> bytes
PyObject* attn_workspace(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded("attn_workspace", n, 7, [&]() -> PyObject* {
    const at::Tensor &q = tensor(o[0], "q"), &kc = tensor(o[1], "k_cache");
    if (q.dim() != 4) value_error("q must be [B, Hq, n, D]");
    if (kc.dim() != 4) value_error("k_cache must be [pages, Hkv, page_size, D]");
    const CacheArgs a = cache_args(kc, tensor(o[2], "v_cache"), maybe(o[5], "k_scale"), maybe(o[6], "v_scale"),
                                   tensor(o[3], "table"), tensor(o[4], "kv_len"), nullptr, q.size(0), kc.size(1),
                                   q.size(3));
    const muse_shape sh = shape(q.size(0), q.size(1), kc.size(1), q.size(2), q.size(3),
                                compute_dtype(q.scalar_type()));
    const size_t size = muse_attn_cache_workspace_size(&sh, &a.ca, &a.ix);
    if (size == 0) check(MUSE_ERR_INVALID_ARG);
    return PyLong_FromSize_t(size);
  });
}

// (q, k_cache, v_cache, table, kv_len, new_len, scale, causal, window, k_scale, v_scale, out,
//  lse (None, True or a tensor), workspace, device_error, stream) -> o or (o, lse)
PyObject* attn_cache(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded("attn_cache", n, 16, [&]() -> PyObject* {
    const at::Tensor &q = tensor(o[0], "q"), &kc = tensor(o[1], "k_cache");
    if (q.dim() != 4) value_error("q must be [B, Hq, n, D]");
    if (kc.dim() != 4) value_error("k_cache must be [pages, Hkv, page_size, D]");
    const int64_t B = q.size(0), Hq = q.size(1), N = q.size(2), D = q.size(3);
    const CacheArgs a = cache_args(kc, tensor(o[2], "v_cache"), maybe(o[9], "k_scale"), maybe(o[10], "v_scale"),
                                   tensor(o[3], "table"), tensor(o[4], "kv_len"), maybe(o[5], "new_len"), B,
                                   kc.size(1), D);
    on(&q, "q", a.dev);
    const muse_shape sh = shape(B, Hq, kc.size(1), N, D, compute_dtype(q.scalar_type()));
    const double scale = PyFloat_AsDouble(o[6]);
    if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
    const int causal = PyObject_IsTrue(o[7]);
    if (causal < 0) throw Raised{};
    const int window = (int)integer(o[8], "window", 0, INT32_MAX);
    const muse_strides qs = strides(q, "q");
    int32_t* err = error_word(maybe(o[14], "device_error"), a.dev);
    const Place p(a.dev, o[15]);
    p.uses_arguments(o, n);

    // rows that are not there (i >= new_len) of an output made here: o = 0, lse = -inf
    const bool ragged = o[5] != Py_None;
    auto fill = [&](at::Tensor& t, double x) {
      const c10::cuda::CUDAStreamGuard on_it(p.stream);
      at::fill_(t, x);
    };
    at::Tensor out, lse, ws;
    if (o[11] == Py_None) {
      out = at::empty(q.sizes(), q.options());
      p.uses(out);
      if (ragged) fill(out, 0.);
    } else {
      out = tensor(o[11], "out");
      if (out.sizes() != q.sizes() || out.scalar_type() != q.scalar_type())
        value_error("out must have q's shape and dtype");
      on(&out, "out", a.dev);
    }
    if (o[12] == Py_True) {
      lse = at::empty({B, Hq, N}, q.options().dtype(at::kFloat));
      p.uses(lse);
      if (ragged) fill(lse, -INFINITY);
    } else if (o[12] != Py_None) {
      lse = tensor(o[12], "lse");
      if (!has_shape(lse, {B, Hq, N}) || lse.scalar_type() != at::kFloat || !lse.is_contiguous())
        value_error("lse must be contiguous fp32 " + shape_text({B, Hq, N}));
      on(&lse, "lse", a.dev);
    }
    if (o[13] == Py_None) {
      const size_t size = muse_attn_cache_workspace_size(&sh, &a.ca, &a.ix);
      if (size == 0) check(MUSE_ERR_INVALID_ARG);
      ws = at::empty({(int64_t)size}, q.options().dtype(at::kByte));
      p.uses(ws);
    } else {
      ws = tensor(o[13], "workspace");
      if (!ws.is_contiguous()) value_error("workspace must be contiguous");
      on(&ws, "workspace", a.dev);
    }
    const muse_strides os = strides(out, "out");
    check(muse_attn_cache(q.data_ptr(), &qs, out.data_ptr(), &os, lse.defined() ? lse.data_ptr<float>() : nullptr,
                          &sh, &a.ca, &a.ix, (float)scale, causal, window, err, ws.data_ptr(), ws.nbytes(),
                          p.stream.stream()));
    PyObject* po = THPVariable_Wrap(std::move(out));
    if (!lse.defined() || !po) return po;
    PyObject* pl = THPVariable_Wrap(std::move(lse));
    PyObject* r = pl ? PyTuple_Pack(2, po, pl) : nullptr;
    Py_DECREF(po);
    Py_XDECREF(pl);
    return r;
  });
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XSETREF(g_error, type);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"cache_write", (PyCFunction)(void*)cache_write, METH_FASTCALL, nullptr},
    {"cache_read", (PyCFunction)(void*)cache_read, METH_FASTCALL, nullptr},
    {"attn_workspace", (PyCFunction)(void*)attn_workspace, METH_FASTCALL, nullptr},
    {"attn_cache", (PyCFunction)(void*)attn_cache, METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_cache", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_cache(void) { return PyModule_Create(&module); }
