// marshal.cpp -- the operators' calls between Python and the C ABI: checks of
// the tensors, their outputs' allocation, and the call.
//
// A Python module of its own (_marshal.so, beside libq1gemv.so): the operators
// run in a few microseconds, and checking some ten tensors attribute by
// attribute from Python took three to five times that.  Arguments come
// positionally and complete from binding.py, which documents the calls; None
// is a null pointer.  Nothing is kept from one call to the next.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <cmath>
#include <string>

#include "q1gemv.h"

namespace {

PyObject* g_error = nullptr;  // binding.Q1Error

template <size_t N>
using Sizes = std::array<int64_t, N>;

// A Python exception is set; unwinds to the entry point.
struct Refused {};

template <class... A>
[[noreturn]] void refuse(PyObject* type, const char* format, A... a) {
  PyErr_Format(type, format, a...);
  throw Refused{};
}

enum : unsigned { kF32 = 1, kBf16 = 2, kF16 = 4, kI32 = 8, kI8 = 16, kU8 = 32, kScale = 64 };

bool is_type(at::ScalarType t, unsigned types) {
  switch (t) {
    case at::kFloat: return types & kF32;
    case at::kBFloat16: return types & kBf16;
    case at::kHalf: return types & (kF16 | kScale);
    case at::kInt: return types & kI32;
    case at::kChar: return types & kI8;
    case at::kByte: return types & kU8;
    case at::kShort:
    case at::kUInt16: return types & kScale;
    default: return false;
  }
}

std::string names_of(unsigned types) {
  std::string s;
  const auto add = [&](unsigned bit, const char* n) {
    if (types & bit) s += s.empty() ? n : std::string(", ") + n;
  };
  add(kF32, "float32"), add(kBf16, "bfloat16"), add(kF16, "float16"), add(kI32, "int32"), add(kI8, "int8");
  add(kU8, "uint8"), add(kScale, "int16, uint16, float16");
  return s;
}

std::string text_of(at::IntArrayRef sizes) {
  std::string s = "(";
  for (size_t i = 0; i < sizes.size(); ++i) s += (i ? ", " : "") + std::to_string(sizes[i]);
  return s + ")";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

// Device, type and shape; the last axis contiguous, or (whole) all of it.
void* pointer(const at::Tensor& t, const char* name, unsigned types, at::IntArrayRef shape, bool whole = false) {
  if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", name);
  if (!is_type(t.scalar_type(), types))
    refuse(PyExc_TypeError, "%s has dtype %s, expected one of %s", name, at::toString(t.scalar_type()), names_of(types).c_str());
  if (t.sizes() != shape)
    refuse(PyExc_ValueError, "%s has shape %s, expected %s", name, text_of(t.sizes()).c_str(), text_of(shape).c_str());
  if (!t.is_contiguous()) {
    if (whole) refuse(PyExc_ValueError, "%s must be contiguous", name);
    if (t.dim() && t.stride(-1) != 1 && t.size(-1) > 1) refuse(PyExc_ValueError, "the last axis of %s must be contiguous", name);
  }
  return t.data_ptr();
}
void* pointer(PyObject* o, const char* name, unsigned types, at::IntArrayRef shape, bool whole = false) {
  return o == Py_None ? nullptr : pointer(tensor(o, name), name, types, shape, whole);
}

// Stride of an axis; `least` for an axis of one entry, whose stride means nothing
// (one row of a buffer may have any, also one that no kernel takes).
int64_t stride(const at::Tensor& t, int axis, int64_t least) { return t.size(axis) > 1 ? t.stride(axis) : least; }
int64_t row_stride(PyObject* o, int64_t least) {
  return o == Py_None ? 0 : stride(THPVariable_Unpack(o), 0, least);
}

unsigned type_bit(at::ScalarType t) { return t == at::kFloat ? kF32 : t == at::kBFloat16 ? kBf16 : t == at::kHalf ? kF16 : 0; }
int type_code(at::ScalarType t) { return t == at::kFloat ? Q1_F32 : t == at::kBFloat16 ? Q1_BF16 : Q1_F16; }

// `o`, or a new tensor of this shape and type where it is None.
at::Tensor given_or_new(PyObject* o, const char* name, at::IntArrayRef shape, const at::Tensor& like, at::ScalarType type) {
  return o == Py_None ? at::empty(shape, like.options().dtype(type)) : tensor(o, name);
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}

void check(int64_t rc, const char* what) {
  if (rc == Q1_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "Ls", static_cast<long long>(rc),
                                      (std::string(what) + ": " + q1_last_error()).c_str());
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Refused{};
}

// The device of a call: that of its first tensor, and every other one's too
// (addresses of another device would be followed on this one).  Tensors that are
// on no CUDA device are left to `pointer`.
c10::Device one_device(PyObject* const* a, Py_ssize_t count) {
  const at::Tensor* first = nullptr;
  for (Py_ssize_t i = 0; i < count; ++i) {
    if (a[i] == Py_None || PyLong_Check(a[i]) || PyFloat_Check(a[i]) || !THPVariable_Check(a[i])) continue;  // (the check of others is slow)
    const at::Tensor& t = THPVariable_Unpack(a[i]);
    if (!t.is_cuda()) continue;
    if (!first) first = &t;
    if (t.device() != first->device())
      refuse(PyExc_ValueError, "tensors on different devices: %s and %s", first->device().str().c_str(), t.device().str().c_str());
  }
  return first ? first->device() : c10::Device(c10::kCPU);
}

// Runs a call's body with its tensors' device current; whatever it throws becomes a Python exception.
template <class F>
PyObject* guarded(PyObject* const* a, Py_ssize_t given, Py_ssize_t wanted, F&& body) {
  if (given != wanted) return PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", given, wanted);
  try {
    const c10::Device device = one_device(a, given);
    c10::OptionalDeviceGuard current;
    if (device.is_cuda()) {  // (asked once: with one device the guard's calls are for nothing, 0.2 us)
      static const bool several = c10::impl::VirtualGuardImpl(c10::kCUDA).deviceCount() > 1;
      if (several) current.reset_device(device);
    }
    return body();
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "an unknown C++ exception");
  }
  return nullptr;
}

// x, weight, eps, residual, residual_out, want_q8, want_y, y, q, d, stream
PyObject* add_rms_norm(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(a, count, 11, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0], "x");
    if (x.dim() != 2) refuse(PyExc_ValueError, "x must be [nvec, n]");
    const int64_t nvec = x.size(0), n = x.size(1);
    const unsigned type = type_bit(x.scalar_type());
    if (!type) refuse(PyExc_TypeError, "x has dtype %s, expected one of float32, bfloat16, float16", at::toString(x.scalar_type()));
    const bool want_q8 = a[5] == Py_True, want_y = a[6] == Py_True;
    if (want_q8 && n % 32) refuse(PyExc_ValueError, "the q8_0 form needs n to be a multiple of 32");
    const Sizes<2> shape = {nvec, n}, scales = {nvec, n / 32};
    const Sizes<1> width = {n};
    void* px = pointer(x, "x", type, shape);
    void* pw = pointer(a[1], "weight", kF32, width);
    if (!pw) refuse(PyExc_TypeError, "weight must be a torch.Tensor");
    void* pr = pointer(a[3], "residual", type, shape);
    at::Tensor ro, y, q, d;
    if (a[3] != Py_None || a[4] != Py_None) ro = given_or_new(a[4], "residual_out", shape, x, x.scalar_type());
    if (want_y) y = given_or_new(a[7], "y", shape, x, x.scalar_type());
    if (want_q8) {
      q = given_or_new(a[8], "q", shape, x, at::kChar);
      d = given_or_new(a[9], "d", scales, x, at::kShort);
      if (q.numel() != nvec * n || d.numel() != nvec * (n / 32)) refuse(PyExc_ValueError, "q/d sizes do not match x");
    }
    check(q8_add_rms_norm(px, stride(x, 0, n), pr, row_stride(a[3], n), static_cast<const float*>(pw),
                          static_cast<float>(number(a[2])), nvec, n, type_code(x.scalar_type()),
                          ro.defined() ? pointer(ro, "residual_out", type, shape) : nullptr,
                          ro.defined() ? stride(ro, 0, n) : 0, want_y ? pointer(y, "y", type, shape) : nullptr,
                          want_y ? stride(y, 0, n) : 0,
                          want_q8 ? static_cast<int8_t*>(pointer(q, "q", kI8, q.sizes(), true)) : nullptr,
                          want_q8 ? static_cast<uint16_t*>(pointer(d, "d", kScale, d.sizes(), true)) : nullptr,
                          reinterpret_cast<void*>(integer(a[10]))),
          "q8_add_rms_norm");
    return Py_BuildValue("(NNNN)", ro.defined() ? THPVariable_Wrap(ro) : Py_NewRef(Py_None),
                         want_y ? THPVariable_Wrap(y) : Py_NewRef(Py_None), want_q8 ? THPVariable_Wrap(q) : Py_NewRef(Py_None),
                         want_q8 ? THPVariable_Wrap(d) : Py_NewRef(Py_None));
  });
}

// x, a, b, index, scale, ranks, base, out, stream
PyObject* lora_add(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(a, count, 9, [&]() -> PyObject* {
    const at::Tensor &x = tensor(a[0], "x"), &wa = tensor(a[1], "a"), &wb = tensor(a[2], "b");
    if (x.dim() != 2 || wa.dim() != 3 || wb.dim() != 3)
      refuse(PyExc_ValueError, "x must be [nvec, n], a [adapters, rank, n], b [adapters, rows, rank]");
    if (a[6] == Py_None && a[7] == Py_None) refuse(PyExc_ValueError, "lora_add needs base, out or both");
    const int64_t nvec = x.size(0), n = x.size(1), adapters = wb.size(0), rows = wb.size(1), rank = wb.size(2);
    const Sizes<1> each = {adapters}, vectors = {nvec};
    const Sizes<2> out_shape = {nvec, rows}, xs = {nvec, n};
    const Sizes<3> a_shape = {adapters, rank, n};
    void* px = pointer(x, "x", kF32, xs);
    void* pa = pointer(wa, "a", kBf16 | kF16, a_shape, true);
    void* pb = pointer(wb, "b", type_bit(wa.scalar_type()), wb.sizes(), true);
    void* pi = pointer(tensor(a[3], "index"), "index", kI32, vectors, true);
    void* ps = pointer(a[4], "scale", kF32, each, true);
    void* pk = pointer(a[5], "ranks", kI32, each, true);
    at::Tensor out = given_or_new(a[7], "out", out_shape, x, at::kFloat);
    const at::Tensor& base = a[6] == Py_None ? out : tensor(a[6], "base");
    check(q1_lora_add(static_cast<const float*>(px), stride(x, 0, n), nvec, n, rows, pa, pb, type_code(wa.scalar_type()), adapters,
                      rank, static_cast<const int32_t*>(pi), static_cast<const int32_t*>(pk), static_cast<const float*>(ps),
                      static_cast<const float*>(pointer(base, "base", kF32, out_shape)), stride(base, 0, rows),
                      static_cast<float*>(pointer(out, "out", kF32, out_shape)), stride(out, 0, rows),
                      reinterpret_cast<void*>(integer(a[8]))),
          "q1_lora_add");
    return THPVariable_Wrap(out);
  });
}

// cache_k, cache_v, table, kv_len, new_start
q1_paged_kv paged_kv(PyObject* const* a, int64_t total_new) {
  const at::Tensor &k = tensor(a[0], "cache_k"), &v = tensor(a[1], "cache_v"), &table = tensor(a[2], "table");
  if (k.dim() != 4) refuse(PyExc_ValueError, "cache_k must be [pages, page_size, kv_heads, dim]");
  if (table.dim() != 2) refuse(PyExc_ValueError, "table must be [batch, width]");
  if (k.size(3) < 1) refuse(PyExc_ValueError, "the cache's dim is 0");  // (callers divide by it)
  q1_paged_kv p = {};
  p.k = pointer(k, "cache_k", kBf16 | kF16, k.sizes());
  p.v = pointer(v, "cache_v", type_bit(k.scalar_type()), k.sizes());
  for (int i = 0; i < 3; ++i)
    if (stride(k, i, 0) != stride(v, i, 0)) refuse(PyExc_ValueError, "cache_k and cache_v must have the same strides");
  p.pages = k.size(0), p.page_size = k.size(1), p.kv_heads = k.size(2), p.dim = k.size(3);
  p.page_stride = stride(k, 0, p.dim), p.slot_stride = stride(k, 1, p.dim), p.head_stride = stride(k, 2, p.dim);
  p.batch = table.size(0), p.table_width = table.size(1);
  p.table = static_cast<const int32_t*>(pointer(table, "table", kI32, table.sizes()));
  p.table_stride = stride(table, 0, p.table_width);
  const Sizes<1> batch = {p.batch}, bounds = {p.batch + 1};
  p.kv_len = static_cast<const int32_t*>(pointer(tensor(a[3], "kv_len"), "kv_len", kI32, batch, true));
  p.new_start = static_cast<const int32_t*>(pointer(tensor(a[4], "new_start"), "new_start", kI32, bounds, true));
  p.total_new = total_new;
  p.dtype = type_code(k.scalar_type());
  return p;
}

// q, k, v, cos_sin, cache_k, cache_v, table, kv_len, new_start, q_out, interleaved, stream
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(a, count, 12, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &cs = tensor(a[3], "cos_sin");
    if (q.dim() != 2 || cs.dim() != 2) refuse(PyExc_ValueError, "q must be [tokens, heads * dim] and cos_sin [positions, rot]");
    const int64_t total = q.size(0);
    const q1_paged_kv kv = paged_kv(a + 4, total);
    if (q.size(1) % kv.dim) refuse(PyExc_ValueError, "q must be [tokens, heads * dim] and cos_sin [positions, rot]");
    const int64_t heads = q.size(1) / kv.dim, width = kv.kv_heads * kv.dim;
    const Sizes<2> kv_shape = {total, width};
    const Sizes<3> out_shape = {total, heads, kv.dim};
    const at::Tensor& cache = THPVariable_Unpack(a[4]);
    void* pq = pointer(q, "q", kF32, q.sizes());
    at::Tensor out = given_or_new(a[9], "q_out", out_shape, q, cache.scalar_type());
    check(q1_rope_append(static_cast<const float*>(pq), stride(q, 0, heads * kv.dim),
                         static_cast<const float*>(pointer(k, "k", kF32, kv_shape)), stride(k, 0, width),
                         static_cast<const float*>(pointer(v, "v", kF32, kv_shape)), stride(v, 0, width),
                         static_cast<const float*>(pointer(cs, "cos_sin", kF32, cs.sizes(), true)), cs.size(0), cs.size(1),
                         a[10] == Py_True, heads, pointer(out, "q_out", type_bit(cache.scalar_type()), out_shape, true), &kv,
                         reinterpret_cast<void*>(integer(a[11]))),
          "q1_rope_append");
    return THPVariable_Wrap(out);
  });
}

// q, cache_k, cache_v, table, kv_len, new_start, max_new, scale (or None), out, workspace, stream
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(a, count, 11, [&]() -> PyObject* {
    const at::Tensor& q = tensor(a[0], "q");
    if (q.dim() != 3) refuse(PyExc_ValueError, "q must be [tokens, heads, dim]");
    const int64_t total = q.size(0), heads = q.size(1), dim = q.size(2);
    const q1_paged_kv kv = paged_kv(a + 1, total);
    if (kv.dim != dim) refuse(PyExc_ValueError, "q has dim %lld, the cache %lld", (long long)dim, (long long)kv.dim);
    const unsigned type = type_bit(THPVariable_Unpack(a[1]).scalar_type());
    void* pq = pointer(q, "q", type, q.sizes());
    const int64_t max_new = integer(a[6]);
    const double scale = a[7] == Py_None ? 1.0 / std::sqrt(double(dim)) : number(a[7]);
    at::Tensor out = given_or_new(a[8], "out", q.sizes(), q, q.scalar_type());
    at::Tensor ws;
    if (a[9] != Py_None) {
      ws = tensor(a[9], "workspace");
    } else {
      const int64_t bytes = q1_paged_attention_workspace(max_new, heads, kv.kv_heads, dim);
      check(bytes < 0 ? bytes : Q1_OK, "q1_paged_attention");
      ws = at::empty({bytes}, q.options().dtype(at::kByte));
    }
    check(q1_paged_attention(pq, stride(q, 0, heads * dim), stride(q, 1, dim), heads, static_cast<float>(scale), &kv, max_new,
                             pointer(out, "out", type, q.sizes()), stride(out, 0, heads * dim), stride(out, 1, dim),
                             pointer(ws, "workspace", kU8, ws.sizes(), true), ws.numel(), reinterpret_cast<void*>(integer(a[10]))),
          "q1_paged_attention");
    return THPVariable_Wrap(out);
  });
}

// cache_k, cache_v, scale_k, scale_v, table, kv_len, new_start
q1_paged_q8 paged_q8(PyObject* const* a, int64_t total_new) {
  const at::Tensor &k = tensor(a[0], "cache_k"), &v = tensor(a[1], "cache_v"), &ks = tensor(a[2], "scale_k"),
                   &vs = tensor(a[3], "scale_v"), &table = tensor(a[4], "table");
  if (k.dim() != 4) refuse(PyExc_ValueError, "cache_k must be [pages, page_size, kv_heads, dim]");
  if (table.dim() != 2) refuse(PyExc_ValueError, "table must be [batch, width]");
  q1_paged_q8 p = {};
  p.pages = k.size(0), p.page_size = k.size(1), p.kv_heads = k.size(2), p.dim = k.size(3);
  if (p.dim < 1) refuse(PyExc_ValueError, "the cache's dim is 0");  // (callers divide by it)
  if (p.dim % 32) refuse(PyExc_ValueError, "the cache's dim %lld is no multiple of 32", (long long)p.dim);
  const Sizes<4> scales = {p.pages, p.page_size, p.kv_heads, p.dim / 32};
  p.k = static_cast<int8_t*>(pointer(k, "cache_k", kI8, k.sizes()));
  p.v = static_cast<int8_t*>(pointer(v, "cache_v", kI8, k.sizes()));
  p.k_scale = static_cast<uint16_t*>(pointer(ks, "scale_k", kScale, scales));
  p.v_scale = static_cast<uint16_t*>(pointer(vs, "scale_v", kScale, scales));
  for (int i = 0; i < 3; ++i) {
    if (stride(k, i, 0) != stride(v, i, 0)) refuse(PyExc_ValueError, "cache_k and cache_v must have the same strides");
    if (stride(ks, i, 0) != stride(vs, i, 0)) refuse(PyExc_ValueError, "scale_k and scale_v must have the same strides");
  }
  p.page_stride = stride(k, 0, p.dim), p.slot_stride = stride(k, 1, p.dim), p.head_stride = stride(k, 2, p.dim);
  p.scale_page_stride = stride(ks, 0, p.dim / 32), p.scale_slot_stride = stride(ks, 1, p.dim / 32);
  p.scale_head_stride = stride(ks, 2, p.dim / 32);
  p.batch = table.size(0), p.table_width = table.size(1);
  p.table = static_cast<const int32_t*>(pointer(table, "table", kI32, table.sizes()));
  p.table_stride = stride(table, 0, p.table_width);
  const Sizes<1> batch = {p.batch}, bounds = {p.batch + 1};
  p.kv_len = static_cast<const int32_t*>(pointer(tensor(a[5], "kv_len"), "kv_len", kI32, batch, true));
  p.new_start = static_cast<const int32_t*>(pointer(tensor(a[6], "new_start"), "new_start", kI32, bounds, true));
  p.total_new = total_new;
  return p;
}

// The type of a code, for calls that do not take it from a tensor.
at::ScalarType type_of_code(PyObject* o, unsigned types) {
  const int64_t code = integer(o);
  const at::ScalarType t = code == Q1_F32 ? at::kFloat : code == Q1_BF16 ? at::kBFloat16 : code == Q1_F16 ? at::kHalf : at::kByte;
  if (!is_type(t, types)) refuse(PyExc_TypeError, "dtype must be one of %s", names_of(types).c_str());
  return t;
}

// q, k, v, cos_sin, cache_k, cache_v, scale_k, scale_v, table, kv_len, new_start, q_out, interleaved, type code, stream
PyObject* rope_append_q8(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(a, count, 15, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &cs = tensor(a[3], "cos_sin");
    if (q.dim() != 2 || cs.dim() != 2) refuse(PyExc_ValueError, "q must be [tokens, heads * dim] and cos_sin [positions, rot]");
    const int64_t total = q.size(0);
    const q1_paged_q8 kv = paged_q8(a + 4, total);
    if (q.size(1) % kv.dim) refuse(PyExc_ValueError, "q must be [tokens, heads * dim] and cos_sin [positions, rot]");
    const int64_t heads = q.size(1) / kv.dim, width = kv.kv_heads * kv.dim;
    const Sizes<2> kv_shape = {total, width};
    const Sizes<3> out_shape = {total, heads, kv.dim};
    const at::ScalarType type = a[11] == Py_None ? type_of_code(a[13], kBf16 | kF16) : tensor(a[11], "q_out").scalar_type();
    void* pq = pointer(q, "q", kF32, q.sizes());
    at::Tensor out = given_or_new(a[11], "q_out", out_shape, q, type);
    check(q1_rope_append_q8(static_cast<const float*>(pq), stride(q, 0, heads * kv.dim),
                            static_cast<const float*>(pointer(k, "k", kF32, kv_shape)), stride(k, 0, width),
                            static_cast<const float*>(pointer(v, "v", kF32, kv_shape)), stride(v, 0, width),
                            static_cast<const float*>(pointer(cs, "cos_sin", kF32, cs.sizes(), true)), cs.size(0), cs.size(1),
                            a[12] == Py_True, heads, pointer(out, "q_out", kBf16 | kF16, out_shape, true), type_code(type), &kv,
                            reinterpret_cast<void*>(integer(a[14]))),
          "q1_rope_append_q8");
    return THPVariable_Wrap(out);
  });
}

// cache_k, cache_v, scale_k, scale_v, table, kv_len, new_start, tokens, type code, k_out, v_out, stream
PyObject* cache_read_q8(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(a, count, 12, [&]() -> PyObject* {
    const int64_t total = integer(a[7]);
    const q1_paged_q8 kv = paged_q8(a, total);
    if (total < 1) refuse(PyExc_ValueError, "tokens must be positive");
    const unsigned types = kF32 | kBf16 | kF16;
    const Sizes<3> shape = {total, kv.kv_heads, kv.dim};
    const at::ScalarType type = a[9] != Py_None    ? tensor(a[9], "k_out").scalar_type()
                                : a[10] != Py_None ? tensor(a[10], "v_out").scalar_type()
                                                   : type_of_code(a[8], types);
    const at::Tensor& like = THPVariable_Unpack(a[0]);
    at::Tensor k = given_or_new(a[9], "k_out", shape, like, type), v = given_or_new(a[10], "v_out", shape, like, type);
    void* pk = pointer(k, "k_out", types, shape, true);
    check(q1_cache_read_q8(&kv, type_code(type), pk, pointer(v, "v_out", type_bit(type), shape, true),
                           reinterpret_cast<void*>(integer(a[11]))),
          "q1_cache_read_q8");
    return Py_BuildValue("(NN)", THPVariable_Wrap(k), THPVariable_Wrap(v));
  });
}

// Sequences whose copies the attention's own workspace holds at once: a
// gigabyte of them, and one at least.
int64_t copied_at_once(int64_t max_new, int64_t heads, const q1_paged_q8& kv, int dtype) {
  const int64_t tokens = kv.table_width * kv.page_size;
  const int64_t one = q1_paged_attention_q8_workspace(max_new, heads, kv.kv_heads, kv.dim, dtype, tokens, 1);
  const int64_t two = q1_paged_attention_q8_workspace(max_new, heads, kv.kv_heads, kv.dim, dtype, tokens, 2);
  if (one < 0 || two <= one) return 1;
  const int64_t fit = (int64_t(1) << 30) / (two - one);
  return fit < 1 ? 1 : fit < kv.batch ? fit : kv.batch;
}

// q, cache_k, cache_v, scale_k, scale_v, table, kv_len, new_start, max_new, scale (or None), out, workspace, stream
PyObject* paged_attention_q8(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(a, count, 13, [&]() -> PyObject* {
    const at::Tensor& q = tensor(a[0], "q");
    if (q.dim() != 3) refuse(PyExc_ValueError, "q must be [tokens, heads, dim]");
    const int64_t total = q.size(0), heads = q.size(1), dim = q.size(2);
    const q1_paged_q8 kv = paged_q8(a + 1, total);
    if (kv.dim != dim) refuse(PyExc_ValueError, "q has dim %lld, the cache %lld", (long long)dim, (long long)kv.dim);
    void* pq = pointer(q, "q", kBf16 | kF16, q.sizes());
    const unsigned type = type_bit(q.scalar_type());
    const int dtype = type_code(q.scalar_type());
    const int64_t max_new = integer(a[8]);
    const double scale = a[9] == Py_None ? 1.0 / std::sqrt(double(dim)) : number(a[9]);
    at::Tensor out = given_or_new(a[10], "out", q.sizes(), q, q.scalar_type());
    at::Tensor ws;
    if (a[11] != Py_None) {
      ws = tensor(a[11], "workspace");
    } else {
      const int64_t bytes = q1_paged_attention_q8_workspace(max_new, heads, kv.kv_heads, dim, dtype, kv.table_width * kv.page_size,
                                                            copied_at_once(max_new, heads, kv, dtype));
      check(bytes < 0 ? bytes : Q1_OK, "q1_paged_attention_q8");
      ws = at::empty({bytes}, q.options().dtype(at::kByte));
    }
    check(q1_paged_attention_q8(pq, stride(q, 0, heads * dim), stride(q, 1, dim), heads, static_cast<float>(scale),
                                dtype, &kv, max_new, pointer(out, "out", type, q.sizes()),
                                stride(out, 0, heads * dim), stride(out, 1, dim), pointer(ws, "workspace", kU8, ws.sizes(), true),
                                ws.numel(), reinterpret_cast<void*>(integer(a[12]))),
          "q1_paged_attention_q8");
    return THPVariable_Wrap(out);
  });
}

// gate, up, activation code, want_y, want_q8, y, q, d, stream
PyObject* gated_act(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(a, count, 9, [&]() -> PyObject* {
    const at::Tensor &gate = tensor(a[0], "gate"), &up = tensor(a[1], "up");
    if (gate.dim() != 2) refuse(PyExc_ValueError, "gate must be [nvec, n]");
    const int64_t nvec = gate.size(0), n = gate.size(1);
    const unsigned type = type_bit(gate.scalar_type());
    if (!type) refuse(PyExc_TypeError, "gate has dtype %s, expected one of float32, bfloat16, float16", at::toString(gate.scalar_type()));
    const bool want_y = a[3] == Py_True, want_q8 = a[4] == Py_True;
    if (want_q8 && n % 32) refuse(PyExc_ValueError, "the q8_0 form needs n to be a multiple of 32");
    const Sizes<2> shape = {nvec, n}, scales = {nvec, n / 32};
    void* pg = pointer(gate, "gate", type, shape);
    void* pu = pointer(up, "up", type, shape);
    at::Tensor y, q, d;
    if (want_y) y = given_or_new(a[5], "y", shape, gate, gate.scalar_type());
    if (want_q8) q = given_or_new(a[6], "q", shape, gate, at::kChar), d = given_or_new(a[7], "d", scales, gate, at::kShort);
    check(q8_gated_act(pg, stride(gate, 0, n), pu, stride(up, 0, n), nvec, n, type_code(gate.scalar_type()),
                       static_cast<int>(integer(a[2])), want_y ? pointer(y, "y", type, shape) : nullptr, want_y ? stride(y, 0, n) : 0,
                       want_q8 ? static_cast<int8_t*>(pointer(q, "q", kI8, shape, true)) : nullptr,
                       want_q8 ? static_cast<uint16_t*>(pointer(d, "d", kScale, scales, true)) : nullptr,
                       reinterpret_cast<void*>(integer(a[8]))),
          "q8_gated_act");
    return Py_BuildValue("(NNN)", want_y ? THPVariable_Wrap(y) : Py_NewRef(Py_None), want_q8 ? THPVariable_Wrap(q) : Py_NewRef(Py_None),
                         want_q8 ? THPVariable_Wrap(d) : Py_NewRef(Py_None));
  });
}

// logits, uniform, temperature, top_k, top_p, min_p (tensors or numbers), out, stream
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(a, count, 8, [&]() -> PyObject* {
    const at::Tensor& logits = tensor(a[0], "logits");
    if (logits.dim() != 2) refuse(PyExc_ValueError, "logits must be [rows, vocab]");
    const Sizes<1> rows = {logits.size(0)};
    void* pl = pointer(logits, "logits", kF32 | kBf16 | kF16, logits.sizes());
    q1_sampling s = {};
    const auto real = [&](PyObject* o, const char* name, const float** each, float* all) {
      if (!PyFloat_Check(o) && !PyLong_Check(o) && THPVariable_Check(o))
        *each = static_cast<const float*>(pointer(o, name, kF32, rows, true));
      else
        *all = static_cast<float>(number(o));
    };
    real(a[2], "temperature", &s.temperature, &s.temperature_all);
    real(a[4], "top_p", &s.top_p, &s.top_p_all);
    real(a[5], "min_p", &s.min_p, &s.min_p_all);
    if (!PyLong_Check(a[3]) && THPVariable_Check(a[3])) {
      s.top_k = static_cast<const int32_t*>(pointer(a[3], "top_k", kI32, rows, true));
    } else {
      const int64_t k = integer(a[3]);  // beyond any vocabulary: as good as all
      s.top_k_all = k < 0 ? 0 : k > (int64_t(1) << 30) ? 1 << 30 : static_cast<int32_t>(k);
    }
    at::Tensor out = given_or_new(a[6], "out", rows, logits, at::kInt);
    check(q1_sample(pl, logits.size(0) > 1 ? logits.stride(0) : logits.size(1), rows[0], logits.size(1), type_code(logits.scalar_type()),
                    static_cast<const float*>(pointer(tensor(a[1], "uniform"), "uniform", kF32, rows, true)), &s,
                    static_cast<int32_t*>(pointer(out, "out", kI32, rows, true)), reinterpret_cast<void*>(integer(a[7]))),
          "q1_sample");
    return THPVariable_Wrap(out);
  });
}

// cache_k, cache_v, table, kv_len, new_start, total_new -> the bytes of the q1_paged_kv
PyObject* make_paged_kv(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(a, count, 6, [&]() -> PyObject* {
    const q1_paged_kv kv = paged_kv(a, integer(a[5]));
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&kv), sizeof kv);
  });
}

// cache_k, cache_v, scale_k, scale_v, table, kv_len, new_start, total_new -> the bytes of the q1_paged_q8
PyObject* make_paged_q8(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(a, count, 8, [&]() -> PyObject* {
    const q1_paged_q8 kv = paged_q8(a, integer(a[7]));
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&kv), sizeof kv);
  });
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_XSETREF(g_error, Py_NewRef(type));
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"set_error", set_error, METH_O, "The exception that a failed call raises."},
    {"add_rms_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(add_rms_norm)), METH_FASTCALL, nullptr},
    {"lora_add", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(lora_add)), METH_FASTCALL, nullptr},
    {"rope_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(rope_append)), METH_FASTCALL, nullptr},
    {"paged_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_attention)), METH_FASTCALL, nullptr},
    {"paged_kv", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(make_paged_kv)), METH_FASTCALL, nullptr},
    {"rope_append_q8", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(rope_append_q8)), METH_FASTCALL, nullptr},
    {"cache_read_q8", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(cache_read_q8)), METH_FASTCALL, nullptr},
    {"paged_attention_q8", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_attention_q8)), METH_FASTCALL, nullptr},
    {"gated_act", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(gated_act)), METH_FASTCALL, nullptr},
    {"sample", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(sample)), METH_FASTCALL, nullptr},
    {"paged_q8", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(make_paged_q8)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&kModule); }
