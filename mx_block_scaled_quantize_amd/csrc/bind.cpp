// Python binding of the serving entry points (rotary tables, rotation, cache
// append, paged attention) with the interpreter's own C interface.
//
// A decoding step makes a few of these calls per layer, each on kernels of a few
// microseconds, so what a call costs before its launch counts: a call among others takes 4.3
// to 7 us with this (one append, one small rotation), which marshalling in Python would
// multiply.  Checks of tensors are here, those of scalars in the library; the arithmetic is in
// libmx as everywhere else.

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPStream.h>

#include <cmath>

#include "../../include/mx.h"

namespace {

PyObject* g_check = nullptr;      // check(status) of the package: raises what a status stands for

const at::Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_VALUE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
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

mx_dtype_t dtype_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return MX_F32;
    case at::kBFloat16: return MX_BF16;
    case at::kHalf: return MX_F16;
    default: TORCH_CHECK_VALUE(false, "unsupported dtype (expected float32, bfloat16 or float16)");
  }
}

void check_heads(const at::Tensor& t, const char* name, const at::Device& dev) {
  TORCH_CHECK_VALUE(t.dim() == 3 && (t.stride(2) == 1 || t.size(2) <= 1), name,
                    " must be [tokens][heads][dim] with contiguous channels");
  TORCH_CHECK_VALUE(t.device() == dev, name, " must be on the device of the other arguments");
}

// Stride of a dimension; 0 where it has one element, whose stride means nothing but would decide on alignment.
int64_t stride_of(const at::Tensor& t, int dim) { return t.size(dim) > 1 ? t.stride(dim) : 0; }

void check_vector(const at::Tensor& t, const char* name, at::ScalarType dt, int64_t n, const at::Device& dev) {
  TORCH_CHECK_VALUE(t.scalar_type() == dt && t.dim() == 1 && t.size(0) == n && t.is_contiguous() && t.device() == dev, name,
                    " must be a contiguous ", dt, " vector of length ", n, " on the device of the other arguments");
}

void check_table(const at::Tensor& t, const at::Device& dev) {
  TORCH_CHECK_VALUE(t.scalar_type() == at::kFloat && t.dim() == 3 && t.size(2) == 2 && t.is_contiguous() && t.device() == dev,
                    "table must be a contiguous float32 tensor [rows][rot / 2][2] on the device of the other arguments");
}

void check_out(const at::Tensor& t, const char* name, const at::Tensor& like) {
  TORCH_CHECK_VALUE(t.sizes() == like.sizes() && t.scalar_type() == like.scalar_type() && t.is_contiguous() &&
                        t.device() == like.device(),
                    name, " must be contiguous with the shape, dtype and device of q");
}

mx_kv_cache_t cache_of(PyObject* const* a, const at::Device& dev) {
  const at::Tensor &k = tensor(a[0], "cache.k"), &ks = tensor(a[1], "cache.k_scales"), &v = tensor(a[2], "cache.v"),
                   &vs = tensor(a[3], "cache.v_scales");
  TORCH_CHECK_VALUE(k.dim() == 4, "cache codes must be [pages][kv_heads][page][dim]");
  const int64_t scales[4] = {k.size(0), k.size(1), k.size(2), k.size(3) / 32};
  TORCH_CHECK_VALUE(v.sizes() == k.sizes() && ks.sizes() == at::IntArrayRef(scales, 4) && vs.sizes() == ks.sizes(),
                    "cache tensors must be codes [pages][kv_heads][page][dim] and scales [..][dim / 32]");
  for (const at::Tensor* t : {&k, &ks, &v, &vs})
    TORCH_CHECK_VALUE(t->scalar_type() == at::kByte && t->is_contiguous() && t->device() == dev,
                      "cache tensors must be contiguous uint8 tensors on the device of the other arguments");
  for (int i = 1; i < 4; ++i) TORCH_CHECK_VALUE(k.size(i) <= INT32_MAX, "cache shape out of range");
  mx_kv_cache_t c;
  c.k = static_cast<uint8_t*>(k.data_ptr());
  c.k_scales = static_cast<uint8_t*>(ks.data_ptr());
  c.v = static_cast<uint8_t*>(v.data_ptr());
  c.v_scales = static_cast<uint8_t*>(vs.data_ptr());
  c.pages = k.size(0);
  c.kv_heads = int32_t(k.size(1));
  c.page = int32_t(k.size(2));
  c.dim = int32_t(k.size(3));
  return c;
}

int narrow_int(int64_t v, const char* what) {
  TORCH_CHECK_VALUE(v >= INT32_MIN && v <= INT32_MAX, what, " out of range");
  return int(v);
}

// The library launches on the current device: makes it the tensors' own for the
// time of a call, and names their current stream.
struct OnDevice {
  explicit OnDevice(const at::Device& dev) {
    TORCH_CHECK_VALUE(dev.is_cuda(), "libmx works on device tensors only");
    TORCH_CHECK(hipGetDevice(&before) == hipSuccess, "hipGetDevice failed");
    here = dev.has_index() ? dev.index() : before;
    if (here != before) TORCH_CHECK(hipSetDevice(here) == hipSuccess, "hipSetDevice failed");
    stream = c10::hip::getCurrentHIPStream(c10::DeviceIndex(here)).stream();
  }
  ~OnDevice() {
    if (here != before) (void)hipSetDevice(before);
  }
  int before = 0, here = 0;
  hipStream_t stream = nullptr;
};

void check_status(mx_status_t st) {
  if (st == MX_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "i", int(st));
  Py_XDECREF(r);
  if (r) PyErr_SetString(PyExc_RuntimeError, mx_status_str(st));
  throw python_error();
}

void check_args(Py_ssize_t n, Py_ssize_t want) {
  TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n);
}

// rope_table(rows, rot, base, scaling, factor, orig_len, out)
PyObject* rope_table(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_args(n, 7);
  const at::Tensor& out = tensor(a[6], "out");
  OnDevice on(out.device());
  check_status(mx_rope_table(integer(a[0]), narrow_int(integer(a[1]), "rot"), real(a[2]),
                             mx_rope_scaling_t(narrow_int(integer(a[3]), "scaling")), real(a[4]), integer(a[5]),
                             static_cast<float*>(out.data_ptr()), on.stream));
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// rope(x, pos, table, layout, inverse, out or None) -> out
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_args(n, 6);
  const at::Tensor &x = tensor(a[0], "x"), &pos = tensor(a[1], "pos"), &table = tensor(a[2], "table");
  const mx_dtype_t dt = dtype_of(x);
  const at::Device dev = x.device();
  check_heads(x, "x", dev);
  check_table(table, dev);
  check_vector(pos, "pos", at::kInt, x.size(0), dev);
  const bool inverse = truth(a[4]);
  OnDevice on(dev);
  at::Tensor out;
  if (a[5] == Py_None) {
    out = at::empty(x.sizes(), x.options());
  } else {
    out = tensor(a[5], "out");
    check_heads(out, "out", dev);
    TORCH_CHECK_VALUE(out.sizes() == x.sizes() && out.scalar_type() == x.scalar_type(),
                      "out must have the shape and dtype of x");
  }
  check_status(mx_rope(x.data_ptr(), dt, x.size(0), narrow_int(x.size(1), "heads"), narrow_int(x.size(2), "dim"),
                       stride_of(x, 0), stride_of(x, 1), static_cast<const int32_t*>(pos.data_ptr()),
                       static_cast<const float*>(table.data_ptr()), table.size(0), narrow_int(2 * table.size(1), "rot"),
                       mx_rope_layout_t(integer(a[3])), inverse, out.data_ptr(), stride_of(out, 0), stride_of(out, 1),
                       on.stream));
  return THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// kv_append(k, v, cache x 4, slots, pos, table, layout, q, q_out): pos, table, q and q_out may be None
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_args(n, 12);
  const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &slots = tensor(a[6], "slots");
  const mx_dtype_t dt = dtype_of(k);
  const at::Device dev = k.device();
  const mx_kv_cache_t cache = cache_of(a + 2, dev);
  check_heads(k, "k", dev);
  check_heads(v, "v", dev);
  const int64_t tokens = k.size(0);
  TORCH_CHECK_VALUE(v.sizes() == k.sizes() && v.scalar_type() == k.scalar_type() && k.size(1) == cache.kv_heads &&
                        k.size(2) == cache.dim,
                    "k and v must be [tokens][kv_heads][dim] of one dtype, matching the cache");
  check_vector(slots, "slots", at::kLong, tokens, dev);
  const bool rotate = a[8] != Py_None;
  const int32_t* pos = nullptr;
  const float* table = nullptr;
  int64_t rows = 0, rot = 2;
  if (rotate) {
    const at::Tensor& t = tensor(a[8], "table");
    check_table(t, dev);
    // a null table stands for no rotation in the library, and one without rows has no address
    TORCH_CHECK_VALUE(t.size(0) > 0, "a rotation needs a table with rows");
    TORCH_CHECK_VALUE(a[7] != Py_None, "a rotation needs pos");
    const at::Tensor& p = tensor(a[7], "pos");
    check_vector(p, "pos", at::kInt, tokens, dev);
    pos = static_cast<const int32_t*>(p.data_ptr());
    table = static_cast<const float*>(t.data_ptr());
    rows = t.size(0);
    rot = 2 * t.size(1);
  }
  OnDevice on(dev);
  at::Tensor out;
  const void* q = nullptr;
  int64_t heads = 0, qt = 0, qh = 0;
  if (a[10] != Py_None) {
    const at::Tensor& t = tensor(a[10], "q");
    check_heads(t, "q", dev);
    TORCH_CHECK_VALUE(rotate, "q is only rotated: it needs a table");
    TORCH_CHECK_VALUE(t.size(0) == tokens && t.size(2) == cache.dim && t.scalar_type() == k.scalar_type(),
                      "q must be [tokens][heads][dim] with the dtype of k");
    if (a[11] == Py_None) {
      out = at::empty(t.sizes(), t.options());
    } else {
      out = tensor(a[11], "q_out");
      check_out(out, "q_out", t);
    }
    q = t.data_ptr();
    heads = t.size(1);
    qt = stride_of(t, 0);
    qh = stride_of(t, 1);
    if (heads == 0) q = nullptr;
  }
  check_status(mx_kv_append(k.data_ptr(), v.data_ptr(), dt, tokens, stride_of(k, 0), stride_of(k, 1), stride_of(v, 0),
                            stride_of(v, 1), &cache, static_cast<const int64_t*>(slots.data_ptr()), pos, table, rows,
                            narrow_int(rot, "rot"), mx_rope_layout_t(integer(a[9])), q, narrow_int(heads, "heads"), qt, qh,
                            out.defined() ? out.data_ptr() : nullptr, on.stream));
  if (!out.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// paged_attention(q, cache x 4, page_table, cu, lens, window, scale or None, lse, max_q, max_kv, out or None)
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_args(n, 14);
  const at::Tensor &q = tensor(a[0], "q"), &pages = tensor(a[5], "page_table"), &cu = tensor(a[6], "cu"),
                   &lens = tensor(a[7], "lens");
  const mx_dtype_t dt = dtype_of(q);
  const at::Device dev = q.device();
  const mx_kv_cache_t cache = cache_of(a + 1, dev);
  check_heads(q, "q", dev);
  const int64_t tokens = q.size(0), heads = q.size(1), requests = lens.dim() == 1 ? lens.size(0) : -1;
  TORCH_CHECK_VALUE(q.size(2) == cache.dim && cache.kv_heads > 0 && heads % cache.kv_heads == 0,
                    "q must have the cache's dim and a multiple of its heads");
  check_vector(lens, "lens", at::kInt, requests, dev);
  check_vector(cu, "cu", at::kInt, requests + 1, dev);
  TORCH_CHECK_VALUE(pages.scalar_type() == at::kInt && pages.dim() == 2 && pages.size(0) == requests &&
                        (pages.stride(1) == 1 || pages.size(1) <= 1) && pages.device() == dev,
                    "page_table must be an int32 tensor [requests][pages] with contiguous rows");
  const int64_t window = integer(a[8]), max_q = integer(a[11]), max_kv = integer(a[12]);
  const double scale = a[9] == Py_None ? 1.0 / std::sqrt(double(cache.dim)) : real(a[9]);
  const bool want_lse = truth(a[10]);
  OnDevice on(dev);
  at::Tensor out, lse, space;
  if (a[13] == Py_None) {
    out = at::empty(q.sizes(), q.options());
  } else {
    out = tensor(a[13], "out");
    check_out(out, "out", q);
  }
  if (want_lse) lse = at::empty({tokens, heads}, q.options().dtype(at::kFloat));
  int64_t need = 0;
  check_status(mx_paged_attention_workspace(tokens, narrow_int(heads, "heads"), cache.kv_heads, cache.dim, requests, max_q,
                                            max_kv, window, &need));
  if (need) space = at::empty({need}, q.options().dtype(at::kByte));
  check_status(mx_paged_attention(
      q.data_ptr(), dt, tokens, int(heads), stride_of(q, 0), stride_of(q, 1), &cache,
      static_cast<const int32_t*>(pages.data_ptr()), pages.stride(0), pages.size(1),
      static_cast<const int32_t*>(cu.data_ptr()), static_cast<const int32_t*>(lens.data_ptr()), requests, max_q, max_kv,
      window, float(scale), out.data_ptr(), want_lse ? static_cast<float*>(lse.data_ptr()) : nullptr,
      need ? space.data_ptr() : nullptr, need, on.stream));
  if (!want_lse) return THPVariable_Wrap(std::move(out));
  THPObjectPtr o(THPVariable_Wrap(std::move(out))), s(THPVariable_Wrap(std::move(lse)));
  if (!o || !s) throw python_error();
  return PyTuple_Pack(2, o.get(), s.get());
  END_HANDLE_TH_ERRORS
}

// set_check(callable): what raises for a status
PyObject* set_check(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(g_check, f);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef fast(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {fast<rope_table>("rope_table"),
                           fast<rope>("rope"),
                           fast<kv_append>("kv_append"),
                           fast<paged_attention>("paged_attention"),
                           {"set_check", set_check, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&g_module); }
