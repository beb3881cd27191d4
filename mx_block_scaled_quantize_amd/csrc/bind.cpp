// Python binding of the serving entry points (rotary tables, rotation, cache
// append, paged attention, the cache's pages, beam selection) with the interpreter's own C interface.
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
#include <ATen/hip/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPStream.h>

#include <cmath>
#include <vector>

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

// One cache (four tensors) or a sequence of them, one for each layer.
std::vector<mx_kv_cache_t> layers_of(PyObject* o, const char* name, at::Device& dev) {
  THPObjectPtr seq(PySequence_Fast(o, "expected a KVCache or a sequence of KVCaches"));
  if (!seq) throw python_error();
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq.get());
  PyObject** items = PySequence_Fast_ITEMS(seq.get());
  TORCH_CHECK_VALUE(n > 0, name, " must have a layer");
  std::vector<mx_kv_cache_t> caches;
  if (THPVariable_Check(items[0])) {
    TORCH_CHECK_VALUE(n == 4, name, " must be a KVCache or a sequence of KVCaches");
    dev = THPVariable_Unpack(items[0]).device();
    caches.push_back(cache_of(items, dev));
    return caches;
  }
  for (Py_ssize_t l = 0; l < n; ++l) {
    THPObjectPtr one(PySequence_Fast(items[l], "expected a KVCache or a sequence of KVCaches"));
    if (!one) throw python_error();
    TORCH_CHECK_VALUE(PySequence_Fast_GET_SIZE(one.get()) == 4, name, " must be a KVCache or a sequence of KVCaches");
    PyObject** four = PySequence_Fast_ITEMS(one.get());
    if (l == 0) dev = tensor(four[0], name).device();
    caches.push_back(cache_of(four, dev));
  }
  return caches;
}

int layer_count(const std::vector<mx_kv_cache_t>& c) { return narrow_int(int64_t(c.size()), "layers"); }

const int32_t* ints(const at::Tensor& t) { return static_cast<const int32_t*>(t.data_ptr()); }
int32_t* ints_out(const at::Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); }

void check_page_table(const at::Tensor& t, int64_t rows, const at::Device& dev) {
  TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && t.dim() == 2 && t.size(0) == rows &&
                        (t.stride(1) == 1 || t.size(1) <= 1) && t.device() == dev,
                    "page_table must be an int32 tensor [rows][pages] with contiguous rows, a row for each length");
}

// Rows that do not overlap: a table expanded from one row is no table to write or to count twice.
int64_t row_stride(const at::Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

int64_t vector_size(const at::Tensor& t, const char* name) {
  TORCH_CHECK_VALUE(t.dim() == 1, name, " must be a vector");
  return t.size(0);
}

// A new tensor, made without the dispatcher's way to the same function: these calls make up to seven.
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType dt, const at::Device& dev) {
  return at::detail::empty_cuda(shape, dt, dev, std::nullopt);
}

// The n-th of the tensors to write to, or a new one.
at::Tensor out_or_new(PyObject* out, Py_ssize_t n, const char* name, at::IntArrayRef shape, at::ScalarType dt,
                      const at::Device& dev) {
  if (out == Py_None) return fresh(shape, dt, dev);
  const at::Tensor& t = tensor(PyTuple_GET_ITEM(out, n), name);
  TORCH_CHECK_VALUE(t.sizes() == shape && t.scalar_type() == dt && t.is_contiguous() && t.device() == dev, name,
                    " must be a contiguous ", dt, " tensor of shape ", shape, " on the device of the other arguments");
  return t;
}

void check_out_tuple(PyObject* out, Py_ssize_t n) {
  TORCH_CHECK_VALUE(out == Py_None || (PyTuple_Check(out) && PyTuple_GET_SIZE(out) == n), "out must be a tuple of ", n,
                    " tensors");
}

PyObject* wrapped(std::initializer_list<at::Tensor> tensors) {
  THPObjectPtr r(PyTuple_New(Py_ssize_t(tensors.size())));
  if (!r) throw python_error();
  Py_ssize_t i = 0;
  for (const at::Tensor& t : tensors) {
    PyObject* o = Py_None;
    if (t.defined()) {
      o = THPVariable_Wrap(t);
      if (!o) throw python_error();
    } else {
      Py_INCREF(o);
    }
    PyTuple_SET_ITEM(r.get(), i++, o);
  }
  return r.release();
}

// kv_copy(src, src_pages, dst, dst_pages)
PyObject* kv_copy(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_args(n, 4);
  at::Device dev(at::kCPU), other(at::kCPU);
  const std::vector<mx_kv_cache_t> src = layers_of(a[0], "src", dev), dst = layers_of(a[2], "dst", other);
  TORCH_CHECK_VALUE(dev == other, "src and dst must be on one device");
  TORCH_CHECK_VALUE(src.size() == dst.size(), "src and dst must have the same layers");
  const at::Tensor &from = tensor(a[1], "src_pages"), &to = tensor(a[3], "dst_pages");
  const int64_t count = vector_size(from, "src_pages");
  check_vector(from, "src_pages", at::kInt, count, dev);
  check_vector(to, "dst_pages", at::kInt, count, dev);
  OnDevice on(dev);
  check_status(mx_kv_copy(src.data(), dst.data(), layer_count(src), ints(from), ints(to), count, on.stream));
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// kv_fork(caches, refs, page_table, lens, cu or None, parents or None, release, tokens, cols or None, out or None)
PyObject* kv_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_args(n, 10);
  at::Device dev(at::kCPU);
  const std::vector<mx_kv_cache_t> caches = layers_of(a[0], "caches", dev);
  const at::Tensor &refs = tensor(a[1], "refs"), &table = tensor(a[2], "page_table"), &lens = tensor(a[3], "lens");
  const int64_t rows = vector_size(lens, "lens"), pages = caches[0].pages;
  check_vector(refs, "refs", at::kInt, pages, dev);
  check_vector(lens, "lens", at::kInt, rows, dev);
  check_page_table(table, rows, dev);
  int64_t children = rows;
  const int32_t *parents = nullptr, *cu = nullptr;
  if (a[5] != Py_None) {
    const at::Tensor& t = tensor(a[5], "parents");
    TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && t.is_contiguous() && t.device() == dev,
                      "parents must be a contiguous int32 tensor on the device of the other arguments");
    children = t.numel();
    parents = ints(t);
  }
  const int64_t tokens = integer(a[7]);
  TORCH_CHECK_VALUE(tokens >= 0, "tokens must not be negative");
  if (a[4] != Py_None) {
    const at::Tensor& t = tensor(a[4], "cu");
    check_vector(t, "cu", at::kInt, children + 1, dev);
    cu = ints(t);
  }
  const bool release = truth(a[6]);
  PyObject* out = a[9];
  check_out_tuple(out, 4);
  int64_t cols = a[8] == Py_None ? table.size(1) : integer(a[8]);
  if (out != Py_None && a[8] == Py_None) {
    const at::Tensor& t = tensor(PyTuple_GET_ITEM(out, 1), "out's page_table");
    if (t.dim() == 2) cols = t.size(1);
  }
  TORCH_CHECK_VALUE(cols >= table.size(1), "the new table must not be narrower than the old one");
  OnDevice on(dev);
  int64_t need = 0;
  check_status(mx_kv_fork_workspace(pages, rows, children, tokens, caches[0].page, &need));
  at::Tensor r = out_or_new(out, 0, "out's refs", {pages}, at::kInt, dev),
             t = out_or_new(out, 1, "out's page_table", {children, cols}, at::kInt, dev),
             l = out_or_new(out, 2, "out's lens", {children}, at::kInt, dev),
             s = out_or_new(out, 3, "out's slots", {tokens}, at::kLong, dev),
             space = fresh({need}, at::kByte, dev);
  // a parents tensor without elements has no address, which would stand for children that continue their own rows;
  // nothing is read through this one
  if (a[5] != Py_None && children == 0) parents = ints(space);
  check_status(mx_kv_fork(caches.data(), layer_count(caches), ints(refs), ints(table), row_stride(table), table.size(1),
                          ints(lens), rows, parents, children, cu, tokens, release, ints_out(r), ints_out(t), cols,
                          ints_out(l), static_cast<int64_t*>(s.data_ptr()), space.data_ptr(), need, on.stream));
  return wrapped({r, t, l, s});
  END_HANDLE_TH_ERRORS
}

// kv_free(refs, page_table, lens, page, keep or None, out or None)
PyObject* kv_free(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_args(n, 6);
  const at::Tensor &refs = tensor(a[0], "refs"), &table = tensor(a[1], "page_table"), &lens = tensor(a[2], "lens");
  const at::Device dev = refs.device();
  const int64_t rows = vector_size(lens, "lens"), pages = vector_size(refs, "refs");
  check_vector(refs, "refs", at::kInt, pages, dev);
  check_vector(lens, "lens", at::kInt, rows, dev);
  check_page_table(table, rows, dev);
  const int32_t* keep = nullptr;
  if (a[4] != Py_None) {
    const at::Tensor& t = tensor(a[4], "keep");
    check_vector(t, "keep", at::kInt, rows, dev);
    keep = ints(t);
  }
  check_out_tuple(a[5], 2);
  OnDevice on(dev);
  at::Tensor r = out_or_new(a[5], 0, "out's refs", {pages}, at::kInt, dev),
             l = out_or_new(a[5], 1, "out's lens", {rows}, at::kInt, dev);
  const int page = narrow_int(integer(a[3]), "page");
  int64_t need = 0;
  check_status(mx_kv_free_workspace(pages, rows, table.size(1), page, &need));
  at::Tensor space;
  if (need) space = fresh({need}, at::kByte, dev);
  check_status(mx_kv_free(ints(refs), pages, page, ints(table), row_stride(table), table.size(1), ints(lens), rows, keep,
                          ints_out(r), ints_out(l), need ? space.data_ptr() : nullptr, need, on.stream));
  return wrapped({r, l});
  END_HANDLE_TH_ERRORS
}

// kv_compact(caches, refs, page_table, lens, out or None)
PyObject* kv_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_args(n, 5);
  at::Device dev(at::kCPU);
  const std::vector<mx_kv_cache_t> caches = layers_of(a[0], "caches", dev);
  const at::Tensor &refs = tensor(a[1], "refs"), &table = tensor(a[2], "page_table"), &lens = tensor(a[3], "lens");
  const int64_t rows = vector_size(lens, "lens"), pages = caches[0].pages;
  check_vector(refs, "refs", at::kInt, pages, dev);
  check_vector(lens, "lens", at::kInt, rows, dev);
  check_page_table(table, rows, dev);
  check_out_tuple(a[4], 3);
  OnDevice on(dev);
  int64_t need = 0;
  check_status(mx_kv_compact_workspace(pages, &need));
  at::Tensor r = out_or_new(a[4], 0, "out's refs", {pages}, at::kInt, dev),
             t = out_or_new(a[4], 1, "out's page_table", table.sizes(), at::kInt, dev),
             u = out_or_new(a[4], 2, "out's count", {1}, at::kInt, dev), space = fresh({need}, at::kByte, dev);
  check_status(mx_kv_compact(caches.data(), layer_count(caches), ints(refs), ints(table), row_stride(table), table.size(1),
                             ints(lens), rows, ints_out(r), ints_out(t), ints_out(u), space.data_ptr(), need, on.stream));
  return wrapped({r, t, u});
  END_HANDLE_TH_ERRORS
}

// beam_select(logits, scores, width or None, finished or None, eos, pad, history or None, lens or None)
PyObject* beam_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_args(n, 8);
  const at::Tensor &x = tensor(a[0], "logits"), &scores = tensor(a[1], "scores");
  const mx_dtype_t dt = dtype_of(x);
  const at::Device dev = x.device();
  TORCH_CHECK_VALUE(x.dim() == 3 && (x.stride(2) == 1 || x.size(2) <= 1),
                    "logits must be [requests][beams][vocab] with contiguous tokens");
  const int64_t requests = x.size(0), beams = x.size(1);
  const int64_t one[2] = {requests, beams};
  auto check_beams = [&](const at::Tensor& t, const char* name, bool ok) {
    TORCH_CHECK_VALUE(ok && t.sizes() == at::IntArrayRef(one, 2) && t.is_contiguous() && t.device() == dev, name,
                      " must be a contiguous tensor [requests][beams] on the device of the other arguments"
                      " (scores float32, finished bool or uint8, lens int32)");
  };
  check_beams(scores, "scores", scores.scalar_type() == at::kFloat);
  const int64_t width = a[2] == Py_None ? beams : integer(a[2]);
  const uint8_t* finished = nullptr;
  if (a[3] != Py_None) {
    const at::Tensor& t = tensor(a[3], "finished");
    check_beams(t, "finished", t.scalar_type() == at::kBool || t.scalar_type() == at::kByte);
    finished = static_cast<const uint8_t*>(t.data_ptr());
  }
  const int64_t eos = integer(a[4]), pad = integer(a[5]);
  const int32_t *history = nullptr, *lens = nullptr;
  int64_t cols = 0;
  TORCH_CHECK_VALUE((a[6] == Py_None) == (a[7] == Py_None), "history and lens are given together");
  if (a[6] != Py_None) {
    const at::Tensor &h = tensor(a[6], "history"), &l = tensor(a[7], "lens");
    check_beams(l, "lens", l.scalar_type() == at::kInt);
    TORCH_CHECK_VALUE(h.scalar_type() == at::kInt && h.dim() == 3 && h.size(0) == requests && h.size(1) == beams &&
                          h.is_contiguous() && h.device() == dev,
                      "history must be a contiguous int32 tensor [requests][beams][tokens]");
    history = ints(h);
    lens = ints(l);
    cols = h.size(2);
  }
  OnDevice on(dev);
  int64_t need = 0;
  check_status(mx_beam_select_workspace(requests, beams, x.size(2), width, &need));
  at::Tensor s = fresh({requests, width}, at::kFloat, dev), p = fresh({requests, width}, at::kInt, dev),
             t = fresh({requests, width}, at::kInt, dev), f = fresh({requests, width}, at::kBool, dev), h, l,
             space = fresh({need}, at::kByte, dev);
  if (a[6] != Py_None) {
    h = fresh({requests, width, cols}, at::kInt, dev);
    l = fresh({requests, width}, at::kInt, dev);
  }
  check_status(mx_beam_select(x.data_ptr(), dt, requests, beams, x.size(2), stride_of(x, 0), stride_of(x, 1),
                              static_cast<const float*>(scores.data_ptr()), finished, width, eos, pad, history, lens, cols,
                              static_cast<float*>(s.data_ptr()), ints_out(p), ints_out(t),
                              static_cast<uint8_t*>(f.data_ptr()), h.defined() ? ints_out(h) : nullptr,
                              l.defined() ? ints_out(l) : nullptr, space.data_ptr(), need, on.stream));
  return wrapped({s, p, t, f, h, l});
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
                           fast<kv_copy>("kv_copy"),
                           fast<kv_fork>("kv_fork"),
                           fast<kv_free>("kv_free"),
                           fast<kv_compact>("kv_compact"),
                           fast<beam_select>("beam_select"),
                           {"set_check", set_check, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&g_module); }
