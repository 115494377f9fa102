// paged_binding.cpp -- Python binding of the paged-cache entry points (a CPython module over
// torch's C++ tensors): checks, output allocation and the call to the C ABI in one step from
// Python, because a decoding step makes these calls in every layer and their launches take no
// longer than a Python-level marshalling of their arguments would.  paged.py holds the public
// functions.  Every function returns its outputs, or the library's error code as an int.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <exception>

#include "entmax_attn.h"

namespace {

struct Refused {};  // a Python exception is set

[[noreturn]] void refuse(const char* format, ...) {
  va_list a;
  va_start(a, format);
  PyErr_FormatV(PyExc_ValueError, format, a);
  va_end(a);
  throw Refused();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
    throw Refused();
  }
  return THPVariable_Unpack(o);
}

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}

int int32(PyObject* o, const char* name) {
  const long long v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse("%s is out of range", name);
  return static_cast<int>(v);
}

// an int32 CUDA tensor of `dim` dimensions on dev with a unit-stride last dimension
const at::Tensor& ints(PyObject* o, const char* name, int dim, at::Device dev) {
  const at::Tensor& t = tensor(o, name);
  if (!t.is_cuda() || t.device() != dev || t.scalar_type() != at::kInt || t.dim() != dim ||
      (t.size(dim - 1) > 1 && t.stride(dim - 1) != 1 && t.numel() > 0) || t.size(dim - 1) > INT32_MAX)
    refuse("%s must be a %d-D int32 CUDA tensor with a unit-stride last dimension, on the device "
           "of the others", name, dim);
  return t;
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
  return at::detail::empty_cuda(shape, type, dev, c10::nullopt);
}

// Elements [from, from + n) of a 1-D tensor, as a tensor of its own on the same storage.
at::Tensor piece(const at::Tensor& base, int64_t from, int64_t n) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(base.storage()),
                                                          base.key_set(), base.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(from);
  t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
  return t;
}

// The given output, or a new one; what was given has to be contiguous, of this shape and type.
at::Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type,
                  at::Device dev) {
  if (o == Py_None) return empty(shape, type, dev);
  const at::Tensor& t = tensor(o, name);
  if (t.sizes() != shape || t.scalar_type() != type || t.device() != dev || !t.is_contiguous())
    refuse("%s must be contiguous, of the documented shape and dtype, on the device of the inputs",
           name);
  return t;
}

// Whether two tensors of one shape are laid out alike: a dimension of one element may carry any
// stride.
bool same_layout(const at::Tensor& a, const at::Tensor& b) {
  for (int64_t i = 0; i < a.dim(); ++i)
    if (a.size(i) > 1 && a.stride(i) != b.stride(i)) return false;
  return true;
}

struct Cache {
  const at::Tensor& k;
  const at::Tensor& v;
  int pages, heads, page, d, dtype;
  int64_t ps, hs, ss;
  at::Device dev;
};

Cache cache(PyObject* ko, PyObject* vo) {
  const at::Tensor &k = tensor(ko, "k_cache"), &v = tensor(vo, "v_cache");
  if (!k.is_cuda() || k.dim() != 4 || k.stride(3) != 1 ||
      (k.scalar_type() != at::kFloat && k.scalar_type() != at::kBFloat16))
    refuse("k_cache must be a float32 or bfloat16 CUDA tensor [num_pages, Hkv, page_size, d] with "
           "a unit-stride last dimension");
  if (v.sizes() != k.sizes() || !same_layout(k, v) || v.scalar_type() != k.scalar_type() ||
      v.device() != k.device())
    refuse("v_cache must have the shape, strides, dtype and device of k_cache");
  for (int i = 0; i < 4; ++i)
    if (k.size(i) > INT32_MAX) refuse("the cache is too large");
  const int64_t d = k.size(3);
  // a dimension of one element may carry any stride: one that the library accepts
  auto stride = [&](int i) { return k.size(i) > 1 ? k.stride(i) : d; };
  return {k, v, static_cast<int>(k.size(0)), static_cast<int>(k.size(1)),
          static_cast<int>(k.size(2)), static_cast<int>(d),
          k.scalar_type() == at::kFloat ? ENTMAX_ATTN_FP32 : ENTMAX_ATTN_BF16, stride(0),
          stride(1), stride(2), k.device()};
}

// Runs f with below-autograd dispatch and C++ exceptions turned into Python's.
template <typename F>
PyObject* guarded(const F& f) {
  try {
    at::AutoDispatchBelowADInplaceOrView below;
    return f();
  } catch (const Refused&) {
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    PyErr_SetString(type ? type : PyExc_MemoryError, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

bool count(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments expected", want);
  return false;
}

// lens, new_lens, free_pages, free_start, block_tables, page_size, n_new, padded, slots, lens_out,
// cu_new, free_next
PyObject* page_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 12)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Device dev = tensor(a[0], "lens").device();
    const at::Tensor &lens = ints(a[0], "lens", 1, dev), &add = ints(a[1], "new_lens", 1, dev),
                     &pool = ints(a[2], "free_pages", 1, dev),
                     &start = ints(a[3], "free_start", 1, dev),
                     &tables = ints(a[4], "block_tables", 2, dev);
    const int64_t B = tables.size(0), W = tables.size(1);
    if (lens.size(0) != B || add.size(0) != B || start.size(0) != 1 || B > INT32_MAX)
      refuse("lens and new_lens must be [B], free_start [1], block_tables [B, W]");
    const int page = int32(a[5], "page_size"), n_new = int32(a[6], "n_new");
    if (n_new < 0) refuse("n_new must not be negative");
    const int padded = PyObject_IsTrue(a[7]);
    if (padded < 0) throw Refused();
    const c10::cuda::CUDAGuard on(dev);
    const at::Tensor slots = padded ? output(a[8], "slots", {B, n_new}, at::kLong, dev)
                                    : output(a[8], "slots", {n_new}, at::kLong, dev);
    at::Tensor lens_out, cu, next;
    if (a[9] == Py_None && a[10] == Py_None && a[11] == Py_None) {
      // one allocation, each 16-byte aligned (the packed forward pass wants cu_new so)
      const int64_t at_lens = (B + 4) / 4 * 4, at_next = at_lens + (B + 3) / 4 * 4;
      const at::Tensor all = empty({at_next + 1}, at::kInt, dev);
      cu = piece(all, 0, B + 1);
      lens_out = piece(all, at_lens, B);
      next = piece(all, at_next, 1);
    } else {
      lens_out = output(a[9], "lens_out", {B}, at::kInt, dev);
      cu = output(a[10], "cu_new", {B + 1}, at::kInt, dev);
      next = output(a[11], "free_next", {1}, at::kInt, dev);
    }
    const int rc = entmax_attn_page_tables(
        static_cast<const int32_t*>(lens.const_data_ptr()),
        static_cast<const int32_t*>(add.const_data_ptr()),
        static_cast<const int32_t*>(pool.const_data_ptr()), static_cast<int>(pool.size(0)),
        static_cast<const int32_t*>(start.const_data_ptr()),
        static_cast<int32_t*>(tables.mutable_data_ptr()), B > 1 ? tables.stride(0) : W,
        static_cast<int>(W), static_cast<int>(B), page,
        n_new ? static_cast<int64_t*>(slots.mutable_data_ptr()) : nullptr, n_new, padded,
        static_cast<int32_t*>(lens_out.mutable_data_ptr()),
        static_cast<int32_t*>(cu.mutable_data_ptr()),
        static_cast<int32_t*>(next.mutable_data_ptr()),
        c10::cuda::getCurrentCUDAStream(dev.index()).stream());
    if (rc != ENTMAX_ATTN_OK) return PyLong_FromLong(rc);
    return Py_BuildValue("(NNNN)", THPVariable_Wrap(slots), THPVariable_Wrap(lens_out),
                         THPVariable_Wrap(cu), THPVariable_Wrap(next));
  });
}

// k, v, k_cache, v_cache, slots
PyObject* paged_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 5)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Cache c = cache(a[2], a[3]);
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &slots = tensor(a[4], "slots");
    const int64_t dim = k.dim();
    if (dim != 3 && dim != 4) refuse("k must be [B, Hkv, T, d] or packed [Hkv, N, d]");
    const int64_t B = dim == 4 ? k.size(0) : 1, H = k.size(dim - 3), T = k.size(dim - 2);
    if (H != c.heads || k.size(dim - 1) != c.d || k.scalar_type() != c.k.scalar_type() ||
        k.device() != c.dev || k.stride(dim - 1) != 1)
      refuse("k must have the cache's heads, head size, dtype and device, and unit-stride rows");
    if (v.sizes() != k.sizes() || !same_layout(k, v) ||
        v.scalar_type() != k.scalar_type() || v.device() != c.dev)
      refuse("v must have the shape, strides, dtype and device of k");
    if (slots.scalar_type() != at::kLong || slots.device() != c.dev || !slots.is_contiguous() ||
        slots.numel() != B * T)
      refuse("slots must be a contiguous int64 tensor, one per new token");
    if (B * T == 0) Py_RETURN_NONE;
    if (B > INT32_MAX || T > INT32_MAX) refuse("too many tokens");
    const c10::cuda::CUDAGuard on(c.dev);
    const int rc = entmax_attn_paged_append(
        k.const_data_ptr(), v.const_data_ptr(), B > 1 ? k.stride(0) : 0,
        H > 1 ? k.stride(dim - 3) : 0, T > 1 ? k.stride(dim - 2) : 0, c.k.mutable_data_ptr(),
        c.v.mutable_data_ptr(), c.ps, c.hs, c.ss, c.pages, c.page,
        static_cast<const int64_t*>(slots.const_data_ptr()), static_cast<int>(B),
        static_cast<int>(H), static_cast<int>(T), c.d, c.dtype,
        c10::cuda::getCurrentCUDAStream(c.dev.index()).stream());
    if (rc != ENTMAX_ATTN_OK) return PyLong_FromLong(rc);
    Py_RETURN_NONE;
  });
}

// q, k_cache, v_cache, block_tables, seq_lens, alpha, n_iter, max_len, out, tau, workspace
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 11)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Cache c = cache(a[1], a[2]);
    const at::Tensor& q = tensor(a[0], "q");
    const int64_t dim = q.dim();
    if (!(dim == 3 || (dim == 4 && q.size(2) == 1)) || q.size(dim - 1) != c.d ||
        q.scalar_type() != c.k.scalar_type() || q.device() != c.dev ||
        (q.stride(dim - 1) != 1 && q.numel() > 0))
      refuse("q must be [B, Hq, d] or [B, Hq, 1, d] with the cache's head size, dtype and device, "
             "and unit-stride rows");
    const int64_t B = q.size(0), Hq = q.size(1);
    const at::Tensor &tables = ints(a[3], "block_tables", 2, c.dev),
                     &lens = ints(a[4], "seq_lens", 1, c.dev);
    const int64_t W = tables.size(1);
    if (tables.size(0) != B || lens.size(0) != B || B > INT32_MAX || Hq > INT32_MAX)
      refuse("block_tables must be [B, W] and seq_lens [B]");
    const double alpha = PyFloat_AsDouble(a[5]);
    if (alpha == -1.0 && PyErr_Occurred()) throw Refused();
    const int n_iter = int32(a[6], "n_iter");
    const int64_t bound = a[7] == Py_None ? W * c.page : integer(a[7]);
    if (bound > INT32_MAX) refuse("max_len must be below 2^31");
    if (bound < 0) refuse("max_len must not be negative");
    const int max_len = static_cast<int>(bound);
    const c10::cuda::CUDAGuard on(c.dev);
    const at::Tensor out = output(a[8], "out", q.sizes(), q.scalar_type(), c.dev);
    const at::Tensor tau = output(a[9], "tau", q.sizes().slice(0, dim - 1), at::kFloat, c.dev);
    if (B == 0) return Py_BuildValue("(NN)", THPVariable_Wrap(out), THPVariable_Wrap(tau));
    const bool no_keys = max_len == 0;  // takes no workspace
    at::Tensor own;
    if (a[10] == Py_None && !no_keys) {
      const size_t need = entmax_attn_decode_workspace_bytes(
          static_cast<int>(B), static_cast<int>(Hq), c.heads, max_len);
      if (need == 0) return PyLong_FromLong(ENTMAX_ATTN_EINVAL);
      own = empty({static_cast<int64_t>(need)}, at::kByte, c.dev);
    }
    const at::Tensor& ws = a[10] == Py_None ? own : tensor(a[10], "workspace");
    if (ws.defined() && (ws.device() != c.dev || !ws.is_contiguous()))
      refuse("workspace must be a contiguous buffer on the cache's device");
    const int rc = entmax_attn_decode(
        q.const_data_ptr(), B > 1 ? q.stride(0) : 0, Hq > 1 ? q.stride(1) : 0,
        c.k.const_data_ptr(), c.v.const_data_ptr(), c.ps, c.hs, c.ss, c.pages, c.page,
        static_cast<const int32_t*>(tables.const_data_ptr()), B > 1 ? tables.stride(0) : W,
        static_cast<int>(W), static_cast<const int32_t*>(lens.const_data_ptr()),
        out.mutable_data_ptr(), static_cast<float*>(tau.mutable_data_ptr()),
        no_keys ? nullptr : ws.mutable_data_ptr(), no_keys ? 0 : ws.nbytes(), static_cast<int>(B), static_cast<int>(Hq), c.heads,
        max_len, c.d, static_cast<float>(alpha), n_iter, c.dtype,
        c10::cuda::getCurrentCUDAStream(c.dev.index()).stream());
    if (rc != ENTMAX_ATTN_OK) return PyLong_FromLong(rc);
    return Py_BuildValue("(NN)", THPVariable_Wrap(out), THPVariable_Wrap(tau));
  });
}

PyMethodDef kMethods[] = {
    {"page_tables", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(page_tables)),
     METH_FASTCALL, nullptr},
    {"paged_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_append)),
     METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode)), METH_FASTCALL,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&kModule); }
