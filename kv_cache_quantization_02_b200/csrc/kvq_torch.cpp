// kvq_torch.cpp -- the torch side of the paged cache's calls, for kvq.py: checks
// of the tensors, outputs and workspaces, the current stream, and the call of
// the C entry point (include/kvq.h).  A decode step makes these calls for every
// layer, and their kernels take 3 to 10 us where there is little to do; the same
// checks in Python and a call through ctypes took 10 to 16 us.
//
// Wrong tensors raise ValueError; a status of the library is returned as an int,
// from which kvq.py makes its KvqError.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <stdexcept>
#include <string>

#include "kvq.h"

namespace {

struct Wrong : std::runtime_error {
  using std::runtime_error::runtime_error;
};

std::string shape_text(at::IntArrayRef s) {
  std::string o = "(";
  for (size_t i = 0; i < s.size(); ++i) o += (i ? ", " : "") + std::to_string(s[i]);
  return o + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* x, const char* name) {
  if (!THPVariable_Check(x)) throw Wrong(std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(x);
}

// A contiguous tensor of this type and shape on CUDA device `index`.
void need(const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape, int index, const char* name) {
  if (!t.is_cuda()) throw Wrong(std::string(name) + " must be a CUDA tensor");
  if (t.scalar_type() != type)
    throw Wrong(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
  if (t.sizes() != shape)
    throw Wrong(std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
  if (!t.is_contiguous()) throw Wrong(std::string(name) + " must be contiguous");
  if (t.get_device() != index)
    throw Wrong(std::string(name) + " must be on cuda:" + std::to_string(index) + " as the cache");
}

int element_type(at::ScalarType t, const char* name) {
  if (t == at::kHalf) return KVQ_FP16;
  if (t == at::kBFloat16) return KVQ_BF16;
  throw Wrong(std::string(name) + " must be torch.float16 or torch.bfloat16, got " + c10::toString(t));
}

// The C entry points take 32-bit sizes, and counts of tokens below 2^31.
int narrow(int64_t x, const char* name) {
  if (x > INT32_MAX) throw Wrong(std::string(name) + " is too large");
  return static_cast<int>(x);
}

struct Cache {
  const at::Tensor &table, &kc, &vc, &ks, &vs;
  int index, format, B, max_blocks, Hkv, block, D;
  int64_t num_blocks;

  explicit Cache(PyObject* const* a)              // block_table, k_cache, v_cache, k_scales, v_scales
      : table(tensor(a[0], "block_table")), kc(tensor(a[1], "k_cache")), vc(tensor(a[2], "v_cache")),
        ks(tensor(a[3], "k_scales")), vs(tensor(a[4], "v_scales")) {
    if (kc.dim() != 4 || table.dim() != 2)
      throw Wrong("k_cache must be [num_blocks, Hkv, block, D] and block_table [B, max_blocks]");
    const at::ScalarType type = kc.scalar_type();
    if (type == at::kChar) format = KVQ_INT8;
    else if (type == at::kFloat8_e4m3fn) format = KVQ_E4M3;
    else throw Wrong(std::string("k_cache must be torch.int8 or torch.float8_e4m3fn, got ") + c10::toString(type));
    if (!kc.is_cuda()) throw Wrong("k_cache must be a CUDA tensor");
    index = kc.get_device();
    num_blocks = kc.size(0);
    Hkv = narrow(kc.size(1), "Hkv");
    block = narrow(kc.size(2), "block");
    D = narrow(kc.size(3), "D");
    B = narrow(table.size(0), "B");
    max_blocks = narrow(table.size(1), "max_blocks");
    need(kc, type, kc.sizes(), index, "k_cache");
    need(vc, type, kc.sizes(), index, "v_cache");
    const int64_t one[2] = {num_blocks, Hkv};
    need(ks, at::kFloat, one, index, "k_scales");
    need(vs, at::kFloat, one, index, "v_scales");
    const int64_t all[2] = {B, max_blocks};
    need(table, at::kInt, all, index, "block_table");
  }
  const int32_t* table_ptr() const { return static_cast<const int32_t*>(table.const_data_ptr()); }
};

const int32_t* list_of(const at::Tensor& t, int64_t n, int index, const char* name) {
  need(t, at::kInt, at::IntArrayRef(&n, 1), index, name);
  return static_cast<const int32_t*>(t.const_data_ptr());
}

// Token rows [n, heads, D] that may lie apart.
struct Rows {
  int dtype;
  int64_t n, stride;
  int heads;
  Rows(const at::Tensor& x, const char* name, const Cache& c) {
    dtype = element_type(x.scalar_type(), name);
    if (x.dim() != 3 || x.size(2) != c.D)
      throw Wrong(std::string(name) + " must be [tokens, heads, " + std::to_string(c.D) + "], got " +
                  shape_text(x.sizes()));
    if (!x.is_cuda() || x.get_device() != c.index)
      throw Wrong(std::string(name) + " must be on cuda:" + std::to_string(c.index) + " as the cache");
    n = x.size(0);
    heads = narrow(x.size(1), "heads");
    if (x.stride(2) != 1 || (x.stride(1) != c.D && heads > 1))
      throw Wrong(std::string(name) + ": the channels and heads of a token must be contiguous");
    stride = n > 1 ? x.stride(0) : static_cast<int64_t>(heads) * c.D;
  }
};

// A new tensor on the current device, straight from the caching allocator (the
// dispatcher takes as long again, and a read of a few rows makes two of them).
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int index) {
  return at::Tensor(at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(index)),
                                           std::nullopt));
}

at::Tensor output(PyObject* given, at::IntArrayRef shape, at::ScalarType type, int index, const char* name) {
  if (given == Py_None) return fresh(shape, type, index);
  const at::Tensor& t = tensor(given, name);
  need(t, type, shape, index, name);
  return t;
}

// True: a new one of `bytes`; a uint8 tensor: that; anything else: none.
at::Tensor workspace(PyObject* given, int64_t bytes, int index) {
  if (given == Py_True) return bytes > 0 ? fresh(at::IntArrayRef(&bytes, 1), at::kByte, index) : at::Tensor();
  if (!THPVariable_Check(given)) return at::Tensor();
  const at::Tensor& t = THPVariable_Unpack(given);
  const int64_t n = t.numel();
  need(t, at::kByte, at::IntArrayRef(&n, 1), index, "workspace");
  return t;
}

void* stream_of(int index) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream(); }

int as_int(PyObject* x) {
  const long v = PyLong_AsLong(x);
  if (v == -1 && PyErr_Occurred()) throw Wrong("");
  if (v > INT32_MAX || v < INT32_MIN) throw Wrong("window is out of range");
  return static_cast<int>(v);
}
float as_float(PyObject* x) {
  const double v = PyFloat_AsDouble(x);
  if (v == -1.0 && PyErr_Occurred()) throw Wrong("");
  return static_cast<float>(v);
}

// f(args) with C++ exceptions as Python ones.
template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    return f();
  } catch (const Wrong& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::Error&) {                   // torch's own class: callers that run out of memory evict blocks
    if (!PyErr_Occurred()) torch::translate_exception_to_python(std::current_exception());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (k, v, cu_tokens, start, block_table, k_cache, v_cache, k_scales, v_scales) -> status
PyObject* paged_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const Cache c(a + 4);
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const Rows rk(k, "k", c), rv(v, "v", c);
    if (rk.heads != c.Hkv || rv.heads != c.Hkv || rv.n != rk.n || rv.dtype != rk.dtype)
      throw Wrong("k and v must both be [n, " + std::to_string(c.Hkv) + ", " + std::to_string(c.D) +
                  "] of one type, got " + shape_text(k.sizes()) + " and " + shape_text(v.sizes()));
    const int32_t* cu = list_of(tensor(a[2], "cu_tokens"), static_cast<int64_t>(c.B) + 1, c.index, "cu_tokens");
    const int32_t* start = list_of(tensor(a[3], "start"), c.B, c.index, "start");
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.index));
    return PyLong_FromLong(kvq_paged_write(
        k.const_data_ptr(), v.const_data_ptr(), rk.dtype, rk.stride, rv.stride, cu, start, c.table_ptr(), c.B,
        c.max_blocks, rk.n, c.Hkv, c.D, c.block, c.format, c.num_blocks, c.kc.mutable_data_ptr(),
        c.vc.mutable_data_ptr(), static_cast<float*>(c.ks.mutable_data_ptr()),
        static_cast<float*>(c.vs.mutable_data_ptr()), stream_of(c.index)));
  });
}

// (cu_tokens, start, block_table, k_cache, v_cache, k_scales, v_scales, n_tokens, bf16, k_out, v_out) -> (k, v) or status
PyObject* paged_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const Cache c(a + 2);
    const int32_t* cu = list_of(tensor(a[0], "cu_tokens"), static_cast<int64_t>(c.B) + 1, c.index, "cu_tokens");
    const int32_t* start = list_of(tensor(a[1], "start"), c.B, c.index, "start");
    const int64_t tokens = PyLong_AsLongLong(a[7]);
    if (tokens == -1 && PyErr_Occurred()) throw Wrong("");
    if (tokens < 0) throw Wrong("n_tokens must not be negative");
    narrow(tokens, "n_tokens");                   // before outputs of that size are asked for
    const int dtype = a[8] == Py_True ? KVQ_BF16 : KVQ_FP16;
    const at::ScalarType type = dtype == KVQ_BF16 ? at::kBFloat16 : at::kHalf;
    const int64_t shape[3] = {tokens, c.Hkv, c.D};
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.index));
    at::Tensor k = output(a[9], shape, type, c.index, "k_out");
    at::Tensor v = output(a[10], shape, type, c.index, "v_out");
    const int rc = kvq_paged_read(cu, start, c.table_ptr(), c.B, c.max_blocks, tokens, c.Hkv, c.D, c.block, c.format,
                                  c.num_blocks, c.kc.const_data_ptr(), c.vc.const_data_ptr(),
                                  static_cast<const float*>(c.ks.const_data_ptr()),
                                  static_cast<const float*>(c.vs.const_data_ptr()), dtype, k.mutable_data_ptr(),
                                  v.mutable_data_ptr(), stream_of(c.index));
    if (rc != KVQ_OK) return PyLong_FromLong(rc);
    PyObject* pair = PyTuple_New(2);
    if (!pair) return nullptr;
    PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(std::move(k)));
    PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(std::move(v)));
    return pair;
  });
}

// (q, seq_len, block_table, k_cache, v_cache, k_scales, v_scales, sm_scale, window, out, workspace) -> out or status
PyObject* paged_attention_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const Cache c(a + 2);
    const at::Tensor& q = tensor(a[0], "q");
    const Rows r(q, "q", c);
    if (r.n != c.B)
      throw Wrong("q must have one row for each of the " + std::to_string(c.B) + " sequences, got " +
                  std::to_string(r.n));
    const int32_t* lens = list_of(tensor(a[1], "seq_len"), c.B, c.index, "seq_len");
    const float scale = as_float(a[7]);
    const int window = as_int(a[8]);
    const int64_t shape[3] = {r.n, r.heads, c.D};
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.index));
    at::Tensor out = output(a[9], shape, q.scalar_type(), c.index, "out");
    const at::Tensor ws = workspace(
        a[10], a[10] == Py_True ? kvq_paged_decode_workspace_bytes(c.B, c.max_blocks, r.heads, c.Hkv, c.D, c.block, window)
                                : 0, c.index);
    const int rc = kvq_paged_attention_decode(
        q.const_data_ptr(), r.dtype, r.stride, lens, c.table_ptr(), c.B, c.max_blocks, r.heads, c.Hkv, c.D, c.block,
        c.format, c.num_blocks, c.kc.const_data_ptr(), c.vc.const_data_ptr(),
        static_cast<const float*>(c.ks.const_data_ptr()), static_cast<const float*>(c.vs.const_data_ptr()), scale,
        window, out.mutable_data_ptr(), ws.defined() ? ws.mutable_data_ptr() : nullptr, ws.defined() ? ws.numel() : 0,
        stream_of(c.index));
    return rc == KVQ_OK ? THPVariable_Wrap(std::move(out)) : PyLong_FromLong(rc);
  });
}

// (q, cu_q, seq_len, block_table, k_cache, v_cache, k_scales, v_scales, sm_scale, window, out, workspace) -> out or status
PyObject* paged_attention_prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const Cache c(a + 3);
    const at::Tensor& q = tensor(a[0], "q");
    const Rows r(q, "q", c);
    const int32_t* cu = list_of(tensor(a[1], "cu_q"), static_cast<int64_t>(c.B) + 1, c.index, "cu_q");
    const int32_t* lens = list_of(tensor(a[2], "seq_len"), c.B, c.index, "seq_len");
    const float scale = as_float(a[8]);
    const int window = as_int(a[9]);
    const int64_t shape[3] = {r.n, r.heads, c.D};
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.index));
    at::Tensor out = output(a[10], shape, q.scalar_type(), c.index, "out");
    const at::Tensor ws = workspace(a[11], a[11] == Py_True ? kvq_paged_prefill_workspace_bytes(
                                                                  c.B, c.max_blocks, r.n, r.heads, c.Hkv, c.D, c.block,
                                                                  window)
                                                            : 0, c.index);
    const int rc = kvq_paged_attention_prefill(
        q.const_data_ptr(), r.dtype, r.stride, cu, lens, c.table_ptr(), c.B, c.max_blocks, r.n, r.heads, c.Hkv, c.D,
        c.block, c.format, c.num_blocks, c.kc.const_data_ptr(), c.vc.const_data_ptr(),
        static_cast<const float*>(c.ks.const_data_ptr()), static_cast<const float*>(c.vs.const_data_ptr()), scale,
        window, out.mutable_data_ptr(), ws.defined() ? ws.mutable_data_ptr() : nullptr, ws.defined() ? ws.numel() : 0,
        stream_of(c.index));
    return rc == KVQ_OK ? THPVariable_Wrap(std::move(out)) : PyLong_FromLong(rc);
  });
}

#define KVQ_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KVQ_METHOD(paged_write), KVQ_METHOD(paged_read), KVQ_METHOD(paged_attention_decode),
                         KVQ_METHOD(paged_attention_prefill), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kvq_torch", "torch side of the paged cache's calls", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kvq_torch() { return PyModule_Create(&module); }
