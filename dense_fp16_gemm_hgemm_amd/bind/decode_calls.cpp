// The calls of Decode (decode.py) from torch tensors to the C ABI of libmi_decode.
//
// A decode step makes many calls of a few microseconds each.  Checks, output
// and launch from Python with ctypes take 10 us (w4_linear) to 22 (kv_append),
// longer than the kernels; here they take about 5.  A call returns its result,
// or the status of a call that the library refused; arguments that do not fit
// raise ValueError or TypeError.  No C++ exception leaves a function.
#include <algorithm>
#include <cmath>

#include <torch/csrc/autograd/python_variable.h>
#include <ATen/hip/impl/HIPStreamMasqueradingAsCUDA.h>
#include <ATen/ops/empty.h>
#include <c10/core/StreamGuard.h>
#include <c10/hip/HIPStream.h>

#include "mi_decode.h"

namespace {

struct Refused {};  // a Python exception is set

template <typename... A>
[[noreturn]] void refuse(PyObject* kind, const char* format, A... a) {
  PyErr_Format(kind, format, a...);
  throw Refused{};
}

const at::Tensor* tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", name);
  return &THPVariable_Unpack(o);
}
const at::Tensor* maybe(PyObject* o, const char* name) { return o == Py_None ? nullptr : tensor(o, name); }

int64_t number(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}
int32_t number32(PyObject* o, const char* name) {
  const int64_t v = number(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_ValueError, "%s is out of range: %lld", name, (long long)v);
  return (int32_t)v;
}
mi_decode_handle_t handle(PyObject* o) {  // None: a closed handle, which the library refuses
  return o == Py_None ? nullptr : reinterpret_cast<mi_decode_handle_t>(PyLong_AsVoidPtr(o));
}

mi_decode_dtype_t type16(const at::Tensor& x, const char* name) {
  if (x.scalar_type() == at::kHalf) return MI_DECODE_F16;
  if (x.scalar_type() != at::kBFloat16)
    refuse(PyExc_TypeError, "%s must be torch.float16 or torch.bfloat16, got %s", name, c10::toString(x.scalar_type()));
  return MI_DECODE_BF16;
}
void same_type(const at::Tensor& x, const at::Tensor& like, const char* name) {
  if (x.scalar_type() != like.scalar_type())
    refuse(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(like.scalar_type()), c10::toString(x.scalar_type()));
}
void on(const at::Tensor* x, c10::Device device, const char* name) {
  if (x && x->device() != device)
    refuse(PyExc_ValueError, "%s must be on %s, got %s", name, device.str().c_str(), x->device().str().c_str());
}
// Kernels run on the handle's device, and with its workspace; -1: an inspection handle.
void same_device(PyObject* handle_device, c10::Device device) {
  const int64_t d = number(handle_device);
  if (d >= 0 && d != device.index())
    refuse(PyExc_ValueError, "the handle is on cuda:%d, the tensors on cuda:%d", (int)d, (int)device.index());
}
// The stream of a call: the current one, or one that the caller names, which is
// the current one then while the call makes its results.  Their memory belongs
// to it: memory of another stream could still be in use there, or be given out
// there again before the kernel has written it.
struct OnStream {
  void* raw;
  c10::OptionalStreamGuard guard;
  OnStream(PyObject* o, c10::Device device) {
    if (o == Py_None) {
      raw = c10::hip::getCurrentHIPStream(device.index()).stream();
      return;
    }
    raw = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) throw Refused{};
    guard.reset_stream(
        c10::hip::getStreamFromExternalMasqueradingAsCUDA(static_cast<hipStream_t>(raw), device.index()).unwrap());
  }
};

bool is(const at::Tensor& x, at::ScalarType t, std::initializer_list<int64_t> shape) {
  return x.scalar_type() == t && x.sizes() == c10::IntArrayRef(shape) && x.is_contiguous();
}

// [tokens, heads, head_dim] with a contiguous last dimension; the stride of a
// dimension of one element says nothing
mi_decode_rows_t rows(const at::Tensor& x, const char* name, int64_t heads, int64_t D, const at::Tensor& like) {
  if (x.dim() != 3 || x.size(1) != heads || x.size(2) != D)
    refuse(PyExc_ValueError, "%s must have shape [tokens, %lld, %lld]", name, (long long)heads, (long long)D);
  same_type(x, like, name);
  if (x.stride(2) != 1) refuse(PyExc_ValueError, "%s must have a contiguous last dimension", name);
  return {x.data_ptr(), x.size(0) > 1 ? x.stride(0) : heads * D, heads > 1 ? x.stride(1) : D};
}

const int32_t* int32s(const at::Tensor& x, const char* name, int64_t dim) {
  if (x.scalar_type() != at::kInt) refuse(PyExc_TypeError, "%s must be torch.int32, got %s", name, c10::toString(x.scalar_type()));
  if (x.dim() != dim || (x.size(dim - 1) > 1 && x.stride(dim - 1) != 1))
    refuse(PyExc_ValueError, "%s must have %d dimension(s), the last one contiguous", name, (int)dim);
  return static_cast<const int32_t*>(x.data_ptr());
}

// The tokens of a call: tables and lengths as tensors, names as the caller knows them.
mi_decode_batch_t batch_of(PyObject* table_o, PyObject* lens_o, PyObject* cu_o, int64_t tokens, int32_t most,
                           c10::Device device, const char* lens_name, const char* cu_name) {
  const at::Tensor &table = *tensor(table_o, "table"), &lens = *tensor(lens_o, lens_name);
  const at::Tensor* cu = maybe(cu_o, cu_name);
  mi_decode_batch_t t = {};
  t.lens = int32s(lens, lens_name, 1);
  t.table = int32s(table, "table", 2);
  const int64_t B = lens.size(0);
  if (table.size(0) != B) refuse(PyExc_ValueError, "table must have one row a sequence (%lld), got %lld", (long long)B, (long long)table.size(0));
  if (!cu) {
    if (tokens != B || most != 1)
      refuse(PyExc_ValueError, "without %s each of the %lld sequences has one token, got %lld", cu_name, (long long)B, (long long)tokens);
  } else {
    t.cu = int32s(*cu, cu_name, 1);
    if (cu->size(0) != B + 1) refuse(PyExc_ValueError, "%s must have %lld entries, got %lld", cu_name, (long long)(B + 1), (long long)cu->size(0));
  }
  on(&lens, device, lens_name);
  on(&table, device, "table");
  on(cu, device, cu_name);
  if (B > INT32_MAX || tokens > INT32_MAX || table.size(1) > INT32_MAX) refuse(PyExc_ValueError, "too many tokens");
  t.table_stride = B > 1 ? table.stride(0) : table.size(1);
  t.table_cols = (int32_t)table.size(1);
  t.batch = (int32_t)B;
  t.tokens = (int32_t)tokens;
  t.max_tokens = most;
  return t;
}

// The most tokens that a sequence has in the call: with cu alone, all of them.
int32_t longest(PyObject* o, PyObject* cu, int64_t tokens, const char* name) {
  if (o != Py_None) return number32(o, name);
  return cu == Py_None ? 1 : (int32_t)std::min<int64_t>(tokens, INT32_MAX);
}

// A KvCache's numbers: the address of its C struct, and its device.
const mi_decode_cache_t& cache_of(PyObject* o) { return *static_cast<const mi_decode_cache_t*>(PyLong_AsVoidPtr(o)); }
c10::Device device_of(PyObject* o) { return c10::Device(c10::kCUDA, (c10::DeviceIndex)number(o)); }

PyObject* result(mi_decode_status_t st, const at::Tensor& x) {
  return st == MI_DECODE_OK ? THPVariable_Wrap(x) : PyLong_FromLong(st);
}

template <typename F>
PyObject* call(Py_ssize_t got, Py_ssize_t want, F f) {
  try {
    if (got != want) refuse(PyExc_TypeError, "expected %d arguments, got %d", (int)want, (int)got);
    return f();
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// handle, its device, x, qweight, scales, zeros, n, group, bias, out, stream
PyObject* w4_linear(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return call(n_args, 11, [&]() -> PyObject* {
    const at::Tensor &x = *tensor(a[2], "x"), &qw = *tensor(a[3], "qweight"), &sc = *tensor(a[4], "scales");
    const at::Tensor *zeros = maybe(a[5], "zeros"), *bias = maybe(a[8], "bias");
    const int64_t n = number(a[6]), group = number(a[7]);
    if (x.dim() != 2 || (x.size(1) > 1 && x.stride(1) != 1)) refuse(PyExc_ValueError, "x must be 2-D with unit-stride rows");
    const mi_decode_dtype_t type = type16(x, "x");
    if (!x.is_cuda()) refuse(PyExc_ValueError, "x must be on the GPU");
    same_device(a[1], x.device());
    const OnStream stream(a[10], x.device());
    if (n < 0) refuse(PyExc_ValueError, "n must not be negative");
    if (group < 32 || group % 32) refuse(PyExc_ValueError, "group must be a positive multiple of 32, got %lld", (long long)group);
    const int64_t M = x.size(0), K = x.size(1), nb = (n + 15) / 16, kb = (K + 127) / 128, groups = (K + group - 1) / group;
    if (!is(qw, at::kInt, {nb, kb, 64, 4}))
      refuse(PyExc_ValueError, "qweight must be contiguous int32 (%lld, %lld, 64, 4) for n=%lld, K=%lld", (long long)nb, (long long)kb, (long long)n, (long long)K);
    if (!is(sc, x.scalar_type(), {groups, nb * 16}))
      refuse(PyExc_ValueError, "scales must be contiguous, of x's type and (%lld, %lld)", (long long)groups, (long long)(nb * 16));
    if (zeros && !is(*zeros, at::kByte, {groups, nb * 16}))
      refuse(PyExc_ValueError, "zeros must be contiguous uint8 (%lld, %lld)", (long long)groups, (long long)(nb * 16));
    if (bias && (bias->scalar_type() != x.scalar_type() || bias->dim() != 1 || bias->size(0) != n || (n > 1 && bias->stride(0) != 1)))
      refuse(PyExc_ValueError, "bias must be contiguous, of x's type and (%lld,)", (long long)n);
    at::Tensor made;
    const at::Tensor* out = maybe(a[9], "out");
    if (!out) {
      made = at::empty({M, n}, x.options());
      out = &made;
    } else if (out->dim() != 2 || out->size(0) != M || out->size(1) != n || out->scalar_type() != x.scalar_type() || (n > 1 && out->stride(1) != 1)) {
      refuse(PyExc_ValueError, "out must be of x's type and (%lld, %lld) with unit-stride rows", (long long)M, (long long)n);
    }
    on(&qw, x.device(), "qweight");
    on(&sc, x.device(), "scales");
    on(zeros, x.device(), "zeros");
    on(bias, x.device(), "bias");
    on(out, x.device(), "out");
    return result(mi_decode_w4_linear(handle(a[0]), type, M, n, K, group, x.data_ptr(), x.stride(0), qw.data_ptr(),
                                      sc.data_ptr(), zeros ? zeros->data_ptr() : nullptr, bias ? bias->data_ptr() : nullptr,
                                      out->data_ptr(), out->stride(0), stream.raw), *out);
  });
}

// handle, its device, cache, device, k, v, table, past, cu_new, max_new, q, rope, interleaved, q_out, stream, positions
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return call(n_args, 16, [&]() -> PyObject* {
    const mi_decode_cache_t& c = cache_of(a[2]);
    const c10::Device device = device_of(a[3]);
    same_device(a[1], device);
    const OnStream stream(a[14], device);
    const at::Tensor &k = *tensor(a[4], "k"), &v = *tensor(a[5], "v");
    const at::Tensor *q = maybe(a[10], "q"), *rope = maybe(a[11], "rope"), *q_out = maybe(a[13], "q_out");
    const mi_decode_dtype_t type = type16(k, "k");
    const mi_decode_rows_t rk = rows(k, "k", c.kv_heads, c.head_dim, k), rv = rows(v, "v", c.kv_heads, c.head_dim, k);
    const int64_t T = k.size(0);
    if (v.size(0) != T) refuse(PyExc_ValueError, "k and v must have the same tokens");
    const mi_decode_batch_t t = batch_of(a[6], a[7], a[8], T, longest(a[9], a[8], T, "max_new"), device, "past", "cu_new");
    mi_decode_rows_t rq = {}, ro = {};
    at::Tensor made;
    int64_t hq = 0;
    if (q) {
      hq = q->dim() == 3 ? q->size(1) : -1;
      rq = rows(*q, "q", hq, c.head_dim, k);
      if (q->size(0) != T) refuse(PyExc_ValueError, "q must have k's tokens");
      if (!q_out) {
        made = at::empty({T, hq, c.head_dim}, q->options());
        q_out = &made;
      }
      ro = rows(*q_out, "q_out", hq, c.head_dim, k);
      if (q_out->size(0) != T) refuse(PyExc_ValueError, "q_out must have q's tokens");
    }
    if (rope && (rope->scalar_type() != at::kFloat || rope->dim() != 2 || !rope->is_contiguous()))
      refuse(PyExc_ValueError, "rope must be a contiguous float32 [positions, rot_dim] table");
    const at::Tensor* positions = maybe(a[15], "positions");
    const int32_t* turned = positions ? int32s(*positions, "positions", 1) : nullptr;
    if (positions && positions->size(0) != T) refuse(PyExc_ValueError, "positions must have one entry a token (%lld), got %lld", (long long)T, (long long)positions->size(0));
    on(positions, device, "positions");
    if (rope && !positions && rope->size(0) < (int64_t)t.table_cols * c.page_size)
      refuse(PyExc_ValueError, "rope has %lld positions, the table has %lld", (long long)rope->size(0), (long long)t.table_cols * c.page_size);
    on(&k, device, "k");
    on(&v, device, "v");
    on(q, device, "q");
    if (q) on(q_out, device, "q_out");
    on(rope, device, "rope");
    const int on_pairs = PyObject_IsTrue(a[12]);
    if (on_pairs < 0) throw Refused{};
    const mi_decode_status_t st = mi_decode_kv_append_at(
        handle(a[0]), &c, type, &t, &rk, &rv, rope ? static_cast<const float*>(rope->data_ptr()) : nullptr,
        rope ? rope->size(0) : 0, rope ? (int32_t)rope->size(1) : 0, on_pairs, turned, (int32_t)hq, q ? &rq : nullptr,
        q ? &ro : nullptr, stream.raw);
    if (st != MI_DECODE_OK || q) return result(st, q ? *q_out : k);
    Py_RETURN_NONE;
  });
}

// handle, its device, cache, device, table, start, cu, tokens, max_tokens, bf16, stream
PyObject* kv_read(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return call(n_args, 11, [&]() -> PyObject* {
    const mi_decode_cache_t& c = cache_of(a[2]);
    const c10::Device device = device_of(a[3]);
    same_device(a[1], device);
    const OnStream stream(a[10], device);
    const int64_t T = number(a[7]);
    if (T < 0) refuse(PyExc_ValueError, "tokens must not be negative");
    const mi_decode_batch_t t = batch_of(a[4], a[5], a[6], T, longest(a[8], a[6], T, "max_tokens"), device, "start", "cu");
    const bool bf16 = PyObject_IsTrue(a[9]);
    const auto options = at::TensorOptions().dtype(bf16 ? at::kBFloat16 : at::kHalf).device(device);
    const at::Tensor k = at::empty({T, c.kv_heads, c.head_dim}, options), v = at::empty({T, c.kv_heads, c.head_dim}, options);
    const mi_decode_status_t st = mi_decode_kv_read(handle(a[0]), &c, bf16 ? MI_DECODE_BF16 : MI_DECODE_F16, &t, k.data_ptr(),
                                                    v.data_ptr(), stream.raw);
    if (st != MI_DECODE_OK) return PyLong_FromLong(st);
    PyObject *pk = THPVariable_Wrap(k), *pv = THPVariable_Wrap(v), *both = pk && pv ? PyTuple_Pack(2, pk, pv) : nullptr;
    Py_XDECREF(pk);
    Py_XDECREF(pv);
    return both;
  });
}

// handle, its device, cache, device, q, table, lens, cu_q, max_q, max_len, window, sinks, scale, out, stream,
// and for a tree: seen
PyObject* attend(PyObject* const* a, Py_ssize_t n_args, bool tree) {
  return call(n_args, tree ? 16 : 15, [&]() -> PyObject* {
    const mi_decode_cache_t& c = cache_of(a[2]);
    const c10::Device device = device_of(a[3]);
    same_device(a[1], device);
    const OnStream stream(a[14], device);
    const at::Tensor& q = *tensor(a[4], "q");
    const mi_decode_dtype_t type = type16(q, "q");
    const int64_t hq = q.dim() == 3 ? q.size(1) : -1;
    const mi_decode_rows_t rq = rows(q, "q", hq, c.head_dim, q);
    const int64_t T = q.size(0);
    if (hq < 1 || hq % c.kv_heads) refuse(PyExc_ValueError, "q must have a multiple of %d heads, got %lld", c.kv_heads, (long long)hq);
    const int32_t window = number32(a[10], "window"), sinks = number32(a[11], "sinks");
    if (window < 0 || sinks < 0) refuse(PyExc_ValueError, "window and sinks must not be negative");
    const at::Tensor* seen = tree ? tensor(a[15], "seen") : nullptr;
    const int32_t* bits = tree ? int32s(*seen, "seen", 2) : nullptr;
    const int64_t words = tree ? seen->size(1) : 0;
    int32_t most = longest(a[8], a[7], T, "max_q");
    // a row of bits has one for each drafted token of its sequence
    if (tree && a[8] == Py_None) most = (int32_t)std::min<int64_t>(most, std::max<int64_t>(32 * words, 1));
    const mi_decode_batch_t t = batch_of(a[5], a[6], a[7], T, most, device, "lens", "cu_q");
    const int64_t max_len = a[9] == Py_None ? (int64_t)t.table_cols * c.page_size : number(a[9]);
    const double scale = a[12] == Py_None ? 1.0 / std::sqrt((double)c.head_dim) : PyFloat_AsDouble(a[12]);
    if (PyErr_Occurred()) throw Refused{};
    at::Tensor made;
    const at::Tensor* out = maybe(a[13], "out");
    if (!out) {
      made = at::empty({T, hq, c.head_dim}, q.options());
      out = &made;
    } else if (out->dim() != 3 || out->size(0) != T) {
      refuse(PyExc_ValueError, "out must have q's tokens");
    }
    const mi_decode_rows_t ro = rows(*out, "out", hq, c.head_dim, q);
    on(&q, device, "q");
    on(out, device, "out");
    if (!tree)
      return result(mi_decode_kv_attend(handle(a[0]), &c, type, &t, max_len, (int32_t)hq, &rq, &ro, (float)scale, window, sinks,
                                        stream.raw), *out);
    if (seen->size(0) != T) refuse(PyExc_ValueError, "seen must have one row a token (%lld), got %lld", (long long)T, (long long)seen->size(0));
    if (words > INT32_MAX || (T > 0 && words * 32 < t.max_tokens))
      refuse(PyExc_ValueError, "seen has %lld words of 32 bits a token, too few for max_q=%d", (long long)words, t.max_tokens);
    on(seen, device, "seen");
    return result(mi_decode_kv_attend_tree(handle(a[0]), &c, type, &t, max_len, (int32_t)hq, &rq, &ro, bits,
                                           T > 1 ? seen->stride(0) : words, (int32_t)words, (float)scale, window, sinks,
                                           stream.raw), *out);
  });
}
PyObject* kv_attend(PyObject*, PyObject* const* a, Py_ssize_t n_args) { return attend(a, n_args, false); }
PyObject* kv_attend_tree(PyObject*, PyObject* const* a, Py_ssize_t n_args) { return attend(a, n_args, true); }

// handle, its device, cache, device, table, past, keep, cu, max_keep, stream
PyObject* kv_keep(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return call(n_args, 10, [&]() -> PyObject* {
    const mi_decode_cache_t& c = cache_of(a[2]);
    const c10::Device device = device_of(a[3]);
    same_device(a[1], device);
    const OnStream stream(a[9], device);
    const at::Tensor& keep = *tensor(a[6], "keep");
    const int32_t* of = int32s(keep, "keep", 1);
    const int64_t T = keep.size(0);
    const mi_decode_batch_t t = batch_of(a[4], a[5], a[7], T, longest(a[8], a[7], T, "max_keep"), device, "past", "cu_keep");
    on(&keep, device, "keep");
    const mi_decode_status_t st = mi_decode_kv_keep(handle(a[0]), &c, &t, of, stream.raw);
    if (st != MI_DECODE_OK) return PyLong_FromLong(st);
    Py_RETURN_NONE;
  });
}

// handle, its device, cache, device, src, dst, stream
PyObject* kv_copy(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return call(n_args, 7, [&]() -> PyObject* {
    const mi_decode_cache_t& c = cache_of(a[2]);
    const c10::Device device = device_of(a[3]);
    same_device(a[1], device);
    const OnStream stream(a[6], device);
    const at::Tensor &src = *tensor(a[4], "src"), &dst = *tensor(a[5], "dst");
    const int32_t *from = int32s(src, "src", 1), *to = int32s(dst, "dst", 1);
    if (src.size(0) != dst.size(0))
      refuse(PyExc_ValueError, "src and dst must have the same length, got %lld and %lld", (long long)src.size(0), (long long)dst.size(0));
    on(&src, device, "src");
    on(&dst, device, "dst");
    const mi_decode_status_t st = mi_decode_kv_copy(handle(a[0]), &c, from, to, src.size(0), stream.raw);
    if (st != MI_DECODE_OK) return PyLong_FromLong(st);
    Py_RETURN_NONE;
  });
}

// 2-D with unit-stride rows; the distance of rows says nothing where there is one
int64_t row_distance(const at::Tensor& x, const char* name, at::ScalarType type, int64_t rows, int64_t cols) {
  if (x.scalar_type() != type) refuse(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(type), c10::toString(x.scalar_type()));
  if (x.dim() != 2 || x.size(0) != rows || x.size(1) != cols || (cols > 1 && x.stride(1) != 1))
    refuse(PyExc_ValueError, "%s must have shape (%lld, %lld) and unit-stride rows", name, (long long)rows, (long long)cols);
  return rows > 1 ? x.stride(0) : cols;
}
int64_t row_distance(const at::Tensor& x, const char* name) {
  return row_distance(x, name, x.scalar_type(), x.dim() == 2 ? x.size(0) : 0, x.dim() == 2 ? x.size(1) : 0);
}
const void* vector(const at::Tensor* x, const char* name, at::ScalarType type, int64_t n) {
  if (!x) return nullptr;
  if (x->scalar_type() != type) refuse(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(type), c10::toString(x->scalar_type()));
  if (x->dim() != 1 || x->size(0) != n || (n > 1 && x->stride(0) != 1))
    refuse(PyExc_ValueError, "%s must be contiguous with %lld entries", name, (long long)n);
  return x->data_ptr();
}

// handle, its device, x, weight, residual, eps, codes, scales, total, stream
PyObject* rms_norm_f8(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return call(n_args, 10, [&]() -> PyObject* {
    const at::Tensor& x = *tensor(a[2], "x");
    const at::Tensor *weight = maybe(a[3], "weight"), *residual = maybe(a[4], "residual");
    const mi_decode_dtype_t type = type16(x, "x");
    if (!x.is_cuda()) refuse(PyExc_ValueError, "x must be on the GPU");
    same_device(a[1], x.device());
    const OnStream stream(a[9], x.device());
    const int64_t ldx = row_distance(x, "x"), M = x.size(0), K = x.size(1), blocks = (K + 127) / 128;
    const int64_t ldr = residual ? row_distance(*residual, "residual", x.scalar_type(), M, K) : 0;
    const void* g = vector(weight, "weight", x.scalar_type(), K);
    const double eps = PyFloat_AsDouble(a[5]);
    if (PyErr_Occurred()) throw Refused{};
    const at::Tensor *codes = maybe(a[6], "codes"), *scales = maybe(a[7], "scales"), *total = maybe(a[8], "total");
    if (total && !residual) refuse(PyExc_ValueError, "without a residual there is no total");
    at::Tensor made[3];
    auto ready = [&](const at::Tensor*& out, int i, at::ScalarType t, int64_t cols) {
      if (out) return;
      made[i] = at::empty({M, cols}, x.options().dtype(t));
      out = &made[i];
    };
    ready(codes, 0, at::kFloat8_e4m3fn, K);
    ready(scales, 1, at::kFloat, blocks);
    if (residual) ready(total, 2, x.scalar_type(), K);
    const int64_t ldc = row_distance(*codes, "codes", at::kFloat8_e4m3fn, M, K);
    const int64_t lds = row_distance(*scales, "scales", at::kFloat, M, blocks);
    const int64_t ldt = total ? row_distance(*total, "total", x.scalar_type(), M, K) : 0;
    on(weight, x.device(), "weight");
    on(residual, x.device(), "residual");
    on(codes, x.device(), "codes");
    on(scales, x.device(), "scales");
    on(total, x.device(), "total");
    const mi_decode_status_t st = mi_decode_rms_norm_f8(
        handle(a[0]), type, M, K, x.data_ptr(), ldx, residual ? residual->data_ptr() : nullptr, ldr, g, (float)eps,
        codes->data_ptr(), ldc, static_cast<float*>(scales->data_ptr()), lds, total ? total->data_ptr() : nullptr, ldt,
        stream.raw);
    if (st != MI_DECODE_OK) return PyLong_FromLong(st);
    PyObject *pc = THPVariable_Wrap(*codes), *ps = THPVariable_Wrap(*scales);
    PyObject* pt = total ? THPVariable_Wrap(*total) : Py_NewRef(Py_None);
    PyObject* all = pc && ps && pt ? PyTuple_Pack(3, pc, ps, pt) : nullptr;
    Py_XDECREF(pc);
    Py_XDECREF(ps);
    Py_XDECREF(pt);
    return all;
  });
}

// handle, its device, x, x_scales, weight, w_scales, bf16, bias, out, stream
PyObject* f8_linear(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return call(n_args, 10, [&]() -> PyObject* {
    const at::Tensor &x = *tensor(a[2], "x"), &xs = *tensor(a[3], "x_scales"), &w = *tensor(a[4], "weight"), &ws = *tensor(a[5], "w_scales");
    const at::Tensor* bias = maybe(a[7], "bias");
    if (x.scalar_type() != at::kFloat8_e4m3fn) refuse(PyExc_TypeError, "x must be torch.float8_e4m3fn, got %s", c10::toString(x.scalar_type()));
    if (!x.is_cuda()) refuse(PyExc_ValueError, "x must be on the GPU");
    same_device(a[1], x.device());
    const OnStream stream(a[9], x.device());
    const int bf16 = PyObject_IsTrue(a[6]);
    const at::ScalarType type = bf16 ? at::kBFloat16 : at::kHalf;
    const int64_t ldx = row_distance(x, "x"), M = x.size(0), K = x.size(1), kb = (K + 127) / 128;
    const int64_t N = w.dim() == 2 ? w.size(0) : 0, ldw = row_distance(w, "weight", at::kFloat8_e4m3fn, N, K);
    const int64_t ldxs = row_distance(xs, "x_scales", at::kFloat, M, kb);
    const int64_t ldws = row_distance(ws, "w_scales", at::kFloat, (N + 127) / 128, kb);
    const void* b = vector(bias, "bias", type, N);
    at::Tensor made;
    const at::Tensor* out = maybe(a[8], "out");
    if (!out) {
      made = at::empty({M, N}, x.options().dtype(type));
      out = &made;
    }
    const int64_t ldy = row_distance(*out, "out", type, M, N);
    on(&xs, x.device(), "x_scales");
    on(&w, x.device(), "weight");
    on(&ws, x.device(), "w_scales");
    on(bias, x.device(), "bias");
    on(out, x.device(), "out");
    return result(mi_decode_f8_linear(handle(a[0]), bf16 ? MI_DECODE_BF16 : MI_DECODE_F16, M, N, K, x.data_ptr(), ldx,
                                      static_cast<const float*>(xs.data_ptr()), ldxs, w.data_ptr(), ldw,
                                      static_cast<const float*>(ws.data_ptr()), ldws, b, out->data_ptr(), ldy, stream.raw),
                  *out);
  });
}


#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(w4_linear), FAST(kv_append), FAST(kv_read), FAST(kv_attend),
                         FAST(kv_attend_tree), FAST(kv_keep), FAST(kv_copy), FAST(rms_norm_f8), FAST(f8_linear), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_decode_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decode_calls() { return PyModule_Create(&module); }
