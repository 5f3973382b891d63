// Python binding of the serving entry points (include/sage.h, "Serving"): checks torch tensors, allocates the
// outputs and calls the C function whose address the caller passes (the library's or its checked twin's).
//
// Compiled, where the rest of the package goes through ctypes: a decode step's kernels take 4 to 10 us, and
// a call took the host 16 to 22 us with the same checks in Python, 6 to 8 us here.  Nothing is computed here.
//
// Every function returns the output tensors, or the C status as an int; bad arguments raise ValueError.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>

#include "sage.h"

namespace {

using at::Tensor;

struct BadArgument {};  // a Python error is set

[[noreturn]] void bad(const char* format, const char* name = "", const char* more = "") {
  PyErr_Format(PyExc_ValueError, format, name, more);
  throw BadArgument();
}

const Tensor& tensor_of(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad("%s must be a tensor", name);
  return THPVariable_Unpack(o);
}
const Tensor* optional_of(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor_of(o, name); }

long long int_of(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw BadArgument();
  return v;
}
double float_of(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw BadArgument();
  return v;
}
bool bool_of(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw BadArgument();
  return v == 1;
}
int int32_of(PyObject* o, const char* name) {
  const long long v = int_of(o);
  if (v < INT32_MIN || v > INT32_MAX) bad("%s does not fit 32 bits", name);
  return (int)v;
}
template <typename F>
F function_of(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no function");
    throw BadArgument();
  }
  return reinterpret_cast<F>(p);
}

int narrow(int64_t v, const char* name) {
  if (v > INT32_MAX) bad("an extent of %s does not fit 32 bits", name);
  return (int)v;
}

// sage_dtype of a tensor type, or -1
int dtype_code(at::ScalarType t) {
  return t == at::kHalf ? SAGE_FP16 : t == at::kBFloat16 ? SAGE_BF16 : t == at::kFloat ? SAGE_FP32 : -1;
}

void* pointer(const Tensor* t) { return t ? const_cast<void*>(t->const_data_ptr()) : nullptr; }

// Heads: a CUDA tensor of fp16, bf16 (or fp32, which the library answers) with contiguous channels; of the type and
// on the device of `like`.
void check_heads(const Tensor& t, const char* name, const Tensor* like = nullptr) {
  if (!t.is_cuda()) bad("%s must be a CUDA tensor (no CPU path exists)", name);
  if (dtype_code(t.scalar_type()) < 0) bad("unsupported dtype of %s", name);
  if (like && (t.scalar_type() != like->scalar_type() || t.get_device() != like->get_device()))
    bad("%s must have the dtype and the device of the other tensors", name);
  if (t.dim() < 3) bad("%s must have tokens, heads and channels", name);
  if (t.stride(-1) != 1 && t.size(-1) > 1 && t.numel()) bad("the channels (last dimension) of %s must be contiguous", name);
}

void check_ints(const Tensor& t, const char* name, int dims, int dev) {
  if (t.scalar_type() != at::kInt || !t.is_cuda() || t.get_device() != dev || t.dim() != dims)
    bad("%s must be an int32 tensor of %s on the device of the others", name, dims == 1 ? "one dimension" : "two dimensions");
  if (t.size(-1) > 1 && t.stride(-1) != 1) bad("the last dimension of %s must be contiguous", name);
}
void check_vector(const Tensor& t, const char* name, int64_t n, int dev) {
  check_ints(t, name, 1, dev);
  if (t.size(0) != n) bad("%s has the wrong length", name);
}

Tensor empty_like(const Tensor& t) {
  return at::detail::empty_cuda(t.sizes(), t.scalar_type(), t.device(), std::nullopt);
}

// The output of a call: the caller's (checked against `like`), or a new one.
Tensor output(PyObject* o, const char* name, const Tensor& like) {
  if (o == Py_None) return empty_like(like);
  const Tensor& t = tensor_of(o, name);
  if (!t.sizes().equals(like.sizes())) bad("%s has the wrong shape", name);
  check_heads(t, name, &like);
  for (int64_t i = 0; i < t.dim(); ++i)
    if (t.stride(i) == 0 && t.size(i) > 1) bad("%s has elements that share memory", name);
  return t;
}

sage_kv_cache cache_of(PyObject* const* a, int64_t d, int* dev) {
  const Tensor &k8 = tensor_of(a[0], "cache['k8']"), &ks = tensor_of(a[1], "cache['ks']"),
               &v8 = tensor_of(a[2], "cache['v8']"), &vs = tensor_of(a[3], "cache['vs']");
  if (k8.scalar_type() != at::kChar || v8.scalar_type() != at::kByte || ks.scalar_type() != at::kFloat ||
      vs.scalar_type() != at::kFloat)
    bad("the cache holds k8 int8, v8 uint8, ks and vs float32");
  if (!k8.is_cuda()) bad("the cache's arrays must be CUDA tensors (no CPU path exists)");
  if (*dev < 0) *dev = k8.get_device();
  for (const Tensor* t : {&k8, &ks, &v8, &vs})
    if (!t->is_cuda() || t->get_device() != *dev || !t->is_contiguous())
      bad("the cache's arrays must be contiguous and on the device of the other tensors");
  if (k8.dim() != 4 || d < 1 || k8.size(3) != (d + 15) / 16 * 16) bad("the cache does not hold heads of this many channels");
  if (!v8.sizes().equals(k8.sizes()) || !ks.sizes().equals(k8.sizes().slice(0, 3)) || !vs.sizes().equals(ks.sizes()))
    bad("the cache's arrays do not fit one another");
  sage_kv_cache c;
  c.k8 = static_cast<int8_t*>(pointer(&k8)), c.ks = static_cast<float*>(pointer(&ks));
  c.v8 = static_cast<uint8_t*>(pointer(&v8)), c.vs = static_cast<float*>(pointer(&vs));
  c.num_pages = narrow(k8.size(0), "the cache"), c.Hkv = narrow(k8.size(1), "the cache");
  c.page_size = narrow(k8.size(2), "the cache"), c.d = (int)d;
  return c;
}

const float* k_mean_of(PyObject* o, int64_t Hkv, int64_t d, int dev) {
  const Tensor* t = optional_of(o, "k_mean");
  if (t && (t->scalar_type() != at::kFloat || !t->is_cuda() || t->get_device() != dev || t->dim() != 2 ||
            t->size(0) != Hkv || t->size(1) != d || !t->is_contiguous()))
    bad("k_mean must be a contiguous float32 tensor (kv heads, head_dim) on the device of the others");
  return static_cast<const float*>(pointer(t));
}

// cos_sin, q_weight, k_weight, norm, eps, interleaved
sage_norm_rope norm_rope_of(PyObject* const* a, int64_t d, int dev) {
  sage_norm_rope nr = {};
  const Tensor *cs = optional_of(a[0], "cos_sin"), *qw = optional_of(a[1], "q_weight"), *kw = optional_of(a[2], "k_weight");
  nr.norm = bool_of(a[3]), nr.eps = (float)float_of(a[4]), nr.interleaved = bool_of(a[5]);
  nr.weight_dtype = SAGE_FP32;
  if ((qw || kw) && !nr.norm) bad("q_weight and k_weight need norm=True");
  for (const Tensor* w : {qw, kw})
    if (w) {
      if (!w->is_cuda() || w->get_device() != dev || dtype_code(w->scalar_type()) < 0 || w->dim() != 1 ||
          w->size(0) != d || !w->is_contiguous())
        bad("%s must be a contiguous fp16, bf16 or fp32 tensor of head_dim values on the device of the others",
            w == qw ? "q_weight" : "k_weight");
      nr.weight_dtype = (sage_dtype)dtype_code(w->scalar_type());
    }
  if (qw && kw && qw->scalar_type() != kw->scalar_type()) bad("q_weight and k_weight must share one dtype");
  nr.q_weight = pointer(qw), nr.k_weight = pointer(kw);
  if (cs) {
    if (cs->scalar_type() != at::kFloat || !cs->is_cuda() || cs->get_device() != dev || cs->dim() != 2 || !cs->is_contiguous())
      bad("cos_sin must be a contiguous float32 tensor (positions, rotary_dim) on the device of the others");
    if (cs->numel() == 0) bad("cos_sin must not be empty");
    nr.cos_sin = static_cast<const float*>(pointer(cs));
    nr.n_pos = narrow(cs->size(0), "cos_sin"), nr.rot = narrow(cs->size(1), "cos_sin");
  }
  return nr;
}

// The device of a call and its current stream.
struct On {
  c10::cuda::OptionalCUDAGuard guard;
  void* stream;
  explicit On(int dev) {
    if (c10::cuda::current_device() != dev) guard.set_index((c10::DeviceIndex)dev);
    stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
  }
};

PyObject* status(sage_status s) { return PyLong_FromLong(s); }

PyObject* two(const Tensor& a, const Tensor* b) {
  PyObject* x = THPVariable_Wrap(a);
  PyObject* y = b ? THPVariable_Wrap(*b) : Py_NewRef(Py_None);
  PyObject* t = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return t;
}

void want(Py_ssize_t n, Py_ssize_t expected) {
  if (n == expected) return;
  PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", expected, n);
  throw BadArgument();
}

#define SAGE_BINDING_BEGIN \
  HANDLE_TH_ERRORS         \
  try {
#define SAGE_BINDING_END        \
  }                             \
  catch (const BadArgument&) {  \
    return nullptr;             \
  }                             \
  END_HANDLE_TH_ERRORS

struct Extents {
  int64_t B, N, H;
  long long batch, token, head;
};
Extents extents(const Tensor& t, bool hnd) {
  if (t.dim() == 3) return {1, t.size(0), t.size(1), 0, t.stride(0), t.stride(1)};
  if (t.dim() != 4) bad("q and k must be 4-D, or 3-D (tokens, heads, head_dim)");
  if (hnd) return {t.size(0), t.size(2), t.size(1), t.stride(0), t.stride(2), t.stride(1)};
  return {t.size(0), t.size(1), t.size(2), t.stride(0), t.stride(1), t.stride(2)};
}

// (function, q, k, positions, hnd, cos_sin, q_weight, k_weight, norm, eps, interleaved, q_out, k_out) -> (q_out, k_out)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  SAGE_BINDING_BEGIN
  want(n, 13);
  const auto call = function_of<decltype(&sage_qk_norm_rope)>(a[0]);
  const Tensor& q = tensor_of(a[1], "q");
  const Tensor *k = optional_of(a[2], "k"), *positions = optional_of(a[3], "positions");
  check_heads(q, "q");
  const bool hnd = bool_of(a[4]);
  const Extents e = extents(q, hnd);
  const int64_t d = q.size(-1);
  const int dev = q.get_device();
  Extents ek = {};
  if (k) {
    check_heads(*k, "k", &q);
    ek = extents(*k, hnd);
    if (ek.B != e.B || ek.N != e.N || k->size(-1) != d || k->dim() != q.dim()) bad("k's shape does not fit q's");
  } else if (a[12] != Py_None) {
    bad("k_out needs k");
  }
  if (positions) {
    if (a[5] == Py_None) bad("positions need cos_sin");
    const int dims = positions->dim() == 1 ? 1 : 2;
    check_ints(*positions, "positions", dims, dev);
    if (positions->size(-1) != e.N || (dims == 2 && positions->size(0) != e.B)) bad("positions must be (N,) or (B, N)");
  }
  const sage_norm_rope nr = norm_rope_of(a + 5, d, dev);
  const On on(dev);
  const Tensor q_out = output(a[11], "q_out", q);
  const Tensor k_out = k ? output(a[12], "k_out", *k) : Tensor();
  const Extents eq = extents(q_out, hnd), eko = k ? extents(k_out, hnd) : Extents{};
  const long long strides[12] = {e.batch,  e.token,  e.head,  ek.batch,  ek.token,  ek.head,
                                 eq.batch, eq.token, eq.head, eko.batch, eko.token, eko.head};
  const sage_status s =
      call(pointer(&q), pointer(k), pointer(&q_out), k ? pointer(&k_out) : nullptr, strides,
           static_cast<const int32_t*>(pointer(positions)), positions && positions->dim() == 2 ? positions->stride(0) : 0,
           narrow(e.B, "q"), narrow(e.N, "q"), narrow(e.H, "q"), narrow(ek.H, "k"), narrow(d, "q"),
           (sage_dtype)dtype_code(q.scalar_type()), &nr, on.stream);
  return s == SAGE_OK ? two(q_out, k ? &k_out : nullptr) : status(s);
  SAGE_BINDING_END
}

// (function, k8, ks, v8, vs, k, v, page_table, seq_lens, cu_seqlens, q, cos_sin, q_weight, k_weight, norm, eps, interleaved,
//  k_mean, q_out) -> q_out or None
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  SAGE_BINDING_BEGIN
  want(n, 19);
  const auto call = function_of<decltype(&sage_cache_append)>(a[0]);
  const Tensor &k = tensor_of(a[5], "k"), &v = tensor_of(a[6], "v"), &table = tensor_of(a[7], "page_table"),
               &lens = tensor_of(a[8], "seq_lens");
  const Tensor *cu = optional_of(a[9], "cu_seqlens"), *q = optional_of(a[10], "q");
  check_heads(k, "k");
  check_heads(v, "v", &k);
  if (k.dim() != 3 || !v.sizes().equals(k.sizes())) bad("k and v must be 3-D (tokens, heads, head_dim) and of one shape");
  const int64_t T = k.size(0), Hkv = k.size(1), d = k.size(2);
  int dev = k.get_device();
  const sage_kv_cache c = cache_of(a + 1, d, &dev);
  if (c.Hkv != Hkv) bad("k does not have the cache's number of heads");
  check_ints(table, "page_table", 2, dev);
  const int64_t B = table.size(0);
  check_vector(lens, "seq_lens", B, dev);
  if (cu)
    check_vector(*cu, "cu_seqlens", B + 1, dev);
  else if (T != B)
    bad("there is not one token per sequence: pass cu_seqlens");
  if (q) {
    check_heads(*q, "q", &k);
    if (q->dim() != 3 || q->size(0) != T || q->size(2) != d) bad("q's shape does not fit k's");
  } else if (a[18] != Py_None) {
    bad("q_out needs q");
  }
  const float* mean = k_mean_of(a[17], Hkv, d, dev);
  const sage_norm_rope nr = norm_rope_of(a + 11, d, dev);
  const On on(dev);
  const Tensor q_out = q ? output(a[18], "q_out", *q) : Tensor();
  const long long strides[8] = {q ? q->stride(0) : 0, q ? q->stride(1) : 0,
                                k.stride(0),          k.stride(1),
                                v.stride(0),          v.stride(1),
                                q ? q_out.stride(0) : 0, q ? q_out.stride(1) : 0};
  const sage_status s = call(&c, pointer(q), pointer(&k), pointer(&v), q ? pointer(&q_out) : nullptr, strides,
                             static_cast<const int32_t*>(pointer(&table)), table.stride(0),
                             narrow(table.size(1), "page_table"), static_cast<const int32_t*>(pointer(&lens)),
                             static_cast<const int32_t*>(pointer(cu)), mean, narrow(T, "k"), narrow(B, "page_table"),
                             q ? narrow(q->size(1), "q") : 0, (sage_dtype)dtype_code(k.scalar_type()), &nr, on.stream);
  if (s != SAGE_OK) return status(s);
  return q ? THPVariable_Wrap(q_out) : Py_NewRef(Py_None);
  SAGE_BINDING_END
}

// (function, k8, ks, v8, vs, page_table, cu_seqlens, total, head_dim, dtype code, starts, k_mean, k_out, v_out)
// -> (k_out, v_out)
PyObject* cache_gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  SAGE_BINDING_BEGIN
  want(n, 14);
  const auto call = function_of<decltype(&sage_cache_gather)>(a[0]);
  const Tensor &table = tensor_of(a[5], "page_table"), &cu = tensor_of(a[6], "cu_seqlens");
  const int T = int32_of(a[7], "total"), d = int32_of(a[8], "head_dim"), code = int32_of(a[9], "dtype");
  const Tensor* starts = optional_of(a[10], "starts");
  const at::ScalarType type = code == SAGE_FP16 ? at::kHalf : code == SAGE_BF16 ? at::kBFloat16 : at::kFloat;
  int dev = -1;
  const sage_kv_cache c = cache_of(a + 1, d, &dev);
  check_ints(table, "page_table", 2, dev);
  const int64_t B = table.size(0);
  check_vector(cu, "cu_seqlens", B + 1, dev);
  if (starts) check_vector(*starts, "starts", B, dev);
  const float* mean = k_mean_of(a[11], c.Hkv, d, dev);
  if (T < 0) bad("total must not be negative");
  const On on(dev);
  const int64_t shape[3] = {T, c.Hkv, d};
  Tensor out[2];
  for (int i = 0; i < 2; ++i) {
    const char* name = i ? "v_out" : "k_out";
    const Tensor* t = optional_of(a[12 + i], name);
    if (t && (!t->is_cuda() || t->get_device() != dev || t->scalar_type() != type || !t->sizes().equals(shape) ||
              !t->is_contiguous()))
      bad("%s must be a contiguous tensor (total, kv heads, head_dim) of the given dtype on the cache's device", name);
    out[i] = t ? *t : Tensor(at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, (c10::DeviceIndex)dev), std::nullopt));
  }
  const sage_status s =
      call(&c, static_cast<const int32_t*>(pointer(&table)), table.stride(0), narrow(table.size(1), "page_table"),
           static_cast<const int32_t*>(pointer(&cu)), static_cast<const int32_t*>(pointer(starts)), mean,
           pointer(&out[0]), pointer(&out[1]), T, narrow(B, "page_table"), (sage_dtype)code, on.stream);
  return s == SAGE_OK ? two(out[0], &out[1]) : status(s);
  SAGE_BINDING_END
}

// (function, k8, ks, v8, vs, q, page_table, seq_lens, max_seqlen, sm_scale, out) -> out
PyObject* attn_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  SAGE_BINDING_BEGIN
  want(n, 11);
  const auto call = function_of<decltype(&sage_attn_decode)>(a[0]);
  const Tensor &q = tensor_of(a[5], "q"), &table = tensor_of(a[6], "page_table"), &lens = tensor_of(a[7], "seq_lens");
  check_heads(q, "q");
  if (q.dim() != 3) bad("q must be 3-D (sequences, heads, head_dim)");
  const int64_t B = q.size(0), d = q.size(2);
  int dev = q.get_device();
  const sage_kv_cache c = cache_of(a + 1, d, &dev);
  check_ints(table, "page_table", 2, dev);
  if (table.size(0) != B) bad("page_table must have a row for every sequence");
  check_vector(lens, "seq_lens", B, dev);
  const int most = int32_of(a[8], "max_seqlen");
  const float scale = (float)float_of(a[9]);
  const On on(dev);
  const Tensor out = output(a[10], "out", q);
  if (!out.is_contiguous()) bad("out must be contiguous");
  const sage_status s =
      call(pointer(&q), q.stride(0), q.stride(1), &c, static_cast<const int32_t*>(pointer(&table)), table.stride(0),
           narrow(table.size(1), "page_table"), static_cast<const int32_t*>(pointer(&lens)), pointer(&out),
           narrow(B, "q"), narrow(q.size(1), "q"), most, (sage_dtype)dtype_code(q.scalar_type()), scale, on.stream);
  return s == SAGE_OK ? THPVariable_Wrap(out) : status(s);
  SAGE_BINDING_END
}

#define SAGE_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {SAGE_METHOD(qk_norm_rope), SAGE_METHOD(cache_append), SAGE_METHOD(cache_gather),
                         SAGE_METHOD(attn_decode), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_sage_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sage_binding() { return PyModule_Create(&module); }
