// Native half of paged.py: checks the tensors of the paged serving calls, allocates their results through PyTorch's
// allocator and calls the C entry points of libzyfa.so on the current stream of the tensors' device.
//
// The calls are made once per layer and token, and small ones run for a few microseconds on the GPU: the same checks
// written in Python took 8 to 20 us of host time per call.  Errors are Python exceptions as elsewhere in the package:
// TypeError for a wrong type or layout, ValueError for wrong sizes or devices, ZyfaError for a status of the library.
#include <Python.h>

#include <ATen/Functions.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <optional>
#include <vector>

#include "zyfa.h"

namespace {

using at::Tensor;

PyObject* g_zyfa_error = nullptr;  // ZyfaError, set when the module is created

#define NEED_TYPE(cond, ...) TORCH_CHECK_TYPE(cond, __VA_ARGS__)
#define NEED_VALUE(cond, ...) TORCH_CHECK_VALUE(cond, __VA_ARGS__)

struct StatusError {
  int status;
  const char* what;
};

void succeed(zyfa_status_t st, const char* what) {
  if (st != ZYFA_OK) throw StatusError{static_cast<int>(st), what};
}

const Tensor& tensor(PyObject* o, const char* name) {
  NEED_TYPE(THPVariable_Check(o), name, " must be a CUDA tensor");
  const Tensor& t = THPVariable_Unpack(o);
  NEED_TYPE(t.layout() == at::kStrided, name, " must be a dense tensor");
  return t;
}

const Tensor* optional(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

int cuda_index(const Tensor& t) { return t.is_cuda() ? t.get_device() : -1; }

int64_t integer(PyObject* o, const char* name) {
  const int64_t x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw python_error();
  NEED_VALUE(x >= -(1ll << 31) && x < (1ll << 31), name, " is out of range");
  return x;
}

// A contiguous tensor of this type, device and shape.
void* exact(const Tensor& t, const char* name, at::ScalarType type, int dev, at::IntArrayRef shape) {
  NEED_TYPE(t.scalar_type() == type && t.is_contiguous(), name, " must be a contiguous ", type, " CUDA tensor");
  NEED_VALUE(dev >= 0 && cuda_index(t) == dev, name, " must be on the same CUDA device as the other tensors");
  NEED_VALUE(t.sizes() == shape, name, " must have shape ", shape, ", got ", t.sizes());
  return t.data_ptr();
}

int code_of(at::ScalarType t) {
  return t == at::kFloat8_e4m3fn || t == at::kByte ? ZYFA_DTYPE_E4M3 : t == at::kBFloat16 ? ZYFA_DTYPE_BF16 : -1;
}

struct Cache {
  zyfa_paged_cache_t c;
  int dev;
  at::ScalarType type;
};

Cache cache_of(PyObject* ko, PyObject* vo) {
  const Tensor &k = tensor(ko, "k_cache"), &v = tensor(vo, "v_cache");
  const int code = code_of(k.scalar_type());
  NEED_TYPE(code >= 0 && v.scalar_type() == k.scalar_type() && k.dim() == 4 && v.dim() == 4,
            "k_cache and v_cache must be e4m3 or bfloat16 CUDA tensors [num_pages, page_size, H_kv, D] of one type");
  const int dev = cuda_index(k);
  NEED_VALUE(dev >= 0 && cuda_index(v) == dev && v.size(0) == k.size(0) && v.size(1) == k.size(1) && v.size(2) == k.size(2),
             "k_cache and v_cache must agree in pages, page size, heads and CUDA device");
  NEED_VALUE(k.stride(3) == 1 && v.stride(3) == 1, "the last dimension of k_cache and v_cache must be contiguous");
  NEED_VALUE(k.size(1) < (1 << 30) && k.size(2) < (1 << 30) && k.size(3) < (1 << 30) && v.size(3) < (1 << 30),
             "k_cache and v_cache are too large in a dimension");
  Cache r;
  r.dev = dev;
  r.type = k.scalar_type();
  r.c = {k.data_ptr(), v.data_ptr(), static_cast<zyfa_dtype_t>(code), static_cast<int>(k.size(1)), k.size(0),
         static_cast<int>(k.size(2)), static_cast<int>(k.size(3)), static_cast<int>(v.size(3)),
         // a dimension of one element may carry any stride
         k.size(0) > 1 ? k.stride(0) : k.size(3), k.size(1) > 1 ? k.stride(1) : k.size(3), k.size(2) > 1 ? k.stride(2) : k.size(3),
         v.size(0) > 1 ? v.stride(0) : v.size(3), v.size(1) > 1 ? v.stride(1) : v.size(3), v.size(2) > 1 ? v.stride(2) : v.size(3)};
  return r;
}

struct Table {
  int* p;
  int64_t stride;
  int width;
};

// A block table whose rows may be part of a wider tensor.
Table table_of(PyObject* o, int64_t B, int dev) {
  const Tensor& t = tensor(o, "block_table");
  NEED_TYPE(t.scalar_type() == at::kInt && t.dim() == 2, "block_table must be an int32 CUDA tensor [B, max_pages]");
  const int64_t width = t.size(1);
  NEED_VALUE(t.size(0) == B && dev >= 0 && cuda_index(t) == dev, "block_table must have ", B,
             " rows, on the same device as the other tensors");
  NEED_VALUE(width < 2 || t.stride(1) == 1, "block_table rows must be contiguous");
  NEED_VALUE(B < 2 || t.stride(0) >= width, "block_table rows must not overlap");
  NEED_VALUE(width <= (1 << 30), "block_table is too wide");
  return {static_cast<int*>(t.data_ptr()), B > 1 ? t.stride(0) : width, static_cast<int>(width)};
}

struct Descales {
  const float* p[3] = {nullptr, nullptr, nullptr};
  int per_head = 0;  // 0, 1 or 3, as the attention takes them
};

// Three descales, all per tensor, all of `heads` values or all of `requests` times as many.
Descales descales_of(PyObject* const* o, int64_t heads, int64_t requests, int dev) {
  static const char* const names[3] = {"q_descale", "k_descale", "v_descale"};
  Descales d;
  int form = -1;
  for (int i = 0; i < 3; ++i) {
    const Tensor* t = optional(o[i], names[i]);
    if (!t) continue;
    NEED_TYPE(t->scalar_type() == at::kFloat && t->is_contiguous(), names[i], " must be a contiguous float32 CUDA tensor or None");
    NEED_VALUE(cuda_index(*t) == dev, names[i], " must be on the same CUDA device as the other tensors");
    const int64_t n = t->numel();
    NEED_VALUE(n == 1 || n == heads || n == requests * heads, names[i], " must hold 1, ", heads, " or ", requests * heads, " values, got ", n);
    const int mine = n == 1 ? 0 : n == heads ? 3 : 1;
    NEED_VALUE(form < 0 || form == mine, "descales must all be per tensor, all per head or all per request and head");
    form = mine;
    d.p[i] = static_cast<const float*>(t->data_ptr());
  }
  d.per_head = form < 0 ? 0 : form;
  return d;
}

Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int dev) {
  return Tensor(at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt));
}

// `n` elements of a larger allocation, from byte `offset` on, as a tensor of its own.
Tensor piece(const Tensor& all, at::ScalarType type, int64_t offset, int64_t n) {
  Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), c10::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef{n}, at::IntArrayRef{1}, offset / static_cast<int64_t>(c10::elementSize(type)));
  return t;
}

cudaStream_t stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

void count(Py_ssize_t n, Py_ssize_t want) { NEED_TYPE(n == want, "expected ", want, " arguments, got ", n); }

PyObject* pack(std::initializer_list<PyObject*> items) {  // steals its items
  PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
  Py_ssize_t i = 0;
  for (PyObject* x : items) {
    if (t) PyTuple_SET_ITEM(t, i++, x); else Py_XDECREF(x);
  }
  return t;
}

PyObject* keep(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// plan(cached_lens, new_lens, block_table, free_pages, cursor, page_size, max_tokens, out or None, result's tuple type) -> the five results
PyObject* plan(PyObject* const* a, Py_ssize_t n) {
  count(n, 9);
  NEED_TYPE(PyType_Check(a[8]) && PyType_IsSubtype(reinterpret_cast<PyTypeObject*>(a[8]), &PyTuple_Type), "expected a tuple type");
  const Tensor &cached = tensor(a[0], "cached_lens"), &fresh_lens = tensor(a[1], "new_lens"), &pool = tensor(a[3], "free_pages"),
               &cursor = tensor(a[4], "cursor");
  const int dev = cuda_index(cached);
  const int64_t page = integer(a[5], "page_size"), rows = integer(a[6], "max_tokens");
  NEED_VALUE(rows >= 0, "max_tokens must not be negative");
  NEED_TYPE(cached.dim() == 1, "cached_lens must be a contiguous int32 CUDA tensor [B]");
  const int64_t B = cached.size(0);
  NEED_VALUE(B <= (1 << 30), "too many requests");
  int* c = static_cast<int*>(exact(cached, "cached_lens", at::kInt, dev, {B}));
  int* f = static_cast<int*>(exact(fresh_lens, "new_lens", at::kInt, dev, {B}));
  const Table t = table_of(a[2], B, dev);
  NEED_TYPE(pool.dim() == 1, "free_pages must be a contiguous int32 CUDA tensor [num_free]");
  int* p = static_cast<int*>(exact(pool, "free_pages", at::kInt, dev, {pool.size(0)}));
  NEED_VALUE(pool.size(0) < (1ll << 31), "too many free pages");
  int* at_ = static_cast<int*>(exact(cursor, "cursor", at::kInt, dev, {1}));
  const int64_t sizes[5] = {B, B + 1, rows, rows, 1};
  void* o[5];
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  std::optional<Tensor> made[5];
  if (a[7] == Py_None) {
    // one allocation for the five (each costs a microsecond, a third of the kernel), slots first for their alignment
    static const int order[5] = {3, 0, 1, 2, 4};
    int64_t bytes = 0, at_byte[5];
    for (int i : order) {
      at_byte[i] = bytes;
      bytes += sizes[i] * (i == 3 ? 8 : 4);
    }
    const Tensor all = fresh({bytes}, at::kByte, dev);
    for (int i = 0; i < 5; ++i) {
      made[i] = piece(all, i == 3 ? at::kLong : at::kInt, at_byte[i], sizes[i]);
      o[i] = static_cast<char*>(all.data_ptr()) + at_byte[i];
    }
  } else {
    static const char* const names[5] = {"out.seq_lens", "out.cu_tokens", "out.positions", "out.slots", "out.cursor"};
    NEED_TYPE(PyTuple_Check(a[7]) && PyTuple_GET_SIZE(a[7]) == 5, "out must be a PagedPlan");
    for (int i = 0; i < 5; ++i) {
      PyObject* x = PyTuple_GET_ITEM(a[7], i);
      o[i] = exact(tensor(x, names[i]), names[i], i == 3 ? at::kLong : at::kInt, dev, {sizes[i]});
    }
  }
  succeed(zyfa_paged_plan(c, f, static_cast<int>(B), static_cast<int>(page), t.p, t.stride, t.width, p, static_cast<int>(pool.size(0)),
                          at_, static_cast<int*>(o[4]), static_cast<int*>(o[0]), static_cast<int*>(o[1]), static_cast<int*>(o[2]),
                          static_cast<long long*>(o[3]), static_cast<int>(rows), stream_of(dev)),
          "zyfa_paged_plan");
  if (a[7] != Py_None) return keep(a[7]);
  PyTypeObject* type = reinterpret_cast<PyTypeObject*>(a[8]);
  PyObject* out = type->tp_alloc(type, 5);
  if (!out) throw python_error();
  for (int i = 0; i < 5; ++i) {
    PyObject* x = THPVariable_Wrap(std::move(*made[i]));
    if (!x) {
      Py_DECREF(out);
      throw python_error();
    }
    PyTuple_SET_ITEM(out, i, x);
  }
  return out;
}

// A bf16 [N, heads, D] tensor with dense heads: its token stride.
int64_t rows_of(const Tensor& t, const char* name, int64_t N, int64_t heads, int64_t D, int dev) {
  NEED_TYPE(t.scalar_type() == at::kBFloat16 && t.dim() == 3, name, " must be a bfloat16 CUDA tensor [N, heads, D]");
  NEED_VALUE(t.size(0) == N && t.size(1) == heads && t.size(2) == D && cuda_index(t) == dev, name, " must have shape [", N, ", ", heads,
             ", ", D, "] on the cache's device, got ", t.sizes());
  NEED_VALUE(t.stride(2) == 1 && (heads < 2 || t.stride(1) == D), "the heads of one token of ", name, " must be contiguous");
  return N > 1 ? t.stride(0) : heads * D;
}

void* dense(const Tensor& t, const char* name, int code, at::IntArrayRef shape, int dev) {
  NEED_TYPE(code_of(t.scalar_type()) == code && t.is_contiguous(), name, " must be a contiguous CUDA tensor of the cache's type");
  NEED_VALUE(t.sizes() == shape && cuda_index(t) == dev, name, " must have shape ", shape, " on the cache's device, got ", t.sizes());
  return t.data_ptr();
}

// rope(inv_freq, axis_pairs or None, offset, interleaved) -> the checked specification that store() takes
PyObject* rope(PyObject* const* a, Py_ssize_t n) {
  count(n, 4);
  const Tensor& inv = tensor(a[0], "inv_freq");
  NEED_TYPE(inv.scalar_type() == at::kFloat && inv.dim() == 1 && inv.is_contiguous(),
            "inv_freq must be a contiguous float32 CUDA tensor [rot_dim / 2]");
  NEED_VALUE(inv.is_cuda() && inv.size(0) <= 4096, "inv_freq must be a CUDA tensor of at most 4096 pairs");
  integer(a[2], "offset");
  PyObject* pairs = a[1] == Py_None ? Py_BuildValue("(L)", static_cast<long long>(inv.size(0))) : PySequence_Tuple(a[1]);
  if (!pairs) throw python_error();
  const THPObjectPtr holder(pairs);
  const Py_ssize_t axes = PyTuple_GET_SIZE(pairs);
  NEED_VALUE(axes >= 1 && axes <= 4, "axis_pairs must be 1 to 4 counts");
  int64_t total = 0;
  for (Py_ssize_t i = 0; i < axes; ++i) {
    const int64_t x = integer(PyTuple_GET_ITEM(pairs, i), "axis_pairs");
    NEED_VALUE(x >= 0, "axis_pairs must not be negative");
    total += x;
  }
  NEED_VALUE(total == inv.size(0), "axis_pairs must sum to ", inv.size(0), ", got ", total);
  return pack({keep(a[0]), keep(pairs), keep(a[2]), keep(a[3])});
}

// store(q, k, v, k_cache, v_cache, slots, positions, (inv_freq, axis_pairs, offset, interleaved) or None, q_descale, k_descale,
//       v_descale, q_out, k_out, v_out) -> q_out or None
PyObject* store(PyObject* const* a, Py_ssize_t n) {
  count(n, 14);
  const Cache cache = cache_of(a[3], a[4]);
  const int dev = cache.dev, code = cache.c.dtype;
  const int64_t H_kv = cache.c.H_kv, D_qk = cache.c.D_qk, D_v = cache.c.D_v;
  const Tensor *q = optional(a[0], "q"), *k = optional(a[1], "k"), *v = optional(a[2], "v");
  const Tensor* some = q ? q : k;
  NEED_TYPE(some && !k == !v && some->dim() == 3, "q, or k and v, must be given as [N, heads, D]");
  const int64_t N = some->size(0), H = q ? q->size(1) : H_kv;
  NEED_VALUE(H < (1 << 30), "too many heads");
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  const Tensor *qo = optional(a[11], "q_out"), *ko = optional(a[12], "k_out"), *vo = optional(a[13], "v_out");
  int64_t qs = 0, ks = 0, vs = 0;
  std::optional<Tensor> made;
  void* qop = nullptr;
  if (q) {
    qs = rows_of(*q, "q", N, H, D_qk, dev);
    if (!qo) made = fresh({N, H, D_qk}, cache.type, dev);
    qop = qo ? dense(*qo, "q_out", code, {N, H, D_qk}, dev) : made->data_ptr();
    NEED_VALUE(N == 0 || qop != q->data_ptr(), "q_out must not be q");
  } else {
    NEED_VALUE(!qo, "q_out without q");
  }
  if (k) {
    ks = rows_of(*k, "k", N, H_kv, D_qk, dev);
    vs = rows_of(*v, "v", N, H_kv, D_v, dev);
  } else {
    NEED_VALUE(!ko && !vo, "k_out or v_out without k and v");
  }
  void* kop = ko ? dense(*ko, "k_out", code, {N, H_kv, D_qk}, dev) : nullptr;
  void* vop = vo ? dense(*vo, "v_out", code, {N, H_kv, D_v}, dev) : nullptr;
  NEED_VALUE(N == 0 || ((!kop || kop != k->data_ptr()) && (!vop || vop != v->data_ptr())), "k_out and v_out must not be k and v");
  void* slots = exact(tensor(a[5], "slots"), "slots", at::kLong, dev, {N});
  zyfa_rope_t spec = {};
  const int* positions = nullptr;
  int64_t stride = 0;
  const bool turns = a[7] != Py_None;
  if (turns) {
    NEED_TYPE(PyTuple_Check(a[7]) && PyTuple_GET_SIZE(a[7]) == 4 && PyTuple_Check(PyTuple_GET_ITEM(a[7], 1)), "rope must be a Rope");
    const Tensor& inv = tensor(PyTuple_GET_ITEM(a[7], 0), "rope.inv_freq");
    PyObject* pairs = PyTuple_GET_ITEM(a[7], 1);
    NEED_VALUE(inv.dim() == 1 && inv.size(0) <= 4096, "rope.inv_freq must be [rot_dim / 2]");
    spec.inv_freq = static_cast<const float*>(exact(inv, "rope.inv_freq", at::kFloat, dev, {inv.size(0)}));
    spec.rot_dim = static_cast<int>(2 * inv.size(0));
    spec.rot_offset = static_cast<int>(integer(PyTuple_GET_ITEM(a[7], 2), "rope.offset"));
    spec.interleaved = PyObject_IsTrue(PyTuple_GET_ITEM(a[7], 3)) == 1;
    const Py_ssize_t axes = PyTuple_GET_SIZE(pairs);
    NEED_VALUE(axes >= 1 && axes <= 4, "rope.axis_pairs must be 1 to 4 counts");
    spec.num_axes = static_cast<int>(axes);
    for (Py_ssize_t i = 0; i < axes; ++i) spec.axis_pairs[i] = static_cast<int>(integer(PyTuple_GET_ITEM(pairs, i), "rope.axis_pairs"));
    const Tensor* pos = optional(a[6], "positions");
    NEED_TYPE(pos && pos->scalar_type() == at::kInt, "positions must be an int32 CUDA tensor [N] or [axes, N]");
    const bool flat = pos->dim() == 1 && axes == 1;
    NEED_VALUE(cuda_index(*pos) == dev && (flat ? pos->size(0) == N : pos->dim() == 2 && pos->size(0) == axes && pos->size(1) == N) &&
                   (N < 2 || pos->stride(-1) == 1),
               "positions must be [", axes, ", ", N, "] with contiguous rows, on the cache's device");
    positions = static_cast<const int*>(pos->data_ptr());
    stride = axes > 1 ? pos->stride(0) : N;
    NEED_VALUE(stride >= N, "positions rows must not overlap");
  }
  const Descales d = code == ZYFA_DTYPE_E4M3 ? descales_of(a + 8, H_kv, 1, dev) : Descales();
  // (an empty tensor has no address, which the C call would take for one that is not given)
  if (N > 0)
    succeed(zyfa_rope_paged_store(q ? q->data_ptr() : nullptr, k ? k->data_ptr() : nullptr, v ? v->data_ptr() : nullptr, qs, ks, vs, qop,
                                kop, vop, positions, stride, static_cast<const long long*>(slots), N, static_cast<int>(H), &cache.c,
                                turns ? &spec : nullptr, d.p[0], d.p[1], d.p[2], d.per_head != 0, stream_of(dev)),
          "zyfa_rope_paged_store");
  return made ? THPVariable_Wrap(std::move(*made)) : keep(a[11]);
}

// decode(q, k_cache, v_cache, block_table, seq_lens, softmax_scale, q_descale, k_descale, v_descale, out, return_lse, workspace)
PyObject* decode(PyObject* const* a, Py_ssize_t n) {
  count(n, 12);
  const Cache cache = cache_of(a[1], a[2]);
  const int dev = cache.dev, code = cache.c.dtype;
  const int64_t H_kv = cache.c.H_kv, D_qk = cache.c.D_qk, D_v = cache.c.D_v;
  const Tensor& q = tensor(a[0], "q");
  NEED_TYPE(code_of(q.scalar_type()) == code && q.dim() == 3, "q must be a CUDA tensor [B, H, D_qk] of the cache's type");
  const int64_t B = q.size(0), H = q.size(1);
  NEED_VALUE(q.size(2) == D_qk && cuda_index(q) == dev, "q must have ", D_qk, " channels, on the cache's device");
  NEED_VALUE(H >= 1 && H < (1 << 30) && B < (1 << 30) && H_kv >= 1 && H % H_kv == 0, "the number of query heads must be a multiple of ",
             H_kv);
  NEED_VALUE(q.stride(2) == 1 && (H < 2 || q.stride(1) == D_qk), "the heads of one request of q must be contiguous");
  const Table t = table_of(a[3], B, dev);
  void* lens = exact(tensor(a[4], "seq_lens"), "seq_lens", at::kInt, dev, {B});
  double scale = 0.0;
  if (a[5] != Py_None) {
    scale = PyFloat_AsDouble(a[5]);
    if (scale == -1.0 && PyErr_Occurred()) throw python_error();
    NEED_VALUE(scale == 0.0 || static_cast<float>(scale) != 0.0f, "softmax_scale is below the smallest float32");  // 0: the default
  }
  const Descales d = code == ZYFA_DTYPE_E4M3 ? descales_of(a + 6, H_kv, B, dev) : Descales();
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  const Tensor* given = optional(a[9], "out");
  std::optional<Tensor> made, lse;
  if (!given) made = fresh({B, H, D_v}, at::kBFloat16, dev);
  void* out = given ? exact(*given, "out", at::kBFloat16, dev, {B, H, D_v}) : made->data_ptr();
  const int want_lse = PyObject_IsTrue(a[10]);
  if (want_lse < 0) throw python_error();
  if (want_lse) lse = fresh({B, H}, at::kFloat, dev);
  const Tensor* ws = optional(a[11], "workspace");
  std::optional<Tensor> scratch;
  if (ws) {
    NEED_TYPE(ws->scalar_type() == at::kByte && ws->is_contiguous() && cuda_index(*ws) == dev,
              "workspace must be a contiguous uint8 tensor on the cache's device");
  } else {
    const size_t bytes = zyfa_attn_decode_paged_workspace_bytes(static_cast<int>(B), static_cast<int>(H), static_cast<int>(H_kv),
                                                                static_cast<int>(D_v), static_cast<long long>(t.width) * cache.c.page_size);
    scratch = fresh({static_cast<int64_t>(bytes)}, at::kByte, dev);
    ws = &*scratch;
  }
  succeed(zyfa_attn_decode_paged(q.data_ptr(), B > 1 ? q.stride(0) : H * D_qk, &cache.c, t.p, t.stride, t.width,
                                 static_cast<const int*>(lens), out, lse ? static_cast<float*>(lse->data_ptr()) : nullptr,
                                 static_cast<int>(B), static_cast<int>(H), static_cast<float>(scale), d.p[0], d.p[1], d.p[2], d.per_head,
                                 ws->data_ptr(), static_cast<size_t>(ws->numel()), stream_of(dev)),
          "zyfa_attn_decode_paged");
  PyObject* result = made ? THPVariable_Wrap(std::move(*made)) : keep(a[9]);
  return lse ? pack({result, THPVariable_Wrap(std::move(*lse))}) : result;
}

// No C++ exception leaves a C entry: each becomes a Python one.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(args, n);
  } catch (const StatusError& e) {
    PyObject* x = PyObject_CallFunction(g_zyfa_error, "is", e.status, e.what);
    if (x) {
      PyErr_SetObject(g_zyfa_error, x);
      Py_DECREF(x);
    }
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyMethodDef g_methods[] = {
    {"plan", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<plan>)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<rope>)), METH_FASTCALL, nullptr},
    {"store", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<store>)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<decode>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged(void) {
  PyObject* api = PyImport_ImportModule("fp8_causal_prefill_gb300.api");
  if (!api) return nullptr;
  g_zyfa_error = PyObject_GetAttrString(api, "ZyfaError");
  Py_DECREF(api);
  if (!g_zyfa_error) return nullptr;
  return PyModule_Create(&g_module);
}
