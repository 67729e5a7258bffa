// The short way from Python to the cache operators: dense tensors on the current
// device, the current stream, no options.  Each function checks its tensors, fills
// the structs of the C ABI and calls it, or answers None where anything is not as
// expected; cache.py then looks at the arguments one by one, for strides, another
// device or stream, or the reason of a refusal.
//   A decoding step's kernels take 3 to 12 us.  Checked and packed in Python a call
// took 7 to 22 us of host time; here it takes 3 to 11, of which the launches are the most
// (back to back, one token: attention 22.5 -> 14.3 us, append 9.3 -> 4.1).
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cmath>
#include <cstring>

#include "attn_gb300.h"

namespace {

constexpr at::ScalarType kBf16 = at::kBFloat16, kF32 = at::kFloat, kI32 = at::kInt;

// One call's tensors: `get` clears `ok` unless the tensor is plain, dense, of the type
// and on the current device.
struct Args {
  int dev = -1;  // the current one, asked for at the first CUDA tensor
  bool ok = true;

  const at::Tensor* get(PyObject* o, at::ScalarType type, int dims) {
    if (!THPVariable_CheckExact(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (dev < 0 && t.is_cuda()) dev = c10::cuda::current_device();
    if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || t.dim() != dims ||
        t.layout() != at::kStrided || !t.is_contiguous() || t.numel() == 0) {
      ok = false;
      return nullptr;
    }
    return &t;
  }
  const at::Tensor* maybe(PyObject* o, at::ScalarType type, int dims) {
    return o == Py_None ? nullptr : get(o, type, dims);
  }
  int integer(PyObject* o) {
    if (!PyLong_CheckExact(o)) {
      ok = false;
      return 0;
    }
    int over = 0;
    const long long x = PyLong_AsLongLongAndOverflow(o, &over);
    if (over != 0 || x < -0x7FFFFFFFll || x > 0x7FFFFFFFll) ok = false;
    return static_cast<int>(x);
  }
  float scale(PyObject* o, int d) {
    if (o == Py_None) return static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
    if (!PyFloat_CheckExact(o)) ok = false;
    return ok ? static_cast<float>(PyFloat_AS_DOUBLE(o)) : 0.f;
  }
  // A size that the structs' ints hold.
  int size(int64_t n) {
    if (n > 0x7FFFFFFFll) ok = false;
    return static_cast<int>(n);
  }
  void same(bool x) { ok = ok && x; }
};

void* address(const at::Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }

bool shaped(const at::Tensor* t, int64_t a, int64_t b, int64_t c) {
  return t->size(0) == a && t->size(1) == b && t->size(2) == c;
}

// The cache of the tensors; k, or else weights, gives the sizes.
attn_cache cache_of(Args& a, PyObject* k, PyObject* v, PyObject* table, PyObject* lens, PyObject* weights,
                    PyObject* positions) {
  attn_cache c;
  std::memset(&c, 0, sizeof(c));
  c.struct_size = sizeof(c);
  const at::Tensor* const tk = a.maybe(k, kBf16, 4);
  const at::Tensor* const tv = a.maybe(v, kBf16, 4);
  const at::Tensor* const tt = a.get(table, kI32, 2);
  const at::Tensor* const tl = a.maybe(lens, kI32, 1);
  const at::Tensor* const tw = a.maybe(weights, kF32, 3);
  const at::Tensor* const tp = a.maybe(positions, kI32, 3);
  if (!a.ok || (tk == nullptr && tw == nullptr)) {
    a.ok = false;
    return c;
  }
  c.n_seq = a.size(tt->size(0));
  c.max_blocks = a.size(tt->size(1));
  if (tk != nullptr) {
    c.n_pages = a.size(tk->size(0));
    c.page_size = a.size(tk->size(1));
    c.num_kv_heads = a.size(tk->size(2));
    c.d = a.size(tk->size(3));
  } else {
    c.n_pages = a.size(tw->size(0));
    c.num_kv_heads = a.size(tw->size(1));
    c.page_size = a.size(tw->size(2));
  }
  a.same(tv == nullptr || tv->sizes() == tk->sizes());
  a.same(tl == nullptr || tl->size(0) == c.n_seq);
  a.same(tw == nullptr || shaped(tw, c.n_pages, c.num_kv_heads, c.page_size));
  a.same(tp == nullptr || shaped(tp, c.n_pages, c.num_kv_heads, c.page_size));
  c.k = address(tk);
  c.v = address(tv);
  c.block_table = static_cast<const int*>(address(tt));
  c.seq_lens = static_cast<const int*>(address(tl));
  c.weights = static_cast<float*>(address(tw));
  c.positions = static_cast<int*>(address(tp));
  return c;
}

// The new tokens of the tensors: q, or k and v, or all three.
attn_new_tokens tokens_of(Args& a, const attn_cache& c, PyObject* q, PyObject* k, PyObject* v, PyObject* cu) {
  attn_new_tokens x;
  std::memset(&x, 0, sizeof(x));
  x.struct_size = sizeof(x);
  const at::Tensor* const tq = a.maybe(q, kBf16, 3);
  const at::Tensor* const tk = a.maybe(k, kBf16, 3);
  const at::Tensor* const tv = a.maybe(v, kBf16, 3);
  const at::Tensor* const tc = a.get(cu, kI32, 1);
  if (!a.ok) return x;
  const int64_t total = (tq != nullptr ? tq : tk)->size(0);
  x.total = a.size(total);
  x.H = tq != nullptr ? a.size(tq->size(1)) : c.num_kv_heads;
  a.same(tc->size(0) == static_cast<int64_t>(c.n_seq) + 1);
  a.same(tq == nullptr || (tq->size(2) == c.d && x.H % c.num_kv_heads == 0));
  a.same(tk == nullptr || (shaped(tk, total, c.num_kv_heads, c.d) && shaped(tv, total, c.num_kv_heads, c.d)));
  x.q = address(tq);
  x.k = address(tk);
  x.v = address(tv);
  x.cu_seqlens = static_cast<const int*>(address(tc));
  return x;
}

cudaStream_t stream_of(const Args& a) {
  return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(a.dev)).stream();
}

at::Tensor empty(const Args& a, at::IntArrayRef sizes, at::ScalarType type) {
  return at::empty(sizes, at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(a.dev)));
}

PyObject* status(int rc) { return PyLong_FromLong(rc); }

#define CACHE_ARGS(count)                                                       \
  HANDLE_TH_ERRORS                                                              \
  if (n != (count)) {                                                           \
    PyErr_SetString(PyExc_TypeError, "cache binding: wrong number of arguments"); \
    return nullptr;                                                             \
  }                                                                             \
  for (Py_ssize_t i = 0; i < required; ++i)                                     \
    if (p[i] == Py_None) Py_RETURN_NONE;                                        \
  Args a

// (q, k_new, v_new, k, v, table, lens, cu, max_new | parents, scale, out, lse, workspace)
// → (out, lse), a status, or None
PyObject* attend(PyObject*, PyObject* const* p, Py_ssize_t n) {
  constexpr Py_ssize_t required = 9;
  CACHE_ARGS(14);
  const attn_cache c = cache_of(a, p[3], p[4], p[5], p[6], Py_None, Py_None);
  if (!a.ok) Py_RETURN_NONE;
  attn_new_tokens x = tokens_of(a, c, p[0], p[1], p[2], p[7]);
  if (!a.ok) Py_RETURN_NONE;
  x.max_seqlen = a.integer(p[8]);
  const at::Tensor* const parents = a.maybe(p[9], kI32, 1);
  const float scale = a.scale(p[10], c.d);
  const at::Tensor* const out = a.maybe(p[11], kBf16, 3);
  const at::Tensor* const lse = a.maybe(p[12], kF32, 2);
  const at::Tensor* const given = p[13] == Py_None ? nullptr : a.get(p[13], at::kByte, 1);
  if (!a.ok) Py_RETURN_NONE;
  const size_t need = attn_fwd_cache_workspace_size(x.H, c.num_kv_heads, x.max_seqlen, c.d);
  a.same(parents == nullptr || parents->size(0) == x.total);
  a.same(out == nullptr || shaped(out, x.total, x.H, c.d));
  a.same(lse == nullptr || (lse->size(0) == x.H && lse->size(1) == x.total));
  if (!a.ok || need == 0) Py_RETURN_NONE;
  at::Tensor new_out, new_lse, workspace;
  if (out == nullptr) new_out = empty(a, {x.total, x.H, c.d}, kBf16);
  if (lse == nullptr) new_lse = empty(a, {x.H, x.total}, kF32);
  if (given == nullptr) workspace = empty(a, {static_cast<int64_t>(need)}, at::kByte);
  const at::Tensor& ws = given != nullptr ? *given : workspace;
  const int rc = attn_fwd_cache(&c, &x, static_cast<const int*>(address(parents)), scale,
                                out != nullptr ? out->data_ptr() : new_out.data_ptr(),
                                static_cast<float*>(lse != nullptr ? lse->data_ptr() : new_lse.data_ptr()),
                                ws.data_ptr(), static_cast<size_t>(ws.numel()), nullptr, stream_of(a));
  if (rc != ATTN_OK) return status(rc);
  PyObject* const o = out != nullptr ? Py_NewRef(p[11]) : THPVariable_Wrap(new_out);
  PyObject* const l = lse != nullptr ? Py_NewRef(p[12]) : THPVariable_Wrap(new_lse);
  PyObject* const both = o != nullptr && l != nullptr ? PyTuple_Pack(2, o, l) : nullptr;
  Py_XDECREF(o);
  Py_XDECREF(l);
  return both;
  END_HANDLE_TH_ERRORS
}

// (k_new, v_new, k, v, table, lens, cu | rows, weights, positions, seq_pos) → a status, or None
PyObject* append(PyObject*, PyObject* const* p, Py_ssize_t n) {
  constexpr Py_ssize_t required = 7;
  CACHE_ARGS(11);
  const attn_cache c = cache_of(a, p[2], p[3], p[4], p[5], p[8], p[9]);
  if (!a.ok) Py_RETURN_NONE;
  const attn_new_tokens x = tokens_of(a, c, Py_None, p[0], p[1], p[6]);
  const at::Tensor* const rows = a.maybe(p[7], kI32, 1);
  const at::Tensor* const seq_pos = a.maybe(p[10], kI32, 1);
  if (!a.ok) Py_RETURN_NONE;
  a.same(seq_pos == nullptr || seq_pos->size(0) == c.n_seq);
  const int n_rows = rows == nullptr ? 0 : a.size(rows->size(0));
  if (!a.ok) Py_RETURN_NONE;
  return status(attn_cache_append(&c, &x, static_cast<const int*>(address(rows)), n_rows,
                                  static_cast<const int*>(address(seq_pos)), stream_of(a)));
  END_HANDLE_TH_ERRORS
}

// (q, lse, k, table, lens, cu, max_new, out | weights, scale) → a status, or None
PyObject* weigh(PyObject*, PyObject* const* p, Py_ssize_t n) {
  constexpr Py_ssize_t required = 8;
  CACHE_ARGS(10);
  const attn_cache c = cache_of(a, p[2], Py_None, p[3], p[4], p[8], Py_None);
  if (!a.ok) Py_RETURN_NONE;
  attn_new_tokens x = tokens_of(a, c, p[0], Py_None, Py_None, p[5]);
  const at::Tensor* const lse = a.get(p[1], kF32, 2);
  const at::Tensor* const out = a.get(p[7], kF32, 3);
  x.max_seqlen = a.integer(p[6]);
  const float scale = a.scale(p[9], c.d);
  if (!a.ok) Py_RETURN_NONE;
  a.same(lse->size(0) == x.H && lse->size(1) == x.total);
  a.same(shaped(out, c.n_pages, c.num_kv_heads, c.page_size));
  if (!a.ok) Py_RETURN_NONE;
  return status(attn_cache_weights(&c, &x, static_cast<const float*>(address(lse)), scale,
                                   static_cast<float*>(address(out)), nullptr, stream_of(a)));
  END_HANDLE_TH_ERRORS
}

// (weights, table, lens, budget, recent | positions, seq_pos, kept) → kept, a status, or None
PyObject* select(PyObject*, PyObject* const* p, Py_ssize_t n) {
  constexpr Py_ssize_t required = 5;
  CACHE_ARGS(8);
  const attn_cache c = cache_of(a, Py_None, Py_None, p[1], p[2], p[0], p[5]);
  const int budget = a.integer(p[3]), recent = a.integer(p[4]);
  const at::Tensor* const seq_pos = a.maybe(p[6], kI32, 1);
  const at::Tensor* const kept = a.maybe(p[7], kI32, 3);
  if (!a.ok || budget < 1) Py_RETURN_NONE;
  a.same(seq_pos == nullptr || seq_pos->size(0) == c.n_seq);
  a.same(seq_pos != nullptr || p[5] == Py_None);
  a.same(kept == nullptr || shaped(kept, c.n_seq, c.num_kv_heads, budget));
  if (!a.ok) Py_RETURN_NONE;
  at::Tensor fresh;
  if (kept == nullptr) fresh = empty(a, {c.n_seq, c.num_kv_heads, budget}, kI32);
  const int rc = attn_cache_select(&c, static_cast<const int*>(address(seq_pos)), budget, recent,
                                   static_cast<int*>(kept != nullptr ? kept->data_ptr() : fresh.data_ptr()),
                                   stream_of(a));
  if (rc != ATTN_OK) return status(rc);
  return kept != nullptr ? Py_NewRef(p[7]) : THPVariable_Wrap(fresh);
  END_HANDLE_TH_ERRORS
}

// (kept, k, v, table | weights, positions) → a status, or None
PyObject* compact(PyObject*, PyObject* const* p, Py_ssize_t n) {
  constexpr Py_ssize_t required = 4;
  CACHE_ARGS(6);
  const attn_cache c = cache_of(a, p[1], p[2], p[3], Py_None, p[4], p[5]);
  const at::Tensor* const kept = a.get(p[0], kI32, 3);
  if (!a.ok) Py_RETURN_NONE;
  const int budget = a.size(kept->size(2));
  a.same(kept->size(0) == c.n_seq && kept->size(1) == c.num_kv_heads);
  if (!a.ok) Py_RETURN_NONE;
  return status(attn_cache_compact(&c, static_cast<const int*>(address(kept)), budget, stream_of(a)));
  END_HANDLE_TH_ERRORS
}

PyMethodDef kMethods[] = {
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"weigh", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(weigh)), METH_FASTCALL, nullptr},
    {"select", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(select)), METH_FASTCALL, nullptr},
    {"compact", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(compact)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_cache_bind", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cache_bind() {
  PyObject* const m = PyModule_Create(&kModule);
  // PyTorch's C++ classes differ from version to version: cache.py compares.
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
