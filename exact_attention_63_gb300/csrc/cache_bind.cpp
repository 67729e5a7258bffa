// The short way from Python to the cache operators and the rotary positions: dense tensors on the current
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

constexpr at::ScalarType kBf16 = at::kBFloat16, kF32 = at::kFloat, kI32 = at::kInt, kI64 = at::kLong,
                         kF64 = at::kDouble, kCodes = at::kFloat8_e4m3fn, kScales = at::kFloat8_e8m0fnu;

// One call's tensors: `get` clears `ok` unless the tensor is plain, dense, of the type
// and on the current device.
struct Args {
  int dev = -1;  // the current one, asked for at the first CUDA tensor
  bool ok = true;

  // A tensor of the type, of `other` as well where that is given, on the current device.
  const at::Tensor* any(PyObject* o, at::ScalarType type, at::ScalarType other) {
    if (!THPVariable_CheckExact(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (dev < 0 && t.is_cuda()) dev = c10::cuda::current_device();
    if (!t.is_cuda() || t.get_device() != dev || (t.scalar_type() != type && t.scalar_type() != other) ||
        t.layout() != at::kStrided || t.numel() == 0) {
      ok = false;
      return nullptr;
    }
    return &t;
  }
  const at::Tensor* get(PyObject* o, at::ScalarType type, int dims, at::ScalarType other) {
    const at::Tensor* const t = any(o, type, other);
    if (t != nullptr && t->dim() == dims && t->is_contiguous()) return t;
    ok = false;
    return nullptr;
  }
  const at::Tensor* get(PyObject* o, at::ScalarType type, int dims) { return get(o, type, dims, type); }
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

// (x, y), both owned; nullptr where one is.
PyObject* both(PyObject* x, PyObject* y) {
  PyObject* const t = x != nullptr && y != nullptr ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return t;
}

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
  return both(out != nullptr ? Py_NewRef(p[11]) : THPVariable_Wrap(new_out),
              lse != nullptr ? Py_NewRef(p[12]) : THPVariable_Wrap(new_lse));
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

// A cache of codes, and its scales' addresses.
attn_cache codes_of(Args& a, PyObject* k, PyObject* v, PyObject* ks, PyObject* vs, PyObject* table, PyObject* lens,
                    void** k_scales, void** v_scales) {
  attn_cache c;
  std::memset(&c, 0, sizeof(c));
  c.struct_size = sizeof(c);
  const at::Tensor* const tk = a.get(k, kCodes, 4, at::kByte);
  const at::Tensor* const tv = a.get(v, kCodes, 4, at::kByte);
  const at::Tensor* const tks = a.get(ks, kScales, 3, at::kByte);
  const at::Tensor* const tvs = a.get(vs, kScales, 3, at::kByte);
  const at::Tensor* const tt = a.get(table, kI32, 2);
  const at::Tensor* const tl = a.get(lens, kI32, 1);
  if (!a.ok) return c;
  c.n_seq = a.size(tt->size(0));
  c.max_blocks = a.size(tt->size(1));
  c.n_pages = a.size(tk->size(0));
  c.page_size = a.size(tk->size(1));
  c.num_kv_heads = a.size(tk->size(2));
  c.d = a.size(tk->size(3));
  a.same(tv->sizes() == tk->sizes());
  a.same(tl->size(0) == c.n_seq);
  a.same(shaped(tks, c.n_pages, c.num_kv_heads, c.page_size / 16) && tvs->sizes() == tks->sizes());
  c.k = address(tk);
  c.v = address(tv);
  c.block_table = static_cast<const int*>(address(tt));
  c.seq_lens = static_cast<const int*>(address(tl));
  *k_scales = address(tks);
  *v_scales = address(tvs);
  return c;
}

// (q, k_new, v_new, k, v, k_scales, v_scales, table, lens, cu, max_new | parents, scale, out, lse,
// workspace) → (out, lse), a status, or None
PyObject* attend_fp8(PyObject*, PyObject* const* p, Py_ssize_t n) {
  constexpr Py_ssize_t required = 11;
  CACHE_ARGS(16);
  void *ks = nullptr, *vs = nullptr;
  const attn_cache c = codes_of(a, p[3], p[4], p[5], p[6], p[7], p[8], &ks, &vs);
  if (!a.ok) Py_RETURN_NONE;
  attn_new_tokens x = tokens_of(a, c, p[0], p[1], p[2], p[9]);
  if (!a.ok) Py_RETURN_NONE;
  x.max_seqlen = a.integer(p[10]);
  const at::Tensor* const parents = a.maybe(p[11], kI32, 1);
  const float scale = a.scale(p[12], c.d);
  const at::Tensor* const out = a.maybe(p[13], kBf16, 3);
  const at::Tensor* const lse = a.maybe(p[14], kF32, 2);
  const at::Tensor* const given = p[15] == Py_None ? nullptr : a.get(p[15], at::kByte, 1);
  if (!a.ok) Py_RETURN_NONE;
  const size_t need = attn_fwd_cache_fp8_workspace_size(x.H, c.num_kv_heads, x.max_seqlen, c.d);
  a.same(parents == nullptr || parents->size(0) == x.total);
  a.same(out == nullptr || shaped(out, x.total, x.H, c.d));
  a.same(lse == nullptr || (lse->size(0) == x.H && lse->size(1) == x.total));
  if (!a.ok || need == 0) Py_RETURN_NONE;
  at::Tensor new_out, new_lse, workspace;
  if (out == nullptr) new_out = empty(a, {x.total, x.H, c.d}, kBf16);
  if (lse == nullptr) new_lse = empty(a, {x.H, x.total}, kF32);
  if (given == nullptr) workspace = empty(a, {static_cast<int64_t>(need)}, at::kByte);
  const at::Tensor& ws = given != nullptr ? *given : workspace;
  const int rc = attn_fwd_cache_fp8(&c, ks, vs, &x, static_cast<const int*>(address(parents)), scale,
                                    out != nullptr ? out->data_ptr() : new_out.data_ptr(),
                                    static_cast<float*>(lse != nullptr ? lse->data_ptr() : new_lse.data_ptr()),
                                    ws.data_ptr(), static_cast<size_t>(ws.numel()), nullptr, stream_of(a));
  if (rc != ATTN_OK) return status(rc);
  return both(out != nullptr ? Py_NewRef(p[13]) : THPVariable_Wrap(new_out),
              lse != nullptr ? Py_NewRef(p[14]) : THPVariable_Wrap(new_lse));
  END_HANDLE_TH_ERRORS
}

// (k_new, v_new, k, v, k_scales, v_scales, table, lens, cu | rows) → a status, or None
PyObject* append_fp8(PyObject*, PyObject* const* p, Py_ssize_t n) {
  constexpr Py_ssize_t required = 9;
  CACHE_ARGS(10);
  void *ks = nullptr, *vs = nullptr;
  const attn_cache c = codes_of(a, p[2], p[3], p[4], p[5], p[6], p[7], &ks, &vs);
  if (!a.ok) Py_RETURN_NONE;
  const attn_new_tokens x = tokens_of(a, c, Py_None, p[0], p[1], p[8]);
  const at::Tensor* const rows = a.maybe(p[9], kI32, 1);
  if (!a.ok) Py_RETURN_NONE;
  const int n_rows = rows == nullptr ? 0 : a.size(rows->size(0));
  if (!a.ok) Py_RETURN_NONE;
  return status(attn_cache_append_fp8(&c, ks, vs, &x, static_cast<const int*>(address(rows)), n_rows, stream_of(a)));
  END_HANDLE_TH_ERRORS
}

// (k, v, k_scales, v_scales, table, lens, cu, total | k_out, v_out) → (k_out, v_out), a status, or None
PyObject* gather_fp8(PyObject*, PyObject* const* p, Py_ssize_t n) {
  constexpr Py_ssize_t required = 8;
  CACHE_ARGS(10);
  void *ks = nullptr, *vs = nullptr;
  const attn_cache c = codes_of(a, p[0], p[1], p[2], p[3], p[4], p[5], &ks, &vs);
  const at::Tensor* const cu = a.get(p[6], kI32, 1);
  const int total = a.integer(p[7]);
  const at::Tensor* const k_out = a.maybe(p[8], kBf16, 3);
  const at::Tensor* const v_out = a.maybe(p[9], kBf16, 3);
  if (!a.ok || total < 1) Py_RETURN_NONE;
  a.same(cu->size(0) == static_cast<int64_t>(c.n_seq) + 1);
  a.same(k_out == nullptr || shaped(k_out, total, c.num_kv_heads, c.d));
  a.same(v_out == nullptr || shaped(v_out, total, c.num_kv_heads, c.d));
  if (!a.ok) Py_RETURN_NONE;
  at::Tensor new_k, new_v;
  if (k_out == nullptr) new_k = empty(a, {total, c.num_kv_heads, c.d}, kBf16);
  if (v_out == nullptr) new_v = empty(a, {total, c.num_kv_heads, c.d}, kBf16);
  const int rc = attn_cache_gather_fp8(&c, ks, vs, static_cast<const int*>(address(cu)), total,
                                       k_out != nullptr ? k_out->data_ptr() : new_k.data_ptr(),
                                       v_out != nullptr ? v_out->data_ptr() : new_v.data_ptr(), stream_of(a));
  if (rc != ATTN_OK) return status(rc);
  return both(k_out != nullptr ? Py_NewRef(p[8]) : THPVariable_Wrap(new_k),
              v_out != nullptr ? Py_NewRef(p[9]) : THPVariable_Wrap(new_v));
  END_HANDLE_TH_ERRORS
}

// (lens, table, n_blocks, free_pages, n_free, page_size | cu, total, missing, slots, positions)
// → (missing, slots, positions), a status, or None
PyObject* pages(PyObject*, PyObject* const* p, Py_ssize_t n) {
  constexpr Py_ssize_t required = 6;
  CACHE_ARGS(11);
  const at::Tensor* const lens = a.get(p[0], kI32, 1);
  const at::Tensor* const table = a.get(p[1], kI32, 2);
  const at::Tensor* const blocks = a.get(p[2], kI32, 1);
  const at::Tensor* const free_pages = a.get(p[3], kI32, 1);
  const at::Tensor* const n_free = a.get(p[4], kI32, 1);
  const at::Tensor* const cu = a.maybe(p[6], kI32, 1);
  const at::Tensor* const missing = a.maybe(p[8], kI32, 1);
  const at::Tensor* const slots = a.maybe(p[9], kI64, 1);
  const at::Tensor* const positions = a.maybe(p[10], kI32, 1);
  attn_pages t;
  std::memset(&t, 0, sizeof(t));
  t.struct_size = sizeof(t);
  t.page_size = a.integer(p[5]);
  const int total = a.integer(p[7]);
  if (!a.ok || total < 0 || (cu == nullptr) != (total == 0)) Py_RETURN_NONE;
  t.n_seq = a.size(table->size(0));
  t.max_blocks = a.size(table->size(1));
  t.n_pages = a.size(free_pages->size(0));
  a.same(lens->size(0) == t.n_seq && blocks->size(0) == t.n_seq && n_free->size(0) == 1);
  a.same(cu == nullptr || cu->size(0) == static_cast<int64_t>(t.n_seq) + 1);
  a.same(missing == nullptr || missing->size(0) == t.n_seq);
  a.same(slots == nullptr || slots->size(0) == total);
  a.same(positions == nullptr || positions->size(0) == total);
  if (!a.ok) Py_RETURN_NONE;
  t.block_table = static_cast<int*>(address(table));
  t.n_blocks = static_cast<int*>(address(blocks));
  t.free_pages = static_cast<int*>(address(free_pages));
  t.n_free = static_cast<int*>(address(n_free));
  at::Tensor new_missing, new_slots, new_positions;
  if (missing == nullptr) new_missing = empty(a, {t.n_seq}, kI32);
  if (cu != nullptr && slots == nullptr) new_slots = empty(a, {total}, kI64);
  if (cu != nullptr && positions == nullptr) new_positions = empty(a, {total}, kI32);
  const at::Tensor* const to_slots = slots != nullptr ? slots : (cu != nullptr ? &new_slots : nullptr);
  const at::Tensor* const to_positions = positions != nullptr ? positions : (cu != nullptr ? &new_positions : nullptr);
  const int rc = attn_cache_pages(&t, static_cast<const int*>(address(lens)),
                                  static_cast<int*>(missing != nullptr ? missing->data_ptr() : new_missing.data_ptr()),
                                  static_cast<const int*>(address(cu)), total, static_cast<long long*>(address(to_slots)),
                                  static_cast<int*>(address(to_positions)), stream_of(a));
  if (rc != ATTN_OK) return status(rc);
  PyObject* const x = missing != nullptr ? Py_NewRef(p[8]) : THPVariable_Wrap(new_missing);
  PyObject* const y = slots != nullptr || cu == nullptr ? Py_NewRef(p[9]) : THPVariable_Wrap(new_slots);
  PyObject* const z = positions != nullptr || cu == nullptr ? Py_NewRef(p[10]) : THPVariable_Wrap(new_positions);
  PyObject* const all = x != nullptr && y != nullptr && z != nullptr ? PyTuple_Pack(3, x, y, z) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  Py_XDECREF(z);
  return all;
  END_HANDLE_TH_ERRORS
}

// q or k of the rotary positions, and its result (`fresh` where none is given): strided views
// whose rows do not overlap.
attn_rows rows_of(Args& a, PyObject* in, PyObject* out, at::Tensor* fresh) {
  attn_rows r;
  std::memset(&r, 0, sizeof(r));
  r.struct_size = sizeof(r);
  const at::Tensor* const x = a.any(in, kBf16, kBf16);
  const at::Tensor* y = out == Py_None ? nullptr : a.any(out, kBf16, kBf16);
  if (!a.ok || x->dim() < 3 || x->dim() > 4 || (y != nullptr && y->sizes() != x->sizes())) {
    a.ok = false;
    return r;
  }
  if (y == nullptr) {
    *fresh = empty(a, x->sizes(), kBf16);
    y = fresh;
  }
  const int dims = static_cast<int>(x->dim());
  r.heads = a.size(x->size(dims - 2));
  for (int side = 0; side < 2; ++side) {
    const at::Tensor& t = side ? *y : *x;
    long long* const st = side ? r.y_strides : r.x_strides;
    if (t.is_contiguous()) continue;  // zeros: dense
    // From the head inwards out: each stride holds what is inside it.
    int64_t inside = t.size(dims - 1);
    a.same(t.stride(dims - 1) == 1);
    for (int i = 2; i >= 0; --i) {
      const int at = dims - 4 + i;  // (packed rows have no batch)
      const int64_t entries = at < 0 ? 1 : t.size(at), stride = entries > 1 ? t.stride(at) : inside;
      a.same(stride >= inside && stride > 0);
      st[i] = stride;
      inside = stride * entries;
    }
  }
  r.x = x->data_ptr();
  r.y = y->data_ptr();
  return r;
}

// (q, k, positions, inv_freq, interleaved, magnitude, q_out, k_out, inverse) → (q', k'), a status, or None
PyObject* rotary(PyObject*, PyObject* const* p, Py_ssize_t n) {
  constexpr Py_ssize_t required = 1;
  CACHE_ARGS(9);
  const at::Tensor* const freq = a.get(p[3], kF64, 1);
  if (!a.ok || !PyBool_Check(p[4]) || !PyFloat_CheckExact(p[5]) || (p[1] == Py_None && p[7] != Py_None)) Py_RETURN_NONE;
  at::Tensor new_q, new_k;
  const attn_rows q = rows_of(a, p[0], p[6], &new_q);
  attn_rows k;
  if (a.ok && p[1] != Py_None) k = rows_of(a, p[1], p[7], &new_k);
  if (!a.ok) Py_RETURN_NONE;
  const at::Tensor& tq = THPVariable_Unpack(p[0]);
  const int dims = static_cast<int>(tq.dim());
  const int64_t batch = dims == 4 ? tq.size(0) : 1, rows = tq.size(dims - 3), d = tq.size(dims - 1);
  if (p[1] != Py_None) {
    const at::Tensor& tk = THPVariable_Unpack(p[1]);
    a.same(tk.dim() == dims && tk.size(0) == tq.size(0) && tk.size(dims - 3) == rows && tk.size(dims - 1) == d);
  }
  const at::Tensor* positions = nullptr;
  int64_t apart = 0;
  if (p[2] != Py_None) {
    positions = a.any(p[2], kI32, kI32);
    if (!a.ok || !positions->is_contiguous()) Py_RETURN_NONE;
    const bool one = positions->dim() == 1 && positions->size(0) == rows;
    a.same(one || (dims == 4 && positions->dim() == 2 && positions->size(0) == batch && positions->size(1) == rows));
    apart = one ? 0 : rows;
  }
  const int b = a.size(batch), r = a.size(rows), pairs = a.size(freq->size(0));
  if (!a.ok || pairs > 1024) Py_RETURN_NONE;
  const int rc = attn_rotary(&q, p[1] != Py_None ? &k : nullptr, b, r, a.size(d),
                             static_cast<const int*>(address(positions)), apart,
                             static_cast<const double*>(address(freq)), 2 * pairs, p[4] == Py_True,
                             static_cast<float>(PyFloat_AS_DOUBLE(p[5])), p[8] == Py_True, stream_of(a));
  if (rc != ATTN_OK) return status(rc);
  return both(p[6] != Py_None ? Py_NewRef(p[6]) : THPVariable_Wrap(new_q),
              p[1] == Py_None ? Py_NewRef(Py_None) : (p[7] != Py_None ? Py_NewRef(p[7]) : THPVariable_Wrap(new_k)));
  END_HANDLE_TH_ERRORS
}

PyMethodDef kMethods[] = {
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"weigh", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(weigh)), METH_FASTCALL, nullptr},
    {"select", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(select)), METH_FASTCALL, nullptr},
    {"compact", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(compact)), METH_FASTCALL, nullptr},
    {"attend_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend_fp8)), METH_FASTCALL, nullptr},
    {"append_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append_fp8)), METH_FASTCALL, nullptr},
    {"gather_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(gather_fp8)), METH_FASTCALL, nullptr},
    {"pages", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(pages)), METH_FASTCALL, nullptr},
    {"rotary", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rotary)), METH_FASTCALL, nullptr},
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
