// serving_binding.cpp - argument marshalling of the serving operators (serving.py) and of the 8-bit
// integer product (int8.py): tensors checked and unpacked, outputs allocated, the C ABI of
// include/fp8amax_serving.h and include/fp8amax_int8.h called through the addresses serving.py
// hands over.  The same in Python took 4 to 7 us of calls that take 8 to 11,
// where the kernels of a decode step run for 3 to 12.
//
// The functions return what the operator returns, or the status code (an int) of a refused call.
#include <hip/hip_runtime_api.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/Exceptions.h>
#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>

#include <cmath>
#include <map>
#include <string>
#include <utility>

#include "fp8amax_int8.h"
#include "fp8amax_serving.h"

namespace {

decltype(&fp8_paged_plan) plan_fn;
decltype(&fp8_kv_append) append_fn;
decltype(&fp8_rope_append) rope_fn;
decltype(&fp8_attn_prompt) prompt_fn;
decltype(&fp8_attn_paged) paged_fn;
decltype(&fp8_attn_paged_workspace) workspace_fn;
decltype(&int8_quantize_rowwise) quantize8_fn;
decltype(&int8_gemm_scaled_rowwise) gemm8_fn;

std::string shape_of(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), what, " must be a tensor");
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o, const char* what) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    TORCH_CHECK_TYPE(false, what, " must be an integer");
  }
  return v;
}

fp8_dtype_t dtype_of(const at::Tensor& t, const char* what) {
  TORCH_CHECK_TYPE(t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kHalf, what, " must be bfloat16 or float16, got ", t.scalar_type());
  return t.scalar_type() == at::kBFloat16 ? FP8_BF16 : FP8_F16;
}

// A [tokens, heads, dim] operand whose rows the kernels read 16 bytes at a time: as it lies if its
// last index is contiguous, the other strides are multiples of 8 and tokens do not overlap, else a copy.
at::Tensor rows(const at::Tensor& t, const char* what, int64_t dim) {
  TORCH_CHECK_VALUE(t.dim() == 3, what, " must be [tokens, heads, head_dim], got shape ", shape_of(t));
  TORCH_CHECK_VALUE(dim == 0 || t.size(2) == dim, what, " must have head_dim ", dim, ", got ", t.size(2));
  const int64_t ts = t.stride(0), hs = t.stride(1);
  const auto at = reinterpret_cast<uintptr_t>(t.data_ptr());
  if (t.stride(2) == 1 && ((ts | hs) & 7) == 0 && (at & 15) == 0 && ts >= t.size(2) && ts <= 1 << 20) return t;
  at::Tensor c = t.contiguous();
  return reinterpret_cast<uintptr_t>(c.data_ptr()) & 15 ? c.clone() : c;
}

at::Tensor vec(const at::Tensor& t, const char* what, at::ScalarType type, int64_t size) {
  TORCH_CHECK_TYPE(t.scalar_type() == type, what, " must be ", type, ", got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.dim() == 1 && (size < 0 || t.size(0) == size), what, " must have shape (", size < 0 ? "n" : std::to_string(size), "), got ", shape_of(t));
  return t.is_contiguous() ? t : t.contiguous();
}

void dense(const at::Tensor& t, const char* what, at::ScalarType type, at::IntArrayRef shape) {
  TORCH_CHECK_TYPE(t.scalar_type() == type, what, " must be ", type, ", got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.sizes() == shape, what, " must have shape ", shape, ", got ", shape_of(t));
  TORCH_CHECK_VALUE(t.is_contiguous(), what, " must be contiguous");
}

const at::Tensor& table(const at::Tensor& t, int64_t batch) {
  TORCH_CHECK_TYPE(t.scalar_type() == at::kInt, "block_table must be int32, got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.dim() == 2 && t.size(0) == batch && t.is_contiguous(), "block_table must be a contiguous [", batch, ", width], got ", shape_of(t));
  return t;
}

// Checked last: every tensor on the same GPU (the library launches on that GPU's current stream).
void on(const at::Tensor& like, std::initializer_list<std::pair<const at::Tensor*, const char*>> others) {
  TORCH_CHECK_VALUE(like.is_cuda(), "all tensors must be on the GPU");
  for (const auto& o : others)
    TORCH_CHECK_VALUE(o.first->device() == like.device(), o.second, " must be on ", like.device(), ", got ", o.first->device());
}

// Whether a dense output shares memory with an operand.
bool overlaps(const at::Tensor& out, const at::Tensor& t) {
  if (out.numel() == 0 || t.numel() == 0) return false;
  int64_t last = 0;
  for (int64_t i = 0; i < t.dim(); ++i) last += (t.size(i) - 1) * t.stride(i);
  const char *a = static_cast<const char*>(out.data_ptr()), *b = static_cast<const char*>(t.data_ptr());
  return a < b + (last + 1) * t.element_size() && b < a + out.numel() * out.element_size();
}

at::Tensor output(PyObject* given, const at::Tensor& q, std::initializer_list<const at::Tensor*> inputs) {
  if (given == Py_None) return at::empty(q.sizes(), q.options());
  const at::Tensor& out = tensor(given, "out");
  dense(out, "out", q.scalar_type(), q.sizes());
  for (const at::Tensor* t : inputs) TORCH_CHECK_VALUE(!t->defined() || !overlaps(out, *t), "out overlaps an input");
  return out;
}

// Four-bit codes come with scales of one byte for 32 channels: a last index more than e4m3's.
bool is_byte_scale(at::ScalarType t) { return t == at::kByte || t == at::kFloat8_e8m0fnu; }

struct Cache {
  at::Tensor k, v, ks, vs;
  fp8_kv_format_t format;
  int64_t dim;      // channels
};
Cache cache_of(PyObject* k, PyObject* v, PyObject* ks, PyObject* vs, at::ScalarType type) {
  Cache c{tensor(k, "k_cache"), tensor(v, "v_cache"), {}, {}, FP8_KV_SAME, 0};
  TORCH_CHECK_VALUE(c.k.dim() == 4, "k_cache must be [pages, kv_heads, page_size, head_dim], got ", shape_of(c.k));
  const auto kind = c.k.scalar_type();
  dense(c.k, "k_cache", kind, c.k.sizes());
  dense(c.v, "v_cache", kind, c.k.sizes());
  c.dim = c.k.size(3);
  TORCH_CHECK_VALUE((ks == Py_None) == (vs == Py_None), "k_scales and v_scales go together");
  if (ks == Py_None) {
    TORCH_CHECK_TYPE(kind == type, "a cache without scales must be ", type, ", got ", kind);
    return c;
  }
  c.ks = tensor(ks, "k_scales");
  c.vs = tensor(vs, "v_scales");
  const auto scale = c.ks.scalar_type();
  if (is_byte_scale(scale)) {
    TORCH_CHECK_TYPE(kind == at::kByte || kind == at::kFloat4_e2m1fn_x2, "a cache with scales of a byte must be uint8 or float4_e2m1fn_x2, got ", kind);
    c.dim = 2 * c.k.size(3);
    const int64_t shape[4] = {c.k.size(0), c.k.size(1), c.k.size(2), c.dim / 32};
    dense(c.ks, "k_scales", scale, shape);
    dense(c.vs, "v_scales", scale, shape);
    c.format = FP8_KV_MXFP4;
    return c;
  }
  TORCH_CHECK_TYPE(kind == at::kByte || kind == at::kFloat8_e4m3fn, "a cache with scales must be uint8 or float8_e4m3fn, got ", kind);
  dense(c.ks, "k_scales", at::kFloat, c.k.sizes().slice(0, 3));
  dense(c.vs, "v_scales", at::kFloat, c.k.sizes().slice(0, 3));
  c.format = FP8_KV_E4M3;
  return c;
}
void* raw(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// For the calls that write a cache: its tensors share no memory with each other.  `one`: keys and values are the
// same rows, which may go to one cache.
void apart(const Cache& c, bool one) {
  const at::Tensor* const t[4] = {&c.k, &c.v, &c.ks, &c.vs};
  const bool shared = one && c.k.data_ptr() == c.v.data_ptr() && raw(c.ks) == raw(c.vs);
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 4; ++j)
      TORCH_CHECK_VALUE(!t[i]->defined() || !t[j]->defined() || (shared && j - i == 1 && i != 1) || !overlaps(*t[i], *t[j]), "caches or their scales overlap");
}
void on_cache(const at::Tensor& like, const Cache& c) {
  on(like, {{&c.k, "k_cache"}, {&c.v, "v_cache"}});
  if (c.format != FP8_KV_SAME) on(like, {{&c.ks, "k_scales"}, {&c.vs, "v_scales"}});
}

template <typename T>
T* ptr(const at::Tensor& t) { return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr; }

void* stream_of(PyObject* o) { return PyLong_AsVoidPtr(o); }

// A workspace of a stream, its counters zero at first and kept: a call leaves it fit for the next.  A
// call that is being captured in a HIP graph gets its own, since the graph may be replayed on any stream.
at::Tensor workspace_of(const at::Tensor& q, void* stream, int64_t need) {
  static auto& kept = *new std::map<std::pair<int, void*>, at::Tensor>;   // lives as long as the process
  hipStreamCaptureStatus status = hipStreamCaptureStatusNone;
  (void)hipStreamIsCapturing(static_cast<hipStream_t>(stream), &status);
  const bool capturing = status != hipStreamCaptureStatusNone;
  at::Tensor own;
  at::Tensor& have = capturing ? own : kept[{q.get_device(), stream}];
  if (!have.defined() || have.size(0) < need) {
    have = at::empty({std::max<int64_t>(need, FP8_ATTN_COUNTER_BYTES)}, q.options().dtype(at::kByte));
    have.narrow(0, 0, FP8_ATTN_COUNTER_BYTES).zero_();
  }
  return have;
}

PyObject* status(fp8_status_t code) { return PyLong_FromLong(code); }
PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

// A part of an allocation as a tensor of its own (as split and view make it, without their dispatch).
at::Tensor part(const at::Tensor& base, int64_t first_byte, int64_t n, at::ScalarType type) {
  auto impl = c10::make_intrusive<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(base.storage()), base.key_set(),
                                                   c10::scalarTypeToTypeMeta(type));
  impl->set_storage_offset(first_byte / static_cast<int64_t>(c10::elementSize(type)));
  impl->set_sizes_contiguous({n});
  return at::Tensor(std::move(impl));
}

#define ARGS(n) TORCH_CHECK_TYPE(nargs == (n), "expected ", (n), " arguments, got ", nargs)

// cached, added, block_table, free_pages, taken, tokens, page_size, out (None or six tensors), stream
PyObject* paged_plan(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  ARGS(9);
  const at::Tensor cached = vec(tensor(a[0], "cached"), "cached", at::kInt, -1);
  const int64_t batch = cached.size(0);
  const at::Tensor added = vec(tensor(a[1], "added"), "added", at::kInt, batch);
  const at::Tensor& tab = table(tensor(a[2], "block_table"), batch);
  const at::Tensor free = vec(tensor(a[3], "free_pages"), "free_pages", at::kInt, -1);
  const at::Tensor taken = vec(tensor(a[4], "taken"), "taken", at::kInt, 1);
  const int64_t tokens = integer(a[5], "tokens"), page = integer(a[6], "page_size");
  TORCH_CHECK_VALUE(tokens >= 0, "tokens must not be negative, got ", tokens);
  TORCH_CHECK_VALUE(page == static_cast<int32_t>(page), "page_size must be a power of two, 16 .. 1024, got ", page);
  at::Tensor o[6];   // cu_tokens, seq_lens, positions, slots, taken, missing
  if (a[7] == Py_None) {
    on(cached, {{&added, "added"}, {&tab, "block_table"}, {&free, "free_pages"}, {&taken, "taken"}});
    const at::Tensor all = at::empty({3 * tokens + 2 * batch + 3}, cached.options());
    o[3] = part(all, 0, tokens, at::kLong);
    o[2] = part(all, 8 * tokens, tokens, at::kInt);
    o[0] = part(all, 12 * tokens, batch + 1, at::kInt);
    o[1] = part(all, 12 * tokens + 4 * (batch + 1), batch, at::kInt);
    o[4] = part(all, 12 * tokens + 4 * (2 * batch + 1), 1, at::kInt);
    o[5] = part(all, 12 * tokens + 4 * (2 * batch + 2), 1, at::kInt);
  } else {
    static const char* const names[6] = {"out.cu_tokens", "out.seq_lens", "out.positions", "out.slots", "out.taken", "out.missing"};
    const int64_t sizes[6] = {batch + 1, batch, tokens, tokens, 1, 1};
    TORCH_CHECK_TYPE(PyTuple_Check(a[7]) && PyTuple_GET_SIZE(a[7]) == 6, "out must be a PagedPlan");
    for (int i = 0; i < 6; ++i) {
      o[i] = tensor(PyTuple_GET_ITEM(a[7], i), names[i]);
      dense(o[i], names[i], i == 3 ? at::kLong : at::kInt, {sizes[i]});
      for (const at::Tensor* t : {&cached, &added, &tab, &free, &taken}) TORCH_CHECK_VALUE(!overlaps(o[i], *t), names[i], " overlaps an input");
      for (int k = 0; k < i; ++k) TORCH_CHECK_VALUE(!overlaps(o[i], o[k]), names[i], " overlaps ", names[k]);
    }
    on(cached, {{&added, "added"}, {&tab, "block_table"}, {&free, "free_pages"}, {&taken, "taken"}, {&o[0], names[0]}, {&o[1], names[1]},
                {&o[2], names[2]}, {&o[3], names[3]}, {&o[4], names[4]}, {&o[5], names[5]}});
  }
  const c10::DeviceGuard guard(cached.device());   // the launch goes to the tensors' GPU
  const fp8_status_t code = plan_fn(ptr<int32_t>(cached), ptr<int32_t>(added), batch, static_cast<int32_t>(page), ptr<int32_t>(tab), tab.size(1),
                                    ptr<int32_t>(free), free.size(0), ptr<int32_t>(taken), tokens, ptr<int32_t>(o[0]), ptr<int32_t>(o[1]),
                                    ptr<int32_t>(o[2]), ptr<int64_t>(o[3]), ptr<int32_t>(o[4]), ptr<int32_t>(o[5]), stream_of(a[8]));
  if (code != FP8_OK) return status(code);
  if (a[7] != Py_None) {
    Py_INCREF(a[7]);
    return a[7];
  }
  PyObject* r = PyTuple_New(6);
  if (r)
    for (int i = 0; i < 6; ++i) PyTuple_SET_ITEM(r, i, wrap(o[i]));
  return r;
  END_HANDLE_TH_ERRORS
}

// k, v, slots, k_cache, v_cache, k_scales, v_scales, stream
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  ARGS(8);
  const at::Tensor& k0 = tensor(a[0], "k");
  const at::Tensor& v0 = tensor(a[1], "v");
  const fp8_dtype_t dt = dtype_of(k0, "k");
  TORCH_CHECK_VALUE(v0.scalar_type() == k0.scalar_type() && v0.sizes() == k0.sizes(), "v must be like k, got ", v0.scalar_type(), " ", shape_of(v0), " and ",
                    k0.scalar_type(), " ", shape_of(k0));
  const Cache c = cache_of(a[3], a[4], a[5], a[6], k0.scalar_type());
  const int64_t heads = c.k.size(1), dim = c.dim, page = c.k.size(2);
  const bool one = k0.data_ptr() == v0.data_ptr() && k0.strides() == v0.strides();
  const at::Tensor k = rows(k0, "k", dim), v = one ? k : rows(v0, "v", dim);
  TORCH_CHECK_VALUE(k.size(1) == heads, "k has ", k.size(1), " heads, the cache ", heads);
  const at::Tensor slots = vec(tensor(a[2], "slots"), "slots", at::kLong, k.size(0));
  for (const at::Tensor* t : {&c.k, &c.v, &c.ks, &c.vs})
    TORCH_CHECK_VALUE(!t->defined() || (!overlaps(*t, k) && !overlaps(*t, v) && !overlaps(*t, slots)), "a cache overlaps k, v or slots");
  apart(c, one);
  on(k, {{&v, "v"}, {&slots, "slots"}});
  on_cache(k, c);
  const c10::DeviceGuard guard(k.device());   // the launch goes to the tensors' GPU
  return status(append_fn(k.data_ptr(), v.data_ptr(), dt, k.size(0), heads, static_cast<int32_t>(dim), k.stride(0), k.stride(1), v.stride(0), v.stride(1),
                          ptr<int64_t>(slots), c.k.size(0), static_cast<int32_t>(page), c.format, c.k.data_ptr(), c.v.data_ptr(), raw(c.ks),
                          raw(c.vs), stream_of(a[7])));
  END_HANDLE_TH_ERRORS
}

// q (or None), k, v, positions, cos_sin, slots, k_cache, v_cache, k_scales, v_scales, interleaved, out, stream
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  ARGS(13);
  const at::Tensor& k0 = tensor(a[1], "k");
  const at::Tensor& v0 = tensor(a[2], "v");
  const fp8_dtype_t dt = dtype_of(k0, "k");
  TORCH_CHECK_VALUE(v0.scalar_type() == k0.scalar_type() && v0.sizes() == k0.sizes(), "v must be like k, got ", v0.scalar_type(), " ", shape_of(v0), " and ",
                    k0.scalar_type(), " ", shape_of(k0));
  const Cache c = cache_of(a[6], a[7], a[8], a[9], k0.scalar_type());
  const int64_t heads = c.k.size(1), dim = c.dim, page = c.k.size(2);
  const at::Tensor k = rows(k0, "k", dim), v = rows(v0, "v", dim);
  TORCH_CHECK_VALUE(k.size(1) == heads, "k has ", k.size(1), " heads, the cache ", heads);
  const int64_t tokens = k.size(0);
  const bool with_q = a[0] != Py_None;
  TORCH_CHECK_VALUE(with_q || a[11] == Py_None, "out goes with q");
  at::Tensor q;
  if (with_q) {
    const at::Tensor& q0 = tensor(a[0], "q");
    TORCH_CHECK_TYPE(q0.scalar_type() == k0.scalar_type(), "q must be of k's type, got ", q0.scalar_type(), " and ", k0.scalar_type());
    q = rows(q0, "q", dim);
    TORCH_CHECK_VALUE(q.size(0) == tokens, "q has ", q.size(0), " tokens, k ", tokens);
  }
  const at::Tensor positions = vec(tensor(a[3], "positions"), "positions", at::kInt, tokens);
  const at::Tensor& table = tensor(a[4], "cos_sin");
  TORCH_CHECK_VALUE(table.dim() == 2, "cos_sin must be [positions, rotary_dim], got ", shape_of(table));
  dense(table, "cos_sin", at::kFloat, table.sizes());
  const int64_t rotary = table.size(1);
  TORCH_CHECK_VALUE(rotary >= 16 && rotary <= dim && rotary % 16 == 0, "rotary_dim must be a multiple of 16, 16 .. ", dim, ", got ", rotary);
  const at::Tensor slots = vec(tensor(a[5], "slots"), "slots", at::kLong, tokens);
  const int interleaved = PyObject_IsTrue(a[10]);
  if (interleaved < 0) return nullptr;
  for (const at::Tensor* t : {&c.k, &c.v, &c.ks, &c.vs})
    for (const at::Tensor* in : std::initializer_list<const at::Tensor*>{&q, &k, &v, &positions, &table, &slots})
      TORCH_CHECK_VALUE(!t->defined() || !in->defined() || !overlaps(*t, *in), "a cache overlaps an input");
  apart(c, false);
  if (a[11] == Py_None) {
    on(k, {{&v, "v"}, {&positions, "positions"}, {&table, "cos_sin"}, {&slots, "slots"}});
    on_cache(k, c);
    if (with_q) on(k, {{&q, "q"}});
  }
  const at::Tensor out = with_q ? output(a[11], q, {&q, &k, &v, &positions, &table, &slots, &c.k, &c.v, &c.ks, &c.vs}) : at::Tensor();
  if (a[11] != Py_None) {
    on(k, {{&v, "v"}, {&positions, "positions"}, {&table, "cos_sin"}, {&slots, "slots"}, {&q, "q"}, {&out, "out"}});
    on_cache(k, c);
  }
  const c10::DeviceGuard guard(k.device());   // the launch goes to the tensors' GPU
  const fp8_status_t code = rope_fn(
      raw(q), k.data_ptr(), v.data_ptr(), dt, tokens, with_q ? q.size(1) : 0, heads, static_cast<int32_t>(dim), with_q ? q.stride(0) : 0,
      with_q ? q.stride(1) : 0, k.stride(0), k.stride(1), v.stride(0), v.stride(1), ptr<int32_t>(positions), ptr<float>(table), table.size(0),
      static_cast<int32_t>(rotary), interleaved, ptr<int64_t>(slots), c.k.size(0), static_cast<int32_t>(page), c.format,
      c.k.data_ptr(), c.v.data_ptr(), raw(c.ks), raw(c.vs), raw(out), stream_of(a[12]));
  if (code != FP8_OK) return status(code);
  if (!with_q) Py_RETURN_NONE;
  if (a[11] != Py_None) {
    Py_INCREF(a[11]);
    return a[11];
  }
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

struct Scores {
  float scale;
  int64_t window;
  bool lse;
};
Scores scores_of(PyObject* scale, PyObject* window, PyObject* lse, int64_t dim) {
  Scores s{dim > 0 ? 1.0f / std::sqrt(static_cast<float>(dim)) : 1.0f, integer(window, "window"), PyObject_IsTrue(lse) == 1};
  if (scale != Py_None) {
    const double x = PyFloat_AsDouble(scale);
    if (x == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      TORCH_CHECK_TYPE(false, "softmax_scale must be a number");
    }
    s.scale = static_cast<float>(x);
  }
  return s;
}

PyObject* result(const at::Tensor& out, const at::Tensor& lse, PyObject* given) {
  PyObject* o = given != Py_None ? (Py_INCREF(given), given) : wrap(out);
  if (!lse.defined()) return o;
  PyObject* r = PyTuple_New(2);
  if (r) {
    PyTuple_SET_ITEM(r, 0, o);
    PyTuple_SET_ITEM(r, 1, wrap(lse));
  }
  return r;
}

// q, k, v, cu_tokens, softmax_scale, window, out, return_lse, stream
PyObject* attn_prompt(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  ARGS(9);
  const at::Tensor &q0 = tensor(a[0], "q"), &k0 = tensor(a[1], "k"), &v0 = tensor(a[2], "v");
  const fp8_dtype_t dt = dtype_of(q0, "q");
  TORCH_CHECK_VALUE(k0.scalar_type() == q0.scalar_type() && v0.scalar_type() == q0.scalar_type() && v0.sizes() == k0.sizes(),
                    "k and v must be alike and of q's type, got ", k0.scalar_type(), " ", shape_of(k0), " and ", v0.scalar_type(), " ", shape_of(v0));
  const at::Tensor q = rows(q0, "q", 0);
  const int64_t tokens = q.size(0), hq = q.size(1), dim = q.size(2);
  const at::Tensor k = rows(k0, "k", dim), v = rows(v0, "v", dim);
  TORCH_CHECK_VALUE(k.size(0) == tokens, "q has ", tokens, " tokens, k ", k.size(0));
  const at::Tensor cu = vec(tensor(a[3], "cu_tokens"), "cu_tokens", at::kInt, -1);
  TORCH_CHECK_VALUE(cu.size(0) >= 1, "cu_tokens must have batch + 1 entries, got 0");
  const Scores s = scores_of(a[4], a[5], a[7], dim);
  if (a[6] == Py_None) on(q, {{&k, "k"}, {&v, "v"}, {&cu, "cu_tokens"}});
  const at::Tensor out = output(a[6], q, {&q, &k, &v, &cu});
  if (a[6] != Py_None) on(q, {{&k, "k"}, {&v, "v"}, {&cu, "cu_tokens"}, {&out, "out"}});
  const at::Tensor lse = s.lse ? at::empty({tokens, hq}, q.options().dtype(at::kFloat)) : at::Tensor();
  const c10::DeviceGuard guard(q.device());   // the launch goes to the tensors' GPU
  const fp8_status_t code = prompt_fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), dt, tokens, ptr<int32_t>(cu), cu.size(0) - 1, hq, k.size(1),
                                      static_cast<int32_t>(dim), q.stride(0), q.stride(1), k.stride(0), k.stride(1), v.stride(0), v.stride(1), s.scale,
                                      s.window, out.data_ptr(), ptr<float>(lse), stream_of(a[8]));
  return code == FP8_OK ? result(out, lse, a[6]) : status(code);
  END_HANDLE_TH_ERRORS
}

// q, k_cache, v_cache, block_table, seq_lens, cu_tokens, k_scales, v_scales, softmax_scale, window,
// max_new, out, return_lse, workspace, stream
PyObject* attn_paged(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  ARGS(15);
  const at::Tensor& q0 = tensor(a[0], "q");
  const fp8_dtype_t dt = dtype_of(q0, "q");
  const Cache c = cache_of(a[1], a[2], a[6], a[7], q0.scalar_type());
  const int64_t pages = c.k.size(0), hk = c.k.size(1), page = c.k.size(2), dim = c.dim;
  const at::Tensor q = rows(q0, "q", dim);
  const int64_t tokens = q.size(0), hq = q.size(1);
  const at::Tensor lens = vec(tensor(a[4], "seq_lens"), "seq_lens", at::kInt, -1);
  const int64_t batch = lens.size(0);
  const at::Tensor cu = vec(tensor(a[5], "cu_tokens"), "cu_tokens", at::kInt, batch + 1);
  const at::Tensor& tab = table(tensor(a[3], "block_table"), batch);
  const Scores s = scores_of(a[8], a[9], a[12], dim);
  const int64_t most = integer(a[10], "max_new"), width = tab.size(1);
  if (a[11] == Py_None) {
    on(q, {{&tab, "block_table"}, {&lens, "seq_lens"}, {&cu, "cu_tokens"}});
    on_cache(q, c);
  }
  const at::Tensor out = output(a[11], q, {&q, &c.k, &c.v, &c.ks, &c.vs, &tab, &lens, &cu});
  if (a[11] != Py_None) {
    on(q, {{&tab, "block_table"}, {&lens, "seq_lens"}, {&cu, "cu_tokens"}, {&out, "out"}});
    on_cache(q, c);
  }
  const at::Tensor lse = s.lse ? at::empty({tokens, hq}, q.options().dtype(at::kFloat)) : at::Tensor();
  void* stream = stream_of(a[14]);
  at::Tensor ws;
  if (a[13] == Py_None) {
    ws = workspace_of(q, stream, workspace_fn(tokens, batch, hq, hk, static_cast<int32_t>(dim), width, static_cast<int32_t>(page), most));
  } else {
    ws = tensor(a[13], "workspace");
    TORCH_CHECK_TYPE(ws.scalar_type() == at::kByte, "workspace must be uint8, got ", ws.scalar_type());
    TORCH_CHECK_VALUE(ws.dim() == 1 && ws.is_contiguous(), "workspace must be a contiguous vector");
    on(q, {{&ws, "workspace"}});
  }
  const c10::DeviceGuard guard(q.device());   // the launch goes to the tensors' GPU
  const fp8_status_t code = paged_fn(q.data_ptr(), dt, tokens, ptr<int32_t>(cu), batch, hq, hk, static_cast<int32_t>(dim), q.stride(0), q.stride(1), c.format,
                                     c.k.data_ptr(), c.v.data_ptr(), raw(c.ks), raw(c.vs), pages, static_cast<int32_t>(page),
                                     ptr<int32_t>(tab), width, ptr<int32_t>(lens), s.scale, s.window, most, out.data_ptr(), ptr<float>(lse), ws.data_ptr(),
                                     ws.size(0), stream);
  return code == FP8_OK ? result(out, lse, a[11]) : status(code);
  END_HANDLE_TH_ERRORS
}

// A matrix as the kernels read it: dense, from a 16-byte boundary, copied if it is not.
at::Tensor matrix(const at::Tensor& t, const char* what) {
  TORCH_CHECK_VALUE(t.dim() == 2, what, " must be a 2-D tensor, got shape ", shape_of(t));
  at::Tensor c = t.contiguous();
  return reinterpret_cast<uintptr_t>(c.data_ptr()) & 15 ? c.clone() : c;
}
// An output: the caller's (checked later with the devices), or a new one.
at::Tensor output_of(PyObject* given, const char* what, at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
  if (given == Py_None) return at::empty(shape, like.options().dtype(type));
  const at::Tensor& out = tensor(given, what);
  dense(out, what, type, shape);
  return out;
}
PyObject* give(PyObject* given, const at::Tensor& t) { return given != Py_None ? (Py_INCREF(given), given) : wrap(t); }

// x, q, scales, stream
PyObject* quantize8(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  ARGS(4);
  const at::Tensor& x0 = tensor(a[0], "x");
  const fp8_dtype_t dt = dtype_of(x0, "x");
  const at::Tensor x = matrix(x0, "x");
  on(x, {});
  const at::Tensor q = output_of(a[1], "q", x.sizes(), at::kChar, x), scales = output_of(a[2], "scales", {x.size(0)}, at::kFloat, x);
  TORCH_CHECK_VALUE(!overlaps(q, x) && !overlaps(scales, x) && !overlaps(scales, q), "an output overlaps an input or the other output");
  on(x, {{&q, "q"}, {&scales, "scales"}});
  const c10::DeviceGuard guard(x.device());   // the launch goes to the tensors' GPU
  const fp8_status_t code = quantize8_fn(x.data_ptr(), dt, x.size(0), x.size(1), ptr<int8_t>(q), ptr<float>(scales), stream_of(a[3]));
  if (code != FP8_OK) return status(code);
  PyObject* r = PyTuple_New(2);
  if (r) {
    PyTuple_SET_ITEM(r, 0, give(a[1], q));
    PyTuple_SET_ITEM(r, 1, give(a[2], scales));
  }
  return r;
  END_HANDLE_TH_ERRORS
}

// qa, sa, qb, sb, out_dtype is bfloat16, out, stream
PyObject* gemm8(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  ARGS(7);
  const at::Tensor &qa0 = tensor(a[0], "qa"), &qb0 = tensor(a[2], "qb");
  TORCH_CHECK_TYPE(qa0.scalar_type() == at::kChar && qb0.scalar_type() == at::kChar, "operands must be int8, got ", qa0.scalar_type(), " and ", qb0.scalar_type());
  const at::Tensor qa = matrix(qa0, "qa"), qb = matrix(qb0, "qb");
  const int64_t m = qa.size(0), n = qb.size(0), k = qa.size(1);
  TORCH_CHECK_VALUE(qb.size(1) == k, "K mismatch: qa has ", k, ", qb has ", qb.size(1));
  const at::Tensor sa = vec(tensor(a[1], "sa"), "sa", at::kFloat, m), sb = vec(tensor(a[3], "sb"), "sb", at::kFloat, n);
  on(qa, {{&sa, "sa"}, {&qb, "qb"}, {&sb, "sb"}});
  at::Tensor out;
  if (a[5] == Py_None) {
    out = at::empty({m, n}, qa.options().dtype(PyObject_IsTrue(a[4]) == 1 ? at::kBFloat16 : at::kHalf));
  } else {
    out = tensor(a[5], "out");
    dtype_of(out, "out");
    dense(out, "out", out.scalar_type(), {m, n});
    for (const at::Tensor* t : {&qa, &qb, &sa, &sb}) TORCH_CHECK_VALUE(!overlaps(out, *t), "out overlaps an input");
    on(qa, {{&out, "out"}});
  }
  const c10::DeviceGuard guard(qa.device());   // the launch goes to the tensors' GPU
  const fp8_status_t code = gemm8_fn(ptr<int8_t>(qa), ptr<float>(sa), ptr<int8_t>(qb), ptr<float>(sb), m, n, k, out.data_ptr(), dtype_of(out, "out"),
                                     stream_of(a[6]));
  return code == FP8_OK ? give(a[5], out) : status(code);
  END_HANDLE_TH_ERRORS
}

// The addresses of fp8_paged_plan, fp8_kv_append, fp8_rope_append, fp8_attn_prompt, fp8_attn_paged, fp8_attn_paged_workspace,
// int8_quantize_rowwise and int8_gemm_scaled_rowwise.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  ARGS(8);
  plan_fn = reinterpret_cast<decltype(plan_fn)>(PyLong_AsVoidPtr(a[0]));
  append_fn = reinterpret_cast<decltype(append_fn)>(PyLong_AsVoidPtr(a[1]));
  rope_fn = reinterpret_cast<decltype(rope_fn)>(PyLong_AsVoidPtr(a[2]));
  prompt_fn = reinterpret_cast<decltype(prompt_fn)>(PyLong_AsVoidPtr(a[3]));
  paged_fn = reinterpret_cast<decltype(paged_fn)>(PyLong_AsVoidPtr(a[4]));
  workspace_fn = reinterpret_cast<decltype(workspace_fn)>(PyLong_AsVoidPtr(a[5]));
  quantize8_fn = reinterpret_cast<decltype(quantize8_fn)>(PyLong_AsVoidPtr(a[6]));
  gemm8_fn = reinterpret_cast<decltype(gemm8_fn)>(PyLong_AsVoidPtr(a[7]));
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(paged_plan), METHOD(kv_append), METHOD(rope_append), METHOD(attn_prompt), METHOD(attn_paged), METHOD(quantize8), METHOD(gemm8), METHOD(bind), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&module); }
