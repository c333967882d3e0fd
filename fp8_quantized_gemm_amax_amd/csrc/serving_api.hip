// serving_api.hip - the C ABI declared in include/fp8amax_serving.h: host-side validation, then
// kernel launches on the caller's stream.  As in api.hip, validation makes no HIP call.
#include "fp8amax_serving.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "serving.hpp"

namespace {

constexpr int64_t kMaxInt = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxElems = int64_t{1} << 40;
constexpr int64_t kMaxKeys = int64_t{1} << 30;     // of a request: key numbers and their sums stay below 2^31
constexpr int64_t kMaxGroups = (int64_t{1} << 24) - 1;   // workgroups of 256 threads: a launch holds 2^32 - 1

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool valid_dt(fp8_dtype_t dt) { return dt == FP8_BF16 || dt == FP8_F16; }
bool valid_format(fp8_kv_format_t f) { return f == FP8_KV_SAME || f == FP8_KV_E4M3 || f == FP8_KV_MXFP4; }
bool valid_dim(int32_t d) { return d == 64 || d == 128; }
bool valid_page(int32_t p) { return p >= 16 && p <= 1024 && (p & (p - 1)) == 0; }
int shift_of(int32_t p) { return __builtin_ctz(static_cast<unsigned>(p)); }

bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const auto x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a_bytes > 0 && b_bytes > 0 && (x < y ? y - x < static_cast<uint64_t>(a_bytes) : x - y < static_cast<uint64_t>(b_bytes));
}

fp8_status_t finish_launch() { return hipGetLastError() == hipSuccess ? FP8_OK : FP8_ERR_LAUNCH; }

// Token and head strides of a [tokens, heads, dim] tensor: the kernels read 16 bytes at a time.
fp8_status_t check_strides(int64_t tokens, int64_t heads, int64_t ts, int64_t hs) {
  if (ts < 0 || hs < 0) return FP8_ERR_BAD_SHAPE;
  if (ts % 8 != 0 || hs % 8 != 0) return FP8_ERR_MISALIGNED;
  if ((tokens > 0 && ts > kMaxElems / tokens) || hs > kMaxElems / heads) return FP8_ERR_TOO_LARGE;
  return FP8_OK;
}

fp8_status_t check_cache(int64_t pages, int64_t heads, int32_t dim, int32_t page) {
  if (pages < 1 || !valid_page(page)) return FP8_ERR_BAD_SHAPE;
  if (pages > kMaxInt || pages > kMaxElems / (heads * page * dim)) return FP8_ERR_TOO_LARGE;
  return FP8_OK;
}

fp8_status_t check_heads(int64_t tokens, int64_t batch, int64_t hq, int64_t hk, int32_t dim, float scale,
                         int64_t window) {
  if (tokens < 0 || batch < 0 || hq < 1 || hk < 1 || hq % hk != 0 || !valid_dim(dim)) return FP8_ERR_BAD_SHAPE;
  if (!std::isfinite(scale) || scale <= 0.0f || window < 0) return FP8_ERR_BAD_SHAPE;
  if (tokens > kMaxInt || batch > kMaxInt || hq > 65535) return FP8_ERR_TOO_LARGE;
  if (tokens * hq > kMaxInt / 2 || batch * hq > kMaxInt / 2) return FP8_ERR_TOO_LARGE;   // rows and tiles are indexed with int
  return FP8_OK;
}

// The arguments of an append (FP8_OK: `a` is filled, or there are no tokens).
fp8_status_t check_append(const void* k, const void* v, fp8_dtype_t dt, int64_t tokens, int64_t kv_heads, int32_t head_dim,
                          int64_t kts, int64_t khs, int64_t vts, int64_t vhs, const int64_t* slots, int64_t pages,
                          int32_t page_size, fp8_kv_format_t format, void* k_cache, void* v_cache, void* k_scales,
                          void* v_scales, fp8amax::AppendArgs& a) {
  if (tokens < 0 || kv_heads < 1 || !valid_dim(head_dim)) return FP8_ERR_BAD_SHAPE;
  if (tokens > kMaxInt || kv_heads > 65535 || tokens * kv_heads > kMaxInt / 2) return FP8_ERR_TOO_LARGE;
  if (!valid_dt(dt) || !valid_format(format)) return FP8_ERR_BAD_DTYPE;
  fp8_status_t st = check_cache(pages, kv_heads, head_dim, page_size);
  if (st == FP8_OK) st = check_strides(tokens, kv_heads, kts, khs);
  if (st == FP8_OK) st = check_strides(tokens, kv_heads, vts, vhs);
  if (st != FP8_OK) return st;
  if (tokens == 0) return FP8_OK;
  if (fp8amax::kv_append_groups(tokens, kv_heads, head_dim) > kMaxGroups) return FP8_ERR_TOO_LARGE;
  const bool scaled = format != FP8_KV_SAME;
  if (!k || !v || !slots || !k_cache || !v_cache || (scaled && (!k_scales || !v_scales))) return FP8_ERR_NULL_POINTER;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(slots, 8) ||
      (scaled && (!aligned(k_scales, 4) || !aligned(v_scales, 4))))
    return FP8_ERR_MISALIGNED;
  a.k = k; a.v = v; a.kts = kts; a.khs = khs; a.vts = vts; a.vhs = vhs;
  a.tokens = static_cast<int>(tokens); a.heads = static_cast<int>(kv_heads);
  a.slots = slots; a.n_slots = pages * page_size; a.page_shift = shift_of(page_size);
  a.kc = k_cache; a.vc = v_cache; a.ks = k_scales; a.vs = v_scales;
  return FP8_OK;
}

// The caches of keys and values and their scales, which an append writes, stand apart (checked last).  `one`: keys and
// values are the same rows, which may go to one cache.
fp8_status_t check_apart(const fp8amax::AppendArgs& a, int32_t head_dim, fp8_kv_format_t format, bool one) {
  const int64_t rows = a.n_slots * a.heads;
  const int64_t codes = rows * head_dim * (format == FP8_KV_SAME ? 4 : format == FP8_KV_E4M3 ? 2 : 1) / 2;
  const int64_t scales = format == FP8_KV_SAME ? 0 : format == FP8_KV_E4M3 ? rows * 4 : rows * (head_dim / 32);
  const void* const at[4] = {a.kc, a.vc, a.ks, a.vs};
  const bool shared = one && a.kc == a.vc && (scales == 0 || a.ks == a.vs);
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 4; ++j)
      if (!(shared && at[i] == at[j]) && overlap(at[i], i < 2 ? codes : scales, at[j], j < 2 ? codes : scales)) return FP8_ERR_BAD_SHAPE;
  return FP8_OK;
}

// A window that no request can fill is none.
int window_of(int64_t window) { return window >= kMaxKeys ? 0 : static_cast<int>(window); }

}  // namespace

extern "C" {

fp8_status_t fp8_paged_plan(const int32_t* cached, const int32_t* added, int64_t batch, int32_t page_size,
                            int32_t* block_table, int64_t width, const int32_t* free_pages, int64_t n_free,
                            const int32_t* taken_in, int64_t tokens, int32_t* cu_tokens, int32_t* seq_lens,
                            int32_t* positions, int64_t* slots, int32_t* taken_out, int32_t* missing, void* stream) {
  if (batch < 0 || tokens < 0 || n_free < 0 || width < 1 || !valid_page(page_size)) return FP8_ERR_BAD_SHAPE;
  if (batch > fp8amax::kMaxBatch || tokens > kMaxInt - 1024 || n_free > kMaxInt || width > kMaxInt / page_size)
    return FP8_ERR_TOO_LARGE;
  if (!taken_in || !cu_tokens || !taken_out || !missing || (n_free > 0 && !free_pages) ||
      (tokens > 0 && (!positions || !slots)) || (batch > 0 && (!cached || !added || !block_table || !seq_lens)))
    return FP8_ERR_NULL_POINTER;
  if (!aligned(cached, 4) || !aligned(added, 4) || !aligned(block_table, 4) || !aligned(free_pages, 4) ||
      !aligned(taken_in, 4) || !aligned(cu_tokens, 4) || !aligned(seq_lens, 4) || !aligned(positions, 4) ||
      !aligned(slots, 8) || !aligned(taken_out, 4) || !aligned(missing, 4))
    return FP8_ERR_MISALIGNED;
  // What one workgroup writes others still read: outputs, the table among them, stand apart.
  struct Range {
    const void* p;
    int64_t bytes;
  };
  const Range ranges[] = {{block_table, batch * width * 4}, {cu_tokens, batch * 4 + 4}, {seq_lens, batch * 4}, {positions, tokens * 4},
                          {slots, tokens * 8}, {taken_out, 4}, {missing, 4},   // outputs; then inputs
                          {cached, batch * 4}, {added, batch * 4}, {free_pages, n_free * 4}, {taken_in, 4}};
  for (int i = 0; i < 7; ++i)
    for (int j = i + 1; j < 11; ++j)
      if (overlap(ranges[i].p, ranges[i].bytes, ranges[j].p, ranges[j].bytes)) return FP8_ERR_BAD_SHAPE;
  fp8amax::PlanArgs a{};
  a.cached = cached; a.added = added; a.batch = static_cast<int>(batch); a.page_shift = shift_of(page_size);
  a.table = block_table; a.width = static_cast<int>(width);
  a.free_pages = free_pages; a.n_free = static_cast<int>(n_free); a.taken_in = taken_in;
  a.tokens = static_cast<int>(tokens);
  a.cu = cu_tokens; a.lens = seq_lens; a.positions = positions; a.slots = slots;
  a.taken_out = taken_out; a.missing = missing;
  (void)hipGetLastError();
  fp8amax::launch_paged_plan(a, static_cast<hipStream_t>(stream));
  return finish_launch();
}

fp8_status_t fp8_kv_append(const void* k, const void* v, fp8_dtype_t dt, int64_t tokens, int64_t kv_heads,
                           int32_t head_dim, int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                           int64_t v_head_stride, const int64_t* slots, int64_t pages, int32_t page_size,
                           fp8_kv_format_t format, void* k_cache, void* v_cache, void* k_scales, void* v_scales,
                           void* stream) {
  fp8amax::AppendArgs a{};
  fp8_status_t st = check_append(k, v, dt, tokens, kv_heads, head_dim, k_token_stride, k_head_stride, v_token_stride,
                                 v_head_stride, slots, pages, page_size, format, k_cache, v_cache, k_scales, v_scales, a);
  if (st != FP8_OK || tokens == 0) return st;
  const bool one = k == v && k_token_stride == v_token_stride && k_head_stride == v_head_stride;
  if ((st = check_apart(a, head_dim, format, one)) != FP8_OK) return st;
  (void)hipGetLastError();
  fp8amax::launch_kv_append(static_cast<int>(dt), head_dim, format, a, static_cast<hipStream_t>(stream));
  return finish_launch();
}

fp8_status_t fp8_rope_append(const void* q, const void* k, const void* v, fp8_dtype_t dt, int64_t tokens,
                             int64_t q_heads, int64_t kv_heads, int32_t head_dim, int64_t q_token_stride,
                             int64_t q_head_stride, int64_t k_token_stride, int64_t k_head_stride,
                             int64_t v_token_stride, int64_t v_head_stride, const int32_t* positions,
                             const float* cos_sin, int64_t n_positions, int32_t rotary_dim, int32_t interleaved,
                             const int64_t* slots, int64_t pages, int32_t page_size, fp8_kv_format_t format,
                             void* k_cache, void* v_cache, void* k_scales, void* v_scales, void* q_out,
                             void* stream) {
  if (q_heads < 0 || n_positions < 0 || !valid_dim(head_dim) || rotary_dim < 16 || rotary_dim > head_dim || rotary_dim % 16 != 0)
    return FP8_ERR_BAD_SHAPE;
  if (n_positions > kMaxInt || q_heads > 65535) return FP8_ERR_TOO_LARGE;
  fp8amax::RopeArgs a{};
  fp8_status_t st = check_append(k, v, dt, tokens, kv_heads, head_dim, k_token_stride, k_head_stride, v_token_stride,
                                 v_head_stride, slots, pages, page_size, format, k_cache, v_cache, k_scales, v_scales, a.kv);
  if (st != FP8_OK) return st;
  if (q_heads > 0 && (st = check_strides(tokens, q_heads, q_token_stride, q_head_stride)) != FP8_OK) return st;
  if (tokens * q_heads > kMaxInt / 2) return FP8_ERR_TOO_LARGE;
  if (tokens == 0) return FP8_OK;
  if (fp8amax::rope_append_groups(tokens, q_heads, kv_heads, head_dim) > kMaxGroups) return FP8_ERR_TOO_LARGE;
  if (!positions || (n_positions > 0 && !cos_sin) || (q_heads > 0 && (!q || !q_out))) return FP8_ERR_NULL_POINTER;
  if (!aligned(positions, 4) || !aligned(cos_sin, 16) || (q_heads > 0 && (!aligned(q, 16) || !aligned(q_out, 16))))
    return FP8_ERR_MISALIGNED;
  if ((st = check_apart(a.kv, head_dim, format, false)) != FP8_OK) return st;
  a.q = q; a.q_out = q_out; a.qts = q_token_stride; a.qhs = q_head_stride; a.q_heads = static_cast<int>(q_heads);
  a.positions = positions; a.cos_sin = cos_sin; a.n_positions = static_cast<int>(n_positions); a.rotary = rotary_dim;
  (void)hipGetLastError();
  fp8amax::launch_rope_append(static_cast<int>(dt), head_dim, format, interleaved != 0, a, static_cast<hipStream_t>(stream));
  return finish_launch();
}

fp8_status_t fp8_attn_prompt(const void* q, const void* k, const void* v, fp8_dtype_t dt, int64_t tokens,
                             const int32_t* cu_tokens, int64_t batch, int64_t q_heads, int64_t kv_heads,
                             int32_t head_dim, int64_t q_token_stride, int64_t q_head_stride,
                             int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                             int64_t v_head_stride, float softmax_scale, int64_t window, void* out, float* lse,
                             void* stream) {
  fp8_status_t st = check_heads(tokens, batch, q_heads, kv_heads, head_dim, softmax_scale, window);
  if (st != FP8_OK) return st;
  if (!valid_dt(dt)) return FP8_ERR_BAD_DTYPE;
  if ((st = check_strides(tokens, q_heads, q_token_stride, q_head_stride)) != FP8_OK) return st;
  if ((st = check_strides(tokens, kv_heads, k_token_stride, k_head_stride)) != FP8_OK) return st;
  if ((st = check_strides(tokens, kv_heads, v_token_stride, v_head_stride)) != FP8_OK) return st;
  if (tokens > 1 && (k_token_stride < head_dim || v_token_stride < head_dim)) return FP8_ERR_BAD_SHAPE;
  if (k_token_stride > (int64_t{1} << 20) || v_token_stride > (int64_t{1} << 20)) return FP8_ERR_TOO_LARGE;
  if (tokens == 0 || batch == 0) return FP8_OK;
  if (fp8amax::attn_prompt_groups(tokens, batch, q_heads, kv_heads) > kMaxGroups) return FP8_ERR_TOO_LARGE;
  if (!q || !k || !v || !cu_tokens || !out) return FP8_ERR_NULL_POINTER;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(cu_tokens, 4) ||
      !aligned(lse, 4))
    return FP8_ERR_MISALIGNED;
  fp8amax::AttnArgs a{};
  a.q = q; a.k = k; a.v = v; a.cu = cu_tokens; a.out = out; a.lse = lse;
  a.qts = q_token_stride; a.qhs = q_head_stride; a.kts = k_token_stride; a.khs = k_head_stride;
  a.vts = v_token_stride; a.vhs = v_head_stride;
  a.tokens = static_cast<int>(tokens); a.batch = static_cast<int>(batch);
  a.hq = static_cast<int>(q_heads); a.hk = static_cast<int>(kv_heads); a.group = a.hq / a.hk;
  a.window = window_of(window); a.scale = softmax_scale;
  (void)hipGetLastError();
  fp8amax::launch_attn_prompt(static_cast<int>(dt), head_dim, a, static_cast<hipStream_t>(stream));
  return finish_launch();
}

int64_t fp8_attn_paged_workspace(int64_t tokens, int64_t batch, int64_t q_heads, int64_t kv_heads, int32_t head_dim,
                                 int64_t width, int32_t page_size, int64_t max_new) {
  if (check_heads(tokens, batch, q_heads, kv_heads, head_dim, 1.0f, 0) != FP8_OK || !valid_page(page_size) ||
      width < 1 || width > kMaxKeys / page_size || max_new < 0)
    return 0;
  return fp8amax::attn_paged_workspace(FP8_KV_MXFP4, tokens, batch, q_heads, kv_heads, head_dim, width * page_size, max_new);
}

fp8_status_t fp8_attn_paged(const void* q, fp8_dtype_t dt, int64_t tokens, const int32_t* cu_tokens, int64_t batch,
                            int64_t q_heads, int64_t kv_heads, int32_t head_dim, int64_t q_token_stride,
                            int64_t q_head_stride, fp8_kv_format_t format, const void* k_cache, const void* v_cache,
                            const void* k_scales, const void* v_scales, int64_t pages, int32_t page_size,
                            const int32_t* block_table, int64_t width, const int32_t* seq_lens, float softmax_scale,
                            int64_t window, int64_t max_new, void* out, float* lse, void* workspace,
                            int64_t workspace_bytes, void* stream) {
  fp8_status_t st = check_heads(tokens, batch, q_heads, kv_heads, head_dim, softmax_scale, window);
  if (st != FP8_OK) return st;
  if (max_new < 0 || width < 1) return FP8_ERR_BAD_SHAPE;
  if (!valid_dt(dt) || !valid_format(format)) return FP8_ERR_BAD_DTYPE;
  if ((st = check_cache(pages, kv_heads, head_dim, page_size)) != FP8_OK) return st;
  if (width > kMaxKeys / page_size || (batch > 0 && width > kMaxElems / batch)) return FP8_ERR_TOO_LARGE;
  if ((st = check_strides(tokens, q_heads, q_token_stride, q_head_stride)) != FP8_OK) return st;
  if (tokens == 0 || batch == 0) return FP8_OK;
  const bool scaled = format != FP8_KV_SAME;
  if (fp8amax::attn_paged_groups(format, tokens, batch, q_heads, kv_heads, width * page_size, max_new) > kMaxGroups)
    return FP8_ERR_TOO_LARGE;
  const int64_t need = fp8amax::attn_paged_workspace(format, tokens, batch, q_heads, kv_heads, head_dim, width * page_size, max_new);
  if (workspace_bytes < need) return FP8_ERR_BAD_SHAPE;
  if (!q || !cu_tokens || !k_cache || !v_cache || !block_table || !seq_lens || !out || (need > 0 && !workspace) ||
      (scaled && (!k_scales || !v_scales)))
    return FP8_ERR_NULL_POINTER;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(workspace, 16) || !aligned(cu_tokens, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(lse, 4) || (scaled && (!aligned(k_scales, 4) || !aligned(v_scales, 4))))
    return FP8_ERR_MISALIGNED;
  fp8amax::AttnArgs a{};
  a.q = q; a.k = k_cache; a.v = v_cache; a.ks = k_scales; a.vs = v_scales;
  a.cu = cu_tokens; a.table = block_table; a.lens = seq_lens; a.out = out; a.lse = lse;
  a.ws = static_cast<char*>(workspace);
  a.qts = q_token_stride; a.qhs = q_head_stride;
  a.tokens = static_cast<int>(tokens); a.batch = static_cast<int>(batch);
  a.hq = static_cast<int>(q_heads); a.hk = static_cast<int>(kv_heads); a.group = a.hq / a.hk;
  a.pages = static_cast<int>(pages); a.page_shift = shift_of(page_size); a.width = static_cast<int>(width);
  a.window = window_of(window); a.scale = softmax_scale;
  (void)hipGetLastError();
  fp8amax::launch_attn_paged(static_cast<int>(dt), head_dim, format, static_cast<int>(max_new > tokens ? tokens : max_new), a,
                             static_cast<hipStream_t>(stream));
  return finish_launch();
}

}  // extern "C"
