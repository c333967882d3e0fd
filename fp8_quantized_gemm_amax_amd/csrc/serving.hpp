// serving.hpp - host-side launchers of the serving operators (internal; arguments already
// validated), and the arguments their kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8amax_serving.h"

namespace fp8amax {

constexpr int64_t kMaxBatch = 16384;   // the plan holds two prefix sums of the batch in LDS

struct PlanArgs {
  const int *cached, *added;
  int batch, page_shift;
  int* table;
  int width;
  const int* free_pages;
  int n_free;
  const int* taken_in;
  int tokens;
  int *cu, *lens, *positions;
  int64_t* slots;
  int *taken_out, *missing;
};
void launch_paged_plan(const PlanArgs& a, hipStream_t s);

struct AppendArgs {
  const void *k, *v;
  int64_t kts, khs, vts, vhs;   // token and head strides, in elements
  int tokens, heads;
  const int64_t* slots;
  int64_t n_slots;
  int page_shift;
  void *kc, *vc;
  float *ks, *vs;
};
int64_t kv_append_groups(int64_t tokens, int64_t heads, int head_dim);   // workgroups of the launch
void launch_kv_append(int dt, int head_dim, bool e4m3, const AppendArgs& a, hipStream_t s);

// Attention over packed prompts (table == nullptr: k and v strided tensors of the same tokens)
// or over a paged cache.
struct AttnArgs {
  const void *q, *k, *v;
  const float *ks, *vs;         // e4m3 caches only
  const int *cu, *table, *lens; // table, lens: paged only
  void* out;
  float* lse;                   // may be null
  char* ws;                     // paged only
  int64_t qts, qhs, kts, khs, vts, vhs;
  int tokens, batch, hq, hk, group;
  int pages, page_shift, width;
  int window;                   // 0: none
  float scale;
};
void launch_attn_prompt(int dt, int head_dim, const AttnArgs& a, hipStream_t s);
void launch_attn_paged(int dt, int head_dim, bool e4m3, int max_new, const AttnArgs& a, hipStream_t s);
int64_t attn_prompt_groups(int64_t tokens, int64_t batch, int64_t hq, int64_t hk);   // workgroups of the launch
int64_t attn_paged_groups(bool e4m3, int64_t tokens, int64_t batch, int64_t hq, int64_t hk, int64_t capacity, int64_t max_new);
int64_t attn_paged_workspace(int64_t tokens, int64_t batch, int64_t hq, int64_t hk, int head_dim, int64_t capacity,
                             int64_t max_new);

}  // namespace fp8amax
