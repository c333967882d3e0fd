// attention.hip - the choice of kernel for attention over a paged cache, and its workspace.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn_device.hpp"

namespace fp8amax {
namespace attn {
namespace {

// Whether a batch goes to the kernel for few rows: where every request has at most 32 rows a key
// head.  Without max_new, by the average.
bool few_rows(int64_t max_new, int64_t group, int64_t tokens, int64_t batch) {
  return (max_new > 0 ? max_new : (tokens + batch - 1) / (batch > 0 ? batch : 1)) * group <= 32;
}

}  // namespace
}  // namespace attn

void launch_attn_paged(int dt, int head_dim, bool e4m3, int max_new, const AttnArgs& a, hipStream_t s) {
  if (attn::few_rows(max_new, a.group, a.tokens, a.batch)) attn::launch_attn_few(dt, head_dim, e4m3, a, s);
  else attn::launch_attn_tile(dt, head_dim, e4m3, a, s);
}

int64_t attn_paged_workspace(int64_t tokens, int64_t batch, int64_t hq, int64_t hk, int head_dim, int64_t capacity,
                             int64_t max_new) {
  using namespace attn;
  if (!may_split(tokens, hq / hk, batch, hk, capacity)) return 0;
  const bool few = few_rows(max_new, hq / hk, tokens, batch);
  return workspace_bytes(few ? 2 * kFewGroups : 2 * extra_units(hk) * hk, few ? 32 : 128, head_dim);
}

}  // namespace fp8amax
