// attention.hip - attention over a paged cache: the choice of kernel, the workspace, and the join
// of partial results where the keys of a tile of rows were cut.
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

// One wave per row and a workgroup per four rows of a tile: out = sum_i 2^(m_i - m) o_i / sum_i
// 2^(m_i - m) l_i over the tile's partial results, in their order.
template <int DT, int D>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, int size) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = blockIdx.x % a.hk, j = blockIdx.x / a.hk;
  Rows r;
  if (!find_rows(a, j, size, true, r)) return;
  const Workspace ws = workspace(a, size);
  const int2 info = ws.info[static_cast<int64_t>(j) * a.hk + h];
  const int slots = static_cast<int>(slot_bound(a.hk));
  const int count = __builtin_amdgcn_readfirstlane(info.y), slot = __builtin_amdgcn_readfirstlane(info.x);
  if (count <= 1 || slot < 0 || slot + static_cast<int64_t>(count - 1) * a.hk >= slots) return;
  const int local = blockIdx.y * 4 + wave, row = r.row0 + local;
  if (row >= r.rows) return;
  const int tok = row / a.group;
  const int64_t out_row = static_cast<int64_t>(r.begin + tok) * a.hq + h * a.group + (row - tok * a.group);
  float m = -INFINITY;
  for (int i = lane; i < count; i += 64) m = fmaxf(m, ws.stats[((slot + static_cast<int64_t>(i) * a.hk) * size + local) * 2]);
  for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
  const float mb = m == -INFINITY ? 0.0f : m;
  float l = 0.0f, o[D / 64] = {};
  for (int i = 0; i < count; ++i) {
    const int64_t at = (slot + static_cast<int64_t>(i) * a.hk) * size + local;
    const float2 st = *reinterpret_cast<const float2*>(ws.stats + at * 2);
    const float w = __builtin_amdgcn_exp2f(st.x - mb);
    l = __builtin_fmaf(w, st.y, l);
#pragma unroll
    for (int c = 0; c < D / 64; ++c) o[c] = __builtin_fmaf(w, ws.out[at * D + 64 * c + lane], o[c]);
  }
  const bool none = r.pos0 + tok < 0;
  uint16_t* out = static_cast<uint16_t*>(a.out) + out_row * D;
#pragma unroll
  for (int c = 0; c < D / 64; ++c) out[64 * c + lane] = static_cast<uint16_t>(pack2<DT>(none ? 0.0f : o[c] / l, 0.0f));
  if (a.lse && lane == 0) a.lse[out_row] = none ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

template <int DT, int D>
void join(int size, const AttnArgs& a, hipStream_t s) {
  const int64_t tiles = tile_bound(a.tokens, a.group, a.batch, size);
  attn_join_kernel<DT, D><<<dim3(static_cast<unsigned>(tiles * a.hk), size / 4), 256, 0, s>>>(a, size);
}

}  // namespace

void launch_attn_join(int dt, int head_dim, int size, const AttnArgs& a, hipStream_t s) {
  if (dt == DT_BF16) head_dim == 128 ? join<DT_BF16, 128>(size, a, s) : join<DT_BF16, 64>(size, a, s);
  else head_dim == 128 ? join<DT_F16, 128>(size, a, s) : join<DT_F16, 64>(size, a, s);
}

}  // namespace attn

void launch_attn_paged(int dt, int head_dim, bool e4m3, int max_new, const AttnArgs& a, hipStream_t s) {
  if (attn::few_rows(max_new, a.group, a.tokens, a.batch)) attn::launch_attn_few(dt, head_dim, e4m3, a, s);
  else attn::launch_attn_tile(dt, head_dim, e4m3, a, s);
}

int64_t attn_paged_workspace(int64_t tokens, int64_t batch, int64_t hq, int64_t hk, int head_dim, int64_t capacity,
                             int64_t max_new) {
  using namespace attn;
  if (!may_split(batch, capacity)) return 0;
  const int size = few_rows(max_new, hq / hk, tokens, batch) ? 32 : 128;
  return info_bytes(tile_bound(tokens, hq / hk, batch, size), hk) + slot_bound(hk) * size * (head_dim + 2) * 4;
}

}  // namespace fp8amax
