// attention.hip - attention over a paged cache: the choice of kernel, the workspace, and the join of the
// partial results for many rows.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "attn_device.hpp"

namespace fp8amax {
namespace attn {
namespace {

// Whether a batch goes to the kernel for few rows: where its requests have at most 32 rows a key head on
// average (64 over an e4m3 cache and 48 over an mxfp4 one, which the kernel for many rows has to widen on
// the way), and none, as far as max_new says, has more than 512, since that one's keys are read once for
// every 32 rows (16 over mxfp4).
// Kernel for many rows against the one for few, us on one card, 128 channels, requests of equal rows over
// half to all of so many keys:
//   16 bits, rows      4            16           32           40
//     24 x 500   17.1 : 13.0  17.4 : 13.3  17.8 : 13.7  17.9 : 27.9
//      8 x 2000  22.3 : 21.3  21.3 : 23.5  21.1 : 28.9  21.7 : 36.0
//     64 x 4000   155 : 152    153 : 164    154 : 172    156 : 300
//     1 x 100000   97 :  79     96 : 110     92 : 123     95 : 146
//   e4m3, rows         4            32           64           80
//     24 x 500   22.3 : 12.6  23.1 : 13.5  23.6 : 17.7  23.9 : 31.3
//      8 x 2000  27.0 : 16.0  26.8 : 22.8  28.1 : 30.0  30.4 : 31.5
//     64 x 4000   157 :  87    159 : 102    162 : 175    163 : 233
//     1 x 100000  108 :  50    103 :  90    105 :  97    113 : 113
//   mxfp4, rows        4            32           48           64           80
//     24 x 500   19.1 : 10.7  19.2 : 12.1  19.6 : 21.4  19.7 : 22.4  20.2 : 21.7
//      8 x 2000  23.7 : 13.3  22.5 : 18.0  23.9 : 23.7  24.0 : 22.1  27.4 : 28.3
//     64 x 4000   141 :  52    146 :  93    146 : 135    151 : 172    151 : 212
//     1 x 100000   93 :  33     87 :  56     89 :  66     89 :  80     98 :  91
// No number of rows suits every length: at the limits the kernel for few is up to 23% faster over short
// caches and up to 37% slower over long ones in 16 bits (above 12 rows), 25% faster to 8% slower over e4m3,
// 25% faster to 9% slower over mxfp4.
// Nor is the limit of 512 rows right for every length: over mxfp4 such a request reads its keys 32 times.  One of
// 512 rows among 63 (15) single tokens over 2000 to 4000 keys each, many : few: over 1000 keys 125 : 55 (57 : 27),
// over 4000 133 : 64 (63 : 40), over 16000 176 : 119 (111 : 100), over 100000 346 : 549 (260 : 511).
bool few_rows(int format, int64_t max_new, int64_t group, int64_t tokens, int64_t batch) {
  return std::min(max_new, tokens) * group <= 512 && tokens * group <= (format == FP8_KV_SAME ? 32 : format == FP8_KV_E4M3 ? 64 : 48) * batch;
}

// Joins the partial results of the launch for many rows, of 128 rows each: a thread takes one row and
// every eighth (fourth) group of four channels of it, and goes over the row's pieces once:
//   out = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i.
// Workgroup (x, y): the tile whose first partial result is x, quarter y of its channels, four pieces'
// reads in flight.  Bound by the latency of those and its launch: 5 us for 24 mixed requests, 15 us
// for 34 MB of partial results.
constexpr int kQuarters = 4;
template <int DT, int D>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  constexpr int kSize = 128, kEach = D / 4 * kSize / 256 / kQuarters;
  const Workspace ws = workspace(a, kSize);
  const int slot = blockIdx.x;
  if (slot >= *ws.used) return;
  const Partial p = ws.partials[slot];
  if (p.count <= 1) return;
  const Rows r = rows_of(a, p.request, load_request<true>(a, p.request), p.tile, kSize);
  const int row = threadIdx.x & 127, quad0 = blockIdx.y * (D / 4 / kQuarters) + (threadIdx.x >> 7);
  if (r.row0 + row >= r.rows) return;
  const int64_t stride = static_cast<int64_t>(a.hk) * kSize;
  const float* stats = ws.stats + (static_cast<int64_t>(slot) * kSize + row) * 2;
  const float* out = ws.out + static_cast<int64_t>(slot) * kSize * D;
  float m = -INFINITY, l = 0.0f, o[kEach][4] = {};
  for (int i0 = 0; i0 < p.count; i0 += 4) {
    float2 st[4];
    v4f x[4][kEach];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t i = min(i0 + k, p.count - 1);
      st[k] = *reinterpret_cast<const float2*>(stats + i * stride * 2);
      if (i0 + k >= p.count) st[k] = make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int e = 0; e < kEach; ++e) x[k][e] = *reinterpret_cast<const v4f*>(out + i * stride * D + partial_at<D>(row, quad0 + 2 * e));
    }
    const float top = fmaxf(fmaxf(fmaxf(m, st[0].x), fmaxf(st[1].x, st[2].x)), st[3].x);
    const float base = top == -INFINITY ? 0.0f : top, keep = __builtin_amdgcn_exp2f(m - base);
    m = top;
    l *= keep;
#pragma unroll
    for (int e = 0; e < kEach; ++e)
#pragma unroll
      for (int y = 0; y < 4; ++y) o[e][y] *= keep;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (i0 + k >= p.count) break;
      const float f = __builtin_amdgcn_exp2f(st[k].x - base);
      l = __builtin_fmaf(f, st[k].y, l);
#pragma unroll
      for (int e = 0; e < kEach; ++e)
#pragma unroll
        for (int y = 0; y < 4; ++y) o[e][y] = __builtin_fmaf(f, x[k][e][y], o[e][y]);
    }
  }
  const int tok = (r.row0 + row) / a.group;
  const bool none = r.pos0 + tok < 0;
  const float inv = none ? 0.0f : 1.0f / l;
  const int64_t out_row = static_cast<int64_t>(r.begin + tok) * a.hq + p.head * a.group + (r.row0 + row - tok * a.group);
#pragma unroll
  for (int e = 0; e < kEach; ++e)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + out_row * D + 4 * (quad0 + 2 * e)) =
        make_uint2(pack2<DT>(o[e][0] * inv, o[e][1] * inv), pack2<DT>(o[e][2] * inv, o[e][3] * inv));
  if (a.lse && quad0 == 0) a.lse[out_row] = none ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

template <int DT, int D>
void join(const AttnArgs& a, hipStream_t s) {
  attn_join_kernel<DT, D><<<dim3(static_cast<unsigned>(2 * extra_units(a.hk) * a.hk), kQuarters), 256, 0, s>>>(a);
}

}  // namespace

void launch_attn_join(int dt, int head_dim, const AttnArgs& a, hipStream_t s) {
  if (dt == DT_BF16) head_dim == 128 ? join<DT_BF16, 128>(a, s) : join<DT_BF16, 64>(a, s);
  else head_dim == 128 ? join<DT_F16, 128>(a, s) : join<DT_F16, 64>(a, s);
}

}  // namespace attn

void launch_attn_paged(int dt, int head_dim, int format, int max_new, const AttnArgs& a, hipStream_t s) {
  if (!attn::few_rows(format, max_new, a.group, a.tokens, a.batch)) attn::launch_attn_tile(dt, head_dim, format, a, s);
  else if (format == FP8_KV_MXFP4) attn::launch_attn_mx4_few(dt, head_dim, a, s);
  else attn::launch_attn_few(dt, head_dim, format == FP8_KV_E4M3, a, s);
}

int64_t attn_prompt_groups(int64_t tokens, int64_t batch, int64_t hq, int64_t hk) {
  return attn::tile_groups(tokens, batch, hq / hk, hk, false);
}

int64_t attn_paged_groups(int format, int64_t tokens, int64_t batch, int64_t hq, int64_t hk, int64_t capacity, int64_t max_new) {
  using namespace attn;
  const int64_t group = hq / hk;
  const bool split = may_split(tokens, group, batch, hk, capacity);
  if (!few_rows(format, max_new, group, tokens, batch)) return tile_groups(tokens, batch, group, hk, split);
  return format == FP8_KV_MXFP4 ? mx4_groups(tokens, batch, group, hk, capacity, split) : few_groups(tokens, batch, group, hk, capacity, split);
}

int64_t attn_paged_workspace(int format, int64_t tokens, int64_t batch, int64_t hq, int64_t hk, int head_dim, int64_t capacity,
                             int64_t max_new) {
  using namespace attn;
  if (!may_split(tokens, hq / hk, batch, hk, capacity)) return 0;
  // Few rows over mxfp4: a key head has a workgroup at least, each with two partial results.
  const int64_t groups = format == FP8_KV_MXFP4 ? std::max<int64_t>(kFewGroups, hk) : kFewGroups;
  auto bytes = [&](bool few) { return workspace_bytes(few ? 2 * groups : 2 * extra_units(hk) * hk, few ? 32 : 128, head_dim); };
  // Whichever kernel a format's rule chooses; FP8_KV_MXFP4 has the most, which is enough for every format.
  int64_t most = 0;
  for (int format : {FP8_KV_SAME, FP8_KV_E4M3, FP8_KV_MXFP4}) most = std::max(most, bytes(few_rows(format, max_new, hq / hk, tokens, batch)));
  return most;
}

}  // namespace fp8amax
