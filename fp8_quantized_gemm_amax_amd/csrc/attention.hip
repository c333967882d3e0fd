// attention.hip - causal attention with grouped heads over packed prompts and over the pages of
// a key/value cache, gfx950.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8_device.hpp"
#include "serving.hpp"

namespace fp8amax {
namespace {

// The request of packed token t (uniform): the last r with cu[r] <= t; its clamped bounds.
__device__ __forceinline__ int request_of(const AttnArgs& a, int t, int& begin, int& end) {
  int lo = 0, hi = a.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.cu[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  begin = min(max(a.cu[lo], 0), a.tokens);
  end = min(max(a.cu[lo + 1], 0), a.tokens);
  return lo;
}

template <int DT>
__device__ __forceinline__ uint16_t from_f32(float x) {
  if constexpr (DT == DT_BF16) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
  else return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
}

// One wave per token and query head: a key per lane for the scores, a pair of output channels
// per lane for the product with v, 64 keys a round with a running maximum and sum.
template <int DT, int D, bool PAGED, bool E4M3>
__global__ __launch_bounds__(256) void attn_rows_kernel(AttnArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (id >= static_cast<int64_t>(a.tokens) * a.hq) return;
  const int t = static_cast<int>(id / a.hq), h = static_cast<int>(id % a.hq), kh = h / a.group;
  int begin, end;
  const int r = request_of(a, t, begin, end);
  if (t < begin || t >= end) return;
  const int len = PAGED ? min(max(a.lens[r], 0), a.width << a.page_shift) : end - begin;
  const int pos = len - (end - begin) + (t - begin);   // may be negative: no keys
  const int first = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + t * a.qts + h * a.qhs;
  const int mask = (1 << a.page_shift) - 1;
  // Row of key j: its page and offset, or -1 where the table names no page.
  auto row_of = [&](int j) -> int64_t {
    const int page = a.table[static_cast<int64_t>(r) * a.width + (j >> a.page_shift)];
    if (page < 0 || page >= a.pages) return -1;
    return (((static_cast<int64_t>(page) * a.hk + kh) << a.page_shift) + (j & mask));
  };
  auto value = [&](const void* base, int64_t row, int64_t ts, int64_t hs, int j, int d) -> float {
    if constexpr (!PAGED) return in_to_f32<DT>(static_cast<const uint16_t*>(base)[(begin + j) * ts + kh * hs + d]);
    else if constexpr (E4M3) return __builtin_amdgcn_cvt_f32_fp8(static_cast<const uint8_t*>(base)[row * D + d], 0);
    else return in_to_f32<DT>(static_cast<const uint16_t*>(base)[row * D + d]);
  };
  float m = -INFINITY, l = 0.0f, o[D / 64] = {};
  for (int j0 = first & ~63; j0 <= pos; j0 += 64) {
    const int j = j0 + lane;
    const bool seen = j >= first && j <= pos;
    int64_t row = 0;
    float x = -INFINITY;
    float vscale = 1.0f;
    if constexpr (PAGED) row = seen ? row_of(j) : -1;
    if (seen) {
      float dot = 0.0f;
      if (row >= 0) {
        for (int d = 0; d < D; ++d) dot = __builtin_fmaf(in_to_f32<DT>(q[d]), value(a.k, row, a.kts, a.khs, j, d), dot);
        if constexpr (E4M3) {
          dot *= a.ks[row];
          vscale = a.vs[row];
        }
      }
      x = dot * a.scale;
    }
    float top = x;
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    const float m1 = fmaxf(m, top), base = m1 == -INFINITY ? 0.0f : m1;
    const float p = seen ? __expf(x - base) : 0.0f, keep = __expf(m - base);
    l = l * keep + wave_sum(p);
    m = m1;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) o[c] *= keep;
    const int n = min(64, pos + 1 - j0);
    for (int k = max(0, first - j0); k < n; ++k) {
      const float w = __shfl(p, k) * (E4M3 ? __shfl(vscale, k) : 1.0f);
      int64_t vrow = 0;
      if constexpr (PAGED) vrow = __shfl(row, k);
      if (vrow >= 0) {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) o[c] = __builtin_fmaf(w, value(a.v, vrow, a.vts, a.vhs, j0 + k, c * 64 + lane), o[c]);
      }
    }
  }
  uint16_t* out = static_cast<uint16_t*>(a.out) + (static_cast<int64_t>(t) * a.hq + h) * D;
#pragma unroll
  for (int c = 0; c < D / 64; ++c) out[c * 64 + lane] = from_f32<DT>(pos < 0 ? 0.0f : o[c] / l);
  if (a.lse && lane == 0) a.lse[static_cast<int64_t>(t) * a.hq + h] = pos < 0 ? -INFINITY : m + __logf(l);
}

template <int DT, int D, bool PAGED, bool E4M3>
void rows(const AttnArgs& a, hipStream_t s) {
  const int64_t n = static_cast<int64_t>(a.tokens) * a.hq;
  attn_rows_kernel<DT, D, PAGED, E4M3><<<static_cast<unsigned>((n + 3) / 4), 256, 0, s>>>(a);
}

template <int DT, int D>
void paged(bool e4m3, const AttnArgs& a, hipStream_t s) {
  e4m3 ? rows<DT, D, true, true>(a, s) : rows<DT, D, true, false>(a, s);
}

}  // namespace

void launch_attn_prompt(int dt, int head_dim, const AttnArgs& a, hipStream_t s) {
  if (dt == DT_BF16) head_dim == 128 ? rows<DT_BF16, 128, false, false>(a, s) : rows<DT_BF16, 64, false, false>(a, s);
  else head_dim == 128 ? rows<DT_F16, 128, false, false>(a, s) : rows<DT_F16, 64, false, false>(a, s);
}

void launch_attn_paged(int dt, int head_dim, bool e4m3, int max_new, const AttnArgs& a, hipStream_t s) {
  if (dt == DT_BF16) head_dim == 128 ? paged<DT_BF16, 128>(e4m3, a, s) : paged<DT_BF16, 64>(e4m3, a, s);
  else head_dim == 128 ? paged<DT_F16, 128>(e4m3, a, s) : paged<DT_F16, 64>(e4m3, a, s);
}

int64_t attn_paged_workspace(int64_t, int64_t, int64_t, int64_t, int, int64_t, int64_t) { return 0; }

}  // namespace fp8amax
