// paged.hip - the paged key/value cache: a step's block tables, slots and positions, and the
// write of new keys and values into their pages.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "quant_device.hpp"
#include "serving.hpp"

namespace fp8amax {
namespace {

constexpr int kPlanThreads = 256;

// Inclusive sums over the workgroup of two non-negative values per thread; `total` gets the
// last thread's.  `part` holds one pair per wave.
__device__ __forceinline__ void scan2(int64_t& a, int64_t& b, int64_t (*part)[2], int64_t total[2]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t x = __shfl_up(a, d), y = __shfl_up(b, d);
    if (lane >= d) { a += x; b += y; }
  }
  if (lane == 63) { part[wave][0] = a; part[wave][1] = b; }
  __syncthreads();
  total[0] = total[1] = 0;
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    if (w == wave) { a += total[0]; b += total[1]; }
    total[0] += part[w][0];
    total[1] += part[w][1];
  }
  __syncthreads();   // part is written again by the next round
}

// The first i with sums[i] > x, for inclusive sums of n > 0 entries and x < sums[n - 1].
__device__ __forceinline__ int owner(const int* sums, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

__device__ __forceinline__ int pages_for(int64_t len, int shift, int width) {
  const int64_t p = (len + (int64_t{1} << shift) - 1) >> shift;
  return static_cast<int>(min(p, static_cast<int64_t>(width)));
}

// One launch: every workgroup forms the prefix sums of the new tokens and of the new pages over
// the whole batch in LDS (8 bytes a request, from L2 after the first workgroup), then takes its
// share of the tokens and of the new table entries, each found by a search in the sums.  A token
// on a new page takes the page from the free list itself rather than from the table, which other
// workgroups are writing.  Bound by the launch and its chain of reads (lengths, then a page number):
// 64 requests and 64 tokens 5.7 us, 1024 requests and 34000 tokens (0.36 MB) 6.6 us; with 256 requests a
// scan, one scan after the other, it took 14% longer.
__global__ __launch_bounds__(kPlanThreads) void paged_plan_kernel(PlanArgs a) {
  extern __shared__ int sums[];
  int* const cu = sums;                 // inclusive sums of the new tokens, at most 2^31 - 1
  int* const pg = sums + a.batch;       // inclusive sums of the new pages
  __shared__ int64_t part[kPlanThreads / 64][2];
  int64_t base[2] = {0, 0}, lost = 0;
  const bool first = blockIdx.x == 0;
  // Each thread sums a run of requests of its own, one scan over the threads puts the runs in place.
  const int run = (a.batch + kPlanThreads - 1) / kPlanThreads;
  const int begin = min(static_cast<int>(threadIdx.x) * run, a.batch), end = min(begin + run, a.batch);
  int64_t na = 0, np = 0;
  for (int i = begin; i < end; ++i) {
    const int64_t c = max(a.cached[i], 0), n = max(a.added[i], 0);
    na += n;
    np += pages_for(c + n, a.page_shift, a.width) - pages_for(c, a.page_shift, a.width);
    cu[i] = static_cast<int>(min(na, int64_t{0x7fffffff}));
    pg[i] = static_cast<int>(min(np, int64_t{0x7fffffff}));
    if (first) {
      a.lens[i] = static_cast<int>(min(c + n, int64_t{0x7fffffff}));
      const int64_t one = int64_t{1} << a.page_shift;   // entries the table does not have
      lost += max(int64_t{0}, ((c + n + one - 1) >> a.page_shift) - max((c + one - 1) >> a.page_shift, int64_t{a.width}));
    }
  }
  const int64_t own_a = na, own_p = np;
  scan2(na, np, part, base);
  const int64_t before_a = na - own_a, before_p = np - own_p;
  for (int i = begin; i < end; ++i) {
    cu[i] = static_cast<int>(min(before_a + cu[i], int64_t{0x7fffffff}));
    pg[i] = static_cast<int>(min(before_p + pg[i], int64_t{0x7fffffff}));
    if (first) a.cu[i + 1] = cu[i];
  }
  __syncthreads();
  const int taken = max(*a.taken_in, 0);
  const int left = max(a.n_free - taken, 0);
  const int tokens = static_cast<int>(min(base[0], int64_t{a.tokens}));
  const int fresh = static_cast<int>(min(base[1], int64_t{0x7fffffff}));
  if (first) {
    int64_t none = 0, total[2];
    scan2(lost, none, part, total);
    if (threadIdx.x == 0) {
      a.cu[0] = 0;
      *a.taken_out = *a.taken_in + min(fresh, left);
      *a.missing = static_cast<int>(min(total[0] + max(fresh - left, 0), int64_t{0x7fffffff}));
    }
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * kPlanThreads;
  const int64_t start = static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x;
  for (int64_t x = start; x < fresh; x += step) {
    const int i = owner(pg, a.batch, static_cast<int>(x));
    const int rank = static_cast<int>(x) - (i ? pg[i - 1] : 0);
    const int col = pages_for(max(a.cached[i], 0), a.page_shift, a.width) + rank;
    a.table[static_cast<int64_t>(i) * a.width + col] = x < left ? a.free_pages[taken + x] : -1;
  }
  for (int64_t t = start; t < a.tokens; t += step) {
    int position = -1;
    int64_t slot = -1;
    if (t < tokens) {
      const int i = owner(cu, a.batch, static_cast<int>(t));
      const int c = max(a.cached[i], 0);
      const int64_t at = int64_t{c} + (static_cast<int>(t) - (i ? cu[i - 1] : 0));
      position = static_cast<int>(min(at, int64_t{0x7fffffff}));
      const int col = position >> a.page_shift;
      if (at == position && col < a.width) {
        const int had = pages_for(c, a.page_shift, a.width);
        int page;
        if (col < had) {
          page = a.table[static_cast<int64_t>(i) * a.width + col];
        } else {
          const int x = (i ? pg[i - 1] : 0) + col - had;
          page = x < left ? a.free_pages[taken + x] : -1;
        }
        if (page >= 0) slot = (static_cast<int64_t>(page) << a.page_shift) + (position & ((1 << a.page_shift) - 1));
      }
    }
    a.positions[t] = position;
    a.slots[t] = slot;
  }
}

constexpr int kAppendThreads = 256;

// One group of D / 8 lanes per token and head: 16 bytes a lane of the key and of the value, the rows'
// largest magnitudes by DPP within the group, then the codes (8 bytes a lane) and the scales, or
// the 16 bytes as they are.  Bound by memory: 16384 tokens of 8 heads of 128 to e4m3, 102 MB, take
// 23.4 us (4.4 TB/s; a 2 GiB copy runs at 4.9).  Key and value of a row in one thread, so that two
// loads are under way: with one tensor a workgroup it took 23% longer; with two and four rows a
// thread 2% and 20%.
template <int DT, int D, bool E4M3>
__global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(AppendArgs a) {
  constexpr int kLanes = D / 8;
  const int id = blockIdx.x * (kAppendThreads / kLanes) + threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  if (id >= a.tokens * a.heads) return;
  const int t = id / a.heads, h = id - t * a.heads;
  const int64_t slot = a.slots[t];
  const U4 w[2] = {load16(static_cast<const uint16_t*>(a.k) + t * a.kts + h * a.khs + lane * 8),
                   load16(static_cast<const uint16_t*>(a.v) + t * a.vts + h * a.vhs + lane * 8)};
  if (slot < 0 || slot >= a.n_slots) return;   // the whole group together
  const int64_t row = (((slot >> a.page_shift) * a.heads + h) << a.page_shift) + (slot & ((1 << a.page_shift) - 1));
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    void* c = v ? a.vc : a.kc;
    if constexpr (E4M3) {
      const uint32_t key = kLanes == 16 ? max16(key8(w[v])) : max8(key8(w[v]));
      const float s = scale_from_amax(amax_from_key<DT>(key));
      const uint2 q = enc8<DT>(w[v], s, 1.0f / s, fast_scale(s));
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(c) + row * D + lane * 8) = q;
      if (lane == 0) (v ? a.vs : a.ks)[row] = s;
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(c) + row * D + lane * 8) = make_uint4(w[v].x, w[v].y, w[v].z, w[v].w);
    }
  }
}

template <int DT, int D>
void append(bool e4m3, const AppendArgs& a, hipStream_t s) {
  const unsigned grid = static_cast<unsigned>(kv_append_groups(a.tokens, a.heads, D));
  if (e4m3) kv_append_kernel<DT, D, true><<<grid, kAppendThreads, 0, s>>>(a);
  else kv_append_kernel<DT, D, false><<<grid, kAppendThreads, 0, s>>>(a);
}

}  // namespace

void launch_paged_plan(const PlanArgs& a, hipStream_t s) {
  const int groups = max(1, min((a.tokens + kPlanThreads - 1) / kPlanThreads, 1024));
  paged_plan_kernel<<<groups, kPlanThreads, static_cast<size_t>(a.batch) * 8, s>>>(a);
}

int64_t kv_append_groups(int64_t tokens, int64_t heads, int head_dim) {
  const int rows = kAppendThreads / (head_dim / 8);
  return (tokens * heads + rows - 1) / rows;
}

void launch_kv_append(int dt, int head_dim, bool e4m3, const AppendArgs& a, hipStream_t s) {
  if (dt == DT_BF16) head_dim == 128 ? append<DT_BF16, 128>(e4m3, a, s) : append<DT_BF16, 64>(e4m3, a, s);
  else head_dim == 128 ? append<DT_F16, 128>(e4m3, a, s) : append<DT_F16, 64>(e4m3, a, s);
}

}  // namespace fp8amax
