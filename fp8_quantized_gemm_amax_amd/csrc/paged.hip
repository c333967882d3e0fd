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
// thread 2% and 20%.  To mxfp4 a lane's eight channels are a quarter of a block, whose largest magnitude
// four lanes find by DPP, and 4 bytes of codes.  Views of a fused projection, from memory: 16384 tokens into
// pages in order 22.1 us (85 MB, 3.8 TB/s), into shuffled slots, 64 bytes each, 24.4, where e4m3 takes 25.3 and
// 25.5; 64 tokens 2.6 us in a graph (e4m3 2.8, a launch by itself 2).
template <int DT, int D, int FORMAT>
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
    if constexpr (FORMAT == FP8_KV_MXFP4) {     // four lanes hold a block
      float x[8];
      widen8<DT>(w[v], x);
      const uint32_t s = mx4_scale(__float_as_uint(amax_from_key<DT>(max4(key8(w[v])))));
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(c) + row * (D / 2) + lane * 4) = enc8_mx4<DT>(x, s);
      if (lane % 4 == 0) static_cast<uint8_t*>(v ? a.vs : a.ks)[row * (D / 32) + lane / 4] = static_cast<uint8_t>(s);
    } else if constexpr (FORMAT == FP8_KV_E4M3) {
      const uint32_t key = kLanes == 16 ? max16(key8(w[v])) : max8(key8(w[v]));
      const float s = scale_from_amax(amax_from_key<DT>(key));
      const uint2 q = enc8<DT>(w[v], s, 1.0f / s, fast_scale(s));
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(c) + row * D + lane * 8) = q;
      if (lane == 0) static_cast<float*>(v ? a.vs : a.ks)[row] = s;
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(c) + row * D + lane * 8) = make_uint4(w[v].x, w[v].y, w[v].z, w[v].w);
    }
  }
}

template <int DT, int D>
void append(int format, const AppendArgs& a, hipStream_t s) {
  const unsigned grid = static_cast<unsigned>(kv_append_groups(a.tokens, a.heads, D));
  if (format == FP8_KV_E4M3) kv_append_kernel<DT, D, FP8_KV_E4M3><<<grid, kAppendThreads, 0, s>>>(a);
  else if (format == FP8_KV_MXFP4) kv_append_kernel<DT, D, FP8_KV_MXFP4><<<grid, kAppendThreads, 0, s>>>(a);
  else kv_append_kernel<DT, D, FP8_KV_SAME><<<grid, kAppendThreads, 0, s>>>(a);
}

// Two float32 values rounded to nearest even in one dword.
template <int DT>
__device__ __forceinline__ uint32_t round2(float lo, float hi) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  typedef _Float16 v2h __attribute__((ext_vector_type(2)));
  if constexpr (DT == DT_BF16) return __builtin_bit_cast(uint32_t, v2bf{static_cast<__bf16>(lo), static_cast<__bf16>(hi)});
  else return __builtin_bit_cast(uint32_t, v2h{static_cast<_Float16>(lo), static_cast<_Float16>(hi)});
}
template <int DT>
__device__ __forceinline__ void store_rounded8(uint16_t* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(round2<DT>(x[0], x[1]), round2<DT>(x[2], x[3]), round2<DT>(x[4], x[5]), round2<DT>(x[6], x[7]));
}

// A lane's sixteen channels of a head, in two runs of eight: the two sides of eight pairs (the runs
// R / 2 apart, or with PAIRS neighbours), or channels past R.
template <bool PAIRS>
struct RopeLane {
  int first, second;     // first channels of the runs
  bool turns;
  float cos[8], sin[8];
  __device__ __forceinline__ RopeLane(int lane, int rotary) {
    turns = 16 * lane < rotary;
    const bool halves = !PAIRS && turns;
    first = halves ? 8 * lane : 16 * lane;
    second = halves ? rotary / 2 + 8 * lane : 16 * lane + 8;
  }
  // This lane's eight cosines and sines of a position's row.
  __device__ __forceinline__ void load(const float* row, int lane, int rotary) {
#pragma unroll
    for (int i = 0; i < 8; ++i) cos[i] = sin[i] = 0.0f;
    if (!turns) return;
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 c = *reinterpret_cast<const float4*>(row + 8 * lane + i);
      const float4 s = *reinterpret_cast<const float4*>(row + rotary / 2 + 8 * lane + i);
      cos[i] = c.x; cos[i + 1] = c.y; cos[i + 2] = c.z; cos[i + 3] = c.w;
      sin[i] = s.x; sin[i + 1] = s.y; sin[i + 2] = s.z; sin[i + 3] = s.w;
    }
  }
  // x, y: the runs, in and out.  Every product and sum is rounded on its own.
  __device__ __forceinline__ void turn(float (&x)[8], float (&y)[8]) const {
    if (!turns) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float& a = PAIRS ? (i < 4 ? x[2 * i] : y[2 * i - 8]) : x[i];
      float& b = PAIRS ? (i < 4 ? x[2 * i + 1] : y[2 * i - 7]) : y[i];
      const float p = a * cos[i] - b * sin[i], q = b * cos[i] + a * sin[i];
      a = p;
      b = q;
    }
  }
};

template <int N>
__device__ __forceinline__ uint32_t key8_f32(const float (&x)[N]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
  return m;
}

// A head's row in the cache, from float32 values in two runs a lane.  `block` (FP8_KV_MXFP4): the
// lane group's D / 8 entries of LDS, the largest keys of its runs.
template <int DT, int D, int FORMAT>
__device__ __forceinline__ void store_row(void* cache, void* scales, int64_t row, int lane, int first, int second,
                                          const float (&x)[8], const float (&y)[8], uint32_t* block) {
  if constexpr (FORMAT == FP8_KV_SAME) {
    uint16_t* to = static_cast<uint16_t*>(cache) + row * D;
    store_rounded8<DT>(to + first, x);
    store_rounded8<DT>(to + second, y);
  } else if constexpr (FORMAT == FP8_KV_E4M3) {
    const uint32_t own = max(key8_f32(x), key8_f32(y)), key = D == 128 ? max8(own) : max4(own);
    const float s = scale_from_amax(key > 0x7f800000u ? __uint_as_float(kCanonicalNaN) : __uint_as_float(key));
    const bool fast = fast_scale_f32(s);
    const float r = 1.0f / s;
    uint8_t* to = static_cast<uint8_t*>(cache) + row * D;
    *reinterpret_cast<uint2*>(to + first) = enc8_f32(x, s, r, fast);
    *reinterpret_cast<uint2*>(to + second) = enc8_f32(y, s, r, fast);
    if (lane == 0) static_cast<float*>(scales)[row] = s;
  } else {
    // runs of a block of 32 channels lie in any lanes of the head: through LDS, in one wave
    block[first / 8] = key8_f32(x);
    block[second / 8] = key8_f32(y);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    auto scale = [&](int channel) {
      const uint4 k = *reinterpret_cast<const uint4*>(block + channel / 32 * 4);
      return mx4_scale(max(max(k.x, k.y), max(k.z, k.w)));
    };
    const uint32_t sx = scale(first), sy = scale(second);
    uint8_t* to = static_cast<uint8_t*>(cache) + row * (D / 2);
    *reinterpret_cast<uint32_t*>(to + first / 2) = enc8_mx4<DT>(x, sx);
    *reinterpret_cast<uint32_t*>(to + second / 2) = enc8_mx4<DT>(y, sy);
    uint8_t* s = static_cast<uint8_t*>(scales) + row * (D / 32);
    if (first % 32 == 0) s[first / 32] = static_cast<uint8_t>(sx);
    if (second % 32 == 0) s[second / 32] = static_cast<uint8_t>(sy);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();      // before the next row's keys
  }
}

// Rotation and append: of a token at position p, channels a and b of a pair and the pair's angle become
//   a' = a cos - b sin, b' = b cos + a sin   (float32, from the table's row p),
// queries are rounded to their type and keys, with the values as they are, to the cache's format: the
// rotated keys never lie in memory in between, where a call for each of the three would read and write
// them once more.
// A group of D / 16 lanes takes a unit of a token: kRopeHeads query heads, or the keys and values of half
// as many key heads, whose loads are all in flight while the table's row, that comes after the position,
// is on its way.  Bound by memory: 16384 tokens of 32 heads over 8 of 128 channels into an e4m3 cache, 373
// MB, 69 us (5.4 TB/s; the best copy of 1 GiB 5.7), into mxfp4 67 us in pages in order and 73 in shuffled
// slots, 64 channels 45 us; and by the chain of reads where there are few: 64 tokens 3.3 us in a graph.  With four heads a unit and with eight, both
// sizes were slower: 73.8 and 81.2 us, 5.0 and 8.3 us (fewer workgroups, longer each).
constexpr int kRopeHeads = 2;
template <int DT, int D, int FORMAT, bool PAIRS>
__global__ __launch_bounds__(kAppendThreads) void rope_append_kernel(RopeArgs a) {
  constexpr int kLanes = D / 16, kHeads = kRopeHeads;
  __shared__ __attribute__((aligned(16))) uint32_t keys[FORMAT == FP8_KV_MXFP4 ? kAppendThreads / kLanes : 1][D / 8];
  uint32_t* const block = keys[FORMAT == FP8_KV_MXFP4 ? threadIdx.x / kLanes : 0];
  const uint32_t q_units = (a.q_heads + kHeads - 1) / kHeads, units = q_units + (a.kv.heads + kHeads / 2 - 1) / (kHeads / 2);
  const uint32_t id = blockIdx.x * (kAppendThreads / kLanes) + threadIdx.x / kLanes;   // below 2^30: see kMaxGroups
  const int lane = threadIdx.x % kLanes;
  const uint32_t t = id / units, u = id - t * units;
  if (t >= static_cast<uint32_t>(a.kv.tokens)) return;
  const int position = a.positions[t];
  RopeLane<PAIRS> lanes(lane, a.rotary);
  const bool is_q = u < q_units;
  const int h0 = static_cast<int>(is_q ? u * kHeads : (u - q_units) * (kHeads / 2));
  const int64_t slot = is_q ? 0 : a.kv.slots[t];
  U4 w[kHeads][2];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const bool value = !is_q && (i & 1);
    const int h = is_q ? min(h0 + i, a.q_heads - 1) : min(h0 + i / 2, a.kv.heads - 1);
    const uint16_t* p = is_q ? static_cast<const uint16_t*>(a.q) + t * a.qts + h * a.qhs
                      : value ? static_cast<const uint16_t*>(a.kv.v) + t * a.kv.vts + h * a.kv.vhs
                              : static_cast<const uint16_t*>(a.kv.k) + t * a.kv.kts + h * a.kv.khs;
    w[i][0] = load16(p + lanes.first);
    w[i][1] = load16(p + lanes.second);
  }
  if (position < 0 || position >= a.n_positions) return;     // the token's lanes together
  lanes.load(a.cos_sin + static_cast<int64_t>(position) * a.rotary, lane, a.rotary);
  if (is_q) {
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      if (h0 + i >= a.q_heads) break;
      float x[8], y[8];
      widen8<DT>(w[i][0], x);
      widen8<DT>(w[i][1], y);
      lanes.turn(x, y);
      uint16_t* to = static_cast<uint16_t*>(a.q_out) + (static_cast<int64_t>(t) * a.q_heads + h0 + i) * D;
      store_rounded8<DT>(to + lanes.first, x);
      store_rounded8<DT>(to + lanes.second, y);
    }
    return;
  }
  if (slot < 0 || slot >= a.kv.n_slots) return;
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = h0 + i / 2;
    if (h >= a.kv.heads) break;
    const int64_t row = (((slot >> a.kv.page_shift) * a.kv.heads + h) << a.kv.page_shift) + (slot & ((1 << a.kv.page_shift) - 1));
    float x[8], y[8];
    widen8<DT>(w[i][0], x);
    widen8<DT>(w[i][1], y);
    if ((i & 1) == 0) lanes.turn(x, y);
    store_row<DT, D, FORMAT>(i & 1 ? a.kv.vc : a.kv.kc, i & 1 ? a.kv.vs : a.kv.ks, row, lane, lanes.first, lanes.second, x, y, block);
  }
}

template <int DT, int D, int FORMAT>
void rope(bool interleaved, const RopeArgs& a, hipStream_t s) {
  const unsigned grid = static_cast<unsigned>(rope_append_groups(a.kv.tokens, a.q_heads, a.kv.heads, D));
  if (interleaved) rope_append_kernel<DT, D, FORMAT, true><<<grid, kAppendThreads, 0, s>>>(a);
  else rope_append_kernel<DT, D, FORMAT, false><<<grid, kAppendThreads, 0, s>>>(a);
}
template <int DT, int D>
void rope(int format, bool interleaved, const RopeArgs& a, hipStream_t s) {
  if (format == FP8_KV_E4M3) rope<DT, D, FP8_KV_E4M3>(interleaved, a, s);
  else if (format == FP8_KV_MXFP4) rope<DT, D, FP8_KV_MXFP4>(interleaved, a, s);
  else rope<DT, D, FP8_KV_SAME>(interleaved, a, s);
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

void launch_kv_append(int dt, int head_dim, int format, const AppendArgs& a, hipStream_t s) {
  if (dt == DT_BF16) head_dim == 128 ? append<DT_BF16, 128>(format, a, s) : append<DT_BF16, 64>(format, a, s);
  else head_dim == 128 ? append<DT_F16, 128>(format, a, s) : append<DT_F16, 64>(format, a, s);
}

int64_t rope_append_groups(int64_t tokens, int64_t q_heads, int64_t kv_heads, int head_dim) {
  const int64_t units = (q_heads + kRopeHeads - 1) / kRopeHeads + (kv_heads + kRopeHeads / 2 - 1) / (kRopeHeads / 2);
  const int groups = kAppendThreads / (head_dim / 16);
  return (tokens * units + groups - 1) / groups;
}

void launch_rope_append(int dt, int head_dim, int format, bool interleaved, const RopeArgs& a, hipStream_t s) {
  if (dt == DT_BF16) head_dim == 128 ? rope<DT_BF16, 128>(format, interleaved, a, s) : rope<DT_BF16, 64>(format, interleaved, a, s);
  else head_dim == 128 ? rope<DT_F16, 128>(format, interleaved, a, s) : rope<DT_F16, 64>(format, interleaved, a, s);
}

}  // namespace fp8amax
