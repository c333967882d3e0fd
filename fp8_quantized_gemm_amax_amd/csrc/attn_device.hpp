// attn_device.hpp - device pieces shared by the attention kernels, gfx950: which rows and keys a
// workgroup handles, the matrix-instruction layouts, LDS tiles of keys and values, and the
// careful path for values that are not finite.
//
// Rows.  The query heads that share a key head are packed: row r of a request and key head h is
// token r / group, query head h * group + r % group, so one tile of keys serves them all and a
// decode step of 8 heads is 8 rows rather than 8 tiles of one.
//
// Layouts.  The scores are formed transposed, S^T = K Q^T (32x32x16 MFMA: lane l holds column
// (query row) l % 32 and, in register i, key 8 (i / 4) + 4 (l / 32) + i % 4), so a query's
// statistics are sums over a lane's own registers and one exchange with lane l ^ 32.  The same
// registers, rounded to 16 bits, are the B operand of O^T = V^T P^T when the sum over keys is
// taken in the order the lanes hold them: slots 0-3 and 4-7 of step s are keys 16 s + 4 (l / 32)
// + 0..3 and + 8..11.  The A operand V^T comes in that order from the transposing LDS reads.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dma.hpp"
#include "fp8_device.hpp"
#include "gemm_common.hpp"
#include "serving.hpp"

namespace fp8amax {
namespace attn {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

// Where keys and values come from.
enum Source { SRC_PACKED = 0, SRC_PAGED = 1, SRC_E4M3 = 2 };

constexpr int kKeys = 64;                  // keys in an LDS tile
constexpr int kPlane = kKeys * 128;        // bytes of a plane: 64 channels of every key of the tile
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// Reads through the scalar cache of what no kernel of the launch writes (uniform addresses).
__device__ __forceinline__ int scalar_int(const int* p) {
  return *reinterpret_cast<const __attribute__((address_space(4))) int*>(reinterpret_cast<uintptr_t>(p));
}

// Waits for this wave's LDS reads and writes: before what they read may be overwritten by a DMA or,
// after a barrier, by another wave.  Memory accesses stay on their side of it.
__device__ __forceinline__ void wait_lds_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

template <int DT>
__device__ __forceinline__ v16f mfma(const v8s& a, const v8s& b, const v16f& c) {
  if constexpr (DT == DT_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// Two float32 values rounded to nearest even in one dword.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (DT == DT_BF16) return __builtin_bit_cast(uint32_t, v2bf{static_cast<__bf16>(lo), static_cast<__bf16>(hi)});
  else return __builtin_bit_cast(uint32_t, v2h{static_cast<_Float16>(lo), static_cast<_Float16>(hi)});
}

// Eight e4m3 codes as 16-bit values (exact: both types hold every code).
template <int DT>
__device__ __forceinline__ v4u codes8(uint32_t lo, uint32_t hi) {
  if constexpr (DT == DT_BF16)
    return v4u{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true))};
  else
    return v4u{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true))};
}

// {a of lane l % 32, b of lane l % 32} in the low and high half, and the same of lanes 32-63.
__device__ __forceinline__ void swap_halves(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ float max_halves(float x) {
  uint32_t a = __float_as_uint(x), b = a;
  swap_halves(a, b);
  return fmaxf(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ float add_halves(float x) {
  uint32_t a = __float_as_uint(x), b = a;
  swap_halves(a, b);
  return __uint_as_float(a) + __uint_as_float(b);
}

// LDS DMA as dma16, with the wait states that the compiler does not insert for inline asm: one
// between the write of m0 and the load (here), and five between a vector instruction's write of
// the buffer's scalars (readfirstlane) and the load (settle, once per buffer).
__device__ __forceinline__ void settle(v4i& rsrc) { asm volatile("s_nop 4" : "+s"(rsrc)); }
__device__ __forceinline__ void dma16_safe(const v4i& rsrc, uint32_t lds, uint32_t voff) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(voff), "s"(rsrc), "{m0}"(lds) : "memory");
}

// One request's part of a tile of rows (all uniform).
struct Rows {
  int request, begin, tokens;   // its first packed token and its number of new tokens
  int rows, row0;               // tokens * group, and the tile's first row
  int len, pos0;                // its keys, and the position of its first new token
};

__device__ __forceinline__ int clamp_cu(const AttnArgs& a, int i) { return min(max(scalar_int(a.cu + i), 0), a.tokens); }

// The rows of tile j of `size` rows.  Request i owns the tile numbers from cu[i] * group / size + i
// on: the next request's first is at least ceil(rows / size) further, so no table of tiles is
// needed and numbers without rows are few (one a request at most).  False where tile j has none.
__device__ __forceinline__ bool find_rows(const AttnArgs& a, int j, int size, bool paged, Rows& r) {
  int lo = 0, hi = a.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    const int64_t first = static_cast<int64_t>(clamp_cu(a, mid)) * a.group / size + mid;
    if (first <= j) lo = mid;
    else hi = mid - 1;
  }
  r.request = lo;
  r.begin = clamp_cu(a, lo);
  r.tokens = clamp_cu(a, lo + 1) - r.begin;
  r.rows = r.tokens * a.group;
  r.row0 = (j - static_cast<int>(static_cast<int64_t>(r.begin) * a.group / size) - lo) * size;
  if (r.tokens <= 0 || r.row0 >= r.rows || r.row0 < 0) return false;
  r.len = paged ? min(max(scalar_int(a.lens + lo), 0), a.width << a.page_shift) : r.tokens;
  r.pos0 = r.len - r.tokens;
  return true;
}

// Base of the next n <= 16 keys from key `at` on (uniform, at a multiple of 8 inside one page),
// as a buffer whose reads past the request's keys, or of a page that is not there, give zeros.
template <int SRC, int D>
__device__ __forceinline__ v4i key_rows(const AttnArgs& a, const Rows& r, const void* base, int64_t ts, int64_t hs,
                                        int h, int at, int n, int page) {
  constexpr int kElem = SRC == SRC_E4M3 ? 1 : 2;
  const int have = min(max(r.len - at, 0), n);
  if constexpr (SRC == SRC_PACKED) {
    const char* p = static_cast<const char*>(base) + ((r.begin + at) * ts + h * hs) * 2;
    return make_rsrc(p, have > 0 ? static_cast<uint32_t>((have - 1) * ts * 2 + D * 2) : 0u);
  } else {
    const bool there = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.pages);
    const int64_t row = ((static_cast<int64_t>(there ? page : 0) * a.hk + h) << a.page_shift) + (at & ((1 << a.page_shift) - 1));
    return make_rsrc(static_cast<const char*>(base) + row * (D * kElem), there ? static_cast<uint32_t>(have * D * kElem) : 0u);
  }
}

// ------------------------------------------------------------------------------------------
// Splitting a long axis.  Few rows over many keys would leave most of the card idle, so the keys
// of a tile of rows are cut into chunks that different workgroups take, each leaving its maximum,
// sum and output for attn_join.  The requests' lengths are on the device, so the cut is made there:
// every workgroup sums the work of the whole batch (three integers a request) and takes
//   steps of 64 keys a chunk = max(kMinSteps, work / kUnits)
// which cuts long requests into more chunks than short ones and leaves a full batch of equal
// lengths uncut.  Then units (request, tile, chunk) are numbered request by request.
constexpr int kUnits = 1024;       // units wanted on the card, over all key heads
constexpr int kMinSteps = 4;       // no chunk below 256 keys: a unit's start and end cost about that
constexpr int kMaxSplitBatch = 1024;   // above, there are enough units without cuts
constexpr int kMaxSplitHeads = 1024;

struct Unit {
  Rows r;
  int head;
  int j0, j1;       // its keys
  int piece, count; // its chunk and how many there are of the tile (1: the whole)
  int slot;         // where the tile's partial results begin, hk apart
};

// Keys [j0, j1) that the rows of a tile see between them, j0 a multiple of 64.
__device__ __forceinline__ void tile_keys(const AttnArgs& a, const Rows& r, int size, int& j0, int& j1) {
  const int last = (min(r.row0 + size, r.rows) - 1) / a.group;
  j1 = max(r.pos0 + last + 1, 0);
  const int lo = a.window > 0 ? max(0, r.pos0 + r.row0 / a.group - a.window + 1) : 0;
  j0 = min(lo, j1) & ~(kKeys - 1);
}

__host__ __device__ constexpr int64_t tile_bound(int64_t tokens, int64_t group, int64_t batch, int size) {
  return tokens * group / size + batch;
}
// Whether a batch can be cut at all: `capacity` is the most keys a request can have.
__host__ __device__ constexpr bool may_split(int64_t batch, int64_t hk, int64_t capacity) {
  return batch <= kMaxSplitBatch && hk <= kMaxSplitHeads && capacity > kMinSteps * kKeys;
}
// Units per key head are at most the tiles and this many more, and partial results at most twice it.
__host__ __device__ constexpr int64_t extra_units(int64_t hk) { return (kUnits + hk - 1) / hk; }

// The inclusive sum of x over the workgroup's 256 threads; total gets the last one's.
__device__ __forceinline__ int scan256(int x, int* part, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 63) part[wave] = x;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w == wave) x += total;
    total += part[w];
  }
  return x;
}

// Unit `block` of the launch (block = unit * hk + head); `lds`: 4 * (2 * kMaxSplitBatch + 8) bytes,
// free again on return.  False where there is none.
template <int SIZE>
__device__ __forceinline__ bool find_unit(const AttnArgs& a, int block, int* lds, Unit& u) {
  u.head = block % a.hk;
  const int unit = block / a.hk;
  int *ends = lds, *slots = lds + kMaxSplitBatch, *part = lds + 2 * kMaxSplitBatch;
  auto shape = [&](int i, int& tiles, int& steps) {
    const int begin = min(max(a.cu[i], 0), a.tokens), n = min(max(a.cu[i + 1], 0), a.tokens) - begin;
    const int len = min(max(a.lens[i], 0), a.width << a.page_shift);
    tiles = n > 0 ? static_cast<int>((static_cast<int64_t>(n) * a.group + SIZE - 1) / SIZE) : 0;
    const int lo = a.window > 0 ? max(0, len - n - a.window + 1) & ~(kKeys - 1) : 0;
    steps = max(1, (len - lo + kKeys - 1) / kKeys);
  };
  int64_t work = 0;
  for (int i = threadIdx.x; i < a.batch; i += 256) {
    int tiles, steps;
    shape(i, tiles, steps);
    work += static_cast<int64_t>(tiles) * steps;
  }
  for (int d = 1; d < 64; d <<= 1) work += __shfl_xor(work, d);
  int64_t* sums = reinterpret_cast<int64_t*>(part);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = work;
  __syncthreads();
  work = sums[0] + sums[1] + sums[2] + sums[3];
  const int64_t want = (work * a.hk + kUnits - 1) / kUnits;
  const int chunk = static_cast<int>(max(want, int64_t{kMinSteps}));
  int before = 0, before_slots = 0;
  for (int i0 = 0; i0 < a.batch; i0 += 256) {
    const int i = i0 + threadIdx.x;
    int tiles = 0, steps = 1;
    if (i < a.batch) shape(i, tiles, steps);
    const int chunks = (steps + chunk - 1) / chunk;
    int total, total_slots;
    const int e = scan256(tiles * chunks, part, total);
    const int s = scan256(chunks > 1 ? tiles * chunks : 0, part, total_slots);
    if (i < a.batch) {
      ends[i] = before + e;
      slots[i] = before_slots + s;
    }
    before += total;
    before_slots += total_slots;
  }
  __syncthreads();
  // more units than the launch holds: cu_tokens decreases somewhere, and nothing is computed
  if (unit >= before || static_cast<int64_t>(before) * a.hk > gridDim.x) return false;
  int lo = 0, hi = a.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > unit) hi = mid;
    else lo = mid + 1;
  }
  const int i = __builtin_amdgcn_readfirstlane(lo);
  int tiles, steps;
  shape(i, tiles, steps);
  const int chunks = (steps + chunk - 1) / chunk;
  const int local = unit - (ends[i] - tiles * chunks);
  // the last tiles see the most keys: they go first
  const int tile = __builtin_amdgcn_readfirstlane(tiles - 1 - local / chunks), piece = __builtin_amdgcn_readfirstlane(local % chunks);
  const int first_slot = __builtin_amdgcn_readfirstlane(slots[i]) - tiles * chunks;
  __syncthreads();
  Rows& r = u.r;
  r.request = i;
  r.begin = clamp_cu(a, i);
  r.tokens = clamp_cu(a, i + 1) - r.begin;
  r.rows = r.tokens * a.group;
  r.row0 = tile * SIZE;
  r.len = min(max(scalar_int(a.lens + i), 0), a.width << a.page_shift);
  r.pos0 = r.len - r.tokens;
  int j0, j1;
  tile_keys(a, r, SIZE, j0, j1);
  const int own = (j1 - j0 + kKeys - 1) / kKeys;
  const int per = max(1, (own + chunks - 1) / chunks);
  u.count = max(1, (own + per - 1) / per);
  if (piece >= u.count) return false;
  u.j0 = j0 + piece * per * kKeys;
  u.j1 = min(j1, u.j0 + per * kKeys);
  u.piece = piece;
  u.slot = (first_slot + tile * chunks) * a.hk + u.head;
  return true;
}

// The workspace: a counter for every partial result, then the partial results' maxima and sums
// [slot][row][2], then their outputs [slot][row][D], float32.  The counters are zero between calls.
constexpr int64_t kCounterBytes = FP8_ATTN_COUNTER_BYTES;
static_assert(kCounterBytes >= 4 * 2 * (kUnits + kMaxSplitHeads), "slot_bound is at most 2 (kUnits + hk - 1)");
__host__ __device__ inline int64_t slot_bound(int64_t hk) { return 2 * extra_units(hk) * hk; }
struct Workspace {
  int* counters;
  float* stats;
  float* out;
};
__device__ __forceinline__ Workspace workspace(const AttnArgs& a, int size) {
  Workspace w;
  w.counters = reinterpret_cast<int*>(a.ws);
  w.stats = reinterpret_cast<float*>(a.ws + kCounterBytes);
  w.out = w.stats + slot_bound(a.hk) * size * 2;
  return w;
}

// Partial results pass between workgroups of one launch, whose XCDs' L2 caches do not see each
// other: they are written and read with agent-scope accesses, which go through to memory, and a
// writer waits for its stores before it counts itself.  (Fences in their place write back and
// empty the whole L2: measured, they doubled the time of every split case.)
__device__ __forceinline__ void leave2(float* p, float x, float y) {
  const uint64_t v = static_cast<uint64_t>(__float_as_uint(x)) | static_cast<uint64_t>(__float_as_uint(y)) << 32;
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 pick2(const float* p) {
  const uint64_t v = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return make_float2(__uint_as_float(static_cast<uint32_t>(v)), __uint_as_float(static_cast<uint32_t>(v >> 32)));
}

// After a workgroup's partial result is stored: the workgroup that finds itself the last of its
// tile joins them all, in their order, so the result does not depend on who that is:
//   out = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i.
// D / 4 lanes take a row's channels; with few rows, several such groups share a row's partial
// results.  `flag` and `lds` (8 KB) are LDS that nothing else uses any more.
template <int DT, int D, int SIZE>
__device__ __forceinline__ void join_partials(const AttnArgs& a, const Unit& u, int* flag, float* lds) {
  constexpr int kLanes = D / 4, kTeams = 256 / kLanes;
  const Workspace ws = workspace(a, SIZE);
  const Rows& r = u.r;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // every thread's stores before the count
  __syncthreads();
  if (threadIdx.x == 0) {
    int* n = ws.counters + u.slot;
    const bool last = __hip_atomic_fetch_add(n, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == u.count - 1;
    if (last) __hip_atomic_store(n, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *flag = last;
  }
  __syncthreads();
  if (!*flag) return;
  const int rows = min(SIZE, r.rows - r.row0);
  const int lane = threadIdx.x % kLanes, team = threadIdx.x / kLanes;
  int share = 1;        // teams to a row
  while (2 * share * rows <= kTeams) share *= 2;
  const int part = team % share;
  const int passes = (rows * share + kTeams - 1) / kTeams;
  for (int pass = 0; pass < passes; ++pass) {
    const int local = (pass * kTeams + team) / share;
    const bool on = local < rows;
    const int64_t at = static_cast<int64_t>(u.slot) * SIZE + (on ? local : 0), step = static_cast<int64_t>(a.hk) * SIZE;
    float m = -INFINITY;
    for (int i = lane; i < u.count; i += kLanes) m = fmaxf(m, pick2(ws.stats + (at + i * step) * 2).x);
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    const float mb = m == -INFINITY ? 0.0f : m;
    float l = 0.0f;
    v4f o;
    o = 0.0f;
#pragma unroll 4
    for (int i = part; i < u.count; i += share) {
      const float2 st = pick2(ws.stats + (at + i * step) * 2);
      const float* from = ws.out + (at + i * step) * D + 4 * lane;
      const float2 x0 = pick2(from), x1 = pick2(from + 2);
      const float x[4] = {x0.x, x0.y, x1.x, x1.y};
      const float w = __builtin_amdgcn_exp2f(st.x - mb);
      l = __builtin_fmaf(w, st.y, l);
#pragma unroll
      for (int y = 0; y < 4; ++y) o[y] = __builtin_fmaf(w, x[y], o[y]);
    }
    if (share > 1) {    // one pass only
      float* to = lds + (team * kLanes + lane) * 8;
      *reinterpret_cast<v4f*>(to) = o;
      to[4] = l;
      __syncthreads();
      if (part == 0)
        for (int k = 1; k < share; ++k) {
          const float* from = to + k * kLanes * 8;
          const v4f x = *reinterpret_cast<const v4f*>(from);
#pragma unroll
          for (int y = 0; y < 4; ++y) o[y] += x[y];
          l += from[4];
        }
    }
    if (!on || part != 0) continue;
    const int row = r.row0 + local, tok = row / a.group;
    const int64_t out_row = static_cast<int64_t>(r.begin + tok) * a.hq + u.head * a.group + (row - tok * a.group);
    const bool none = r.pos0 + tok < 0;
    const float inv = none ? 0.0f : 1.0f / l;
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + out_row * D + 4 * lane) =
        make_uint2(pack2<DT>(o[0] * inv, o[1] * inv), pack2<DT>(o[2] * inv, o[3] * inv));
    if (a.lse && lane == 0) a.lse[out_row] = none ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
  }
}

// ------------------------------------------------------------------------------------------
// Values that are not finite.  The product with v multiplies a masked key's value by a weight of
// zero, which is right unless that value is infinite or NaN.  A workgroup with a result that is not
// finite goes over its keys once more: such values enter the product as zeros, so rows that do not
// see them get the bits they would have had, and rows whose weight for them is not zero get what
// they hold added afterwards.
template <int DT>
struct Odd {
  static constexpr short kExp = DT == DT_BF16 ? 0x7f80 : 0x7c00;
  static constexpr short kOne = DT == DT_BF16 ? 0x3f80 : 0x3c00;
  // 1 where the value is of kind 0: +inf, 1: -inf, 2: NaN, else 0.
  static __device__ __forceinline__ v8s is(const v8s& x, int kind) {
    v8s r;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool odd = (x[i] & kExp) == kExp, nan = (x[i] & 0x7fff) > kExp;
      r[i] = odd && (nan ? kind == 2 : kind == (x[i] < 0)) ? kOne : 0;
    }
    return r;
  }
  static __device__ __forceinline__ v8s without(const v8s& x) {
    v8s r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = (x[i] & kExp) == kExp ? 0 : x[i];
    return r;
  }
  static __device__ __forceinline__ v8s seen(const v8s& p) {
    v8s r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = (p[i] & 0x7fff) ? kOne : 0;
    return r;
  }
};

template <int DT>
__device__ __forceinline__ v16f mfma_odd(const v8s& v, const v8s& p, v16f o) {
  o = mfma<DT>(Odd<DT>::without(v), p, o);
  const v8s w = Odd<DT>::seen(p);
#pragma unroll 1
  for (int kind = 0; kind < 3; ++kind) {
    v16f n;
    n = 0.0f;
    n = mfma<DT>(Odd<DT>::is(v, kind), w, n);
    const float add = kind == 0 ? INFINITY : kind == 1 ? -INFINITY : __uint_as_float(kCanonicalNaN);
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] += n[i] > 0.0f ? add : 0.0f;
  }
  return o;
}

// Host side: the paged kernels for many rows and for few.
void launch_attn_tile(int dt, int head_dim, bool e4m3, const AttnArgs& a, hipStream_t s);
void launch_attn_few(int dt, int head_dim, bool e4m3, const AttnArgs& a, hipStream_t s);

}  // namespace attn
}  // namespace fp8amax
