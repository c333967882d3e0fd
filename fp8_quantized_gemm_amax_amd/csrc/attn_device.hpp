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
enum Source { SRC_PACKED = 0, SRC_PAGED = 1, SRC_E4M3 = 2, SRC_MXFP4 = 3 };

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

template <int DT>
__device__ __forceinline__ v8s pack8(const float (&x)[8]) {
  return __builtin_bit_cast(v8s, v4u{pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]), pack2<DT>(x[4], x[5]), pack2<DT>(x[6], x[7])});
}

// Eight e4m3 codes as 16-bit values (exact: both types hold every code), times a power of two.
template <int DT>
__device__ __forceinline__ v4u codes8(uint32_t lo, uint32_t hi, float power = 1.0f) {
  if constexpr (DT == DT_BF16)
    return v4u{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, power, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, power, true)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, power, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, power, true))};
  else
    return v4u{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, power, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, power, true)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, power, false)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, power, true))};
}

// Eight e2m1 codes, the first in the low bits, times the power of two of a scale byte (mx4_power).
template <int DT>
__device__ __forceinline__ v4u mx4_values8(uint32_t w, float power) {
  if constexpr (DT == DT_BF16)
    return v4u{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, power, 0)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, power, 1)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, power, 2)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, power, 3))};
  else
    return v4u{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, power, 0)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, power, 1)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, power, 2)),
               __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, power, 3))};
}
__device__ __forceinline__ float mx4_power(uint32_t byte) { return __uint_as_float(byte << 23); }

// fp16 queries over an e4m3 cache.  A weight times its value's scale can lie far outside fp16's range,
// next to another key's above all, so the scale is split into 2^e and the rest: the power of two goes
// to the codes, where it is exact for -14 <= e <= 7 (every code times it is an fp16 number), and the
// rest, 1 to 2 for a scale in that range, to the weight.  So the values are what an fp16 cache would
// hold, no key's scale touches another's product, and a rest or a product beyond fp16 shows as an
// output that is not finite.
constexpr bool splits_scale(int dt, bool codes) { return codes && dt == DT_F16; }
struct SplitScale {
  float power, rest;
};
__device__ __forceinline__ SplitScale split_scale(float scale) {
  const uint32_t e = min(max((__float_as_uint(scale) >> 23) & 0xff, 127u - 14), 127u + 7);
  return {__uint_as_float(e << 23), scale * __uint_as_float((254 - e) << 23)};
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

// The 16 keys from key `at` on (uniform, a multiple of 16, so inside one page) as a buffer whose reads
// past the request's keys, or of a page that is not there, give zeros.
template <int SRC, int D>
__device__ __forceinline__ v4i key_rows(const AttnArgs& a, const Rows& r, const void* base, int h, int at, int page) {
  constexpr int kElem = SRC == SRC_E4M3 ? 1 : 2;
  const bool there = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.pages);
  const int64_t row = ((static_cast<int64_t>(there ? page : 0) * a.hk + h) << a.page_shift) + (at & ((1 << a.page_shift) - 1));
  const int have = there ? min(max(r.len - at, 0), 16) : 0;
  return make_rsrc(static_cast<const char*>(base) + row * (D * kElem), static_cast<uint32_t>(have * D * kElem));
}

// ------------------------------------------------------------------------------------------
// Splitting a long axis.  Few rows over many keys would leave most of the card idle, so the keys
// of a tile of rows are cut into pieces that different workgroups take, each leaving its maximum,
// sum and output, which the last of them joins.  The requests' lengths are on the device, so the
// cut is made there: every workgroup sums the batch's work (three integers a request).
// The most requests whose sums the workgroups hold in LDS.  Above, nothing is cut, which costs nothing
// where requests are alike (1100 e4m3 requests of up to 300 keys: 184 us with a limit of 1024 or 2048)
// and much where one is long (131072 keys among them: 1368 us and 256).
constexpr int kMaxSplitBatch = 1024;
constexpr int kMaxSplitHeads = 1024;
constexpr int kMinKeys = 256;          // no piece below (one request of 701 keys, 32 heads: 128, 256, 512 keys 11.2, 11.5, 17.5 us)
constexpr int kMaxSlots = 4096;        // partial results of a launch

struct Unit {
  Rows r;
  int head;
  int j0, j1;        // its keys
  int piece, count;  // its piece and how many there are of the tile (1: the whole)
  int slot0, slot1, slot_step;   // the tile's partial results: slot0, then slot1 and every slot_step
  __device__ __forceinline__ int64_t slot(int p) const { return p == 0 ? slot0 : slot1 + static_cast<int64_t>(p - 1) * slot_step; }
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
// Whether a batch is cut at all: `capacity` is the most keys a request can have.
__host__ __device__ constexpr bool may_split(int64_t tokens, int64_t group, int64_t batch, int64_t hk, int64_t capacity) {
  return batch <= kMaxSplitBatch && hk <= kMaxSplitHeads && capacity > kMinKeys &&
         tile_bound(tokens, group, batch, 32) * (capacity / kKeys + 1) < (int64_t{1} << 30) / hk;   // steps are counted in int
}

// A request's bounds as the kernels use them.
struct Request {
  int begin, tokens, len;   // first packed token, new tokens (not negative), keys
  bool bad;                 // cu_tokens decreases here
};
template <bool PAGED>
__device__ __forceinline__ Request load_request(const AttnArgs& a, int i) {
  const int lo = a.cu[i], hi = a.cu[i + 1];
  Request q;
  q.begin = min(max(lo, 0), a.tokens);
  q.tokens = max(min(max(hi, 0), a.tokens) - q.begin, 0);
  q.len = PAGED ? min(max(a.lens[i], 0), a.width << a.page_shift) : q.tokens;
  q.bad = hi < lo;
  return q;
}
// Its tiles, and steps of `step` keys that its rows see between them.
struct Shape {
  int tiles, steps, low;   // low: the first key
};
template <int SIZE>
__device__ __forceinline__ Shape shape_of(const AttnArgs& a, const Request& q, int step) {
  Shape s;
  s.tiles = static_cast<int>((static_cast<int64_t>(q.tokens) * a.group + SIZE - 1) / SIZE);
  s.low = a.window > 0 ? max(0, q.len - q.tokens - a.window + 1) & ~(kKeys - 1) : 0;
  s.steps = max(1, (q.len - s.low + step - 1) / step);
  return s;
}

// The inclusive sum of x over a wave: within rows of 16 lanes, then across them.
template <int CTRL, int ROWS>
__device__ __forceinline__ int shifted(int x) { return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, false); }
__device__ __forceinline__ int scan64(int x) {
  x += shifted<0x111, 0xf>(x);      // row_shr 1, 2, 4, 8
  x += shifted<0x112, 0xf>(x);
  x += shifted<0x114, 0xf>(x);
  x += shifted<0x118, 0xf>(x);
  x += shifted<0x142, 0xa>(x);      // row_bcast 15 into rows 1 and 3
  return x + shifted<0x143, 0xc>(x);   // row_bcast 31 into rows 2 and 3
}
// The same over the workgroup's 256 threads; total gets the last one's.
__device__ __forceinline__ int scan256(int x, int* part, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  x = scan64(x);
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

// Inclusive sums over the requests of a number each has: in the lanes of every wave for up to 64
// requests (no barrier), else in LDS (`ends`, kMaxSplitBatch, and `part`, 4 integers).
// A batch whose cu_tokens decreases somewhere has a total of 0: nothing is computed for it.
template <bool PAGED>
struct Sums {
  int *ends, *part;
  int mine, total;
  Request lane_request;    // up to 64 requests: each lane's, loaded once
  __device__ __forceinline__ Sums(const AttnArgs& a, int* lds) : ends(lds), part(lds + kMaxSplitBatch), mine(0), total(0), lane_request{0, 0, 0, false} {
    const int lane = threadIdx.x & 63;
    if (a.batch <= 64 && lane < a.batch) lane_request = load_request<PAGED>(a, lane);
  }
  // Request i (uniform).
  __device__ __forceinline__ Request request(const AttnArgs& a, int i) const {
    Request q = lane_request;
    if (a.batch > 64) q = load_request<PAGED>(a, i);
    const int from = a.batch > 64 ? 0 : i;
    return {__builtin_amdgcn_readlane(q.begin, from), __builtin_amdgcn_readlane(q.tokens, from), __builtin_amdgcn_readlane(q.len, from), false};
  }
  template <typename F>
  __device__ __forceinline__ void make(const AttnArgs& a, F number) {
    bool bad = false;
    if (a.batch <= 64) {
      const int lane = threadIdx.x & 63;
      mine = scan64(lane < a.batch ? number(lane_request) : 0);
      total = __any(lane_request.bad) ? 0 : __builtin_amdgcn_readlane(mine, 63);
      return;
    }
    auto at = [&](int i) {
      const Request q = load_request<PAGED>(a, i);
      bad |= q.bad;
      return number(q);
    };
    int before = 0;
    for (int i0 = 0; i0 < a.batch; i0 += 256) {
      const int i = i0 + threadIdx.x;
      int sum;
      const int e = scan256(i < a.batch ? at(i) : 0, part, sum);
      if (i < a.batch) ends[i] = before + e;
      before += sum;
    }
    total = __syncthreads_or(bad) ? 0 : before;
  }
  // The first request whose sum is above x < total, and the sum up to it (uniform).
  __device__ __forceinline__ int find(int batch, int x, int& end) const {
    if (batch <= 64) {
      const int i = __builtin_ctzll(__ballot(mine > x) | (uint64_t{1} << 63));
      end = __builtin_amdgcn_readlane(mine, i);
      return i;
    }
    int lo = 0, hi = batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (ends[mid] > x) hi = mid;
      else lo = mid + 1;
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    end = __builtin_amdgcn_readfirstlane(ends[lo]);
    return lo;
  }
};

// Tile `tile` of request i.
__device__ __forceinline__ Rows rows_of(const AttnArgs& a, int i, const Request& q, int tile, int size) {
  return {i, q.begin, q.tokens, q.tokens * a.group, tile * size, q.len, q.len - q.tokens};
}

// Packed prompts of up to 64 requests: tile `rank` of them all in the order of their index in their
// request, the last first, so that the tiles that see the most keys start first whatever request
// they are of (hardware starts workgroups in order).  Up to kSlots workgroups are all on the card at
// once, two to a CU: there the second of a CU is the lightest left, not the next.  12 prompts of up to
// 2048 tokens: 59 us so, 64 in the order of the requests.
constexpr int kSlots = 512;
template <int SIZE>
__device__ __forceinline__ bool find_ranked(const AttnArgs& a, Unit& u) {
  const int lane = threadIdx.x & 63;
  u.head = blockIdx.x % a.hk;
  int rank = blockIdx.x / a.hk, tiles = 0, most = 0;
  const Sums<false> requests(a, nullptr);
  if (lane < a.batch) tiles = shape_of<SIZE>(a, requests.lane_request, kKeys).tiles;
  auto sum = [&](int x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
    return __builtin_amdgcn_readfirstlane(x);
  };
  const int total = sum(tiles);
  if (rank >= total) return false;
  const int first = kSlots / 2 / a.hk;
  if (total * a.hk <= kSlots && rank >= first) rank = total - 1 - (rank - first);
  // the largest index k that more than `rank` tiles reach: tiles of index k or above
  int above = 0;
  for (int bit = static_cast<int>(0x80000000u >> __builtin_clz(total)); bit; bit >>= 1) {
    const int n = sum(max(tiles - (most + bit), 0));
    if (n > rank) most += bit;
    else above = n;
  }
  const bool on = tiles > most;
  const uint64_t mask = __ballot(on);
  const int order = __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(mask >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0));
  const int i = __builtin_ctzll(__ballot(on && order == rank - above) | (uint64_t{1} << 63));
  u.r = rows_of(a, i, requests.request(a, i), most, SIZE);
  tile_keys(a, u.r, SIZE, u.j0, u.j1);
  u.piece = 0;
  u.count = 1;
  return true;
}

// The workspace: a counter for every partial result (zero between calls), how many partial results
// a launch for many rows has and of which tiles they are, then the partial results' maxima and sums
// [slot][row][2] and their outputs, float32.  An output lies as the matrix unit leaves it, so that
// whole lines are written: [slot][row / 32][channel / 32][channel % 32 / 8][channel % 8 / 4][row % 32]
// [channel % 4].
constexpr int64_t kCounterBytes = FP8_ATTN_COUNTER_BYTES, kHeadBytes = 16 + 16 * kMaxSlots;
static_assert(kCounterBytes >= 4 * kMaxSlots, "a counter a slot");
struct Partial {
  int request, tile, head, count;   // count 0 in all places of a tile but its first
};
struct Workspace {
  int *counters, *used;
  Partial* partials;
  float* stats;
  float* out;
};
__device__ __forceinline__ Workspace workspace(const AttnArgs& a, int size) {
  Workspace w;
  w.counters = reinterpret_cast<int*>(a.ws);
  w.used = reinterpret_cast<int*>(a.ws + kCounterBytes);
  w.partials = reinterpret_cast<Partial*>(a.ws + kCounterBytes + 16);
  w.stats = reinterpret_cast<float*>(a.ws + kCounterBytes + kHeadBytes);
  w.out = w.stats + static_cast<int64_t>(kMaxSlots) * size * 2;
  return w;
}
__host__ __device__ constexpr int64_t workspace_bytes(int64_t slots, int size, int head_dim) {
  return kCounterBytes + kHeadBytes + int64_t{kMaxSlots} * size * 8 + slots * size * head_dim * 4;
}
// Where four channels 4 quad .. of a row lie in an output of D channels.
template <int D>
__device__ __forceinline__ int64_t partial_at(int row, int quad) {
  return ((row >> 5) * (D / 32) + (quad >> 3)) * 1024 + ((quad >> 1) & 3) * 256 + (quad & 1) * 128 + (row & 31) * 4;
}

// The cut for many rows, where the work of tiles differs (a prompt's last rows see the most keys)
// and the hardware's own order of workgroups balances it: pieces of
//   max(kMinTileKeys, work / kUnits)
// keys, numbered request by request, the tiles that see the most first.  A full batch of equal
// lengths stays uncut.  A second launch joins the partial results: 128 rows of them are too much for
// one workgroup at the end of the first (2 tiles a head over 100000 keys took 2.3 times as long that way).
// One unit a CU rather than the two that fit, since a partial result of 128 rows is 64 KB to write and
// to read: with 512, 256 and 192 units 3442 tokens over up to 16000 keys take 489, 455 and 456 us, 16
// over 100000 110, 99 and 109, 16 x 64 over up to 4096 53, 48 and 51.  Pieces of at least 512 keys: 24
// mixed requests of up to 2000 keys take 26.7 us (e4m3) and 21.1 (16 bits); with 256 27.0 and 21.1, with
// 1024 33.1 and 25.2.
constexpr int kUnits = 256;
constexpr int kMinTileKeys = 512;
// Units per key head are at most the tiles and this many more, and partial results at most twice it.
__host__ __device__ constexpr int64_t extra_units(int64_t hk) { return (kUnits + hk - 1) / hk; }
static_assert(2 * (kUnits + kMaxSplitHeads) <= kMaxSlots, "partial results of the cut for many rows");

// Unit `block` of the launch (block = unit * hk + head).  `lds`: 4 * (kMaxSplitBatch + 4) bytes, free
// again on return.  False where there is none.
template <int SIZE>
__device__ __forceinline__ bool find_unit(const AttnArgs& a, int block, int* lds, Unit& u) {
  u.head = block % a.hk;
  const int unit = block / a.hk;
  Sums<true> sums(a, lds);
  sums.make(a, [&](const Request& q) {
    const Shape s = shape_of<SIZE>(a, q, kKeys);
    return s.tiles * s.steps;
  });
  const int most = max((sums.total * a.hk + kUnits - 1) / kUnits, kMinTileKeys / kKeys);   // steps a piece
  sums.make(a, [&](const Request& q) {
    const Shape s = shape_of<SIZE>(a, q, kKeys);
    return s.tiles * ((s.steps + most - 1) / most);
  });
  if (unit >= sums.total) {
    if (block == 0 && threadIdx.x == 0) *workspace(a, SIZE).used = 0;
    return false;
  }
  int end;
  const int i = sums.find(a.batch, unit, end);
  const Request q = sums.request(a, i);
  const Shape s = shape_of<SIZE>(a, q, kKeys);
  const int pieces = (s.steps + most - 1) / most, tiles = s.tiles;
  const int local = unit - (end - tiles * pieces);
  const int tile = tiles - 1 - local / pieces;
  u.piece = local % pieces;
  u.slot0 = 0;
  if (pieces > 1 || block == 0) {
    sums.make(a, [&](const Request& y) {
      const Shape x = shape_of<SIZE>(a, y, kKeys);
      const int n = (x.steps + most - 1) / most;
      return n > 1 ? x.tiles * n : 0;
    });
    int slots;
    if (a.batch <= 64) slots = __builtin_amdgcn_readlane(sums.mine, i);
    else slots = __builtin_amdgcn_readfirstlane(sums.ends[i]);
    if (pieces > 1) u.slot0 = (slots - tiles * pieces + tile * pieces) * a.hk + u.head;
    if (block == 0 && threadIdx.x == 0) *workspace(a, SIZE).used = sums.total * a.hk;
  }
  if (a.batch > 64) __syncthreads();
  u.r = rows_of(a, i, q, tile, SIZE);
  int j0, j1;
  tile_keys(a, u.r, SIZE, j0, j1);
  const int own = (j1 - j0 + kKeys - 1) / kKeys;
  const int per = max(1, (own + pieces - 1) / pieces);
  u.count = max(1, (own + per - 1) / per);
  u.slot1 = u.slot0 + a.hk;
  u.slot_step = a.hk;
  if (pieces > 1 && threadIdx.x == 0)
    workspace(a, SIZE).partials[u.slot(u.piece)] = {i, tile, u.head, u.piece == 0 && u.count > 1 ? u.count : 0};
  if (u.piece >= u.count) return false;
  u.j0 = j0 + u.piece * per * kKeys;
  u.j1 = min(j1, u.j0 + per * kKeys);
  return true;
}

// The cut for few rows, where the keys are read once and every step costs the same: the batch's
// steps in one line, an equal stretch for each of kFewGroups workgroups (two to a CU: with 256, 512
// and 1024 the 64-request e4m3 batch takes 88.9, 73.9 and 81.7 us, 4 requests of up to 131072 keys 171,
// 179 and 189).
constexpr int kFewGroups = 512;
static_assert(2 * kFewGroups <= kMaxSlots, "partial results of the cut for few rows");

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
// A lane's 16 outputs of 32 channels: `to` the block of its 32 rows and 32 channels.
__device__ __forceinline__ void leave_block(float* to, const v16f& o) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    leave2(to + g * 256 + lane * 4, o[4 * g], o[4 * g + 1]);
    leave2(to + g * 256 + lane * 4 + 2, o[4 * g + 2], o[4 * g + 3]);
  }
}

// A sum of weights and four outputs relative to the largest exponent met.
struct Joined {
  float m, l, o[4];
  __device__ __forceinline__ void add(float m2, float l2, const float* x) {
    const float top = fmaxf(m, m2), base = top == -INFINITY ? 0.0f : top;
    const float f = __builtin_amdgcn_exp2f(m - base), g = __builtin_amdgcn_exp2f(m2 - base);
    l = __builtin_fmaf(g, l2, l * f);
#pragma unroll
    for (int y = 0; y < 4; ++y) o[y] = __builtin_fmaf(g, x[y], o[y] * f);
    m = top;
  }
};

// After a workgroup's partial result is stored: the workgroup that finds itself the last of its
// tile joins them all, in an order that does not depend on who that is:
//   out = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i.
// A thread takes four channels of a row, and has eight pieces' reads in flight (they go to memory, at
// more than a microsecond each); with few rows, several threads share a row's pieces.  `lds` is
// kJoinBytes of LDS that nothing else uses any more.  A place for a partial result holds SIZE rows,
// of which a tile has ROWS at most.
constexpr int kJoinBytes = 16 + 256 * 8 * 4;
template <int DT, int D, int SIZE, int ROWS = SIZE>
__device__ __forceinline__ void join_partials(const AttnArgs& a, const Unit& u, char* lds) {
  constexpr int kPieces = 8;
  int* const flag = reinterpret_cast<int*>(lds);
  float* const shared = reinterpret_cast<float*>(lds + 16) + threadIdx.x * 8;
  const Workspace ws = workspace(a, SIZE);
  const Rows& r = u.r;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // every thread's stores before the count
  __syncthreads();
  if (threadIdx.x == 0) {
    int* n = ws.counters + u.slot0;
    const bool last = __hip_atomic_fetch_add(n, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == u.count - 1;
    if (last) __hip_atomic_store(n, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *flag = last;
  }
  __syncthreads();
  if (!*flag) return;
  const int rows = min(ROWS, r.rows - r.row0);
  int bits = 0;                       // rows, rounded up to a power of two
  while ((1 << bits) < rows) ++bits;
  const int items = (D / 4) << bits;  // item n: row n % 2^bits, channels 4 (n >> bits) .. + 3
  const int share = items < 256 ? 256 / items : 1;
  const int part = share > 1 ? threadIdx.x / items : 0;
#pragma unroll 1
  for (int n = threadIdx.x - part * items; n < items; n += 256) {
    const bool on = (n & ((1 << bits) - 1)) < rows;
    const int row = on ? n & ((1 << bits) - 1) : 0, quad = n >> bits;
    const float* stats = ws.stats + row * 2;
    const float* out = ws.out + partial_at<D>(row, quad);
    Joined j{-INFINITY, 0.0f, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll 1
    for (int i0 = part; i0 < u.count; i0 += kPieces * share) {
      float2 st[kPieces], x[kPieces][2];
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int64_t slot = u.slot(min(i0 + k * share, u.count - 1));
        st[k] = pick2(stats + slot * (SIZE * 2));
        x[k][0] = pick2(out + slot * (SIZE * D));
        x[k][1] = pick2(out + slot * (SIZE * D) + 2);
      }
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const float y[4] = {x[k][0].x, x[k][0].y, x[k][1].x, x[k][1].y};
        if (i0 + k * share < u.count) j.add(st[k].x, st[k].y, y);
      }
    }
    if (share > 1) {    // one pass only
      *reinterpret_cast<v4f*>(shared) = v4f{j.o[0], j.o[1], j.o[2], j.o[3]};
      *reinterpret_cast<float2*>(shared + 4) = make_float2(j.m, j.l);
      __syncthreads();
      if (part != 0) continue;
      for (int k = 1; k < share; ++k) {
        const float* from = shared + k * items * 8;
        j.add(from[4], from[5], from);
      }
    }
    if (!on) continue;
    const int tok = (r.row0 + row) / a.group;
    const int64_t out_row = static_cast<int64_t>(r.begin + tok) * a.hq + u.head * a.group + (r.row0 + row - tok * a.group);
    const bool none = r.pos0 + tok < 0;
    const float inv = none ? 0.0f : 1.0f / j.l;
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + out_row * D + 4 * quad) =
        make_uint2(pack2<DT>(j.o[0] * inv, j.o[1] * inv), pack2<DT>(j.o[2] * inv, j.o[3] * inv));
    if (a.lse && quad == 0) a.lse[out_row] = none ? -INFINITY : (j.m + __builtin_amdgcn_logf(j.l)) * kLn2;
  }
}

// ------------------------------------------------------------------------------------------
// Values that are not finite.  The product with v multiplies a masked key's value by a weight of
// zero, which is right unless that value is infinite or NaN.  A workgroup with a result that is not
// finite goes over its keys once more: such values enter the product as zeros, so rows that do not
// see them get the bits they would have had, and rows that see them, however small the weight, get
// what they hold added afterwards.
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
  // 1 where bit i of `seen` is set.
  static __device__ __forceinline__ v8s ones(uint32_t seen) {
    v8s r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = seen >> i & 1 ? kOne : 0;
    return r;
  }
};

// Eight fp16 values of few bits (codes times powers of two) as bf16.
__device__ __forceinline__ v8s as_bf16(const v8s& x) {
  const v8h h = __builtin_bit_cast(v8h, x);
  v8bf r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = static_cast<__bf16>(static_cast<float>(h[i]));
  return __builtin_bit_cast(v8s, r);
}

// The product of eight keys' values v with their weights z, of type DT; bit i of `seen`: the row sees
// key i (a weight is 0 where it does not).  SPLIT (fp16): weights beyond
// fp16's range are taken out of it, and multiplied as two bf16, their rounding and what it left.
template <int DT, bool SPLIT>
__device__ __forceinline__ v16f mfma_odd(const v8s& v, const float (&z)[8], uint32_t seen, v16f o) {
  float x[8];
  bool any = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool in = !SPLIT || __builtin_fabsf(z[i]) < 65520.0f;     // rounds to an fp16 number; false for NaN
    x[i] = in ? z[i] : 0.0f;
    any |= !in;
  }
  o = mfma<DT>(Odd<DT>::without(v), pack8<DT>(x), o);
  if (SPLIT && __any(any)) {
    float big[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) big[i] = __builtin_fabsf(z[i]) < 65520.0f ? 0.0f : z[i];
    const v8s w = as_bf16(Odd<DT>::without(v)), near = pack8<DT_BF16>(big);
    o = mfma<DT_BF16>(w, near, o);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = static_cast<float>(__builtin_bit_cast(v8bf, near)[i]);
      big[i] = __builtin_isfinite(y) ? big[i] - y : 0.0f;
    }
    o = mfma<DT_BF16>(w, pack8<DT_BF16>(big), o);
  }
  const v8s ones = Odd<DT>::ones(seen);
#pragma unroll 1
  for (int kind = 0; kind < 3; ++kind) {
    v16f n;
    n = 0.0f;
    n = mfma<DT>(Odd<DT>::is(v, kind), ones, n);
    const float add = kind == 0 ? INFINITY : kind == 1 ? -INFINITY : __uint_as_float(kCanonicalNaN);
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] += n[i] > 0.0f ? add : 0.0f;
  }
  return o;
}

// The same for a tile of 16 channels and 16 rows, 32 keys at a time (16x16x32).
template <int DT>
__device__ __forceinline__ v4f mfma16(const v8s& a, const v8s& b, const v4f& c) {
  if constexpr (DT == DT_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}
template <int DT>
__device__ __forceinline__ v4f mfma16_odd(const v8s& v, const v8s& p, uint32_t seen, v4f o) {
  o = mfma16<DT>(Odd<DT>::without(v), p, o);
  const v8s ones = Odd<DT>::ones(seen);
#pragma unroll 1
  for (int kind = 0; kind < 3; ++kind) {
    const v4f n = mfma16<DT>(Odd<DT>::is(v, kind), ones, v4f{0.0f, 0.0f, 0.0f, 0.0f});
    const float add = kind == 0 ? INFINITY : kind == 1 ? -INFINITY : __uint_as_float(kCanonicalNaN);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] += n[i] > 0.0f ? add : 0.0f;
  }
  return o;
}

// Host side: workgroups of a launch for many rows and for few, and the launches.
inline int64_t tile_groups(int64_t tokens, int64_t batch, int64_t group, int64_t hk, bool split) {
  return (tile_bound(tokens, group, batch, 128) + (split ? extra_units(hk) : 0)) * hk;
}
inline int64_t few_groups(int64_t tokens, int64_t batch, int64_t group, int64_t hk, int64_t capacity, bool split) {
  const int64_t tiles = tile_bound(tokens, group, batch, 32) * hk, pieces = tiles * ((capacity + kMinKeys - 1) / kMinKeys);
  if (!split) return tiles;
  return pieces < kFewGroups ? pieces : kFewGroups;   // no more than the pieces have work
}
// Over an mxfp4 cache: tiles of kMx4Rows rows; when cut, a key head's workgroups and all of them.
constexpr int kMx4Rows = 16;
inline int64_t mx4_head_groups(int64_t tokens, int64_t batch, int64_t group, int64_t hk, int64_t capacity) {
  const int64_t pieces = tile_bound(tokens, group, batch, kMx4Rows) * ((capacity + kMinKeys - 1) / kMinKeys);
  const int64_t most = hk < kFewGroups ? kFewGroups / hk : 1;
  return pieces < most ? pieces : most;
}
inline int64_t mx4_groups(int64_t tokens, int64_t batch, int64_t group, int64_t hk, int64_t capacity, bool split) {
  return (split ? mx4_head_groups(tokens, batch, group, hk, capacity) : tile_bound(tokens, group, batch, kMx4Rows)) * hk;
}
static_assert(2 * kFewGroups <= kMaxSlots && 2 * kMaxSplitHeads <= kMaxSlots, "partial results of the cut for few rows");
void launch_attn_tile(int dt, int head_dim, int format, const AttnArgs& a, hipStream_t s);
void launch_attn_few(int dt, int head_dim, bool e4m3, const AttnArgs& a, hipStream_t s);
void launch_attn_mx4_few(int dt, int head_dim, const AttnArgs& a, hipStream_t s);
void launch_attn_join(int dt, int head_dim, const AttnArgs& a, hipStream_t s);   // after launch_attn_tile's

}  // namespace attn
}  // namespace fp8amax
