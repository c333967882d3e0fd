// attn_mx4.hip - attention over a paged mxfp4 cache for few packed rows a request and key head, 16 at a
// time: the keys are the work.  The recurrence of attn_few.hip,
//   m' = max(m, max_j s_j), l' = 2^(m - m') l + sum_j 2^(s_j - m'), o' = 2^(m - m') o + sum_j 2^(s_j - m') v_j,
// over codes of 4 bits, which the conversion instruction turns into 16-bit numbers with their scale in
// one step.  S^T = K Q^T and O^T = V^T P^T are formed with 16x16x32 products: lane l holds query row
// l % 16 and, in register i of a group of 16 keys, key 4 (l / 16) + i.
//   K: a key's channels lie in its lanes' order as they are in the page: lane l reads piece l / 16 of
//      key l % 16 (16 keys a load, 1 KB of a page), straight into the product's operand.
//   V: the product wants eight keys of one channel in a lane, and a scale belongs to 32 channels of one
//      key, so V is converted key by key, put into LDS as 16-bit numbers and read with the transposing
//      read, 32 keys at a time.
// A workgroup of four waves takes one unit of keys; each wave walks over its own tiles of 64 without a
// barrier, and the four results are joined in LDS at the end.  The next tile's codes are on their way
// while this one is multiplied.
// Bound by the reads of the cache, 136 bytes a key and head of 128 channels, once their number is large.
// Measured on one card, 32 heads on 8 of 128 channels, bf16, one new token a request, everything from
// memory: 16, 32, 64 and 128 requests of 4096 to 8192 keys 28.1, 49.6, 89.2 and 170 us (104, 210, 429 and 870
// MB), four of 32768, 65536 and 131072 34.7, 59.5 and 109 us (143, 285 and 570 MB): 5.5 and 5.8 TB/s for what
// is added, and some 10 us that do not depend on the keys: the launch, the cut (one microsecond), the first
// reads' latency, the join of the waves and of the pieces.  One request of 701 keys 8.4 us.  Every 16 rows of
// a request are a tile of their own, which reads the keys again: 64 requests of 2000 to 4000 keys, 4, 8, 16, 32
// and 48 rows 51.5, 52.1, 55.2, 85.9 and 115 us.  Of other arrangements, one wider (32 rows for a tile of 64
// keys) spilled and took 153 us where two passes over 16 rows take 65; a second tile on its way, three waves a
// SIMD, eight waves a workgroup and 768 to 2048 workgroups were all slower than this with two workgroups a CU.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "attn_device.hpp"

namespace fp8amax {
namespace attn {
namespace {

constexpr int kWaves = 4, kRows = kMx4Rows;
constexpr int kTileKeys = 64, kGroups = kTileKeys / 16;   // keys a wave takes at a time, 16 to a load
constexpr int kStep = kWaves * kTileKeys;                 // and the workgroup: the least that is cut off
static_assert(kStep == kMinKeys, "pieces of the cut");
// Up to this many keys a tile is not worth cutting.  One request over 4 key heads, 400, 701 and 1000 keys:
// whole 8.7, 10.2 and 12.0 us, cut 9.0, 9.2 and 9.4; 16 requests over 8: whole 9.1, 10.8 and 15.3, cut
// 11.8, 12.9 and 13.0.  Up to 64 requests, whose lengths are in the lanes: 64 of 450 keys over two key heads
// 9.2 us, 65 13.4, over one 9.2 and 11.0.
constexpr int kWholeKeys = 512;
// What a tile costs a workgroup besides its keys (finding it, its queries, the first codes' latency, the
// join and the result: 3.7 us, measured inside 64 requests' step), in steps; counted where a workgroup has
// kManySteps of them or more.  With it and without, 32 heads: 64 ragged requests of up to 8192 keys 49.4
// and 52.8 us, 128 of them 92.2 and 95.6, 32 of up to 2048 with a key head a head 34.5 and 40.4, 64 of up
// to 4096 over 4 heads of 64 channels 16.8 and 20.2.  From two steps on rather than three, 64 of up to 3000
// over 4 heads of 128: 18.6, not 21.7, 16 of 2000 keys each, two whole steps a workgroup: 16.9, not 15.1.
template <int D>
constexpr int kTileCost = D == 64 ? 2 : 1;
constexpr int kManySteps = 2;
// The last of a tile's workgroups reads its pieces eight at a time, each time at memory's latency, so a tile
// of more than kManyPieces is cut into longer ones, up to the square root of a kPieceLength-th of its steps:
// one request of 131072 keys over one key head 30.9 us, in 512 pieces 78.6; of 20635 over four heads 22.1
// (26.1 in 81), of 60000 over eight 31.1 (34.8).  With 16 pieces and 64 and lengths of a 2nd and a 4th the
// same calls took 31 to 41, 22 to 24 and 31 to 34 us.  Up to 64 requests, as above: one of 131072 keys among ones
// of 100, over one key head 37.9 us with 64 requests and 70.6 with 65, over four 35.4 and 37.4.
constexpr int kManyPieces = 24, kPieceLength = 8;
#define FP8_GLOBAL __attribute__((address_space(1)))

// x / d by d's reciprocal, x and d not negative: the quotient is off by one or two where it is below 2^22.
__device__ __forceinline__ int quotient(int x, int d, float inverse) {
  int q = static_cast<int>(static_cast<float>(x) * inverse), r = x - q * d;
  while (r < 0) { --q; r += d; }
  while (r >= d) { ++q; r -= d; }
  return q;
}
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Largest and sum over the four lanes l % 16 + {0, 16, 32, 48}.
__device__ __forceinline__ float max_quarters(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return max_halves(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float add_quarters(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return add_halves(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

template <int DT, int D>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_mx4_few_kernel(AttnArgs a, bool split) {
  constexpr int kSteps = D / 32, kBlocks = D / 16, kWords = D / 32;   // dwords of a piece
  // 32 keys' values, 16 bits; the second 64 channels a row further, so that they use the other banks
  constexpr int kPlaneBytes = 32 * 128 + 128, kHalf = (D / 64) * kPlaneBytes;
  constexpr int kOwn = kBlocks / kWaves;                              // blocks of a wave in the join
  static_assert(kHalf >= kBlocks * 1024 && kWaves * kHalf >= kJoinBytes, "the joins' LDS");
  __shared__ __attribute__((aligned(1024))) char lds[kWaves * kHalf];
  __shared__ float stats[2][kWaves][kRows];
  __shared__ int ends[kMaxSplitBatch + 4];
  typedef uint32_t Piece __attribute__((ext_vector_type(kWords)));
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int quarter = lane >> 4, col = lane & 15;
  char* const vt = lds + wave * kHalf;
  const float per_group = 1.0f / static_cast<float>(a.group);
  auto token_of = [&](int row) { return quotient(row, a.group, per_group); };

  // where this lane's pieces and scale bytes lie in 16 keys of the cache
  const uint32_t koff = col * (D / 2) + quarter * (D / 8), kscale = col * (D / 32) + quarter * (D / 32) / 4;
  const uint32_t voff = lane * (D / 8), vscale = (lane >> 2) * (D / 32) + (lane & 3) * (D / 32) / 4;
  // V in LDS, 32 keys at a time: rows of 64 channels, chunk c of eight of them at c ^ swz(key % 16); where
  // this lane writes (key lane / 4 of 16, chunks from (lane % 4) D / 32 on) and reads (key 4 quarter + lane % 16 / 4)
  const int wkey = lane >> 2, wchunk = (lane & 3) * (D / 32);
  char* const vwrite = vt + (wchunk >> 3) * kPlaneBytes + wkey * 128;
  const int rkey = 4 * quarter + (col >> 2);
  const char* const vread = vt + rkey * 128 + (lane & 1) * 8;
  const int rchunk = ((lane & 3) >> 1) ^ gemm::swz(rkey);

  auto run = [&](const Unit& unit) {
    const Rows& r = unit.r;
    const int h = unit.head, j0 = unit.j0, j1 = unit.j1;
    const int last_row = min(r.row0 + kRows - 1, r.rows - 1);
    const int row = min(r.row0 + col, last_row), tok = token_of(row), pos = r.pos0 + tok;
    const int first_pos = __builtin_amdgcn_readlane(pos, 0), last_pos = __builtin_amdgcn_readlane(pos, 15);
    v8s q[kSteps];
    const uint16_t* qp = static_cast<const uint16_t*>(a.q) + (r.begin + tok) * a.qts + (h * a.group + row - tok * a.group) * a.qhs;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) q[s] = *reinterpret_cast<const v8s*>(qp + quarter * (D / 4) + 8 * s);

    // A tile's four groups of 16 keys, each in one page: the pages' numbers, and from them the groups'
    // places in the cache, counted in groups (a cache has 2^40 numbers at most, so 2^30 of them); a group
    // whose page is not in the cache gets place 0 and a bit in `holes`.  Pages of 64 keys or more hold a
    // tile whole: one number.
    const bool whole = a.page_shift >= 6;
    const uint32_t page_groups = static_cast<uint32_t>(a.hk) << (a.page_shift - 4), head_groups = static_cast<uint32_t>(h) << (a.page_shift - 4);
    const int* const table = a.table + static_cast<int64_t>(r.request) * a.width;
    auto pages_of = [&](int t, int (&pages)[kGroups]) {
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        if (g > 0 && whole) break;
        pages[g] = scalar_int(table + (min(t + 16 * g, j1 - 1) >> a.page_shift));   // past the unit's keys: its last page, masked
      }
    };
    struct Place {
      uint32_t group[kGroups], holes;
    };
    auto place = [&](int t, const int (&pages)[kGroups]) -> Place {
      Place to;
      to.holes = 0;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        if (g > 0 && whole) break;
        const uint32_t page = uniform(pages[g]);
        const bool there = page < static_cast<uint32_t>(a.pages);
        to.holes |= there ? 0u : (whole ? 15u : 1u << g);
        to.group[g] = (there ? page : 0u) * page_groups + head_groups + (((t + 16 * g) & ((1 << a.page_shift) - 1)) >> 4);
      }
      return to;
    };
    struct Codes {
      Piece c[kGroups];
      uint32_t s[kGroups];     // whole dwords: of a byte, the compiler masks what it has just asked for, and waits
    };
    // A tile's codes and scales.  Sixteen keys of a page are always in the cache, so all are read; those
    // past the request's keys, whose places may hold anything, and those without a page become zeros.
    auto fetch = [&](const void* p, const void* sp, uint32_t off, uint32_t soff, const Place& at, Codes& to) {
      soff &= ~3u;
      asm("" : "+v"(off), "+v"(soff));      // scalar bases and a lane's 32-bit offsets
      auto read = [&](const FP8_GLOBAL char* codes, const FP8_GLOBAL char* scales, int g, int skip) {
        to.c[g] = *reinterpret_cast<const FP8_GLOBAL Piece*>(codes + off + skip * (16 * D / 2));
        to.s[g] = *reinterpret_cast<const FP8_GLOBAL uint32_t*>(scales + soff + skip * (16 * D / 32));
      };
      auto base = [&](const void* p, uint32_t group, int bytes) {
        const FP8_GLOBAL char* from = (const FP8_GLOBAL char*)p + static_cast<uint64_t>(group) * bytes;
        asm("" : "+s"(from));
        return from;
      };
      if (whole) {
        const auto* codes = base(p, at.group[0], 16 * D / 2);
        const auto* scales = base(sp, at.group[0], 16 * D / 32);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) read(codes, scales, g, g);
      } else {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) read(base(p, at.group[g], 16 * D / 2), base(sp, at.group[g], 16 * D / 32), g, 0);
      }
    };
    auto clear = [&](int key, int t, uint32_t holes, Codes& to) {
      if (t + kTileKeys <= r.len && holes == 0) return;
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
        if ((holes >> g & 1) != 0 || t + 16 * g + key >= r.len) {
          to.c[g] = 0;
          to.s[g] = 127u * 0x01010101u;
        }
    };
    // Scores of a tile's keys, 16 a group.
    auto score = [&](const Codes& k, v4f (&s)[kGroups]) {
      float power[kGroups];
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        power[g] = mx4_power(k.s[g] >> (8 * (kscale & 3)) & 0xff);
        s[g] = 0.0f;
      }
#pragma unroll
      for (int x = 0; x < kSteps; ++x)
#pragma unroll
        for (int g = 0; g < kGroups; ++g) s[g] = mfma16<DT>(__builtin_bit_cast(v8s, mx4_values8<DT>(k.c[g][x], power[g])), q[x], s[g]);
    };
    auto mask = [&](int t, v4f (&s)[kGroups]) {
      if (t + kTileKeys - 1 <= first_pos && !(a.window > 0 && t < last_pos - a.window + 1)) return;
      const int hi = pos - t - 4 * quarter, lo = a.window > 0 ? hi - a.window + 1 : -t - 4 * quarter;
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[g][i] = 16 * g + i <= hi && 16 * g + i >= lo ? s[g][i] : -INFINITY;
    };
    // 32 of a tile's values into LDS, and eight keys of a block of 16 channels out of it.
    auto put = [&](const Codes& v, int w) {
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const float power = mx4_power(v.s[2 * w + g] >> (8 * (vscale & 3)) & 0xff);
#pragma unroll
        for (int x = 0; x < kWords; ++x)
          *reinterpret_cast<v4u*>(vwrite + g * 2048 + ((((wchunk & 7) + x) ^ gemm::swz(wkey)) << 4)) = mx4_values8<DT>(v.c[2 * w + g][x], power);
      }
    };
    auto take = [&](int i) -> v8s {
      const char* at = vread + (i / 4) * kPlaneBytes + ((rchunk ^ ((i & 3) << 1)) << 4);
      const v4s y0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)at);
      const v4s y1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(at + 2048));
      return __builtin_shufflevector(y0, y1, 0, 1, 2, 3, 4, 5, 6, 7);
    };

    const float c = a.scale * kLog2e;
    v4f o[kBlocks];
    float m, l;
    // A tile's weights from its scores: the running maximum and what it rescales, the sum.
    auto weigh = [&](auto& o, const v4f (&s)[kGroups], v8s (&p)[kTileKeys / 32]) {
      float top = s[0][0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i / 4][i % 4]);
      top = max_quarters(top) * c;
      if (__any(top > m)) {
        const float m1 = fmaxf(m, top);
        const float keep = m == m1 ? 1.0f : __builtin_amdgcn_exp2f(m - m1);
        m = m1;
        l *= keep;
#pragma unroll
        for (auto& block : o)
#pragma unroll
          for (int x = 0; x < 4; ++x) block[x] *= keep;
      }
      const float mb = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int w = 0; w < kTileKeys / 32; ++w) {
        float z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          z[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * w + i / 4][i % 4], c, -mb));
          l += z[i];
        }
        p[w] = pack8<DT>(z);
      }
    };
    auto walk = [&]() {
      m = -INFINITY;
      l = 0.0f;
#pragma unroll
      for (int i = 0; i < kBlocks; ++i) o[i] = 0.0f;
      int pages[kGroups];
      Codes k, v;
      Place at;
      int t = j0 + wave * kTileKeys;
      if (t < j1) {
        pages_of(t, pages);
        at = place(t, pages);
        fetch(a.k, a.ks, koff, kscale, at, k);
        fetch(a.v, a.vs, voff, vscale, at, v);
        pages_of(t + kStep, pages);
      }
      // The queries arrive here: still on their way in the loop, they would be waited for there, and every
      // load behind them with them.
#pragma unroll
      for (int s = 0; s < kSteps; ++s) asm volatile("" : "+v"(q[s]));
      // One tile; MORE: the wave has another one behind it, whose codes are fetched meanwhile.  (As a
      // condition inside, the waits would have to fit both ways, and those for V would be for the next K.)
      auto step = [&](auto more_c) {
        constexpr bool MORE = decltype(more_c)::value;
        const uint32_t holes = at.holes;
        if constexpr (MORE) {
          at = place(t + kStep, pages);
          __builtin_amdgcn_sched_barrier(0);     // scalar loads return in any order: a wait for these would be for the next
          pages_of(t + 2 * kStep, pages);
        }
        clear(col, t, holes, k);
        clear(lane >> 2, t, holes, v);
        v4f s[kGroups];
        score(k, s);
        // The first half's values go through LDS while the scores come out of the matrix unit and the
        // weights are formed.  A wave's LDS accesses take effect in their order, so the second half's
        // values are written behind the first half's reads without a wait.
        v8s y[kBlocks];
        put(v, 0);
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) y[i] = take(i);
        put(v, 1);
        if constexpr (MORE) {
          fetch(a.k, a.ks, koff, kscale, at, k);
          fetch(a.v, a.vs, voff, vscale, at, v);
        }
        mask(t, s);
        v8s p[kTileKeys / 32];
        weigh(o, s, p);
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
          o[i] = mfma16<DT>(y[i], p[0], o[i]);
          y[i] = take(i);
        }
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) o[i] = mfma16<DT>(y[i], p[1], o[i]);
        t += kStep;
      };
      while (t + kStep < j1) step(std::true_type{});
      if (t < j1) step(std::false_type{});
    };
    // Once more, with the values that are not finite kept apart: 16 channels at a time and one tile after
    // the other (few registers, so that the code above keeps its own).
    auto walk_odd = [&]() {
#pragma unroll 1
      for (int x = 0; x < kBlocks; ++x) {
        v4f part[1];
        m = -INFINITY;
        l = 0.0f;
        part[0] = 0.0f;
#pragma unroll 1
        for (int t = j0 + wave * kTileKeys; t < j1; t += kStep) {
          int pages[kGroups];
          pages_of(t, pages);
          const Place at = place(t, pages);
          Codes codes;
          fetch(a.k, a.ks, koff, kscale, at, codes);
          clear(col, t, at.holes, codes);
          v4f s[kGroups];
          score(codes, s);
          fetch(a.v, a.vs, voff, vscale, at, codes);
          mask(t, s);
          const int hi = pos - t - 4 * quarter, lo = a.window > 0 ? hi - a.window + 1 : -t - 4 * quarter;
          uint32_t seen = 0;       // by the keys' places: also one whose score is -infinity
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int key = 16 * (i / 4) + i % 4;
            seen |= (key <= hi && key >= lo ? 1u : 0u) << i;
          }
          v8s p[kTileKeys / 32];
          weigh(part, s, p);
          clear(lane >> 2, t, at.holes, codes);
#pragma unroll
          for (int w = 0; w < kTileKeys / 32; ++w) {
            put(codes, w);
            part[0] = mfma16_odd<DT>(take(x), p[w], seen >> (8 * w), part[0]);
          }
        }
#pragma unroll
        for (int y = 0; y < kBlocks; ++y)
          if (y == x) o[y] = part[0];
      }
    };
    // Joins the waves: wave w adds up the blocks of 16 channels from w kOwn on and keeps them in front.
    auto join = [&]() {
      __syncthreads();
      l = add_quarters(l);
#pragma unroll
      for (int i = 0; i < kBlocks; ++i) *reinterpret_cast<v4f*>(lds + (wave * kBlocks + i) * 1024 + lane * 16) = o[i];
      if (quarter == 0) {
        stats[0][wave][col] = m;
        stats[1][wave][col] = l;
      }
      __syncthreads();
      float mw[kWaves];
      m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) m = fmaxf(m, mw[w] = stats[0][w][col]);
      l = 0.0f;
#pragma unroll
      for (int i = 0; i < kOwn; ++i) o[i] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = mw[w] == m ? 1.0f : __builtin_amdgcn_exp2f(mw[w] - m);
        l = __builtin_fmaf(f, stats[1][w][col], l);
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
          const v4f x = *reinterpret_cast<const v4f*>(lds + (w * kBlocks + wave * kOwn + i) * 1024 + lane * 16);
#pragma unroll
          for (int y = 0; y < 4; ++y) o[i][y] = __builtin_fmaf(f, x[y], o[i][y]);
        }
      }
    };
    walk();
    join();
    bool fine = true;
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
#pragma unroll
      for (int y = 0; y < 4; ++y) fine &= __builtin_isfinite(o[i][y]);
    if (__syncthreads_or(!fine)) {
      walk_odd();
      join();
    }

    if (unit.count > 1) {
      if (r.row0 + col < r.rows) {
        const Workspace ws = workspace(a, 32);
        const int64_t slot = unit.slot(unit.piece);
        if (wave == 0 && quarter == 0) leave2(ws.stats + (slot * 32 + col) * 2, m, l);
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
          float* to = ws.out + slot * (32 * D) + partial_at<D>(col, 4 * (wave * kOwn + i) + quarter);
          leave2(to, o[i][0], o[i][1]);
          leave2(to + 2, o[i][2], o[i][3]);
        }
      }
      join_partials<DT, D, 32, kRows>(a, unit, lds);
      return;
    }
    if (r.row0 + col >= r.rows) return;
    const int64_t out_row = static_cast<int64_t>(r.begin + tok) * a.hq + h * a.group + (row - tok * a.group);
    const float inv = pos < 0 ? 0.0f : 1.0f / l;
    if (a.lse && wave == 0 && quarter == 0) a.lse[out_row] = pos < 0 ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
    uint16_t* out = static_cast<uint16_t*>(a.out) + out_row * D + wave * (16 * kOwn) + 4 * quarter;
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      *reinterpret_cast<uint2*>(out + 16 * i) = make_uint2(pack2<DT>(o[i][0] * inv, o[i][1] * inv), pack2<DT>(o[i][2] * inv, o[i][3] * inv));
  };

  if (!split) {      // a workgroup takes a whole tile
    Unit unit;
    unit.head = blockIdx.x % a.hk;
    if (!find_rows(a, blockIdx.x / a.hk, kRows, true, unit.r)) return;
    tile_keys(a, unit.r, kRows, unit.j0, unit.j1);
    unit.piece = 0;
    unit.count = 1;
    run(unit);
    return;
  }
  // The work of a key head (blockIdx.y) as one line of steps, request by request, in tiles of kRows rows,
  // cut into stretches that differ by a step at most, one for each of the head's workgroups: a stretch may
  // end one tile, hold others whole and begin the next.  Where there are many steps, a tile begins with
  // `cost` steps without keys, so that a workgroup with more tiles has fewer keys.  Where there are few steps
  // and no tile has more than kWholeKeys, a tile is one step and stays whole.  Every workgroup makes the cut for itself; a
  // division costs as much as a tenth of a tile, so there are few, by reciprocals.
  Sums<true> sums(a, ends);
  bool cut_tiles = true;
  int cost = 0;
  auto shape = [&](const Request& q) {
    Shape s;
    s.tiles = static_cast<int>((static_cast<int64_t>(q.tokens) * a.group + kRows - 1) / kRows);
    s.low = a.window > 0 ? max(0, q.len - q.tokens - a.window + 1) & ~(kKeys - 1) : 0;
    s.steps = cut_tiles ? max(1, (q.len - s.low + kStep - 1) / kStep) : 1;
    return s;
  };
  auto work = [&](const Request& q) {
    const Shape s = shape(q);
    return s.tiles * (s.steps + cost);
  };
  sums.make(a, work);
  const int groups = gridDim.x;
  if (sums.total / kManySteps >= groups) {
    cost = kTileCost<D>;
    sums.make(a, work);
  }
  if (a.batch <= 64 && sums.total <= 2 * groups) {
    const Shape s = shape(sums.lane_request);
    if (!__any(lane < a.batch && s.tiles > 0 && s.steps * kStep > kWholeKeys)) {
      cut_tiles = false;
      sums.make(a, work);
    }
  }
  const int total = sums.total;
  // Workgroup b has the steps from cut(b) to cut(b + 1), `each` of them, the first `more` one more.
  int each = max(uniform(quotient(total, groups, 1.0f / static_cast<float>(groups))), 1);
  if (a.batch <= 64 && groups > kManyPieces) {
    const Shape s = shape(sums.lane_request);
    while (__any(lane < a.batch && s.tiles > 0 && (s.steps - 1) / kManyPieces >= each &&
                 (s.steps - 1) / kPieceLength >= static_cast<int64_t>(each) * each)) ++each;
  }
  const int more = max(total - each * groups, 0), b = blockIdx.x;
  const float per_each = 1.0f / static_cast<float>(each), per_wide = 1.0f / static_cast<float>(each + 1);
  auto cut = [&](int b) { return b * each + min(b, more); };
  auto owner = [&](int x) {
    const int wide = more * (each + 1);
    return uniform(x < wide ? quotient(x, each + 1, per_wide) : more + quotient(x - wide, each, per_each));
  };
  const int begin = cut(b), to = min(total, cut(b + 1));
  for (int from = begin; from < to;) {
    Unit unit;
    unit.head = blockIdx.y;
    int end;
    const int i = sums.find(a.batch, from, end);
    const Request q = sums.request(a, i);
    const Shape s = shape(q);
    const int all = s.steps + cost, local = from - (end - s.tiles * all);
    const int tile = uniform(quotient(local, all, 1.0f / static_cast<float>(all))), at = local - tile * all;
    const int n = min(to - from, all - at);      // of them `cost` without keys in front
    const int start = from - at, stop = start + all;
    from += n;
    if (at + n <= cost) continue;                // (then the stretch ends here)
    const int step = max(at - cost, 0), steps = at + n - cost - step;
    unit.r = rows_of(a, i, q, tile, kRows);
    const int last = uniform(token_of(min(unit.r.row0 + kRows, unit.r.rows) - 1));
    const int low = a.window > 0 ? max(0, unit.r.pos0 + uniform(token_of(unit.r.row0)) - a.window + 1) : 0;
    unit.j1 = max(unit.r.pos0 + last + 1, 0);
    unit.j0 = min(low, unit.j1) & ~(kKeys - 1);
    if (cut_tiles) {
      unit.j0 = max(unit.j0, s.low + step * kStep);
      unit.j1 = min(unit.j1, s.low + (step + steps) * kStep);
    }
    // the tile's pieces: a workgroup has at most two partial results, of its first tile and its last
    const int first = start + cost >= begin ? b : owner(start + cost), final = stop <= cut(b + 1) ? b : owner(stop - 1);
    const int slots = 2 * static_cast<int>(blockIdx.y) * groups;
    unit.piece = b - first;
    unit.count = final - first + 1;
    unit.slot0 = slots + 2 * first + (start <= cut(first) ? 0 : 1);
    unit.slot1 = slots + 2 * (first + 1);
    unit.slot_step = 2;
    run(unit);
    if (from < to) __syncthreads();   // before the next tile takes the LDS over
  }
}

template <int DT, int D>
void launch(const AttnArgs& a, hipStream_t s) {
  const int64_t capacity = static_cast<int64_t>(a.width) << a.page_shift;
  const bool split = may_split(a.tokens, a.group, a.batch, a.hk, capacity);
  const dim3 grid = split ? dim3(static_cast<unsigned>(mx4_head_groups(a.tokens, a.batch, a.group, a.hk, capacity)), a.hk)
                          : dim3(static_cast<unsigned>(mx4_groups(a.tokens, a.batch, a.group, a.hk, capacity, false)));
  attn_mx4_few_kernel<DT, D><<<grid, 64 * kWaves, 0, s>>>(a, split);
}

}  // namespace

void launch_attn_mx4_few(int dt, int head_dim, const AttnArgs& a, hipStream_t s) {
  if (dt == DT_BF16) head_dim == 128 ? launch<DT_BF16, 128>(a, s) : launch<DT_BF16, 64>(a, s);
  else head_dim == 128 ? launch<DT_F16, 128>(a, s) : launch<DT_F16, 64>(a, s);
}

}  // namespace attn
}  // namespace fp8amax
