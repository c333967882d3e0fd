// attn_mx4.hip - attention over a paged mxfp4 cache for few packed rows a request and key head, 16 or
// 32 rows at a time: the keys are the work.  The recurrence of attn_few.hip,
//   m' = max(m, max_j s_j), l' = 2^(m - m') l + sum_j 2^(s_j - m'), o' = 2^(m - m') o + sum_j 2^(s_j - m') v_j,
// over codes of 4 bits, which the conversion instruction turns into 16-bit numbers with their scale in
// one step.  S^T = K Q^T and O^T = V^T P^T are formed with 16x16x32 products: lane l holds query row
// l % 16 and, in register i of a tile of 16 keys, key 4 (l / 16) + i.
//   K: a key's channels lie in its lanes' order as they are in the page: lane l reads piece l / 16 of
//      key l % 16 (16 keys a load, 1 KB of a page), straight into the product's operand.
//   V: the product wants eight keys of one channel in a lane, and a scale belongs to 32 channels of one
//      key, so V is converted key by key, put into LDS as 16-bit numbers (16 KB a wave) and read with
//      the transposing read.
// A workgroup of four waves takes one unit of keys; each wave walks over its own tiles of 64 without a
// barrier, and the four results are joined in LDS at the end.  The next tile's codes are on their way
// while this one is multiplied.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "attn_device.hpp"

namespace fp8amax {
namespace attn {
namespace {

constexpr int kTileKeys = 64, kGroups = kTileKeys / 16;   // keys a wave takes at a time, 16 to a load

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

template <int DT, int D, int NR>
__global__ __launch_bounds__(256, 2) void attn_mx4_few_kernel(AttnArgs a, bool split) {
  constexpr int kRows = 16 * NR, kSteps = D / 32, kBlocks = D / 16, kWords = D / 32;   // dwords of a piece
  constexpr int kPlaneBytes = kTileKeys * 128, kTile = (D / 64) * kPlaneBytes;
  static_assert(kJoinBytes <= 4 * kTile && NR * kBlocks * 1024 <= kTile, "the joins' LDS");
  __shared__ __attribute__((aligned(1024))) char lds[4 * kTile];
  __shared__ float stats[2][4][kRows];
  __shared__ int ends[kMaxSplitBatch + 4];
  typedef uint32_t Piece __attribute__((ext_vector_type(kWords)));
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int quarter = lane >> 4, col = lane & 15;
  char* const vt = lds + wave * kTile;

  // where this lane's pieces and scale bytes lie in 16 keys of the cache
  const uint32_t koff = col * (D / 2) + quarter * (D / 8), kscale = col * (D / 32) + quarter * (D / 32) / 4;
  const uint32_t voff = lane * (D / 8), vscale = (lane >> 2) * (D / 32) + (lane & 3) * (D / 32) / 4;
  // V in LDS: rows of 64 channels, chunk c of eight of them at c ^ swz(key % 16); where this lane writes
  // (key lane / 4 of 16, chunks from (lane % 4) D / 32 on) and reads (key 4 quarter + lane % 16 / 4)
  const int wkey = lane >> 2, wchunk = (lane & 3) * (D / 32);
  char* const vwrite = vt + (wchunk >> 3) * kPlaneBytes + wkey * 128;
  const int rkey = 4 * quarter + (col >> 2);
  const uint32_t vread = rkey * 128 + ((((lane & 3) >> 1) ^ gemm::swz(rkey)) << 4) + (lane & 1) * 8;

  auto run = [&](const Unit& unit) {
    const Rows& r = unit.r;
    const int h = unit.head, j0 = unit.j0, j1 = unit.j1;
    const int last_row = min(r.row0 + kRows - 1, r.rows - 1);
    const int first_pos = r.pos0 + r.row0 / a.group, last_pos = r.pos0 + last_row / a.group;
    int tok[NR], row[NR], pos[NR], low[NR];
    v8s q[NR][kSteps];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      row[n] = min(r.row0 + 16 * n + col, last_row);
      tok[n] = row[n] / a.group;
      pos[n] = r.pos0 + tok[n];
      low[n] = a.window > 0 ? pos[n] - a.window + 1 : 0;
      const uint16_t* qp = static_cast<const uint16_t*>(a.q) + (r.begin + tok[n]) * a.qts + (h * a.group + row[n] - tok[n] * a.group) * a.qhs;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) q[n][s] = *reinterpret_cast<const v8s*>(qp + quarter * (D / 4) + 8 * s);
    }

    // The cache rows of the 16 keys from key `at` on, which lie in one page; -1 where they are not there.
    auto page_of = [&](int at) -> int {
      return at < j1 ? scalar_int(a.table + static_cast<int64_t>(r.request) * a.width + (at >> a.page_shift)) : -1;
    };
    auto row_of = [&](int at, int page) -> int64_t {
      const bool there = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.pages);
      return there ? ((static_cast<int64_t>(page) * a.hk + h) << a.page_shift) + (at & ((1 << a.page_shift) - 1)) : -1;
    };
    struct Codes {
      Piece c[kGroups];
      uint32_t s[kGroups];
    };
    // A tile's codes and scales.  Sixteen keys of a page are always in the cache, so all are read; those
    // past the request's keys, whose places may hold anything, and those without a page become zeros.
    auto fetch = [&](const void* p, const void* sp, uint32_t off, uint32_t soff, int key, int t, const int64_t (&rows)[kGroups], Codes& to) {
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int64_t at = max(rows[g], int64_t{0});
        to.c[g] = *reinterpret_cast<const Piece*>(static_cast<const char*>(p) + at * (D / 2) + off);
        to.s[g] = *reinterpret_cast<const uint8_t*>(static_cast<const char*>(sp) + at * (D / 32) + soff);
      }
      if (t + kTileKeys > r.len || (rows[0] | rows[1] | rows[2] | rows[3]) < 0) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
          if (rows[g] < 0 || t + 16 * g + key >= r.len) {
            to.c[g] = 0;
            to.s[g] = 127;
          }
      }
    };

    const float c = a.scale * kLog2e;
    v4f o[NR][kBlocks];
    float m[NR], l[NR];
    auto walk = [&](auto odd_c) {
      constexpr bool ODD = decltype(odd_c)::value;
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        m[n] = -INFINITY;
        l[n] = 0.0f;
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) o[n][i] = 0.0f;
      }
      int64_t rows[kGroups];
      int pages[kGroups];
      Codes k, v;
      int t = j0 + wave * kTileKeys;
      if (t < j1) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) rows[g] = row_of(t + 16 * g, page_of(t + 16 * g));
        fetch(a.k, a.ks, koff, kscale, col, t, rows, k);
        fetch(a.v, a.vs, voff, vscale, lane >> 2, t, rows, v);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) pages[g] = page_of(t + 4 * kTileKeys + 16 * g);
      }
      for (; t < j1; t += 4 * kTileKeys) {
        const int t1 = t + 4 * kTileKeys;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) rows[g] = row_of(t1 + 16 * g, pages[g]);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) pages[g] = page_of(t1 + 4 * kTileKeys + 16 * g);
        v4f s[NR][kGroups];
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          const float power = mx4_power(k.s[g]);
#pragma unroll
          for (int n = 0; n < NR; ++n) s[n][g] = 0.0f;
#pragma unroll
          for (int x = 0; x < kSteps; ++x) {
            const v8s key = __builtin_bit_cast(v8s, mx4_values8<DT>(k.c[g][x], power));
#pragma unroll
            for (int n = 0; n < NR; ++n) s[n][g] = mfma16<DT>(key, q[n][x], s[n][g]);
          }
        }
        if (t1 < j1) fetch(a.k, a.ks, koff, kscale, col, t1, rows, k);
        if (t + kTileKeys - 1 > first_pos || (a.window > 0 && t < last_pos - a.window + 1)) {
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            const int hi = pos[n] - t - 4 * quarter, lo = low[n] - t - 4 * quarter;
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[n][g][i] = 16 * g + i <= hi && 16 * g + i >= lo ? s[n][g][i] : -INFINITY;
          }
        }
        uint32_t seen[NR];     // ODD: the keys that this lane's row sees
        v8s p[NR][kTileKeys / 32];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          seen[n] = 0;
          if constexpr (ODD) {
#pragma unroll
            for (int i = 0; i < 16; ++i) seen[n] |= (s[n][i / 4][i % 4] == -INFINITY ? 0u : 1u) << i;
          }
          float top = s[n][0][0];
#pragma unroll
          for (int i = 1; i < 16; ++i) top = fmaxf(top, s[n][i / 4][i % 4]);
          top = max_quarters(top) * c;
          if (__any(top > m[n])) {
            const float m1 = fmaxf(m[n], top);
            const float keep = m[n] == m1 ? 1.0f : __builtin_amdgcn_exp2f(m[n] - m1);
            m[n] = m1;
            l[n] *= keep;
#pragma unroll
            for (int i = 0; i < kBlocks; ++i)
#pragma unroll
              for (int x = 0; x < 4; ++x) o[n][i][x] *= keep;
          }
          const float mb = m[n] == -INFINITY ? 0.0f : m[n];
#pragma unroll
          for (int w = 0; w < kTileKeys / 32; ++w) {
            float z[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              z[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][2 * w + i / 4][i % 4], c, -mb));
              l[n] += z[i];
            }
            p[n][w] = pack8<DT>(z);
          }
        }
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          const float power = mx4_power(v.s[g]);
#pragma unroll
          for (int x = 0; x < kWords; ++x)
            *reinterpret_cast<v4u*>(vwrite + g * 2048 + ((((wchunk & 7) + x) ^ gemm::swz(wkey)) << 4)) = mx4_values8<DT>(v.c[g][x], power);
        }
        if (t1 < j1) fetch(a.v, a.vs, voff, vscale, lane >> 2, t1, rows, v);
        wait_lds_reads();
#pragma unroll
        for (int w = 0; w < kTileKeys / 32; ++w)
#pragma unroll
          for (int i = 0; i < kBlocks; ++i) {
            const char* at = vt + (i / 4) * kPlaneBytes + w * 4096 + (vread ^ ((i & 3) << 5));
            const v4s y0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)at);
            const v4s y1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(at + 2048));
            const v8s y = __builtin_shufflevector(y0, y1, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
            for (int n = 0; n < NR; ++n) {
              if constexpr (ODD) o[n][i] = mfma16_odd<DT>(y, p[n][w], seen[n] >> (8 * w), o[n][i]);
              else o[n][i] = mfma16<DT>(y, p[n][w], o[n][i]);
            }
          }
        wait_lds_reads();     // before the next tile's values take their place
      }
      // join the four waves: wave w adds up blocks w kBlocks / 4 .. of 16 channels and keeps them in front
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        l[n] = add_quarters(l[n]);
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) *reinterpret_cast<v4f*>(lds + ((wave * NR + n) * kBlocks + i) * 1024 + lane * 16) = o[n][i];
        if (quarter == 0) {
          stats[0][wave][16 * n + col] = m[n];
          stats[1][wave][16 * n + col] = l[n];
        }
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        float mw[4];
        m[n] = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) m[n] = fmaxf(m[n], mw[w] = stats[0][w][16 * n + col]);
        l[n] = 0.0f;
#pragma unroll
        for (int i = 0; i < kBlocks / 4; ++i) o[n][i] = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float f = mw[w] == m[n] ? 1.0f : __builtin_amdgcn_exp2f(mw[w] - m[n]);
          l[n] = __builtin_fmaf(f, stats[1][w][16 * n + col], l[n]);
#pragma unroll
          for (int i = 0; i < kBlocks / 4; ++i) {
            const v4f x = *reinterpret_cast<const v4f*>(lds + ((w * NR + n) * kBlocks + wave * (kBlocks / 4) + i) * 1024 + lane * 16);
#pragma unroll
            for (int y = 0; y < 4; ++y) o[n][i][y] = __builtin_fmaf(f, x[y], o[n][i][y]);
          }
        }
      }
    };
    walk(std::false_type{});
    bool fine = true;
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int i = 0; i < kBlocks / 4; ++i)
#pragma unroll
        for (int y = 0; y < 4; ++y) fine &= __builtin_isfinite(o[n][i][y]);
    if (__syncthreads_or(!fine)) walk(std::true_type{});

    if (unit.count > 1) {
      const Workspace ws = workspace(a, 32);
      const int64_t slot = unit.slot(unit.piece);
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        if (r.row0 + 16 * n + col >= r.rows) continue;
        if (wave == 0 && quarter == 0) leave2(ws.stats + (slot * 32 + 16 * n + col) * 2, m[n], l[n]);
#pragma unroll
        for (int i = 0; i < kBlocks / 4; ++i) {
          float* to = ws.out + slot * (32 * D) + partial_at<D>(16 * n + col, 4 * (wave * (kBlocks / 4) + i) + quarter);
          leave2(to, o[n][i][0], o[n][i][1]);
          leave2(to + 2, o[n][i][2], o[n][i][3]);
        }
      }
      join_partials<DT, D, 32, kRows>(a, unit, lds);
      return;
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      if (r.row0 + 16 * n + col >= r.rows) continue;
      const int64_t out_row = static_cast<int64_t>(r.begin + tok[n]) * a.hq + h * a.group + (row[n] - tok[n] * a.group);
      const float inv = pos[n] < 0 ? 0.0f : 1.0f / l[n];
      if (a.lse && wave == 0 && quarter == 0) a.lse[out_row] = pos[n] < 0 ? -INFINITY : (m[n] + __builtin_amdgcn_logf(l[n])) * kLn2;
      uint16_t* out = static_cast<uint16_t*>(a.out) + out_row * D + wave * (D / 4) + 4 * quarter;
#pragma unroll
      for (int i = 0; i < kBlocks / 4; ++i)
        *reinterpret_cast<uint2*>(out + 16 * i) = make_uint2(pack2<DT>(o[n][i][0] * inv, o[n][i][1] * inv), pack2<DT>(o[n][i][2] * inv, o[n][i][3] * inv));
    }
  };
  walk_few<kRows, 4 * kTileKeys>(a, split, ends, run);
}

template <int DT, int D>
void launch(const AttnArgs& a, hipStream_t s) {
  const int64_t capacity = static_cast<int64_t>(a.width) << a.page_shift;
  const bool split = may_split(a.tokens, a.group, a.batch, a.hk, capacity);
  const int rows = mx4_rows(a.tokens, a.group, a.batch);
  const unsigned groups = static_cast<unsigned>(few_groups(a.tokens, a.batch, a.group, a.hk, capacity, split, rows));
  if (rows == 16) attn_mx4_few_kernel<DT, D, 1><<<groups, 256, 0, s>>>(a, split);
  else attn_mx4_few_kernel<DT, D, 2><<<groups, 256, 0, s>>>(a, split);
}

}  // namespace

void launch_attn_mx4_few(int dt, int head_dim, const AttnArgs& a, hipStream_t s) {
  if (dt == DT_BF16) head_dim == 128 ? launch<DT_BF16, 128>(a, s) : launch<DT_BF16, 64>(a, s);
  else head_dim == 128 ? launch<DT_F16, 128>(a, s) : launch<DT_F16, 64>(a, s);
}

}  // namespace attn
}  // namespace fp8amax
