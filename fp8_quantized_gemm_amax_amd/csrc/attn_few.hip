// attn_few.hip - attention over a paged cache for few packed rows a request and key head (single
// tokens, short drafts, and such next to some chunks), 32 rows at a time: the keys are the work.
//   m' = max(m, max_j s_j), l' = 2^(m - m') l + sum_j 2^(s_j - m'), o' = 2^(m - m') o + sum_j 2^(s_j - m') v_j
// over tiles of keys, s_j = scale log2(e) q.k_j, and out = o / l, all float32; a weight is rounded to
// 16 bits for its product with v.  A workgroup of four waves takes one unit of keys; each wave walks
// over its own tiles of them, through its own LDS without a barrier, for all rows, and the four
// results are joined in LDS at the end.  K of the next tile is under way while V of this one is
// multiplied, V while the next scores are: 16 KB a wave, two workgroups a CU, so 128 KB of reads in
// flight a CU.
// Long caches are bound by HBM: 4 requests of up to 131072 keys, 8 heads of 128 in bf16, 977 MB,
// take 180 us (5.4 TB/s; a plain read of 1 GiB reaches 7.0, a copy 4.9 with its writes); 64 e4m3
// requests of up to 8192 keys, 322 MB, 74 us (4.4 TB/s).  Short ones are bound by a chain of dependent reads of 1
// to 2 us each (lengths, table, K and V, partial results): one request of 701 keys, 32 heads of 128,
// 11.5 MB, takes 11.7 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "attn_device.hpp"

namespace fp8amax {
namespace attn {
namespace {

constexpr int kRows = 32;
// Up to this many keys a tile is not worth cutting: the join costs what walking over them does.  64
// requests of up to 300 keys, e4m3: cut 17.6 us, whole 13.1; of up to 500, 16 bits: 18.5 and 15.2; one
// request of 500: 10.8 and 11.1.  At 768: 16 e4m3 requests of up to 700 keys, cut 11.6, whole 14.5.
constexpr int kWholeKeys = 512;

// One dword from `p` into LDS at to + lane where `on` holds for the lane, 0 where it does not.
__device__ __forceinline__ void dma4_lane(const float* p, float* to, bool on) {
  if (on) asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(p), "{m0}"(lds_addr(to)) : "memory");
  else to[threadIdx.x & 63] = 0.0f;
}

template <int DT, int D, int SRC>
__global__ __launch_bounds__(256, 2) void attn_few_kernel(AttnArgs a, bool split) {
  constexpr bool kCodes = SRC == SRC_E4M3, kSplit = splits_scale(DT, kCodes);
  constexpr int kTileKeys = !kCodes && D == 128 ? 32 : 64;   // keys a wave takes at a time: 8 KB of K (4: codes of 64 channels)
  constexpr int kSub = kTileKeys / 32, kGroups = kTileKeys / 16, kSteps = D / 16;
  constexpr int kRowBytes = kCodes && D == 64 ? 64 : 128;    // of a key in a plane
  constexpr int kPlanes = !kCodes && D == 128 ? 2 : 1;
  constexpr int kPlaneBytes = kTileKeys * kRowBytes, kTile = kPlanes * kPlaneBytes;
  constexpr int kDma = kTile / 1024;                         // DMA instructions of a tile
  static_assert(kJoinBytes <= 8 * kTile, "the join's LDS");
  __shared__ __attribute__((aligned(1024))) char lds[4 * 2 * kTile];
  __shared__ __attribute__((aligned(16))) float scales[kCodes ? 4 : 1][2][64];
  __shared__ __attribute__((aligned(16))) _Float16 powers[kSplit ? 4 : 1][64];
  __shared__ float stats[2][4][32];
  __shared__ int ends[kMaxSplitBatch + 4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, col = lane & 31;
  char* const kt = lds + wave * 2 * kTile;
  char* const vt = kt + kTile;
  const uint32_t kbase = lds_addr(kt), vbase = kbase + kTile;
  float* const my_ks = scales[kCodes ? wave : 0][0];
  float* const my_vs = scales[kCodes ? wave : 0][1];

  // Chunk of 16 bytes at position x of key row i in LDS; rows of 64 bytes hold four.
  auto chunk_of = [](int x, int i) { return kRowBytes == 128 ? x ^ gemm::swz(i & 15) : x ^ ((i >> 1) & 3); };
  uint32_t off[2];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int i = kRowBytes == 128 ? 8 * g + (lane >> 3) : lane >> 2;
    off[g] = i * (kCodes ? D : 2 * D) + chunk_of(lane & (kRowBytes / 16 - 1), i) * 16;
  }
  auto run = [&](const Unit& unit) {
    const Rows& r = unit.r;
    const int h = unit.head, j0 = unit.j0, j1 = unit.j1;
    const int last_row = min(r.row0 + 31, r.rows - 1);
    const int first_pos = r.pos0 + r.row0 / a.group, last_pos = r.pos0 + last_row / a.group;
    const int row = min(r.row0 + col, last_row), tok = row / a.group, pos = r.pos0 + tok;
    const int low = a.window > 0 ? pos - a.window + 1 : 0;
    const uint16_t* qp = static_cast<const uint16_t*>(a.q) + (r.begin + tok) * a.qts + (h * a.group + row - tok * a.group) * a.qhs;
    v8s q[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s)   // codes are read 16 channels at a time: their order over two steps
      q[s] = *reinterpret_cast<const v8s*>(qp + (kCodes ? 32 * (s / 2) + 16 * half + 8 * (s & 1) : 16 * s + 8 * half));

    auto page_of = [&](int at) -> int {
      return at < j1 ? scalar_int(a.table + static_cast<int64_t>(r.request) * a.width + (at >> a.page_shift)) : -1;
    };
    auto bring = [&](const void* p, int t, const int (&pages)[kGroups], uint32_t to) {
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        v4i rs = key_rows<SRC, D>(a, r, p, h, t + 16 * g, pages[g]);
        settle(rs);
#pragma unroll
        for (int x = 0; x < kPlanes; ++x)
#pragma unroll
          for (int y = 0; y < kRowBytes / 64; ++y)
            dma16(rs, to + x * kPlaneBytes + g * 16 * kRowBytes + y * 1024, off[y] + x * 128);
      }
    };
    // The scales of a tile's keys; 0 where there is no key or its page is not in the cache, whose codes read as 0 too.
    auto bring_scales = [&](const float* p, int t, const int (&pages)[kGroups], float* to) {
      int page = pages[0];
#pragma unroll
      for (int g = 1; g < kGroups; ++g) {   // as a value of its own: a choice of addresses would put the array into memory
        const int other = __builtin_amdgcn_readfirstlane(pages[g]);
        page = lane >> 4 == g ? other : page;
      }
      const int at = t + lane;
      const int64_t x = ((static_cast<int64_t>(page) * a.hk + h) << a.page_shift) + (at & ((1 << a.page_shift) - 1));
      dma4_lane(p + x, to, at < r.len && static_cast<uint32_t>(page) < static_cast<uint32_t>(a.pages));
    };

    // this lane's operands in LDS
    const int vr = kCodes ? 4 * half + ((lane >> 1) & 3) + 8 * ((lane >> 3) & 1) : 4 * half + ((lane & 15) >> 2);
    const int vdsub = (lane >> 4) & 1;

    const float c = a.scale * kLog2e;
    v16f o[D / 32];
    float m, l;
    auto walk = [&](auto odd_c) {
      constexpr bool ODD = decltype(odd_c)::value;
      m = -INFINITY;
      l = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o[i] = 0.0f;
      int pages[kGroups];
      int t = j0 + wave * kTileKeys;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) pages[g] = page_of(t + 16 * g);
      if (t < j1) {
        if constexpr (kCodes) bring_scales(a.ks, t, pages, my_ks);
        bring(a.k, t, pages, kbase);
        if constexpr (kCodes) bring_scales(a.vs, t, pages, my_vs);
        bring(a.v, t, pages, vbase);
      }
      for (; t < j1; t += 4 * kTileKeys) {
        const int t1 = t + 4 * kTileKeys;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) pages[g] = page_of(t1 + 16 * g);
        wait_vmcnt<kDma>();      // K and the scales are there: at least the DMAs of V came after them
        asm volatile("" ::: "memory");
        v16f s[kSub];
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
          s[u] = 0.0f;
          const int i = 32 * u + col;
          if constexpr (kCodes) {
#pragma unroll
            for (int x = 0; x < kSteps / 2; ++x) {
              const v4u w = *reinterpret_cast<const v4u*>(kt + i * kRowBytes + (chunk_of(2 * x + half, i) << 4));
              s[u] = mfma<DT>(__builtin_bit_cast(v8s, codes8<DT>(w[0], w[1])), q[2 * x], s[u]);
              s[u] = mfma<DT>(__builtin_bit_cast(v8s, codes8<DT>(w[2], w[3])), q[2 * x + 1], s[u]);
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const v4f x = *reinterpret_cast<const v4f*>(my_ks + 32 * u + 8 * g + 4 * half);
#pragma unroll
              for (int y = 0; y < 4; ++y) s[u][4 * g + y] *= x[y];
            }
          } else {
#pragma unroll
            for (int x = 0; x < kSteps; ++x) {
              const v8s k = *reinterpret_cast<const v8s*>(kt + (x / 4) * kPlaneBytes + i * 128 + (chunk_of(2 * (x & 3) + half, i) << 4));
              s[u] = mfma<DT>(k, q[x], s[u]);
            }
          }
        }
        wait_lds_reads();
        if (t1 < j1) {
          if constexpr (kCodes) bring_scales(a.ks, t1, pages, my_ks);
          bring(a.k, t1, pages, kbase);
        }
        if constexpr (kSplit) {
          const SplitScale y = split_scale(my_vs[lane]);
          my_vs[lane] = y.rest;
          powers[wave][lane] = static_cast<_Float16>(y.power);
        }
        if (t + kTileKeys - 1 > first_pos || (a.window > 0 && t < last_pos - a.window + 1)) {
          const int hi = pos - t - 4 * half, lo = low - t - 4 * half;
#pragma unroll
          for (int u = 0; u < kSub; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int key = 32 * u + 8 * (i / 4) + i % 4;
              s[u][i] = key <= hi && key >= lo ? s[u][i] : -INFINITY;
            }
        }
        uint32_t seen = 0;      // ODD: the keys that this lane's row sees
        if constexpr (ODD) {
#pragma unroll
          for (int i = 0; i < 16 * kSub; ++i) seen |= (s[i / 16][i % 16] == -INFINITY ? 0u : 1u) << i;
        }
        float top = s[0][0];
#pragma unroll
        for (int i = 1; i < 16 * kSub; ++i) top = fmaxf(top, s[i / 16][i % 16]);
        top = max_halves(top) * c;
        if (__any(top > m)) {
          const float m1 = fmaxf(m, top);
          const float keep = m == m1 ? 1.0f : __builtin_amdgcn_exp2f(m - m1);
          m = m1;
          l *= keep;
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int x = 0; x < 16; ++x) o[i][x] *= keep;
        }
        const float mb = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            s[u][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][i], c, -mb));
            l += s[u][i];
          }
        // V is there: at least the DMAs of the next K came after it, if there is one
        if (t1 < j1) wait_vmcnt<kDma>();
        else wait_vmcnt<0>();
        asm volatile("" ::: "memory");
#pragma unroll
        for (int w = 0; w < kTileKeys / 16; ++w) {
          float z[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = s[w / 2][8 * (w & 1) + i];
          if constexpr (kCodes) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const v4f x = *reinterpret_cast<const v4f*>(my_vs + 16 * w + 8 * g + 4 * half);
#pragma unroll
              for (int y = 0; y < 4; ++y) z[4 * g + y] = ODD && !(seen >> (8 * w + 4 * g + y) & 1) ? 0.0f : z[4 * g + y] * x[y];
            }
          }
          const v8s p = pack8<DT>(z);
          v8h power;
          if constexpr (kSplit) {
            typedef _Float16 v4h __attribute__((ext_vector_type(4)));
            power = __builtin_shufflevector(*reinterpret_cast<const v4h*>(powers[wave] + 16 * w + 4 * half),
                                            *reinterpret_cast<const v4h*>(powers[wave] + 16 * w + 4 * half + 8), 0, 1, 2, 3, 4, 5, 6, 7);
          }
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            v8s v;
            if constexpr (kCodes) {
              typedef int v2i __attribute__((ext_vector_type(2)));
              const int key = 16 * w + vr;
              const char* at = vt + key * kRowBytes + (chunk_of(2 * i + vdsub, key) << 4) + (lane & 1) * 8;
              const v2i y = __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) v2i*)at);
              v = __builtin_bit_cast(v8s, codes8<DT>(y[0], y[1]));
              if constexpr (kSplit) v = __builtin_bit_cast(v8s, __builtin_bit_cast(v8h, v) * power);
            } else {
              const int chunk = (i & 1) * 4 + vdsub * 2 + ((lane & 3) >> 1);
              const char* at = vt + (i / 2) * kPlaneBytes + (lane & 1) * 8;
              const int k0 = 16 * w + vr, k1 = k0 + 8;
              const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(at + k0 * 128 + (chunk_of(chunk, k0) << 4)));
              const v4s z = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(at + k1 * 128 + (chunk_of(chunk, k1) << 4)));
              v = __builtin_shufflevector(y, z, 0, 1, 2, 3, 4, 5, 6, 7);
            }
            if constexpr (ODD) o[i] = mfma_odd<DT, kSplit>(v, z, seen >> (8 * w), o[i]);
            else o[i] = mfma<DT>(v, p, o[i]);
          }
        }
        wait_lds_reads();
        if (t1 < j1) {
          if constexpr (kCodes) bring_scales(a.vs, t1, pages, my_vs);
          bring(a.v, t1, pages, vbase);
        }
      }
      l = add_halves(l);
      // join the four waves: wave w adds up channels 32 w .. 32 w + 31 and keeps them in o[0]
      __syncthreads();
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<v4f*>(lds + (wave * (D / 32) + i) * 4096 + g * 1024 + lane * 16) =
              v4f{o[i][4 * g], o[i][4 * g + 1], o[i][4 * g + 2], o[i][4 * g + 3]};
      if (half == 0) {
        stats[0][wave][col] = m;
        stats[1][wave][col] = l;
      }
      __syncthreads();
      float mw[4];
      m = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) m = fmaxf(m, mw[w] = stats[0][w][col]);
      l = 0.0f;
      o[0] = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = mw[w] == m ? 1.0f : __builtin_amdgcn_exp2f(mw[w] - m);
        l = __builtin_fmaf(f, stats[1][w][col], l);
        if (wave < D / 32) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const v4f x = *reinterpret_cast<const v4f*>(lds + (w * (D / 32) + wave) * 4096 + g * 1024 + lane * 16);
#pragma unroll
            for (int y = 0; y < 4; ++y) o[0][4 * g + y] = __builtin_fmaf(f, x[y], o[0][4 * g + y]);
          }
        }
      }
    };
    walk(std::false_type{});
    bool fine = true;
#pragma unroll
    for (int x = 0; x < 16; ++x) fine &= __builtin_isfinite(o[0][x]);
    if (__syncthreads_or(!fine)) walk(std::true_type{});

    const bool mine = wave < D / 32 && r.row0 + col < r.rows;
    if (unit.count > 1) {
      if (mine) {
        const Workspace ws = workspace(a, kRows);
        const int64_t slot = unit.slot(unit.piece);
        if (wave == 0 && half == 0) leave2(ws.stats + (slot * kRows + col) * 2, m, l);
        leave_block(ws.out + slot * (kRows * D) + wave * 1024, o[0]);
      }
      join_partials<DT, D, kRows>(a, unit, lds);
      return;
    }
    if (!mine) return;
    const int64_t out_row = static_cast<int64_t>(r.begin + tok) * a.hq + h * a.group + (row - tok * a.group);
    const float inv = pos < 0 ? 0.0f : 1.0f / l;
    if (a.lse && wave == 0 && half == 0) a.lse[out_row] = pos < 0 ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
    uint16_t* out = static_cast<uint16_t*>(a.out) + out_row * D + 32 * wave + 4 * half;
#pragma unroll
    for (int g = 0; g < 4; ++g)
      *reinterpret_cast<uint2*>(out + 8 * g) = make_uint2(pack2<DT>(o[0][4 * g] * inv, o[0][4 * g + 1] * inv),
                                                          pack2<DT>(o[0][4 * g + 2] * inv, o[0][4 * g + 3] * inv));
  };

  // The work of the batch as one line of steps, head by head, request by request, cut into one equal
  // stretch for each workgroup: a stretch may end one tile, hold others whole and begin the next.
  // Where there are few steps and no tile has more than kWholeKeys, a tile is one step and stays whole.
  // Without cuts a workgroup takes a whole tile.
  constexpr int kStep = 4 * kTileKeys, kLeast = kMinKeys > kStep ? kMinKeys / kStep : 1;
  Sums<true> sums(a, ends);
  int step_keys = kStep, least = kLeast;
  auto make = [&] {
    sums.make(a, [&](const Request& q) {
      const Shape s = shape_of<kRows>(a, q, step_keys);
      return s.tiles * s.steps;
    });
  };
  if (split) {
    make();
    auto longer = [&] {
      const Shape s = shape_of<kRows>(a, sums.lane_request, kStep);
      return lane < a.batch && s.tiles > 0 && s.steps * kStep > kWholeKeys;
    };
    if (a.batch <= 64 && sums.total * a.hk <= 2 * static_cast<int>(gridDim.x) && !__any(longer())) {
      step_keys = 1 << 30;
      least = 1;
      make();
    }
  }
  const int total = split ? sums.total * a.hk : gridDim.x;
  const int each = split ? max((total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x), least) : 1;
  const int to = min(total, static_cast<int>(blockIdx.x + 1) * each);
  for (int from = static_cast<int>(blockIdx.x) * each; from < to;) {
    Unit unit;
    int n = 1;
    if (split) {
      unit.head = from / sums.total;
      int end;
      const int x = from - unit.head * sums.total;
      const int i = sums.find(a.batch, x, end);
      const Request q = sums.request(a, i);
      const Shape s = shape_of<kRows>(a, q, step_keys);
      const int steps = s.steps, local = x - (end - s.tiles * steps), tile = local / steps, step = local - tile * steps;
      n = min(to - from, steps - step);
      unit.r = rows_of(a, i, q, tile, kRows);
      tile_keys(a, unit.r, kRows, unit.j0, unit.j1);
      unit.j0 = max(unit.j0, s.low + step * step_keys);
      unit.j1 = min(unit.j1, s.low + (step + n) * step_keys);
      // the tile's pieces: a workgroup has at most two partial results, of its first tile and its last
      const int begin = from - step, first = begin / each, last = (begin + steps - 1) / each;
      unit.piece = static_cast<int>(blockIdx.x) - first;
      unit.count = last - first + 1;
      unit.slot0 = 2 * first + (begin == first * each ? 0 : 1);
      unit.slot1 = 2 * (first + 1);
      unit.slot_step = 2;
    } else {
      unit.head = blockIdx.x % a.hk;
      if (!find_rows(a, blockIdx.x / a.hk, kRows, true, unit.r)) return;
      tile_keys(a, unit.r, kRows, unit.j0, unit.j1);
      unit.piece = 0;
      unit.count = 1;
    }
    run(unit);
    from += n;
    if (from < to) __syncthreads();   // before the next tile takes the LDS over
  }
}

template <int DT, int D, int SRC>
void launch(const AttnArgs& a, hipStream_t s) {
  const int64_t capacity = static_cast<int64_t>(a.width) << a.page_shift;
  const bool split = may_split(a.tokens, a.group, a.batch, a.hk, capacity);
  const int64_t groups = few_groups(a.tokens, a.batch, a.group, a.hk, capacity, split);
  attn_few_kernel<DT, D, SRC><<<static_cast<unsigned>(groups), 256, 0, s>>>(a, split);
}

template <int SRC>
void launch_typed(int dt, int head_dim, const AttnArgs& a, hipStream_t s) {
  if (dt == DT_BF16) head_dim == 128 ? launch<DT_BF16, 128, SRC>(a, s) : launch<DT_BF16, 64, SRC>(a, s);
  else head_dim == 128 ? launch<DT_F16, 128, SRC>(a, s) : launch<DT_F16, 64, SRC>(a, s);
}

}  // namespace

void launch_attn_few(int dt, int head_dim, bool e4m3, const AttnArgs& a, hipStream_t s) {
  e4m3 ? launch_typed<SRC_E4M3>(dt, head_dim, a, s) : launch_typed<SRC_PAGED>(dt, head_dim, a, s);
}

}  // namespace attn
}  // namespace fp8amax
