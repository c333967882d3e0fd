// attn_tile.hip - attention for many rows: a workgroup of four waves takes 128 packed rows (32 a
// wave) of one key head and walks over the keys in tiles of 64 that all four waves share in LDS.
//   S^T = K Q^T, P^T = 2^(c S^T - m), l += sum P, O^T += V^T P^T, c = scale log2(e),
// one pass with a running maximum m; S, l, m and O are float32 in registers, P is rounded to 16 bits
// for its product with V, and O / l once to the output's type.
// Per tile and wave, 128 channels: 32 MFMAs of 32 cycles each and 187 vector instructions, 32 of them
// exponentials of 8 cycles, so the matrix and the vector unit are both in demand; tile i's weights are
// formed while tile i + 1's keys and the weights that are ready are multiplied (3% of 16384 tokens'
// time).  64 KB of LDS a workgroup, so two share a CU and one's barriers hide behind the
// other's work; one workgroup a CU with tiles further ahead, or with two teams of four waves that
// take turns, was slower.
// Measured on one card, 32 heads on 8 of 128 channels, bf16: 16384 tokens 2.02 ms, 1090 TFLOP/s, where a
// library product of 8192^3 reaches 1240: power bounds both, with inputs of zeros they run at 1528 and
// 1768.  12 packed prompts of up to 2048 tokens 58 us: 41 steps of 64 keys a CU at 0.95 us where two
// workgroups share it are 39 us, the rest is that the longest tiles, 32 steps, share to their end.  3442
// new tokens of four requests over up to 16000 cached keys 455 us (1032 TFLOP/s).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "attn_device.hpp"

namespace fp8amax {
namespace attn {
namespace {

constexpr int kWaves = 4;
constexpr int kRows = 32 * kWaves;
// The running maximum follows a larger score only past this much (in powers of two): weights are then
// at most 2^8 rather than 1, which float32 sums and 16-bit weights hold as well, and most tiles leave
// o as it is.  Without slack (0) 16384 tokens take 2058 us instead of 1988, 3442 over up to 16000 keys
// 472 instead of 455 (one card).
constexpr float kSlack = 8.0f;

// The workgroup's unit: cut from the batch's work (find_unit) or a whole tile of rows.
template <int SIZE, bool PAGED>
__device__ __forceinline__ bool unit_of(const AttnArgs& a, bool split, char* lds, Unit& u) {
  if constexpr (PAGED) {
    if (split) return find_unit<SIZE>(a, blockIdx.x, reinterpret_cast<int*>(lds), u);
  } else {
    if (a.batch <= 64) return find_ranked<SIZE>(a, u);
  }
  u.head = blockIdx.x % a.hk;
  // heavy tiles first: a prompt's last rows see the most keys
  if (!find_rows(a, gridDim.x / a.hk - 1 - blockIdx.x / a.hk, SIZE, PAGED, u.r)) return false;
  tile_keys(a, u.r, SIZE, u.j0, u.j1);
  u.piece = 0;
  u.count = 1;
  return true;
}

template <int DT, int D, int SRC>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_tile_kernel(AttnArgs a, bool split) {
  constexpr int kPlanes = D / 64, kTile = kPlanes * kPlane, kSteps = D / 16;
  constexpr bool kPaged = SRC != SRC_PACKED, kCodes = SRC == SRC_E4M3, kSplit = splits_scale(DT, kCodes);
  __shared__ __attribute__((aligned(1024))) char lds[4 * kTile];   // K, K, V, V
  __shared__ __attribute__((aligned(16))) float kscale[kCodes ? 4 : 1][kKeys], vscale[kCodes ? 2 : 1][kKeys];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Unit unit;
  if (!unit_of<kRows, kPaged>(a, split, lds, unit)) return;
  const Rows& r = unit.r;
  const int h = unit.head, j0 = unit.j0, j1 = unit.j1;

  const float c = a.scale * kLog2e;
  v16f o[D / 32];
  float m, l;     // running maximum (times c) and this lane's share of the sum

  // Over the keys; ODD: again, with the values that are not finite kept apart.
  auto pass = [&](auto odd_c, const int lane) {
    constexpr bool ODD = decltype(odd_c)::value;
    const int half = lane >> 5, col = lane & 31;
    // this wave's rows, and this lane's
    const int w0 = min(r.row0 + 32 * wave, r.rows - 1), w1 = min(w0 + 31, r.rows - 1);
    const int wave_first = r.pos0 + w0 / a.group, wave_last = r.pos0 + w1 / a.group;
    const int row = min(r.row0 + 32 * wave + col, r.rows - 1);
    const int tok = row / a.group, pos = r.pos0 + tok;
    const int low = a.window > 0 ? pos - a.window + 1 : 0;
    const uint16_t* qp = static_cast<const uint16_t*>(a.q) + (r.begin + tok) * a.qts + (h * a.group + row - tok * a.group) * a.qhs;
    v8s q[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) q[s] = *reinterpret_cast<const v8s*>(qp + 16 * s + 8 * half);

    // A tile into LDS: this wave brings keys 16 wave .. 16 wave + 15, 16-bit ones by DMA, codes
    // through registers, where they are converted (exactly) once for all four waves.
    const uint32_t base = lds_addr(lds);
    uint32_t koff[2], voff[2];
    if constexpr (!kCodes) {
      const uint32_t kb = kPaged ? D * 2 : static_cast<uint32_t>(a.kts * 2), vb = kPaged ? D * 2 : static_cast<uint32_t>(a.vts * 2);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint32_t c = gemm::dma_chunk(lane, g) * 16;
        koff[g] = (8 * g + (lane >> 3)) * kb + c;
        voff[g] = (8 * g + (lane >> 3)) * vb + c;
      }
    }
    auto page_of = [&](int t) -> int {
      if constexpr (!kPaged) return 0;
      const int at = t + 16 * wave;
      return at < r.len ? scalar_int(a.table + static_cast<int64_t>(r.request) * a.width + (at >> a.page_shift)) : -1;
    };
    // Where the wave's 16 keys of the tile at key t lie: their first row, and how many there are.
    struct Place {
      int64_t row;
      int n;
    };
    auto place = [&](int t, int page) -> Place {
      const int at = t + 16 * wave, have = min(max(r.len - at, 0), 16);
      if constexpr (!kPaged) return {r.begin + at, have};
      const bool there = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.pages);
      return {((static_cast<int64_t>(there ? page : 0) * a.hk + h) << a.page_shift) + (at & ((1 << a.page_shift) - 1)), there ? have : 0};
    };
    auto bring = [&](const void* p, int64_t ts, int64_t hs, const uint32_t (&off)[2], const Place& at, int buffer) {
      const char* from = static_cast<const char*>(p) + (kPaged ? at.row * D : at.row * ts + h * hs) * 2;
      v4i rs = make_rsrc(from, at.n > 0 ? static_cast<uint32_t>((at.n - 1) * (kPaged ? D : ts) * 2 + D * 2) : 0u);
      settle(rs);
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int x = 0; x < kPlanes; ++x)
          dma16(rs, base + buffer * kTile + x * kPlane + (2 * wave + g) * 1024, off[g] + x * 128);
    };
    // codes in flight: a lane's D / 4 bytes of one key and one scale
    struct Codes {
      v4i c[kPlanes];
      float s;
    };
    auto fetch = [&](const void* p, const float* sp, const Place& at, Codes& to) {
      auto buffer = [&](const void* q, int each) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(static_cast<const char*>(q)) + at.row * each, 0, at.n * each, kRsrcWord3);
      };
      const auto rc = buffer(p, D);
#pragma unroll
      for (int x = 0; x < kPlanes; ++x) to.c[x] = __builtin_amdgcn_raw_buffer_load_b128(rc, lane * (D / 4) + 16 * x, 0, 0);
      to.s = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(buffer(sp, 4), (lane & 15) * 4, 0, 0));
    };
    auto put = [&](auto value, const Codes& from, int buffer, float* to_scale) {
      constexpr bool SPLIT = kSplit && decltype(value)::value;   // a value's power of two goes to its codes
      const int key = 16 * wave + (lane >> 2);
      float power = 1.0f, scale = from.s;
      if constexpr (SPLIT) {
        const SplitScale y = split_scale(scale);
        scale = y.rest;
        power = __shfl(y.power, lane >> 2);
      }
#pragma unroll
      for (int x = 0; x < kPlanes; ++x) {
        const int c = (lane & 3) * (D / 32) + 2 * x;       // first of the two chunks of eight channels
        char* to = lds + buffer * kTile + (c >> 3) * kPlane + key * 128;
        *reinterpret_cast<v4u*>(to + (((c & 7) ^ gemm::swz(key & 15)) << 4)) = codes8<DT>(from.c[x][0], from.c[x][1], power);
        *reinterpret_cast<v4u*>(to + (((c & 7) + 1) ^ gemm::swz(key & 15)) * 16) = codes8<DT>(from.c[x][2], from.c[x][3], power);
      }
      if (lane < 16) to_scale[16 * wave + lane] = scale;
    };

    // LDS addresses of this lane's operands
    const uint32_t ka = (lane & 31) * 128 + ((half ^ gemm::swz(lane & 15)) << 4);      // ^ (2 s % 8) * 16
    const int vr = 4 * half + ((lane & 15) >> 2);                                      // + 16 s (+ 8)
    const uint32_t vc = (((lane >> 4) & 1) * 2 + ((lane & 3) >> 1)), vb = (lane & 1) * 8;   // chunk (^ 4: odd 32 channels)
    const uint32_t va0 = vr * 128 + ((vc ^ gemm::swz(vr)) << 4) + vb;
    const uint32_t va1 = (vr + 8) * 128 + ((vc ^ gemm::swz(vr + 8)) << 4) + vb;

    // Scores of 32 of a tile's keys: A operands of steps 4 q .. 4 q + 3, and their products.
    auto read_k = [&](int buffer, int w, v8s (&k)[kSteps / 2]) {
#pragma unroll
      for (int i = 0; i < kSteps / 2; ++i) {
        const int x = (w & 1) * (kSteps / 2) + i;
        k[i] = *reinterpret_cast<const v8s*>(lds + buffer * kTile + (x / 4) * kPlane + (w / 2) * 4096 + (ka ^ ((2 * x % 8) << 4)));
      }
    };
    auto score = [&](int w, const v8s (&k)[kSteps / 2], v16f (&s)[2]) {
      if ((w & 1) == 0) s[w / 2] = 0.0f;
#pragma unroll
      for (int i = 0; i < kSteps / 2; ++i) s[w / 2] = mfma<DT>(k[i], q[(w & 1) * (kSteps / 2) + i], s[w / 2]);
    };
    auto read_v1 = [&](int buffer, int w, int i) -> v8s {      // 16 keys, channels 32 i ..
      const uint32_t flip = (i & 1) << 6;
      const char* at = lds + (2 + buffer) * kTile + (i / 2) * kPlane + w * 2048;
      const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(at + (va0 ^ flip)));
      const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(at + (va1 ^ flip)));
      return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    auto read_v = [&](int buffer, int w, v8s (&v)[D / 32]) {
#pragma unroll
      for (int i = 0; i < D / 32; ++i) v[i] = read_v1(buffer, w, i);
    };

    // The steps from a tile's scores to its weights: the keys' scales; the mask; the running maximum
    // and what it rescales; 16 keys' weights for the product with their values, and their share of
    // the sum.
    auto scale_scores = [&](v16f (&s)[2], const float* scale) {
      if constexpr (kCodes) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const v4f x = *reinterpret_cast<const v4f*>(scale + 32 * u + 8 * g + 4 * half);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[u][4 * g + i] *= x[i];
          }
      }
    };
    auto mask_scores = [&](v16f (&s)[2], int t) {
      if (t + kKeys - 1 > wave_first || (a.window > 0 && t < wave_last - a.window + 1)) {
        const int hi = pos - t - 4 * half, lo = low - t - 4 * half;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int key = 32 * u + 8 * (i / 4) + i % 4;
            s[u][i] = key <= hi && key >= lo ? s[u][i] : -INFINITY;
          }
      }
    };
    auto follow_maximum = [&](v16f (&s)[2], auto& o) {
      constexpr int kBlocks = sizeof(o) / sizeof(v16f);
      float top = s[0][0];
#pragma unroll
      for (int i = 1; i < 32; ++i) top = fmaxf(top, s[i / 16][i % 16]);
      top = max_halves(top) * c;
      const bool above = top > m + kSlack;
      if (__any(above)) {      // each row by its own scores: another row's change nothing in it
        const float m1 = above ? top : m;
        const float keep = above ? __builtin_amdgcn_exp2f(m - m1) : 1.0f;
        m = m1;
        l *= keep;
#pragma unroll
        for (int i = 0; i < kBlocks; ++i)
#pragma unroll
          for (int x = 0; x < 16; ++x) o[i][x] *= keep;
      }
    };
    auto weigh = [&](auto odd_c, const v16f (&s)[2], int w, float mb, const float* scale, float (&x)[8]) {
      constexpr bool ODD = decltype(odd_c)::value;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[w / 2][8 * (w & 1) + i], c, -mb));
        l += x[i];
      }
      if constexpr (kCodes) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const v4f y = *reinterpret_cast<const v4f*>(scale + 16 * w + 8 * g + 4 * half);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float z = x[4 * g + i] * y[i];
            x[4 * g + i] = ODD && s[w / 2][8 * (w & 1) + 4 * g + i] == -INFINITY ? 0.0f : z;
          }
        }
      }
    };

    // Over the keys once.  Tile i's weights are formed while the matrix unit multiplies tile i + 1's
    // keys and the weights that are ready with tile i's values: K runs one tile ahead of V.
    auto walk = [&]() {
      m = -INFINITY;
      l = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o[i] = 0.0f;
      if (j0 >= j1) return;
      v16f s0[2], s1[2];
      Codes ck, cv;
      const Place at0 = place(j0, page_of(j0));
      Place at1 = place(j0 + kKeys, page_of(j0 + kKeys));   // of the tile whose V comes next
      int page = page_of(j0 + 2 * kKeys);                   // of the tile whose K comes next
      if constexpr (kCodes) {
        Codes first;
        fetch(a.k, a.ks, at0, first);
        fetch(a.k, a.ks, at1, ck);
        fetch(a.v, a.vs, at0, cv);
        put(std::false_type{}, first, 0, kscale[0]);
        put(std::false_type{}, ck, 1, kscale[kCodes ? 1 : 0]);
        put(std::true_type{}, cv, 2, vscale[0]);
        const Place at2 = place(j0 + 2 * kKeys, page);
        fetch(a.k, a.ks, at2, ck);
        fetch(a.v, a.vs, at1, cv);
        at1 = at2;
        page = page_of(j0 + 3 * kKeys);
      } else {
        bring(a.k, a.kts, a.khs, koff, at0, 0);
        bring(a.k, a.kts, a.khs, koff, at1, 1);
        bring(a.v, a.vts, a.vhs, voff, at0, 2);
        wait_vmcnt<4 * kPlanes>();      // the first K tile: the next one's and V's DMAs came after it
      }
      wait_lds_reads();
      stage_barrier();
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        v8s k[kSteps / 2];
        read_k(0, w, k);
        score(w, k, s0);
      }
      int t = j0, tile = 0;
      auto step = [&](auto parity, v16f (&s)[2], v16f (&next)[2]) {
        constexpr int B = decltype(parity)::value;      // tile i's buffer
        wait_lds_reads();
        if constexpr (!kCodes) wait_vmcnt<0>();
        stage_barrier();
        if constexpr (kCodes) {
          put(std::false_type{}, ck, B, kscale[kCodes ? (tile + 2) & 3 : 0]);
          put(std::true_type{}, cv, 2 + (B ^ 1), vscale[kCodes ? B ^ 1 : 0]);
          const Place at = place(t + 3 * kKeys, page);
          fetch(a.k, a.ks, at, ck);
          fetch(a.v, a.vs, at1, cv);
          at1 = at;
          page = page_of(t + 4 * kKeys);
        } else if (t + kKeys < j1) {
          const Place at = place(t + 2 * kKeys, page);
          bring(a.k, a.kts, a.khs, koff, at, B);
          bring(a.v, a.vts, a.vhs, voff, at1, 2 + (B ^ 1));
          at1 = at;
          page = page_of(t + 3 * kKeys);
        }
        v8s k[2][kSteps / 2], v[2][D / 32];
        read_k(B ^ 1, 0, k[0]);
        scale_scores(s, kscale[kCodes ? tile & 3 : 0]);
        mask_scores(s, t);
        follow_maximum(s, o);
        const float mb = m == -INFINITY ? 0.0f : m;
        v8s p[2];
#pragma unroll
        for (int w = 0; w < 4; ++w) {      // 16 keys
          if (w < 3) read_k(B ^ 1, w + 1, k[(w + 1) & 1]);
          read_v(B, w, v[w & 1]);
          float z[8];
          weigh(std::false_type{}, s, w, mb, vscale[kCodes ? B : 0], z);
          p[w & 1] = pack8<DT>(z);
          score(w, k[w & 1], next);
          if (w > 0) {
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
              o[i] = mfma<DT>(v[(w + 1) & 1][i], p[(w + 1) & 1], o[i]);
          }
#pragma unroll
          for (int n = 0; n < kSteps / 2 + (w > 0 ? D / 32 : 0); ++n) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);    // MFMA
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);    // LDS reads
            __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);    // VALU
            __builtin_amdgcn_sched_group_barrier(0x400, 1, 0);    // exponentials
          }
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) o[i] = mfma<DT>(v[1][i], p[1], o[i]);
        t += kKeys;
        ++tile;
      };
      while (true) {
        step(std::integral_constant<int, 0>{}, s0, s1);
        if (t >= j1) break;
        step(std::integral_constant<int, 1>{}, s1, s0);
        if (t >= j1) break;
      }
    };
    // Once more, with the values that are not finite kept apart: 32 channels at a time and one tile
    // after the other (few registers, so that the code above keeps its own).
    auto walk_odd = [&]() {
#pragma unroll 1
      for (int x = 0; x < D / 32; ++x) {
        v16f part[1];
        part[0] = 0.0f;
        m = -INFINITY;
        l = 0.0f;
  #pragma unroll 1
        for (int t = j0; t < j1; t += kKeys) {
          const Place at = place(t, page_of(t));
          wait_lds_reads();
          stage_barrier();
          if constexpr (kCodes) {
            Codes codes;
            fetch(a.k, a.ks, at, codes);
            put(std::false_type{}, codes, 0, kscale[0]);
            fetch(a.v, a.vs, at, codes);
            put(std::true_type{}, codes, 2, vscale[0]);
          } else {
            bring(a.k, a.kts, a.khs, koff, at, 0);
            bring(a.v, a.vts, a.vhs, voff, at, 2);
            wait_vmcnt<0>();
          }
          wait_lds_reads();
          stage_barrier();
          v16f s[2];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            v8s k[kSteps / 2];
            read_k(0, w, k);
            score(w, k, s);
          }
          scale_scores(s, kscale[0]);
          mask_scores(s, t);
          follow_maximum(s, part);
          const float mb = m == -INFINITY ? 0.0f : m;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            float z[8];
            weigh(std::true_type{}, s, w, mb, vscale[0], z);
            uint32_t seen = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) seen |= (s[w / 2][8 * (w & 1) + i] == -INFINITY ? 0u : 1u) << i;
            part[0] = mfma_odd<DT, kSplit>(read_v1(0, w, x), z, seen, part[0]);
          }
        }
#pragma unroll
        for (int y = 0; y < D / 32; ++y)
          if (y == x) o[y] = part[0];
      }
    };
    if constexpr (ODD) walk_odd();
    else walk();
  };
  pass(std::false_type{}, lane);
  bool fine = true;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int x = 0; x < 16; ++x) fine &= __builtin_isfinite(o[i][x]);
  if (__syncthreads_or(!fine)) {
    int again = lane;      // nothing of the first pass is kept for it in registers
    asm volatile("" : "+v"(again));
    pass(std::true_type{}, again);
  }
  const int half = lane >> 5, col = lane & 31;
  const int row = min(r.row0 + 32 * wave + col, r.rows - 1), tok = row / a.group, pos = r.pos0 + tok;

  l = add_halves(l);
  const int64_t out_row = static_cast<int64_t>(r.begin + tok) * a.hq + h * a.group + (row - tok * a.group);
  const bool store = r.row0 + 32 * wave + col < r.rows;
  if (kPaged && unit.count > 1) {      // a partial result: maximum, sum and output as they are
    if (store) {
      const Workspace ws = workspace(a, kRows);
      const int64_t slot = unit.slot(unit.piece);
      if (half == 0) *reinterpret_cast<float2*>(ws.stats + (slot * kRows + 32 * wave + col) * 2) = make_float2(m, l);
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<v4f*>(ws.out + slot * (kRows * D) + ((wave * (D / 32) + i) * 4 + g) * 256 + lane * 4) =
              v4f{o[i][4 * g], o[i][4 * g + 1], o[i][4 * g + 2], o[i][4 * g + 3]};
    }
    return;
  }
  if (r.row0 + 32 * wave >= r.rows) return;
  const float inv = pos < 0 ? 0.0f : 1.0f / l;
  if (a.lse && store && half == 0) a.lse[out_row] = pos < 0 ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
  uint16_t* out = static_cast<uint16_t*>(a.out) + out_row * D + 8 * half;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int g = 0; g < 4; g += 2) {
      // lane l holds channels 8 g + 4 (l / 32) + 0..3 of groups g and g + 1: exchanged so that each
      // half has eight in a row
      uint32_t a0 = pack2<DT>(o[i][4 * g] * inv, o[i][4 * g + 1] * inv), a1 = pack2<DT>(o[i][4 * g + 2] * inv, o[i][4 * g + 3] * inv);
      uint32_t b0 = pack2<DT>(o[i][4 * g + 4] * inv, o[i][4 * g + 5] * inv), b1 = pack2<DT>(o[i][4 * g + 6] * inv, o[i][4 * g + 7] * inv);
      swap_halves(a0, b0);
      swap_halves(a1, b1);
      if (store) *reinterpret_cast<v4u*>(out + 32 * i + 8 * g) = v4u{a0, a1, b0, b1};
    }
}

template <int DT, int D, int SRC>
void launch(const AttnArgs& a, hipStream_t s) {
  const bool split = SRC != SRC_PACKED && may_split(a.tokens, a.group, a.batch, a.hk, static_cast<int64_t>(a.width) << a.page_shift);
  const int64_t groups = tile_groups(a.tokens, a.batch, a.group, a.hk, split);
  attn_tile_kernel<DT, D, SRC><<<static_cast<unsigned>(groups), 64 * kWaves, 0, s>>>(a, split);
  if (split) launch_attn_join(DT, D, a, s);
}

template <int SRC>
void launch_typed(int dt, int head_dim, const AttnArgs& a, hipStream_t s) {
  if (dt == DT_BF16) head_dim == 128 ? launch<DT_BF16, 128, SRC>(a, s) : launch<DT_BF16, 64, SRC>(a, s);
  else head_dim == 128 ? launch<DT_F16, 128, SRC>(a, s) : launch<DT_F16, 64, SRC>(a, s);
}

}  // namespace

void launch_attn_tile(int dt, int head_dim, bool e4m3, const AttnArgs& a, hipStream_t s) {
  e4m3 ? launch_typed<SRC_E4M3>(dt, head_dim, a, s) : launch_typed<SRC_PAGED>(dt, head_dim, a, s);
}

}  // namespace attn

void launch_attn_prompt(int dt, int head_dim, const AttnArgs& a, hipStream_t s) {
  attn::launch_typed<attn::SRC_PACKED>(dt, head_dim, a, s);
}

}  // namespace fp8amax
