// attn_tile.hip - attention for many rows: a workgroup of four waves takes 128 packed rows (32 a
// wave) of one key head and walks over the keys in tiles of 64 that all four waves share in LDS.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "attn_device.hpp"

namespace fp8amax {
namespace attn {
namespace {

constexpr int kWaves = 4;
constexpr int kRows = 32 * kWaves;
constexpr float kSlack = 8.0f;

// The workgroup's unit: cut from the batch's work (find_unit) or a whole tile of rows.
template <int SIZE, bool PAGED>
__device__ __forceinline__ bool unit_of(const AttnArgs& a, bool split, char* lds, Unit& u) {
  if (PAGED && split) return find_unit<SIZE, PAGED>(a, blockIdx.x, reinterpret_cast<int*>(lds), u);
  if (!PAGED && a.batch <= 64) return find_ranked<SIZE>(a, u);
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
  constexpr bool kPaged = SRC != SRC_PACKED, kCodes = SRC == SRC_E4M3, kRange = kCodes && DT == DT_F16;
  __shared__ __attribute__((aligned(1024))) char lds[4 * kTile];   // K, K, V, V
  __shared__ __attribute__((aligned(16))) float scales[kCodes ? 2 : 1][2][kKeys];   // of the tile's keys and values
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, col = lane & 31;
  Unit unit;
  if (!unit_of<kRows, kPaged>(a, split, lds, unit)) return;
  const Rows& r = unit.r;
  const int h = unit.head, j0 = unit.j0, j1 = unit.j1;

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
  auto bring = [&](const void* p, int64_t ts, int64_t hs, const uint32_t (&off)[2], int t, int page, int buffer) {
    v4i rs = key_rows<SRC, D>(a, r, p, ts, hs, h, t + 16 * wave, 16, page);
    settle(rs);
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int x = 0; x < kPlanes; ++x)
        dma16_safe(rs, base + buffer * kTile + x * kPlane + (2 * wave + g) * 1024, off[g] + x * 128);
  };
  // codes in flight: a lane's D / 4 bytes of one key, of K and V, and one scale of each
  v4i ck[kPlanes], cv[kPlanes];
  float sk = 0.0f, sv = 0.0f;
  auto fetch = [&](int t, int page) {
    const int at = t + 16 * wave, have = min(max(r.len - at, 0), 16);
    const bool there = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.pages);
    const int64_t first = ((static_cast<int64_t>(there ? page : 0) * a.hk + h) << a.page_shift) + (at & ((1 << a.page_shift) - 1));
    const int n = there ? have : 0;
    auto buffer = [&](const void* p, int64_t bytes, int each) {
      return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(static_cast<const char*>(p)) + bytes * each, 0, n * each, kRsrcWord3);
    };
    const auto rk = buffer(a.k, first, D), rv = buffer(a.v, first, D);
#pragma unroll
    for (int x = 0; x < kPlanes; ++x) {
      ck[x] = __builtin_amdgcn_raw_buffer_load_b128(rk, lane * (D / 4) + 16 * x, 0, 0);
      cv[x] = __builtin_amdgcn_raw_buffer_load_b128(rv, lane * (D / 4) + 16 * x, 0, 0);
    }
    sk = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(buffer(a.ks, first, 4), (lane & 15) * 4, 0, 0));
    sv = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(buffer(a.vs, first, 4), (lane & 15) * 4, 0, 0));
  };
  auto put = [&](int buffer) {
    const int key = 16 * wave + (lane >> 2);
#pragma unroll
    for (int x = 0; x < kPlanes; ++x) {
      const int c = (lane & 3) * (D / 32) + 2 * x;       // first of the two chunks of eight channels
      char* to = lds + (c >> 3) * kPlane + key * 128;
      const int c0 = ((c & 7) ^ gemm::swz(key & 15)) << 4, c1 = (((c & 7) + 1) ^ gemm::swz(key & 15)) << 4;
      *reinterpret_cast<v4u*>(to + buffer * kTile + c0) = codes8<DT>(ck[x][0], ck[x][1]);
      *reinterpret_cast<v4u*>(to + buffer * kTile + c1) = codes8<DT>(ck[x][2], ck[x][3]);
      *reinterpret_cast<v4u*>(to + (2 + buffer) * kTile + c0) = codes8<DT>(cv[x][0], cv[x][1]);
      *reinterpret_cast<v4u*>(to + (2 + buffer) * kTile + c1) = codes8<DT>(cv[x][2], cv[x][3]);
    }
    if (lane < 16) {
      scales[kCodes ? buffer : 0][0][16 * wave + lane] = sk;
      scales[kCodes ? buffer : 0][1][16 * wave + lane] = sv;
    }
  };

  // LDS addresses of this lane's operands
  const uint32_t ka = (lane & 31) * 128 + ((half ^ gemm::swz(lane & 15)) << 4);      // ^ (2 s % 8) * 16
  const int vr = 4 * half + ((lane & 15) >> 2);                                      // + 16 s (+ 8)
  const uint32_t vc = (((lane >> 4) & 1) * 2 + ((lane & 3) >> 1)), vb = (lane & 1) * 8;   // chunk (^ 4: odd 32 channels)
  const uint32_t va0 = vr * 128 + ((vc ^ gemm::swz(vr)) << 4) + vb;
  const uint32_t va1 = (vr + 8) * 128 + ((vc ^ gemm::swz(vr + 8)) << 4) + vb;

  const float c = a.scale * kLog2e;
  v16f o[D / 32];
  float m, l;     // running maximum (times c) and this lane's share of the sum
  int unit_exp;   // kRange: o is in units of 2^unit_exp

  // Over the keys once; ODD: again, with the values that are not finite kept apart.
  auto walk = [&](auto odd_c) {
    constexpr bool ODD = decltype(odd_c)::value;
    m = -INFINITY;
    l = 0.0f;
    unit_exp = -200;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = 0.0f;
    int page = page_of(j0);
    if (j0 < j1) {
      if constexpr (kCodes) {
        fetch(j0, page);
        put(0);
        fetch(j0 + kKeys, page_of(j0 + kKeys));
      } else {
        bring(a.k, a.kts, a.khs, koff, j0, page, 0);
        bring(a.v, a.vts, a.vhs, voff, j0, page, 2);
      }
    }
    page = page_of(j0 + (kCodes ? 2 : 1) * kKeys);
    int buf = 0;
    for (int t = j0; t < j1; t += kKeys, buf ^= 1) {
      wait_lds_reads();
      if constexpr (!kCodes) wait_vmcnt<0>();
      stage_barrier();
      if constexpr (!kCodes) {
        if (t + kKeys < j1) {
          bring(a.k, a.kts, a.khs, koff, t + kKeys, page, buf ^ 1);
          bring(a.v, a.vts, a.vhs, voff, t + kKeys, page, 2 + (buf ^ 1));
          page = page_of(t + 2 * kKeys);
        }
      } else {
        if (t + kKeys < j1) {
          put(buf ^ 1);
          fetch(t + 2 * kKeys, page);
          page = page_of(t + 3 * kKeys);
        }
      }
      if (t > wave_last) continue;      // this wave sees none of them (uniform; the barriers stay common)
      const char* kt = lds + buf * kTile;
      v16f s[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        s[u] = 0.0f;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const v8s k = *reinterpret_cast<const v8s*>(kt + (i / 4) * kPlane + u * 4096 + (ka ^ ((2 * i % 8) << 4)));
          s[u] = mfma<DT>(k, q[i], s[u]);
        }
      }
      if constexpr (kCodes) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const v4f x = *reinterpret_cast<const v4f*>(&scales[buf][0][32 * u + 8 * g + 4 * half]);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[u][4 * g + i] *= x[i];
          }
      }
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
      float top = s[0][0];
#pragma unroll
      for (int i = 1; i < 32; ++i) top = fmaxf(top, s[i / 16][i % 16]);
      top = max_halves(top) * c;
      if (__any(top > m + kSlack)) {
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
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[u][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][i], c, -mb));
          l += s[u][i];
        }
      if constexpr (kCodes) {
        // a weight's share of its value's scale; for fp16, in units of a power of two at least the
        // largest scale met, so that no product leaves fp16's range
        float unit_inv = 1.0f;
        if constexpr (kRange) {
          float most = 0.0f;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const v4f x = *reinterpret_cast<const v4f*>(&scales[buf][1][32 * u + 8 * g + 4 * half]);
              most = fmaxf(fmaxf(fmaxf(most, x[0]), fmaxf(x[1], x[2])), x[3]);
            }
          most = max_halves(most);
          const int e = min(max(__builtin_amdgcn_frexp_expf(most), -120), 120);
          if (e > unit_exp) {      // the same in every lane: the scales are
            const float keep = __builtin_ldexpf(1.0f, max(unit_exp - e, -200));
            unit_exp = e;
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
#pragma unroll
              for (int x = 0; x < 16; ++x) o[i][x] *= keep;
          }
          unit_inv = __builtin_ldexpf(1.0f, -unit_exp);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const v4f x = *reinterpret_cast<const v4f*>(&scales[buf][1][32 * u + 8 * g + 4 * half]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float y = s[u][4 * g + i] * (kRange ? x[i] * unit_inv : x[i]);
              s[u][4 * g + i] = ODD && s[u][4 * g + i] == 0.0f ? 0.0f : y;
            }
          }
      }
      v8s p[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        v4u x;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = pack2<DT>(s[w / 2][8 * (w & 1) + 2 * i], s[w / 2][8 * (w & 1) + 2 * i + 1]);
        p[w] = __builtin_bit_cast(v8s, x);
      }
      const char* vt = lds + (2 + buf) * kTile;
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint32_t flip = (i & 1) << 6;
          const char* at = vt + (i / 2) * kPlane + w * 2048;
          const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(at + (va0 ^ flip)));
          const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(at + (va1 ^ flip)));
          const v8s v = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
          if constexpr (ODD) o[i] = mfma_odd<DT>(v, p[w], o[i]);
          else o[i] = mfma<DT>(v, p[w], o[i]);
        }
    }
  };
  walk(std::false_type{});
  bool fine = true;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int x = 0; x < 16; ++x) fine &= __builtin_isfinite(o[i][x]);
  if (__syncthreads_or(!fine)) walk(std::true_type{});

  l = add_halves(l);
  if constexpr (kRange) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int x = 0; x < 16; ++x) o[i][x] = __builtin_ldexpf(o[i][x], unit_exp);
  }
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
  const int64_t tiles = tile_bound(a.tokens, a.group, a.batch, kRows);
  const bool split = SRC != SRC_PACKED && may_split(a.tokens, a.group, a.batch, a.hk, static_cast<int64_t>(a.width) << a.page_shift);
  const int64_t units = (tiles + (split ? extra_units(a.hk) : 0)) * a.hk;
  attn_tile_kernel<DT, D, SRC><<<static_cast<unsigned>(units), 64 * kWaves, 0, s>>>(a, split);
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
