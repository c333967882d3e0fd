// quant_device.hpp - element-wise steps of the quantizers, shared by every kernel that
// writes e4m3 codes (the quantize kernels and the fused one-token decode step): 16-byte
// loads of eight 16-bit inputs, their magnitude keys, the cast of eight inputs with a
// group's scale (the fast quotient or the exact path), and a group's scale and its store.
//
// Steps: Transformer Engine page "Что такое FP8 инференс на H100 (Transformer Engine)?",
// section 3 steps 2-4 (amax, scale = amax / 448, x / scale rounded to e4m3); UE8M0
// scales from the fine-grained FP8 page ("FP8 chi tiết", UE8M0 scale format).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8_device.hpp"

namespace fp8amax {

struct U4 { uint32_t x, y, z, w; };

__device__ __forceinline__ U4 load16(const void* p) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  return {v.x, v.y, v.z, v.w};
}

__device__ __forceinline__ uint32_t key8(const U4& v) {
  uint32_t m = key_max_pair(0u, v.x);
  m = key_max_pair(m, v.y);
  m = key_max_pair(m, v.z);
  return key_max_pair(m, v.w);
}

template <int DT>
__device__ __forceinline__ float lo16(uint32_t w) { return in_to_f32<DT>(w & 0xffffu); }
template <int DT>
__device__ __forceinline__ float hi16(uint32_t w) { return in_to_f32<DT>(w >> 16); }

// Exact path: IEEE division and the software encoder, element by element.  Used for
// groups whose scale is NaN, infinite or below 2^-100.
template <int DT>
__device__ __forceinline__ uint32_t enc4_exact(uint32_t w0, uint32_t w1, float s) {
  return e4m3_encode(lo16<DT>(w0) / s) | (e4m3_encode(hi16<DT>(w0) / s) << 8) |
         (e4m3_encode(lo16<DT>(w1) / s) << 16) | (e4m3_encode(hi16<DT>(w1) / s) << 24);
}

template <int DT>
__device__ __forceinline__ uint32_t enc4_fast(uint32_t w0, uint32_t w1, float s, float r) {
  return cvt4(quot_fast(lo16<DT>(w0), s, r), quot_fast(hi16<DT>(w0), s, r),
              quot_fast(lo16<DT>(w1), s, r), quot_fast(hi16<DT>(w1), s, r));
}

// Eight 16-bit inputs -> eight e4m3 codes.  `fast` = fast_scale(s), r = 1/s.
template <int DT>
__device__ __forceinline__ uint2 enc8(const U4& v, float s, float r, bool fast) {
  if (fast) return make_uint2(enc4_fast<DT>(v.x, v.y, s, r), enc4_fast<DT>(v.z, v.w, s, r));
  return make_uint2(enc4_exact<DT>(v.x, v.y, s), enc4_exact<DT>(v.z, v.w, s));
}

// One element (ragged paths).
template <int DT>
__device__ __forceinline__ uint8_t enc1(uint32_t h, float s, float r, bool fast) {
  const float x = in_to_f32<DT>(h);
  if (fast) {
    const float q = quot_fast(x, s, r);
    return static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(q, q, 0, false) & 0xff);
  }
  return static_cast<uint8_t>(e4m3_encode(x / s));
}

// A group's scale from its amax, and the value stored for it: the float32 scale amax / 448,
// or (E8M0) the power-of-two scale and its e8m0fnu code.
template <bool E8M0>
struct GroupScale {
  float scale;
  uint32_t code;
  __device__ __forceinline__ explicit GroupScale(float amax) {
    if constexpr (E8M0) {
      code = e8m0_from_amax(amax);
      scale = e8m0_value(code);
    } else {
      scale = scale_from_amax(amax);
      code = 0;
    }
  }
  // Store the scale of group (row, col) of a grid with `ncols` groups per row: float32
  // rows are ncols long; UE8M0 rows are `stride` bytes (ncols rounded up to whole 32-bit
  // words), and the group that ends a row also sets the row's padding bytes to 127 (2^0).
  __device__ __forceinline__ void store(void* out, int64_t row, int64_t col, int64_t ncols,
                                        int64_t stride) const {
    if constexpr (E8M0) {
      uint8_t* o = static_cast<uint8_t*>(out) + row * stride;
      o[col] = static_cast<uint8_t>(code);
      if (col == ncols - 1)
        for (int64_t p = ncols; p < stride; ++p) o[p] = 127;
    } else {
      static_cast<float*>(out)[row * ncols + col] = scale;
    }
  }
};

// Eight float32 values -> eight e4m3 codes.  The fast quotient wants a scale of at least 2^-60 here:
// a float32 value has 24 bits, and the remainder of its quotient must not reach the subnormal numbers.
__device__ __forceinline__ bool fast_scale_f32(float s) { return s >= 0x1p-60f && s <= 3.40282347e38f; }
__device__ __forceinline__ uint2 enc8_f32(const float (&x)[8], float s, float r, bool fast) {
  if (fast)
    return make_uint2(cvt4(quot_fast(x[0], s, r), quot_fast(x[1], s, r), quot_fast(x[2], s, r), quot_fast(x[3], s, r)),
                      cvt4(quot_fast(x[4], s, r), quot_fast(x[5], s, r), quot_fast(x[6], s, r), quot_fast(x[7], s, r)));
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = e4m3_encode(x[i] / s);
  return make_uint2(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24, c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
}

// ------------------------------------------------------------------------------------
// e2m1 codes with a power-of-two scale for 32 values (OCP MX, FP4).  A magnitude key is the bits of
// |x| as float32; NaN sorts above infinity, which sorts above the rest.

// The scale byte s of a block whose largest key is `key`: 2^(s - 127) the smallest power of two from
// 2^-127 not below amax / 6; 127 for a block of zeros, 255 for one with a value that is not finite.
// Integer work on amax = (1 + f) 2^E: 6 = 1.5 * 2^2, so E - 2 where 1 + f <= 1.5 and E - 1 above.
__device__ __forceinline__ uint32_t mx4_scale(uint32_t key) {
  if (key >= 0x7f800000u) return 255u;
  if (key == 0u) return 127u;
  return static_cast<uint32_t>(max(static_cast<int>(key >> 23) - 2 + ((key & 0x7fffffu) > 0x400000u ? 1 : 0), 0));
}

// The largest code's value: 6, or 3 where 4 times the scale is past the 16-bit type's range (2^14 with
// fp16, 2^126 with bf16), which rounding would reach from 3.5.
template <int DT>
__device__ __forceinline__ float mx4_limit(uint32_t s) {
  return s >= (DT == DT_BF16 ? 127u + 126 : 127u + 14) ? 3.0f : 6.0f;
}

// Eight float32 values -> eight codes in one dword, the first in the low bits: round to nearest even
// on the grid 0, 0.5, 1, 1.5, 2, 3, 4, 6.  The product with the power of two is exact, or so small
// that the code is 0.
template <int DT>
__device__ __forceinline__ uint32_t enc8_mx4(const float (&x)[8], uint32_t s) {
  if (s == 255u) return 0u;
  const float r = __uint_as_float((254u - s) << 23), top = mx4_limit<DT>(s);
  uint32_t w = 0;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __builtin_amdgcn_fmed3f(x[i] * r, -top, top);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[0], y[1], 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[2], y[3], 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[4], y[5], 1.0f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[6], y[7], 1.0f, 3);
}

// Eight 16-bit inputs as float32.
template <int DT>
__device__ __forceinline__ void widen8(const U4& v, float (&x)[8]) {
  x[0] = lo16<DT>(v.x); x[1] = hi16<DT>(v.x); x[2] = lo16<DT>(v.y); x[3] = hi16<DT>(v.y);
  x[4] = lo16<DT>(v.z); x[5] = hi16<DT>(v.z); x[6] = lo16<DT>(v.w); x[7] = hi16<DT>(v.w);
}

// Max over each aligned group of four lanes.
__device__ __forceinline__ uint32_t max4(uint32_t v) {
  v = max(v, dpp_u32<0xB1>(v));    // quad_perm [1,0,3,2]
  return max(v, dpp_u32<0x4E>(v));   // quad_perm [2,3,0,1]
}

}  // namespace fp8amax
