// Rows of float32 / bf16 / float16 values eight at a time, and MXFP8 codes of
// them, shared by the quantisers (quantize.hip) and the norm (norm.hip).
#pragma once

#include "gq_device.hpp"
#include "../../include/gq.h"

namespace gq {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
// the same vectors at the alignment of one element: rows may start anywhere
// (the memory pipeline takes unaligned dword accesses)
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Eight values of 16 bits each as float32 (exact).
template <int kType>
__device__ __forceinline__ void widen8(u32x4 a, float (&v)[8]) {
  static_assert(kType != GQ_F32);
  if constexpr (kType == GQ_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16lo_to_f32(a[i]);
      v[2 * i + 1] = bf16hi_to_f32(a[i]);
    }
  } else {
    const f16x8 h = __builtin_bit_cast(f16x8, a);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
  }
}

// Eight consecutive values of a row as float32 (exact).
template <int kType>
__device__ __forceinline__ void load8(const void* p, float (&v)[8]) {
  if constexpr (kType == GQ_F32) {
    const u32x4_a4* q = static_cast<const u32x4_a4*>(p);
    const u32x4 a = q[0], b = q[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(a[i]);
      v[4 + i] = __uint_as_float(b[i]);
    }
  } else {
    widen8<kType>(*static_cast<const u32x4_a2*>(p), v);
  }
}

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_umax(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, false));
}

// Largest magnitude, as bits, of the 32 values that a quad of lanes holds
// (infinity and NaN compare above every number).
__device__ __forceinline__ uint32_t quad_amax(const float (&v)[8]) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  m = dpp_umax<0xB1>(m);                                    // quad_perm [1,0,3,2]
  return dpp_umax<0x4E>(m);                                 // quad_perm [2,3,0,1]
}

// MXFP8 of the eight values of quad member `lane % 4` of a block: e4m3 codes in
// element order and the block's scale byte X + 127, X the smallest exponent with
// amax 2^-X <= 448, the largest e4m3 magnitude (no code saturates); -127 for a
// zero block, 255 with codes 0 for a block with an infinity or NaN.
__device__ __forceinline__ u32x2 quantize8_e4m3(const float (&v)[8], uint32_t& scale) {
  const uint32_t m = quad_amax(v);
  const int e = (int)(m >> 23);
  const int X = max(e - 135 + ((m & 0x7FFFFFu) > 0x600000u ? 1 : 0), -127);
  const bool bad = e == 255;
  scale = bad ? 255u : (uint32_t)(X + 127);
  auto s = [&](int i) { return __builtin_amdgcn_ldexpf(v[i], -X); };
  int a = __builtin_amdgcn_cvt_pk_fp8_f32(s(0), s(1), 0, false);
  a = __builtin_amdgcn_cvt_pk_fp8_f32(s(2), s(3), a, true);
  int b = __builtin_amdgcn_cvt_pk_fp8_f32(s(4), s(5), 0, false);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(s(6), s(7), b, true);
  return bad ? u32x2{0u, 0u} : u32x2{(uint32_t)a, (uint32_t)b};
}

// The values that eight e4m3 codes stand for under scale byte `scale`, as bf16
// pairs: exact, but for magnitudes below 2^-133, which round to bf16's steps.
__device__ __forceinline__ u32x4 e4m3_bf16_scaled(u32x2 q, uint32_t scale) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int w = (int)(i < 2 ? q.x : q.y);
    const f32x2 p = (i & 1) ? __builtin_amdgcn_cvt_pk_f32_fp8(w, true)
                            : __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
    const uint32_t r = pack_bf16x2(__builtin_amdgcn_ldexpf(p.x, (int)scale - 127),
                                   __builtin_amdgcn_ldexpf(p.y, (int)scale - 127));
    o[i] = scale == 255u ? 0x7FC07FC0u : r;
  }
  return o;
}

}  // namespace gq
