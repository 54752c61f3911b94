// MXFP4 quantisation: rows of float32 / bf16 / float16 values -> e2m1 codes
// and one e8m0 scale per 32 values (the layout every MXFP4 entry point
// reads), and on request the values that the codes stand for, as bf16.
//
// Per block of 32 values (OCP Microscaling formats v1.0):
//   X    = clamp(floor(log2 amax) - 2, -127, 127);  amax = 0: X = -127
//   code = sign | nearest e2m1 magnitude of |v| * 2^-X, ties to the even
//          code, magnitudes above 6 become 6
//   scale byte = X + 127, value = e2m1(code) * 2^X (exact in bf16)
// A block with an infinity or a NaN gets scale 255 and codes 0: every value
// of it decodes to NaN.
//
// Bound by HBM: each value is read once, 0.53 bytes (and 2 for the values)
// are written.  Four neighbouring lanes own a block, eight values each: a
// lane's load is one or two 16-byte pieces, a wave's code store 256
// contiguous bytes and its value store 1 KB.  The block maximum is taken on
// the bit patterns (NaN and infinity compare above every number) with two
// DPP moves.
#include "gq_device.hpp"
#include "gq_host.hpp"
#include "../../include/gq.h"

namespace gq {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
// the same vectors at the alignment of one element: rows may start anywhere
// (the memory pipeline takes unaligned dword loads)
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

constexpr int kQuantThreads = 256;

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
    const u32x4 a = *static_cast<const u32x4_a2*>(p);
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
}

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_umax(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, false));
}

// Codes of the eight values of lane quad member `lane % 4` of a block (in
// element order, low nibble first) and the block's scale byte.
__device__ __forceinline__ uint32_t quantize8(const float (&v)[8], uint32_t& scale) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  m = dpp_umax<0xB1>(m);                                    // quad_perm [1,0,3,2]
  m = dpp_umax<0x4E>(m);                                    // quad_perm [2,3,0,1]
  const int e = (int)(m >> 23);                             // 255: infinity or NaN
  const int X = max(e - 129, -127);
  const bool bad = e == 255;
  scale = bad ? 255u : (uint32_t)(X + 127);
  uint32_t c = 0u;
  // 2^-X by ldexp (exact where the result matters: what underflows rounds
  // to zero anyway), then the converter at scale 1: round to nearest even,
  // saturating, sign kept
  auto s = [&](int i) { return __builtin_amdgcn_ldexpf(v[i], -X); };
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, s(0), s(1), 1.0f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, s(2), s(3), 1.0f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, s(4), s(5), 1.0f, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, s(6), s(7), 1.0f, 3);
  return bad ? 0u : c;
}

// Threads of a workgroup: 2^lgx chunks of eight values along a row, the rest
// along rows; the grid strides over rows.  Chunks per row is a multiple of 4
// and chunk % 4 == lane % 4, so a quad of lanes is always one block (lgx >=
// 2) and is active or idle as a whole.
template <int kType>
__global__ __launch_bounds__(kQuantThreads) void mxfp4_quantize_kernel(
    const void* __restrict__ x, int64_t rows, int64_t chunks, int64_t stride_bytes, int lgx,
    uint32_t* __restrict__ codes, uint8_t* __restrict__ scales, u32x4* __restrict__ values) {
  constexpr int kSize = kType == GQ_F32 ? 4 : 2;
  const int64_t c = ((int64_t)blockIdx.x << lgx) + (threadIdx.x & ((1 << lgx) - 1));
  if (c >= chunks) return;
  const int64_t rstep = (int64_t)gridDim.y * (kQuantThreads >> lgx);
  for (int64_t r = (int64_t)blockIdx.y * (kQuantThreads >> lgx) + (threadIdx.x >> lgx); r < rows;
       r += rstep) {
    float v[8];
    load8<kType>(static_cast<const char*>(x) + r * stride_bytes + c * (8 * kSize), v);
    uint32_t s;
    const uint32_t q = quantize8(v, s);
    const int64_t o = r * chunks + c;
    codes[o] = q;
    if ((threadIdx.x & 3) == 0) scales[o >> 2] = (uint8_t)s;
    if (values) {
      const float f = e8m0_to_f32(s);
      values[o] = u32x4{e2m1_pair_bf16_scaled(q, 0, f), e2m1_pair_bf16_scaled(q, 1, f),
                        e2m1_pair_bf16_scaled(q, 2, f), e2m1_pair_bf16_scaled(q, 3, f)};
    }
  }
}

}  // namespace gq

extern "C" int gq_mxfp4_quantize(const void* x, int32_t x_dtype, int64_t rows, int32_t K,
                                 int64_t x_stride, uint8_t* blocks, uint8_t* scales,
                                 uint16_t* values, hipStream_t stream) {
  using namespace gq;
  if (x_dtype != GQ_F32 && x_dtype != GQ_BF16 && x_dtype != GQ_F16) return kInvalid;
  if (rows < 0 || K <= 0 || K % 32 || x_stride < K) return kInvalid;
  if (rows == 0) return kOk;
  const int size = x_dtype == GQ_F32 ? 4 : 2;
  if (!x || !blocks || !scales || (reinterpret_cast<uintptr_t>(x) & (size - 1))) return kInvalid;
  if (!aligned16(blocks) || (values && !aligned16(values))) return kInvalid;
  if (x_stride > INT64_MAX / 8 / rows) return kNotSupported;
  // rows without gaps are one long row, up to the threads that a launch takes
  int64_t chunks = K / 8, n = rows;
  if (x_stride == K && chunks * rows <= most_groups(kQuantThreads) * kQuantThreads) {
    chunks *= rows;
    n = 1;
  }
  int lgx = 2;
  while (lgx < 8 && ((int64_t)1 << lgx) < chunks) ++lgx;
  const int64_t bx = ceil_div64(chunks, (int64_t)1 << lgx);
  const int64_t by = ceil_div64(n, kQuantThreads >> lgx);
  // (a row has at most 2^28 chunks; beyond 65535 groups of rows the kernel strides)
  const dim3 grid((unsigned)bx, (unsigned)(by < 65535 ? by : 65535));
  auto* c = reinterpret_cast<uint32_t*>(blocks);
  auto* v = reinterpret_cast<u32x4*>(values);
  switch (x_dtype) {
    case GQ_F32:
      hipLaunchKernelGGL(mxfp4_quantize_kernel<GQ_F32>, grid, dim3(kQuantThreads), 0, stream, x, n,
                         chunks, x_stride * size, lgx, c, scales, v);
      break;
    case GQ_BF16:
      hipLaunchKernelGGL(mxfp4_quantize_kernel<GQ_BF16>, grid, dim3(kQuantThreads), 0, stream, x,
                         n, chunks, x_stride * size, lgx, c, scales, v);
      break;
    default:
      hipLaunchKernelGGL(mxfp4_quantize_kernel<GQ_F16>, grid, dim3(kQuantThreads), 0, stream, x, n,
                         chunks, x_stride * size, lgx, c, scales, v);
      break;
  }
  return launch_status();
}
