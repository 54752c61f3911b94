// MXFP4 and MXFP8 quantisation: rows of float32 / bf16 / float16 values -> e2m1
// or e4m3 codes and one e8m0 scale per 32 values (the layout that the entry
// points of the format read), and on request the values that the codes stand
// for, as bf16.
//
// MXFP4, per block of 32 values (OCP Microscaling formats v1.0):
//   X    = clamp(floor(log2 amax) - 2, -127, 127);  amax = 0: X = -127
//   code = sign | nearest e2m1 magnitude of |v| * 2^-X, ties to the even
//          code, magnitudes above 6 become 6
//   scale byte = X + 127, value = e2m1(code) * 2^X (exact in bf16)
// MXFP8 (values.hpp): X the smallest exponent with amax 2^-X <= 448, as in the
// first term of the two-term split, so that no code saturates; code = e4m3 of
// v 2^-X, ties to even.
// A block with an infinity or a NaN gets scale 255 and codes 0: every value
// of it decodes to NaN.
//
// Bound by HBM: each value is read once, 0.53 or 1.03 bytes (and 2 for the
// values) are written.  Four neighbouring lanes own a block, eight values each: a
// lane's load is one or two 16-byte pieces, a wave's code store 256
// (or 512) contiguous bytes and its value store 1 KB.  The block maximum is taken on
// the bit patterns (NaN and infinity compare above every number) with two
// DPP moves.
#include <type_traits>

#include "values.hpp"
#include "gq_host.hpp"

namespace gq {

constexpr int kQuantThreads = 256;

// Codes of the eight values of lane quad member `lane % 4` of a block (in
// element order, low nibble first) and the block's scale byte.
__device__ __forceinline__ uint32_t quantize8(const float (&v)[8], uint32_t& scale) {
  const uint32_t m = quad_amax(v);
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
template <int kType, bool k8>
__global__ __launch_bounds__(kQuantThreads) void mx_quantize_kernel(
    const void* __restrict__ x, int64_t rows, int64_t chunks, int64_t stride_bytes, int lgx,
    std::conditional_t<k8, u32x2, uint32_t>* __restrict__ codes, uint8_t* __restrict__ scales, u32x4* __restrict__ values) {
  constexpr int kSize = kType == GQ_F32 ? 4 : 2;
  const int64_t c = ((int64_t)blockIdx.x << lgx) + (threadIdx.x & ((1 << lgx) - 1));
  if (c >= chunks) return;
  const int64_t rstep = (int64_t)gridDim.y * (kQuantThreads >> lgx);
  for (int64_t r = (int64_t)blockIdx.y * (kQuantThreads >> lgx) + (threadIdx.x >> lgx); r < rows;
       r += rstep) {
    float v[8];
    load8<kType>(static_cast<const char*>(x) + r * stride_bytes + c * (8 * kSize), v);
    uint32_t s;
    const int64_t o = r * chunks + c;
    if constexpr (k8) {
      const u32x2 q = quantize8_e4m3(v, s);
      codes[o] = q;
      if (values) values[o] = e4m3_bf16_scaled(q, s);
    } else {
      const uint32_t q = quantize8(v, s);
      codes[o] = q;
      if (values) {
        const float f = e8m0_to_f32(s);
        values[o] = u32x4{e2m1_pair_bf16_scaled(q, 0, f), e2m1_pair_bf16_scaled(q, 1, f),
                          e2m1_pair_bf16_scaled(q, 2, f), e2m1_pair_bf16_scaled(q, 3, f)};
      }
    }
    if ((threadIdx.x & 3) == 0) scales[o >> 2] = (uint8_t)s;
  }
}

template <bool k8>
static int quantize_entry(const void* x, int32_t x_dtype, int64_t rows, int32_t K,
                          int64_t x_stride, uint8_t* codes, uint8_t* scales, uint16_t* values,
                          hipStream_t stream) {
  if (x_dtype != GQ_F32 && x_dtype != GQ_BF16 && x_dtype != GQ_F16) return kInvalid;
  if (rows < 0 || K <= 0 || K % 32 || x_stride < K) return kInvalid;
  if (rows == 0) return kOk;
  const int size = x_dtype == GQ_F32 ? 4 : 2;
  if (!x || !codes || !scales || (reinterpret_cast<uintptr_t>(x) & (size - 1))) return kInvalid;
  if (!aligned16(codes) || (values && !aligned16(values))) return kInvalid;
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
  auto* c = reinterpret_cast<std::conditional_t<k8, u32x2, uint32_t>*>(codes);
  auto* v = reinterpret_cast<u32x4*>(values);
  auto go = [&](auto type) {
    hipLaunchKernelGGL((mx_quantize_kernel<decltype(type)::value, k8>), grid, dim3(kQuantThreads),
                       0, stream, x, n, chunks, x_stride * size, lgx, c, scales, v);
  };
  if (x_dtype == GQ_F32) go(std::integral_constant<int, GQ_F32>{});
  else if (x_dtype == GQ_BF16) go(std::integral_constant<int, GQ_BF16>{});
  else go(std::integral_constant<int, GQ_F16>{});
  return launch_status();
}

}  // namespace gq

extern "C" int gq_mxfp4_quantize(const void* x, int32_t x_dtype, int64_t rows, int32_t K,
                                 int64_t x_stride, uint8_t* blocks, uint8_t* scales,
                                 uint16_t* values, hipStream_t stream) {
  return gq::quantize_entry<false>(x, x_dtype, rows, K, x_stride, blocks, scales, values, stream);
}

extern "C" int gq_mxfp8_quantize(const void* x, int32_t x_dtype, int64_t rows, int32_t K,
                                 int64_t x_stride, uint8_t* codes, uint8_t* scales,
                                 uint16_t* values, hipStream_t stream) {
  return gq::quantize_entry<true>(x, x_dtype, rows, K, x_stride, codes, scales, values, stream);
}
