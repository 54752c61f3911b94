// Expert routing: the topk largest logits of each token with their softmax
// weights, and the gradient of the weights to the logits.
//
//   forward   ids = the topk largest logits, largest first, ties to the lower
//             index; w_s = exp(z_s - peak) / sum, the sum over the chosen
//             logits (renormalize) or over all of the row's
//   backward  p = the same softmax; with g the gradient of the weights
//             (scattered to the experts) dz = p (g - sum p g); experts that a
//             renormalised softmax leaves out get 0
//
// One wave per token: E <= 1024 logits are at most 16 registers per lane, the
// selection is topk rounds of a wave maximum (DPP) and a ballot, the sums are
// DPP sums: no LDS, no atomics, fixed order.  Bound by the latency of the
// rounds for a few tokens and by their VALU time for many.
#include <type_traits>

#include "topk.hpp"
#include "gq_host.hpp"
#include "../../include/gq.h"

namespace gq {

constexpr int kRouterThreads = 256;

template <int kType>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (kType == GQ_F32) return static_cast<const float*>(p)[i];
  else if constexpr (kType == GQ_BF16)
    return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  else return (float)static_cast<const _Float16*>(p)[i];
}
template <int kType>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if constexpr (kType == GQ_F32) static_cast<float*>(p)[i] = v;
  else if constexpr (kType == GQ_BF16) static_cast<uint16_t*>(p)[i] = f32_to_bf16_bits(v);
  else static_cast<_Float16*>(p)[i] = (_Float16)v;
}

template <int kType, int C>
__global__ __launch_bounds__(kRouterThreads) void moe_topk_kernel(
    const void* __restrict__ logits, int64_t rows, int E, int64_t stride, int topk, int renorm,
    int32_t* __restrict__ ids, float* __restrict__ weights) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t row =
      (int64_t)blockIdx.x * (kRouterThreads / kWave) +
      __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  if (row >= rows) return;
  uint32_t key[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = 64 * c + lane;
    const float z = load1<kType>(logits, row * stride + min(e, E - 1));
    key[c] = e < E ? logit_key(z) : 0u;
  }
  uint32_t all[C];
#pragma unroll
  for (int c = 0; c < C; ++c) all[c] = key[c];
  int id;
  float z;
  wave_topk<C>(key, topk, id, z);
  const float peak = row_peak(z, id);
  const float part = id >= 0 ? expf(z - peak) : 0.f;
  float total = part;
  if (!renorm) {
    total = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
      total += all[c] > kDeadKey ? expf(key_logit(all[c]) - peak) : 0.f;
  }
  total = wave_fsum(total);
  if (lane < topk) {
    ids[row * topk + lane] = id;
    weights[row * topk + lane] = id >= 0 ? part / total : 0.f;
  }
}

template <int kType, int C>
__global__ __launch_bounds__(kRouterThreads) void moe_topk_backward_kernel(
    const float* __restrict__ dw, const void* __restrict__ logits, int64_t rows, int E,
    int64_t stride, const int32_t* __restrict__ ids, int topk, int renorm,
    void* __restrict__ dz) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t row =
      (int64_t)blockIdx.x * (kRouterThreads / kWave) +
      __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  if (row >= rows) return;
  const float kInf = __builtin_inff();
  // slot `lane`: its expert (-1: none), logit and weight gradient
  int id = lane < topk ? ids[row * topk + lane] : -1;
  id = (unsigned)id < (unsigned)E ? id : -1;
  float g = 0.f, zs = -kInf;
  if (id >= 0) {
    g = dw[row * topk + lane];
    zs = load1<kType>(logits, row * stride + id);
    if (zs == -kInf) { id = -1; g = 0.f; }               // a masked expert has no weight
  }
  uint32_t key[C];
#pragma unroll
  for (int c = 0; c < C; ++c) key[c] = 0u;
  uint32_t best = id >= 0 ? logit_key(zs) : 0u;
  if (!renorm) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = 64 * c + lane;
      const float z = load1<kType>(logits, row * stride + min(e, E - 1));
      key[c] = e < E ? logit_key(z) : 0u;
      best = max(best, key[c]);
    }
  }
  const uint32_t m = wave_umax(best);
  const float peak = m > kDeadKey ? key_logit(m) : 0.f;
  const float part = id >= 0 ? expf(zs - peak) : 0.f;
  float p[C];
  float sum = part;
  if (!renorm) {
    sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      p[c] = key[c] > kDeadKey ? expf(key_logit(key[c]) - peak) : 0.f;
      sum += p[c];
    }
  }
  const float total = wave_fsum(sum);
  const float inv = m > kDeadKey ? 1.f / total : 0.f;    // no live expert: no gradient
  const float w = part * inv;                            // slot weight
  const float dot = wave_fsum(w * g);
  // what slot s adds to its expert, in slot order
  const float add = renorm ? w * (g - dot) : g;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = 64 * c + lane;
    if (64 * c >= E) break;
    float acc = 0.f;
    for (int s = 0; s < topk; ++s) {
      const int is = __builtin_amdgcn_readlane(id, s);
      const float as = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(add), s));
      acc += is == e ? as : 0.f;
    }
    if (!renorm) acc = p[c] * inv * (acc - dot);
    if (e < E) store1<kType>(dz, row * E + e, acc);
  }
}

template <int kType, typename F>
static void by_width(int E, F&& f) {
  if (E <= 64) f(std::integral_constant<int, 1>{});
  else if (E <= 128) f(std::integral_constant<int, 2>{});
  else if (E <= 256) f(std::integral_constant<int, 4>{});
  else if (E <= 512) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

static int router_checks(const void* logits, int32_t dtype, int64_t rows, int32_t E,
                         int64_t stride, int32_t topk, const void* a, const void* b,
                         const void* c, int64_t& blocks) {
  if (dtype != GQ_F32 && dtype != GQ_BF16 && dtype != GQ_F16) return kInvalid;
  if (rows < 0 || E < 1 || topk < 1 || stride < E) return kInvalid;
  if (E > kTopkMaxExperts || topk > kTopkMax) return kNotSupported;
  if (rows == 0) return kOk;
  const uintptr_t mask = dtype == GQ_F32 ? 3 : 1;
  if (!logits || !a || !b || !c || (reinterpret_cast<uintptr_t>(logits) & mask)) return kInvalid;
  blocks = ceil_div64(rows, kRouterThreads / kWave);
  if (blocks > INT32_MAX || stride > INT64_MAX / 4 / rows) return kNotSupported;
  return kOk;
}

}  // namespace gq

extern "C" int gq_moe_topk(const void* logits, int32_t dtype, int64_t rows, int32_t num_experts,
                           int64_t stride, int32_t topk, int32_t renormalize, int32_t* topk_ids,
                           float* topk_weights, hipStream_t stream) {
  using namespace gq;
  int64_t blocks = 0;
  if (topk > num_experts) return kInvalid;
  const int st = router_checks(logits, dtype, rows, num_experts, stride, topk, topk_ids,
                               topk_weights, logits, blocks);
  if (st != kOk || rows == 0) return st;
  if (!aligned4(topk_ids) || !aligned4(topk_weights)) return kInvalid;
  auto go = [&](auto type) {
    constexpr int T = decltype(type)::value;
    by_width<T>(num_experts, [&](auto c) {
      hipLaunchKernelGGL((moe_topk_kernel<T, decltype(c)::value>), dim3((unsigned)blocks),
                         dim3(kRouterThreads), 0, stream, logits, rows, num_experts, stride, topk,
                         renormalize, topk_ids, topk_weights);
    });
  };
  if (dtype == GQ_F32) go(std::integral_constant<int, GQ_F32>{});
  else if (dtype == GQ_BF16) go(std::integral_constant<int, GQ_BF16>{});
  else go(std::integral_constant<int, GQ_F16>{});
  return launch_status();
}

extern "C" int gq_moe_topk_backward(const float* d_weights, const void* logits, int32_t dtype,
                                    int64_t rows, int32_t num_experts, int64_t stride,
                                    const int32_t* topk_ids, int32_t topk, int32_t renormalize,
                                    void* d_logits, hipStream_t stream) {
  using namespace gq;
  int64_t blocks = 0;
  const int st = router_checks(logits, dtype, rows, num_experts, stride, topk, d_weights,
                               topk_ids, d_logits, blocks);
  if (st != kOk || rows == 0) return st;
  const uintptr_t mask = dtype == GQ_F32 ? 3 : 1;
  if (!aligned4(d_weights) || !aligned4(topk_ids) ||
      (reinterpret_cast<uintptr_t>(d_logits) & mask))
    return kInvalid;
  auto go = [&](auto type) {
    constexpr int T = decltype(type)::value;
    by_width<T>(num_experts, [&](auto c) {
      hipLaunchKernelGGL((moe_topk_backward_kernel<T, decltype(c)::value>),
                         dim3((unsigned)blocks), dim3(kRouterThreads), 0, stream, d_weights,
                         logits, rows, num_experts, stride, topk_ids, topk, renormalize, d_logits);
    });
  };
  if (dtype == GQ_F32) go(std::integral_constant<int, GQ_F32>{});
  else if (dtype == GQ_BF16) go(std::integral_constant<int, GQ_BF16>{});
  else go(std::integral_constant<int, GQ_F16>{});
  return launch_status();
}
