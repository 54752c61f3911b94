// Pieces shared by the router's kernels (router.hip: softmax top-k and the
// gradients; moe_route.hip: scores of either kind, groups, a balancing bias):
// one element of a row, launches over rows, argument checks.
#pragma once

#include <type_traits>

#include "topk.hpp"
#include "gq_host.hpp"
#include "../../include/gq.h"

namespace gq {

constexpr int kRouterThreads = 256;
constexpr int kWaveRows = kRouterThreads / kWave;        // rows of a workgroup, a wave each

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

// sigmoid(z) 2^(-m log2 e), i.e. sigmoid(z) times e^-m, for z <= 0 or m = 0: scores
// that are all tiny keep their ratios under m, the largest of their logits.
__device__ __forceinline__ float sigmoid_over(float z, float m) {
  return z > 0.f ? 1.0f / (1.0f + expf(-z)) : expf(z - m) / (1.0f + expf(z));
}

template <typename F>
static void by_width(int E, F&& f) {
  if (E <= 64) f(std::integral_constant<int, 1>{});
  else if (E <= 128) f(std::integral_constant<int, 2>{});
  else if (E <= 256) f(std::integral_constant<int, 4>{});
  else if (E <= 512) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

// launch(first row, rows) over pieces of the rows: a launch takes 2^24 - 1
// workgroups of `group` rows (2^26 - 4 rows a wave each, 2^28 - 16 sixteen lanes).
template <typename F>
static void by_rows(int64_t rows, int group, F&& launch) {
  const int64_t most = most_groups(kRouterThreads) * group;
  for (int64_t at = 0; at < rows; at += most) launch(at, rows - at < most ? rows - at : most);
}
template <int kType>
static inline const void* row_at(const void* p, int64_t element) {
  return static_cast<const char*>(p) + element * (kType == GQ_F32 ? 4 : 2);
}
template <int kType>
static inline void* row_at(void* p, int64_t element) {
  return static_cast<char*>(p) + element * (kType == GQ_F32 ? 4 : 2);
}

static inline int router_checks(const void* logits, int32_t dtype, int64_t rows, int32_t E,
                         int64_t stride, int32_t topk, const void* a, const void* b,
                         const void* c) {
  if (dtype != GQ_F32 && dtype != GQ_BF16 && dtype != GQ_F16) return kInvalid;
  if (rows < 0 || E < 1 || topk < 1 || stride < E) return kInvalid;
  if (E > kTopkMaxExperts || topk > kTopkMax) return kNotSupported;
  if (rows == 0) return kOk;
  const uintptr_t mask = dtype == GQ_F32 ? 3 : 1;
  if (!logits || !a || !b || !c || (reinterpret_cast<uintptr_t>(logits) & mask)) return kInvalid;
  if (rows > (int64_t)1 << 33 || stride > INT64_MAX / 4 / rows) return kNotSupported;
  return kOk;
}

}  // namespace gq
