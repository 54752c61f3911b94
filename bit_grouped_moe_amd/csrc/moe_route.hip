// Expert routing with scores of either kind, a balancing bias and groups.
//
//   s = softmax(z) or sigmoid(z);  c = s + bias (without a bias: in the order of z)
//   a group of E / groups neighbouring experts counts as its largest c, or as the
//   sum of its two largest; the topk_groups largest groups are open
//   ids = the topk largest c of the open groups, largest first
//   w = scale s, or scale s / sum of the chosen s (renormalize)
//
// Ties go to the lower index; an expert whose logit or choice is -inf is masked.
// Which of two experts is larger is decided in 64 bits: the selection of a row
// then does not depend on the last bits of a float32 exponential.  Weights are
// float32, from the chosen logits.
//
// One wave a row, at most 16 experts a lane, expert 64 c + l in lane l.
#include "router.hpp"

namespace gq {

constexpr int kRouteMaxGroups = kWave;                   // a lane each

struct RouteArgs {
  const float* bias;             // [E] or null
  int E, topk, sigmoid, groups, topk_groups, group_top, renorm;
  uint32_t size_magic;           // expert / (E / groups) = expert * size_magic >> 20
  float scale;
  int32_t* ids;
  float* weights;
};

// Order-preserving key of a double, as logit_key: NaN above all, -inf (a masked
// expert or group) kDeadKey64 and below every other; 0 past the row's experts.
constexpr uint64_t kDeadKey64 = 0x000FFFFFFFFFFFFFull;
__device__ __forceinline__ uint64_t key64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
  return v != v ? ~0ull : b ^ ((b >> 63) ? ~0ull : 0x8000000000000000ull);
}
__device__ __forceinline__ double key_value(uint64_t k) {
  return __builtin_bit_cast(double, k == ~0ull ? 0x7FF8000000000000ull
                                               : (k >> 63) ? k ^ 0x8000000000000000ull : ~k);
}
__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
  const uint32_t hi = wave_umax((uint32_t)(v >> 32));
  const uint32_t lo = wave_umax((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
  return v;
}

// The selection in 64 bits: slot `lane`'s expert and logit (-1 and -inf: none).
// z holds the row's logits, -inf past its experts; keys: C * 64 words of LDS.
template <int C>
__device__ __forceinline__ void select64(const RouteArgs& g, const float (&z)[C], int lane,
                                         uint64_t* keys, int& id, float& logit) {
  uint64_t key[C];
  double total = 1.0, peak = 0.0;
  if (!g.sigmoid && (g.bias || g.group_top > 1)) {
    uint32_t best = 0u;
#pragma unroll
    for (int c = 0; c < C; ++c) best = max(best, logit_key(z[c]));
    const uint32_t m = wave_umax(best);
    peak = m > kDeadKey ? (double)key_logit(m) : 0.0;
    total = 0.0;
#pragma unroll
    for (int c = 0; c < C; ++c) total += z[c] == -__builtin_inff() ? 0.0 : exp((double)z[c] - peak);
    total = wave_sum64(total);
  }
  auto score = [&](float v) {
    return g.sigmoid ? 1.0 / (1.0 + exp(-(double)v)) : exp((double)v - peak) / total;
  };
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = 64 * c + lane;
    uint64_t k = 0ull, two = 0ull;
    if (e < g.E) {
      k = kDeadKey64;
      if (z[c] != -__builtin_inff()) k = key64(g.bias ? score(z[c]) + (double)g.bias[e] : (double)z[c]);
      // a sum of two is one of scores, also where the experts' order is the logits'
      two = g.group_top > 1 && !g.bias && k > kDeadKey64 ? key64(score(z[c])) : k;
    }
    key[c] = k;
    if (g.groups > 1) keys[e] = two;
  }
  if (g.groups > 1) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    uint64_t first = 0ull, second = 0ull;
    if (lane < g.groups) {
      const int size = g.E / g.groups;
      for (int i = 0; i < size; ++i) {
        const uint64_t k = keys[lane * size + i];
        second = max(second, min(first, k));
        first = max(first, k);
      }
      if (g.group_top > 1 && second > kDeadKey64) first = key64(key_value(first) + key_value(second));
    }
    int before = 0;                                      // groups ahead of this one
    for (int j = 0; j < g.groups; ++j) {
      const uint64_t k =
          ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(first >> 32), j) << 32) |
          (uint32_t)__builtin_amdgcn_readlane((int)first, j);
      before += k > first || (k == first && j < lane);
    }
    const uint64_t open = __ballot(lane < g.groups && before < g.topk_groups);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = 64 * c + lane;
      if (!((open >> (((uint32_t)e * g.size_magic) >> 20 & 63u)) & 1ull)) key[c] = 0ull;
    }
  }
  uint32_t ids = 0xFFFFFFFFu, won = __float_as_uint(-__builtin_inff());
  for (int s = 0; s < g.topk; ++s) {
    uint64_t best = key[0];
#pragma unroll
    for (int c = 1; c < C; ++c) best = max(best, key[c]);
    const uint64_t m = wave_max64(best);
    if (m <= kDeadKey64) break;                          // uniform
    bool open = true;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint64_t at = __ballot(key[c] == m);
      if (open && at) {                                  // uniform
        open = false;
        const int l = __builtin_ctzll(at);
        if (lane == l) key[c] = 0ull;
        ids = wave_writelane((uint32_t)(64 * c + l), s, ids);
        won = wave_writelane(
            (uint32_t)__builtin_amdgcn_readlane(__float_as_int(z[c]), l), s, won);
      }
    }
  }
  id = (int)ids;
  logit = __uint_as_float(won);
}

template <int kType, int C>
__global__ __launch_bounds__(kRouterThreads) void moe_route_kernel(
    const void* __restrict__ logits, int64_t rows, int64_t stride, RouteArgs g) {
  __shared__ uint64_t keys[kWaveRows][C * kWave];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t row = (int64_t)blockIdx.x * kWaveRows + wave;
  if (row >= rows) return;
  const float kInf = __builtin_inff();
  float z[C];
#pragma unroll
  for (int c = 0; c < C; ++c) z[c] = load1<kType>(logits, row * stride + min(64 * c + lane, g.E - 1));
#pragma unroll
  for (int c = 0; c < C; ++c)
    if (64 * c + lane >= g.E) z[c] = -kInf;
  int id;
  float zs;
  select64<C>(g, z, lane, keys[wave], id, zs);
  // weights: over the largest logit of the slots, or of the row
  uint32_t best = id >= 0 ? logit_key(zs) : 0u;
  bool broken = false;                                   // a softmax with a NaN or +inf
  if (!g.sigmoid) {
    uint32_t all = 0u;
#pragma unroll
    for (int c = 0; c < C; ++c) all = max(all, logit_key(z[c]));
    broken = wave_umax(all) >= 0xFF800000u;              // the key of +inf
    if (!g.renorm) best = all;
  }
  const uint32_t m = wave_umax(best);
  const float peak = broken ? __uint_as_float(0x7FC00000u) : m > kDeadKey ? key_logit(m) : 0.f;
  const float part = id < 0 ? 0.f
                     : g.sigmoid ? sigmoid_over(zs, g.renorm && peak <= 0.f ? peak : 0.f)
                                 : expf(zs - peak);
  float total = part;
  if (!g.sigmoid && !g.renorm) {
    total = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) total += z[c] == -kInf ? 0.f : expf(z[c] - peak);
  }
  total = g.sigmoid && !g.renorm ? 1.f : wave_fsum(total);
  if (lane < g.topk) {
    g.ids[row * g.topk + lane] = id;
    g.weights[row * g.topk + lane] = id >= 0 ? part / total * g.scale : 0.f;
  }
}

}  // namespace gq

extern "C" int gq_moe_route(const void* logits, int32_t dtype, int64_t rows, int32_t num_experts,
                            int64_t stride, const float* bias, int32_t topk, int32_t score,
                            int32_t groups, int32_t topk_groups, int32_t group_top,
                            int32_t renormalize, float scale, int32_t* topk_ids,
                            float* topk_weights, hipStream_t stream) {
  using namespace gq;
  if (score != GQ_SOFTMAX && score != GQ_SIGMOID) return kInvalid;
  if (num_experts < 1 || groups < 1 || num_experts % groups || topk_groups < 1 ||
      topk_groups > groups || group_top < 1 || group_top > 2)
    return kInvalid;
  if (topk > topk_groups * (num_experts / groups)) return kInvalid;
  if (!(scale > -3.4e38f && scale < 3.4e38f)) return kInvalid;
  const int st = router_checks(logits, dtype, rows, num_experts, stride, topk, topk_ids,
                               topk_weights, logits);
  if (st == kOk && groups > kRouteMaxGroups) return kNotSupported;
  if (st != kOk || rows == 0) return st;
  if (!aligned4(topk_ids) || !aligned4(topk_weights) || !aligned4(bias)) return kInvalid;
  RouteArgs g{};
  g.bias = bias;
  g.E = num_experts; g.topk = topk; g.sigmoid = score == GQ_SIGMOID;
  g.groups = groups; g.topk_groups = topk_groups; g.group_top = group_top;
  g.renorm = renormalize != 0; g.scale = scale;
  // exact for every expert below 1024: the error of an expert e's quotient is
  // below e / 2^20 < 1 / size
  g.size_magic = (1u << 20) / (uint32_t)(num_experts / groups) + 1;
  auto go = [&](auto type) {
    constexpr int T = decltype(type)::value;
    by_width(num_experts, [&](auto c) {
      by_rows(rows, kWaveRows, [&](int64_t at, int64_t n) {
        g.ids = topk_ids + at * topk;
        g.weights = topk_weights + at * topk;
        hipLaunchKernelGGL((moe_route_kernel<T, decltype(c)::value>),
                           dim3((unsigned)ceil_div64(n, kWaveRows)), dim3(kRouterThreads), 0,
                           stream, row_at<T>(logits, at * stride), n, stride, g);
      });
    });
  };
  if (dtype == GQ_F32) go(std::integral_constant<int, GQ_F32>{});
  else if (dtype == GQ_BF16) go(std::integral_constant<int, GQ_BF16>{});
  else go(std::integral_constant<int, GQ_F16>{});
  return launch_status();
}
