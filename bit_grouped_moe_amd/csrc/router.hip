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
// Two variants.  One wave a row, at most 16 logits per lane, a round of the
// selection being a wave maximum (DPP) and a ballot: short for few rows, and
// for any number of experts and slots.  Sixteen lanes a row
// (moe_topk_group_kernel below): a quarter of the instructions and a longer
// chain, for many rows of up to 256 experts and 16 slots.  Sums are DPP sums
// in a fixed order.
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
  wave_keys<C>(E, lane, [&](int e) { return load1<kType>(logits, row * stride + e); }, key);
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
    wave_keys<C>(E, lane, [&](int e) { return load1<kType>(logits, row * stride + e); }, key);
#pragma unroll
    for (int c = 0; c < C; ++c) best = max(best, key[c]);
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

// ---- many rows of up to 256 experts and 16 slots: sixteen lanes a row ----------
// Lane l of a row holds experts C l .. C l + C - 1 as keys that no two experts
// share (logit, then lower index), sorted once in the lane (Batcher's
// merge-exchange network).  A round is four DPP maxima over the lanes' first
// keys; the lane that held the maximum moves its list up by one.  A 16-bit
// logit and the index fit 32 bits, a float32 logit takes 64.  A round of four
// rows is 15 instructions for 128 experts in bf16, where a wave of the other
// variant spends 20 on one row.  Bound by VALU time.
//
// Measured, top-8, wave -> group, us (graph-replayed, launch included):
//                    bf16 E = 128   bf16 E = 256   f32 E = 128    f32 E = 256
//   256 rows forward  2.89 -> 2.69   3.44 -> 3.28   2.88 -> 3.84   3.37 -> 5.71
//   4096     forward  3.86 -> 2.86   4.73 -> 3.50   3.82 -> 4.39   4.62 -> 6.06
//   8192     forward  5.14 -> 3.13   6.62 -> 4.18   5.15 -> 4.81   6.50 -> 9.42
//   16384    forward  8.22 -> 4.16  10.56 -> 5.75   7.86 -> 6.63  10.43 -> 12.85
//   256     backward  2.76 -> 2.72   3.27 -> 2.86   2.59 -> 2.69   3.31 -> 3.22
//   4096    backward  3.66 -> 2.93   4.79 -> 3.27   3.67 -> 3.11   5.12 -> 4.31
//   16384   backward  8.00 -> 3.64  12.12 -> 4.95   8.56 -> 4.68  12.70 -> 9.29
// Below 4096 rows the softmax over all experts (not renormalised) is up to
// 0.8 us slower in sixteen lanes; hence kGroupFrom.  The 64-bit keys of float32
// pay from 64 rows an expert on and not at all above 128 experts.
constexpr int kGroup = 16;
constexpr int kGroupRows = kRouterThreads / kGroup;
constexpr int kGroupMaxExperts = 16 * kGroup;
constexpr int kGroupFrom = 4096;                         // rows

__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  auto step = [&](auto ctrl) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, 0xF, 0xF,
                                                     false));
  };
  step(std::integral_constant<int, 0xB1>{});
  step(std::integral_constant<int, 0x4E>{});
  step(std::integral_constant<int, 0x141>{});
  step(std::integral_constant<int, 0x140>{});
  return v;
}
__device__ __forceinline__ uint64_t group_max(uint64_t v) {
  const uint32_t hi = group_max((uint32_t)(v >> 32));
  const uint32_t lo = group_max((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return ((uint64_t)hi << 32) | lo;
}

// Keys of a logit and its expert: larger logit, larger key; equal logits, lower
// expert.  The order of the logits is logit_key's.
template <int kType>
struct GroupKey {                                        // bf16, f16: 16 bits and the index
  using type = uint32_t;
  static constexpr uint32_t kDead = kType == GQ_BF16 ? 0x007Fu : 0x03FFu;   // -inf
  static __device__ __forceinline__ uint32_t make(uint16_t raw, int e) {
    uint32_t k;
    if constexpr (kType == GQ_BF16) {
      k = logit_key(__uint_as_float((uint32_t)raw << 16)) >> 16;
    } else {
      const uint32_t b = raw == 0x8000u ? 0u : raw;
      k = b ^ ((b >> 15) ? 0xFFFFu : 0x8000u);
      k = (raw & 0x7FFFu) > 0x7C00u ? 0xFFFFu : k;
    }
    return (k << 16) | (0xFFFFu - (uint32_t)e);
  }
  static __device__ __forceinline__ bool live(uint32_t k) { return (k >> 16) > kDead; }
  static __device__ __forceinline__ int expert(uint32_t k) { return 0xFFFF - (int)(k & 0xFFFFu); }
  static __device__ __forceinline__ float logit(uint32_t k) {
    if constexpr (kType == GQ_BF16) {
      return key_logit((k >> 16) == 0xFFFFu ? 0xFFFFFFFFu : (k & 0xFFFF0000u) |
                                                  ((k >> 31) ? 0u : 0xFFFFu));
    } else {
      const uint32_t v = k >> 16;
      if (v == 0xFFFFu) return __uint_as_float(0x7FC00000u);
      const uint16_t b = (uint16_t)((v >> 15) ? v ^ 0x8000u : ~v);
      return (float)__builtin_bit_cast(_Float16, b);
    }
  }
};
template <>
struct GroupKey<GQ_F32> {
  using type = uint64_t;
  static __device__ __forceinline__ uint64_t make(uint32_t raw, int e) {
    return ((uint64_t)logit_key(__uint_as_float(raw)) << 32) | (0xFFFFFFFFu - (uint32_t)e);
  }
  static __device__ __forceinline__ bool live(uint64_t k) { return (uint32_t)(k >> 32) > kDeadKey; }
  static __device__ __forceinline__ int expert(uint64_t k) {
    return (int)(0xFFFFFFFFu - (uint32_t)k);
  }
  static __device__ __forceinline__ float logit(uint64_t k) { return key_logit((uint32_t)(k >> 32)); }
};

// A lane's C raw logits: one or more wide loads where every row's and lane's
// place allows them (`wide`, from the host), else C narrow ones.  Lanes and
// elements past the row's experts load some of the row's own.
template <int kType, int C>
struct GroupRow {
  using raw = std::conditional_t<kType == GQ_F32, uint32_t, uint16_t>;
  static constexpr int kBytes = C * (int)sizeof(raw);
  static constexpr int kUnit = kBytes < 16 ? kBytes : 16;
  typedef uint32_t vec __attribute__((ext_vector_type(kUnit / 4)));
  union {
    vec v[kBytes / kUnit];
    raw r[C];
  };
  __device__ __forceinline__ void load(const void* row, int l, int E, bool wide) {
    const raw* p = static_cast<const raw*>(row);
    if (wide) {
      const vec* q = reinterpret_cast<const vec*>(p + (C * l < E ? C * l : 0));
#pragma unroll
      for (int i = 0; i < kBytes / kUnit; ++i) v[i] = q[i];
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) r[c] = p[min(C * l + c, E - 1)];
    }
  }
  __device__ __forceinline__ void store(void* row, int l, int E, bool wide) const {
    raw* p = static_cast<raw*>(row) + C * l;
    if (wide) {
      if (C * l < E) {
#pragma unroll
        for (int i = 0; i < kBytes / kUnit; ++i) reinterpret_cast<vec*>(p)[i] = v[i];
      }
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (C * l + c < E) p[c] = r[c];
    }
  }
  static __device__ __forceinline__ float value(raw b) {
    if constexpr (kType == GQ_F32) return __uint_as_float(b);
    else if constexpr (kType == GQ_BF16) return __uint_as_float((uint32_t)b << 16);
    else return (float)__builtin_bit_cast(_Float16, b);
  }
  static __device__ __forceinline__ raw bits(float v) {
    if constexpr (kType == GQ_F32) return __float_as_uint(v);
    else if constexpr (kType == GQ_BF16) return f32_to_bf16_bits(v);
    else return __builtin_bit_cast(uint16_t, (_Float16)v);
  }
};

template <int kType, int C>
__global__ __launch_bounds__(kRouterThreads) void moe_topk_group_kernel(
    const void* __restrict__ logits, int64_t rows, int E, int64_t stride, int topk, int renorm,
    int wide, int32_t* __restrict__ ids, float* __restrict__ weights) {
  using Row = GroupRow<kType, C>;
  using Key = GroupKey<kType>;
  using key_t = typename Key::type;
  const int l = threadIdx.x & (kGroup - 1);
  const int64_t own = (int64_t)blockIdx.x * kGroupRows + threadIdx.x / kGroup;
  const int64_t row = own < rows ? own : rows - 1;       // every lane takes part in the maxima
  Row x;
  x.load(static_cast<const typename Row::raw*>(logits) + row * stride, l, E, wide);
  key_t key[C];
#pragma unroll
  for (int c = 0; c < C; ++c) key[c] = C * l + c < E ? Key::make(x.r[c], C * l + c) : (key_t)0;
#pragma unroll
  for (int p = 1; p < C; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < C; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i) {
          const int u = i + j, v = i + j + k;
          if (v < C && u / (2 * p) == v / (2 * p)) {
            const bool swap = key[u] < key[v];
            const key_t hi = swap ? key[v] : key[u], lo = swap ? key[u] : key[v];
            key[u] = hi;
            key[v] = lo;
          }
        }
  const key_t first = group_max(key[0]);
  const float peak = Key::live(first) ? Key::logit(first) : 0.f;
  float total = 0.f;
  if (!renorm) {
#pragma unroll
    for (int c = 0; c < C; ++c) total += Key::live(key[c]) ? expf(Key::logit(key[c]) - peak) : 0.f;
  }
  key_t won = 0;
  for (int s = 0; s < topk; ++s) {
    const key_t m = group_max(key[0]);
    won = l == s ? m : won;
    const bool mine = key[0] == m;
#pragma unroll
    for (int c = 0; c < C; ++c) key[c] = mine ? (c + 1 < C ? key[c + 1] : (key_t)0) : key[c];
  }
  const bool live = Key::live(won);
  const float part = live ? expf(Key::logit(won) - peak) : 0.f;
  total = group_sum_last(renorm ? part : total, kGroup);
  if (l < topk && own < rows) {
    ids[row * topk + l] = live ? Key::expert(won) : -1;
    weights[row * topk + l] = live ? part / total : 0.f;
  }
}

// Gradients of the slots meet in the row's floats in LDS, added slot by slot
// (one lane a row at a time, so an expert that is named twice adds in slot
// order), and every lane then writes its experts' gradients.
template <int kType, int C>
__global__ __launch_bounds__(kRouterThreads) void moe_topk_backward_group_kernel(
    const float* __restrict__ dw, const void* __restrict__ logits, int64_t rows, int E,
    int64_t stride, const int32_t* __restrict__ ids, int topk, int renorm, int wide_in,
    int wide_out, void* __restrict__ dz) {
  using Row = GroupRow<kType, C>;
  using raw = typename Row::raw;
  __shared__ __align__(16) float acc[kGroupRows][C * kGroup];
  const int l = threadIdx.x & (kGroup - 1);
  const int64_t own = (int64_t)blockIdx.x * kGroupRows + threadIdx.x / kGroup;
  const int64_t row = own < rows ? own : rows - 1;
  float* sums = acc[threadIdx.x / kGroup];
  const raw* z = static_cast<const raw*>(logits) + row * stride;
  const float kInf = __builtin_inff();
#pragma unroll
  for (int c = 0; c < C; ++c) sums[C * l + c] = 0.f;
  int id = l < topk ? ids[row * topk + l] : -1;
  id = (unsigned)id < (unsigned)E ? id : -1;
  float g = 0.f, zs = -kInf;
  if (id >= 0) {
    g = dw[row * topk + l];
    zs = Row::value(z[id]);
    if (zs == -kInf) { id = -1; g = 0.f; }               // a masked expert has no weight
  }
  uint32_t best = id >= 0 ? logit_key(zs) : 0u;
  Row x;
  if (!renorm) {
    x.load(z, l, E, wide_in);
#pragma unroll
    for (int c = 0; c < C; ++c)
      best = max(best, C * l + c < E ? logit_key(Row::value(x.r[c])) : 0u);
  }
  const uint32_t m = group_max(best);
  const float peak = m > kDeadKey ? key_logit(m) : 0.f;
  const float part = id >= 0 ? expf(zs - peak) : 0.f;
  float p[C];
  float sum = part;
  if (!renorm) {
    sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float v = Row::value(x.r[c]);
      p[c] = C * l + c < E && v != -kInf ? expf(v - peak) : 0.f;
      sum += p[c];
    }
  }
  const float total = group_sum_last(sum, kGroup);
  const float inv = m > kDeadKey ? 1.f / total : 0.f;    // no live expert: no gradient
  const float w = part * inv;                            // slot weight
  const float dot = group_sum_last(w * g, kGroup);
  const float add = renorm ? w * (g - dot) : g;
  for (int s = 0; s < topk; ++s) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (l == s && id >= 0) sums[id] += add;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  if (own >= rows) return;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float v = sums[C * l + c];
    if (!renorm) v = p[c] * inv * (v - dot);
    x.r[c] = Row::bits(v);
  }
  x.store(static_cast<raw*>(dz) + row * E, l, E, wide_out);
}

template <int kMost, typename F>
static void by_group(int E, F&& f) {
  if (E <= 4 * kGroup) f(std::integral_constant<int, 4>{});
  else if (E <= 8 * kGroup) f(std::integral_constant<int, 8>{});
  else if constexpr (kMost > 8 * kGroup) f(std::integral_constant<int, 16>{});
}

// Whether rows of E elements of the type, `pitch` elements apart, can be read or
// written C elements at once.
template <int kType, int C>
static bool group_wide(const void* p, int E, int64_t pitch) {
  constexpr int kSize = (int)sizeof(typename GroupRow<kType, C>::raw);
  constexpr uintptr_t kMask = GroupRow<kType, C>::kUnit - 1;
  return E % C == 0 && ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(pitch * kSize)) & kMask) == 0;
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
static const void* row_at(const void* p, int64_t element) {
  return static_cast<const char*>(p) + element * (kType == GQ_F32 ? 4 : 2);
}
template <int kType>
static void* row_at(void* p, int64_t element) {
  return static_cast<char*>(p) + element * (kType == GQ_F32 ? 4 : 2);
}

static int router_checks(const void* logits, int32_t dtype, int64_t rows, int32_t E,
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

extern "C" int gq_moe_topk(const void* logits, int32_t dtype, int64_t rows, int32_t num_experts,
                           int64_t stride, int32_t topk, int32_t renormalize, int32_t* topk_ids,
                           float* topk_weights, hipStream_t stream) {
  using namespace gq;
  if (topk > num_experts) return kInvalid;
  const int st = router_checks(logits, dtype, rows, num_experts, stride, topk, topk_ids,
                               topk_weights, logits);
  if (st != kOk || rows == 0) return st;
  if (!aligned4(topk_ids) || !aligned4(topk_weights)) return kInvalid;
  auto go = [&](auto type) {
    constexpr int T = decltype(type)::value;
    constexpr int kMost = T == GQ_F32 ? 8 * kGroup : kGroupMaxExperts;
    if (num_experts <= kMost && topk <= kGroup && rows >= kGroupFrom &&
        (T != GQ_F32 || rows >= 64 * (int64_t)num_experts)) {
      by_group<kMost>(num_experts, [&](auto c) {
        constexpr int C = decltype(c)::value;
        by_rows(rows, kGroupRows, [&](int64_t at, int64_t n) {
          hipLaunchKernelGGL((moe_topk_group_kernel<T, C>),
                             dim3((unsigned)ceil_div64(n, kGroupRows)), dim3(kRouterThreads), 0,
                             stream, row_at<T>(logits, at * stride), n, num_experts, stride, topk,
                             renormalize, (int)group_wide<T, C>(logits, num_experts, stride),
                             topk_ids + at * topk, topk_weights + at * topk);
        });
      });
      return;
    }
    by_width(num_experts, [&](auto c) {
      by_rows(rows, kWaveRows, [&](int64_t at, int64_t n) {
        hipLaunchKernelGGL((moe_topk_kernel<T, decltype(c)::value>),
                           dim3((unsigned)ceil_div64(n, kWaveRows)), dim3(kRouterThreads), 0,
                           stream, row_at<T>(logits, at * stride), n, num_experts, stride, topk,
                           renormalize, topk_ids + at * topk, topk_weights + at * topk);
      });
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
  const int st = router_checks(logits, dtype, rows, num_experts, stride, topk, d_weights,
                               topk_ids, d_logits);
  if (st != kOk || rows == 0) return st;
  const uintptr_t mask = dtype == GQ_F32 ? 3 : 1;
  if (!aligned4(d_weights) || !aligned4(topk_ids) ||
      (reinterpret_cast<uintptr_t>(d_logits) & mask))
    return kInvalid;
  auto go = [&](auto type) {
    constexpr int T = decltype(type)::value;
    if (num_experts <= kGroupMaxExperts && topk <= kGroup && rows >= kGroupFrom) {
      by_group<kGroupMaxExperts>(num_experts, [&](auto c) {
        constexpr int C = decltype(c)::value;
        by_rows(rows, kGroupRows, [&](int64_t at, int64_t n) {
          hipLaunchKernelGGL((moe_topk_backward_group_kernel<T, C>),
                             dim3((unsigned)ceil_div64(n, kGroupRows)), dim3(kRouterThreads), 0,
                             stream, d_weights + at * topk, row_at<T>(logits, at * stride), n,
                             num_experts, stride, topk_ids + at * topk, topk, renormalize,
                             (int)group_wide<T, C>(logits, num_experts, stride),
                             (int)group_wide<T, C>(d_logits, num_experts, num_experts),
                             row_at<T>(d_logits, at * num_experts));
        });
      });
      return;
    }
    by_width(num_experts, [&](auto c) {
      by_rows(rows, kWaveRows, [&](int64_t at, int64_t n) {
        hipLaunchKernelGGL((moe_topk_backward_kernel<T, decltype(c)::value>),
                           dim3((unsigned)ceil_div64(n, kWaveRows)), dim3(kRouterThreads), 0,
                           stream, d_weights + at * topk, row_at<T>(logits, at * stride), n,
                           num_experts, stride, topk_ids + at * topk, topk, renormalize,
                           row_at<T>(d_logits, at * num_experts));
      });
    });
  };
  if (dtype == GQ_F32) go(std::integral_constant<int, GQ_F32>{});
  else if (dtype == GQ_BF16) go(std::integral_constant<int, GQ_BF16>{});
  else go(std::integral_constant<int, GQ_F16>{});
  return launch_status();
}
