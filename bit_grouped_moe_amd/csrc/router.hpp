// Pieces shared by the router's kernels (router.hip: softmax top-k and the
// gradients; moe_route.hip: scores of either kind, groups, a balancing bias):
// one element of a row, launches over rows, argument checks.
#pragma once

#include <type_traits>
#include <utility>

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

// ---- sixteen lanes a row -------------------------------------------------------
constexpr int kGroup = 16;
constexpr int kGroupRows = kRouterThreads / kGroup;
constexpr int kGroupMaxExperts = 16 * kGroup;

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

// Batcher's merge-exchange network for C keys, as a list of pairs.
template <int C>
struct SortNetwork {
  int count = 0;
  int u[C * C] = {}, v[C * C] = {};
  constexpr SortNetwork() {
    for (int p = 1; p < C; p *= 2)
      for (int k = p; k >= 1; k /= 2)
        for (int j = k % p; j + k < C; j += 2 * k)
          for (int i = 0; i < k; ++i)
            if (i + j + k < C && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
              u[count] = i + j;
              v[count++] = i + j + k;
            }
  }
};
template <typename F, int... k>
__device__ __forceinline__ void each_of(F&& f, std::integer_sequence<int, k...>) {
  (f(std::integral_constant<int, k>{}), ...);            // f(0), f(1), ...
}

// A lane's keys, largest first.
template <int C, typename key_t>
__device__ __forceinline__ void sort_down(key_t (&key)[C]) {
  constexpr SortNetwork<C> net;
  each_of(
      [&](auto at) {
        constexpr int u = net.u[decltype(at)::value], v = net.v[decltype(at)::value];
        const bool swap = key[u] < key[v];
        const key_t hi = swap ? key[v] : key[u], lo = swap ? key[u] : key[v];
        key[u] = hi;
        key[v] = lo;
      },
      std::make_integer_sequence<int, net.count>{});
}

// A lane's list without its first key, where `mine`.  (By a mask that the compiler
// does not see through: a selection between neighbours becomes a variable index,
// and the list leaves the registers; 16384 rows of 256 bf16 logits, top-8, 26 us.)
template <int C, typename key_t>
__device__ __forceinline__ void drop_first(key_t (&key)[C], bool mine) {
  uint32_t half = mine ? 0xFFFFFFFFu : 0u;
  asm("" : "+v"(half));
  const key_t mask = sizeof(key_t) == 8 ? (key_t)(((uint64_t)half << 32) | half) : (key_t)half;
#pragma unroll
  for (int c = 0; c < C; ++c) key[c] = ((c + 1 < C ? key[c + 1] : (key_t)0) & mask) | (key[c] & ~mask);
}

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
