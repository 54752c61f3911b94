// Selection of the largest logits of a row by one wave, shared by the router
// kernels and the decode layer.
#pragma once

#include <type_traits>

#include "gq_device.hpp"

namespace gq {

// v with lane `lane` (uniform) set to `value` (uniform): v_writelane_b32, which
// the compiler offers as an intrinsic only.
__device__ uint32_t wave_writelane(uint32_t value, uint32_t lane, uint32_t v) __asm(
    "llvm.amdgcn.writelane.i32");

constexpr int kTopkMax = 64;                 // slots: one per lane
constexpr int kTopkMaxExperts = 1024;        // 16 logits per lane

// Order-preserving key of a logit: larger logit, larger key; -0 and +0 are
// one value; NaN is above every number (a NaN logit is chosen and makes its
// row's weights NaN: it is never hidden); -inf, a masked expert, is kDeadKey
// and is never chosen.  A slot past the row's experts has key 0.
constexpr uint32_t kDeadKey = 0x007FFFFFu;
__device__ __forceinline__ uint32_t logit_key(float z) {
  const uint32_t b = __float_as_uint(z + 0.0f);
  const uint32_t k = b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
  return z != z ? 0xFFFFFFFFu : k;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  if (k == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
  return __uint_as_float((k >> 31) ? k ^ 0x80000000u : ~k);
}

// Keys of a row: lane l takes experts 64 c + l, load(e) a logit.  All loads are
// in flight before the first is used: left to itself, the compiler puts each
// behind the test of its expert and waits for one before it asks for the next
// (one-token NF4 layer 14.1 -> 13.8 us).
template <int C, typename F>
__device__ __forceinline__ void wave_keys(int E, int lane, F&& load, uint32_t (&key)[C]) {
  float z[C];
#pragma unroll
  for (int c = 0; c < C; ++c) z[c] = load(min(64 * c + lane, E - 1));
#pragma unroll
  for (int c = 0; c < C; ++c) asm volatile("" : "+v"(z[c]));
#pragma unroll
  for (int c = 0; c < C; ++c) key[c] = 64 * c + lane < E ? logit_key(z[c]) : 0u;
}

// Maximum over the wave, in every lane's scalar (uniform) result.
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  auto step = [&](auto ctrl, auto mask) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value,
                                                     decltype(mask)::value, 0xF, false));
  };
  step(std::integral_constant<int, 0xB1>{}, std::integral_constant<int, 0xF>{});
  step(std::integral_constant<int, 0x4E>{}, std::integral_constant<int, 0xF>{});
  step(std::integral_constant<int, 0x141>{}, std::integral_constant<int, 0xF>{});
  step(std::integral_constant<int, 0x140>{}, std::integral_constant<int, 0xF>{});
  step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});
  step(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0x8>{});
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Sum over the wave in a fixed order, the same value in every lane.
__device__ __forceinline__ float wave_fsum(float v) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(group_sum_last(v, 64)), 63));
}

// The topk largest of the row's logits, largest first, equal ones by lower
// index.  Lane l holds experts 64 c + l in key[c]; lane s < topk receives
// slot s (id -1 where only masked experts are left).  A round is a wave
// maximum and C ballots; the place of the first match is scalar, and the
// slot's values and the taken key are written with v_writelane: 20 VALU
// instructions a round for 128 experts, 30 with selects on the lane number
// (graph-replayed, inputs in turn, selects -> this: 16384 rows of 128 experts,
// top-32, 24.5 -> 22.8 us; of 512, top-8, 17.1 -> 16.5; 2048 rows of 128 3.51 ->
// 3.37; one-token layer of 512 experts 12.5 -> 12.2, of 128 the same, 13.9).  No
// memory.
template <int C>
__device__ __forceinline__ void wave_topk(uint32_t (&key)[C], int topk, int& id, float& logit) {
  uint32_t ids = 0xFFFFFFFFu, won = kDeadKey;
  for (int s = 0; s < topk; ++s) {
    uint32_t best = key[0];
#pragma unroll
    for (int c = 1; c < C; ++c) best = max(best, key[c]);
    const uint32_t m = wave_umax(best);
    if (m <= kDeadKey) break;                            // uniform
    won = wave_writelane(m, s, won);
    bool open = true;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint64_t at = __ballot(key[c] == m);
      if (open && at) {                                  // uniform
        open = false;
        const int l = __builtin_ctzll(at);
        key[c] = wave_writelane(0u, l, key[c]);
        ids = wave_writelane((uint32_t)(64 * c + l), s, ids);
      }
    }
  }
  id = (int)ids;
  logit = key_logit(won);
}

// The row's largest logit (slot 0's); 0 where every expert is masked.
__device__ __forceinline__ float row_peak(float logit, int id) {
  const float p = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(logit), 0));
  return __builtin_amdgcn_readlane(id, 0) < 0 ? 0.0f : p;
}

}  // namespace gq
