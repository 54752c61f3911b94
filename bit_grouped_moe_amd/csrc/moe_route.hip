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
// then does not depend on the last bits of a float32 exponential.  That takes
// 64-bit arithmetic only where 32 bits leave a doubt (below).  Weights are float32,
// from the chosen logits.
//
// One wave a row, at most 16 experts a lane, expert 64 c + l in lane l.
#include "router.hpp"

namespace gq {

constexpr int kRouteMaxGroups = kWave;                   // a lane each

struct RouteArgs {
  const float* bias;             // [E] or null
  int E, topk, sigmoid, groups, topk_groups, group_top, renorm;
  uint32_t size_magic;           // expert / (E / groups) = expert * size_magic >> 20
  int share;                     // log2 of the lanes that look through a group
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
    const int group = lane >> g.share;
    if (group < g.groups) {
      const int size = g.E / g.groups;
      for (int i = lane & ((1 << g.share) - 1); i < size; i += 1 << g.share) {
        const uint64_t k = keys[group * size + i];
        second = max(second, min(first, k));
        first = max(first, k);
      }
    }
    for (int by = 1; by < 1 << g.share; by *= 2) {
      const uint64_t f = __shfl_xor(first, by, kWave), s = __shfl_xor(second, by, kWave);
      second = max(min(first, f), max(second, s));
      first = max(first, f);
    }
    if (g.group_top > 1 && second > kDeadKey64) first = key64(key_value(first) + key_value(second));
    int before = 0;                                      // groups ahead of this one
    for (int j = 0; j < g.groups; ++j) {
      const uint64_t k =
          ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(first >> 32), j << g.share) << 32) |
          (uint32_t)__builtin_amdgcn_readlane((int)first, j << g.share);
      before += k > first || (k == first && j < group);
    }
    const uint64_t open = __ballot(group < g.groups && before < g.topk_groups);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = 64 * c + lane;
      if (!((open >> ((((uint32_t)e * g.size_magic) >> 20) << g.share & 63u)) & 1ull)) key[c] = 0ull;
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

// ---- in 32 bits, where that decides -------------------------------------------
// Scores in float32 from the hardware exponential and reciprocal (an ulp each).  A
// sigmoid is off by less than off = 2^-22 (s (1 - s) |z| < 1/4 times the argument's
// rounding, and an ulp each of the exponential, the sum and the reciprocal), the sum
// with the bias by 2^-24 of itself.
// A softmax's score is e^-x / sum, x how far its logit lies below the peak.  Far below,
// where x's rounding counts x times, it is off by several 2^-19 of itself; what is
// needed and holds is a bound on differences of choices, by off = 2^-19 of the row's
// largest score.  In units of 2^-24 of that score: the argument x log2 e is off by 2.3 x
// (x, log2 e and their product rounded), so a numerator by e^-x (2.3 x + 2) <= 2.1, and
// by 1 where it is multiplied by the sum's inverse: 3.1 of a score's own.  The inverse
// is off by 2.3 times the row's mean of x weighted by e^-x (at most 4.5 for 1024
// experts), 2 for the exponentials, 22 additions and 2 for the reciprocal: 37 for the
// largest score and in proportion for every other, the same way for all.  Two scores'
// difference is so off by 37 + 2 3.1 < 64 = 2 off, that of two sums of two by
// 2 37 + 4 3.1 < 128 = 4 off, and one score against its value in 64 bits by
// 37 + 3.1 < 2 off.
// Two choices further apart than that and their sums' roundings are in the order of
// float64; so are choices of equal logits and biases, by index.  A row that this does
// not decide is selected again in 64 bits: one row in 10^3 with random float32 logits
// and biases.
__device__ __forceinline__ float fast_exp(float d) {
  return __builtin_amdgcn_exp2f(d * 1.44269504088896341f);
}
__device__ __forceinline__ float fast_sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + fast_exp(-z));
}
// Whether a choice a (at least) lies clearly above a choice b (at most), the difference
// of whose scores is off by less than 2 `off`; false with a NaN.
__device__ __forceinline__ bool clearly(float a, float b, float off) {
  return a - b > 2.f * off + 0x1p-23f * (fabsf(a) + fabsf(b));
}
// A group's value from the keys of its largest and (sums) second largest choice, as
// a key (0: all masked), and the keys of bounds of what it is in 64 bits.  The
// choices may cancel: their roundings count by their own size, not by their sum's.
struct GroupValue {
  uint32_t key, low, high;
  __device__ __forceinline__ GroupValue(uint32_t first, uint32_t second, float off, bool sums) {
    float v = first > kDeadKey ? key_logit(first) : -__builtin_inff();
    float size = fabsf(v);
    if (sums && second > kDeadKey) {
      const float w = key_logit(second);
      v += w;
      size += fabsf(w);
    }
    key = first > kDeadKey ? logit_key(v) : 0u;
    // off for each choice (against another group's as many); half a step for each, for v
    // and for a bound itself
    const float room = (sums ? 2.f : 1.f) * off + 0x1p-22f * size;
    const bool sound = room < __builtin_inff();          // no NaN, nothing overflowed
    low = sound ? logit_key(v - room) : 0u;
    high = sound ? logit_key(v + room) : ~0u;
  }
};

// The two largest of this lane's two and another lane's.
template <int kCtrl>
__device__ __forceinline__ void two_largest(uint32_t& first, uint32_t& second) {
  const uint32_t f = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)first, kCtrl, 0xF, 0xF, false);
  const uint32_t s = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)second, kCtrl, 0xF, 0xF, false);
  second = max(min(first, f), max(second, s));
  first = max(first, f);
}

// A slot's weight before the division by their sum, from the logit zs of its expert
// id (-1: none), and the peak that the sum is taken over.
struct RowWeights {
  float peak, part;
  // slots, all: the largest key of the slots' logits and (softmax) of the row's
  __device__ __forceinline__ RowWeights(const RouteArgs& g, int id, float zs, uint32_t slots,
                                        uint32_t all) {
    const bool broken = !g.sigmoid && all >= 0xFF800000u;  // a softmax with a NaN or +inf
    const uint32_t m = !g.sigmoid && !g.renorm ? all : slots;
    peak = broken ? __uint_as_float(0x7FC00000u) : m > kDeadKey ? key_logit(m) : 0.f;
    part = id < 0      ? 0.f
           : g.sigmoid ? sigmoid_over(zs, g.renorm && peak <= 0.f ? peak : 0.f)
                       : expf(zs - peak);
  }
};

// One wave a row.  LDS: the larger of 64-bit and 32-bit keys of the row.
template <int kType, int C>
__global__ __launch_bounds__(kRouterThreads) void moe_route_kernel(
    const void* __restrict__ logits, int64_t rows, int64_t stride, RouteArgs g) {
  __shared__ uint64_t keys[kWaveRows][C * kWave];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t row = (int64_t)blockIdx.x * kWaveRows + wave;
  if (row >= rows) return;
  const float kInf = __builtin_inff();
  float z[C], b[C];
#pragma unroll
  for (int c = 0; c < C; ++c) z[c] = load1<kType>(logits, row * stride + min(64 * c + lane, g.E - 1));
#pragma unroll
  for (int c = 0; c < C; ++c) b[c] = g.bias ? g.bias[min(64 * c + lane, g.E - 1)] : 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) asm volatile("" : "+v"(z[c]), "+v"(b[c]));
  uint32_t all = 0u;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (64 * c + lane >= g.E) z[c] = -kInf;
    all = max(all, logit_key(z[c]));
  }
  if (!g.sigmoid) all = wave_umax(all);

  const bool sums = g.groups > 1 && g.group_top > 1;
  float score[C];
  float off = 0x1p-22f;
  if (g.bias || sums) {
    if (g.sigmoid) {
#pragma unroll
      for (int c = 0; c < C; ++c) score[c] = fast_sigmoid(z[c]);
    } else {
      const float peak = all > kDeadKey ? key_logit(all) : 0.f;
      float total = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        score[c] = fast_exp(z[c] - peak);
        total += score[c];
      }
      total = __builtin_amdgcn_rcpf(wave_fsum(total));
      off = 0x1p-19f * total;
#pragma unroll
      for (int c = 0; c < C; ++c) score[c] *= total;
    }
  }
  uint32_t key[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    key[c] = z[c] == -kInf ? kDeadKey : logit_key(g.bias ? score[c] + b[c] : z[c]);
    if (64 * c + lane >= g.E) key[c] = 0u;
  }
  bool sure = true;                                      // uniform
  if (g.groups > 1) {
    uint32_t* k32 = reinterpret_cast<uint32_t*>(keys[wave]);
#pragma unroll
    for (int c = 0; c < C; ++c)
      k32[64 * c + lane] = sums && !g.bias && key[c] > kDeadKey ? logit_key(score[c]) : key[c];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    // 2^share lanes a group (at most 16), each every 2^share-th of its experts
    uint32_t first = 0u, second = 0u;
    const int group = lane >> g.share;
    if (group < g.groups) {
      const int size = g.E / g.groups;
      for (int i = lane & ((1 << g.share) - 1); i < size; i += 1 << g.share) {
        const uint32_t k = k32[group * size + i];
        second = max(second, min(first, k));
        first = max(first, k);
      }
    }
    if (g.share > 0) two_largest<0xB1>(first, second);
    if (g.share > 1) two_largest<0x4E>(first, second);
    if (g.share > 2) two_largest<0x141>(first, second);
    if (g.share > 3) two_largest<0x140>(first, second);
    const GroupValue value(first, second, off, sums);
    const uint32_t mine = value.key;
    int before = 0;                                      // groups ahead of this one
    for (int j = 0; j < g.groups; ++j) {
      const uint32_t k = (uint32_t)__builtin_amdgcn_readlane((int)mine, j << g.share);
      before += k > mine || (k == mine && j < group);
    }
    const bool in = group < g.groups && before < g.topk_groups;
    const uint64_t open = __ballot(in);
    if (g.bias || sums) {
      // the least open and the largest closed group
      const uint32_t least = ~wave_umax(in && mine ? ~value.low : 0u);
      const uint32_t most = wave_umax(group < g.groups && !in && mine ? value.high : 0u);
      sure = most <= kDeadKey || least > most;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = 64 * c + lane;
      const uint32_t bit = (((uint32_t)e * g.size_magic) >> 20) << g.share & 63u;
      if (!((open >> bit) & 1ull)) key[c] = 0u;
    }
  }
  int id = -1;
  float zs = -kInf, won = -kInf;
  if (sure) {
    wave_topk<C>(key, g.topk, id, won);
    zs = g.bias && id >= 0 ? load1<kType>(logits, row * stride + id) : won;
    if (g.bias) {
      uint32_t best = key[0];
#pragma unroll
      for (int c = 1; c < C; ++c) best = max(best, key[c]);
      best = wave_umax(best);                            // the largest that was not chosen
      float next = __shfl_down(won, 1, kWave);
      int next_id = __shfl_down(id, 1, kWave);
      if (lane == g.topk - 1) {
        next = best > kDeadKey ? key_logit(best) : -kInf;
        next_id = -1;
      }
      const bool slot = lane < g.topk && id >= 0 && next != -kInf;
      bool close = slot && !clearly(won, next, off);
      if (__ballot(close)) {
        // slots of equal logits and biases are in the order of their indices
        const float zn = __shfl_down(zs, 1, kWave);
        const float bs = id >= 0 ? g.bias[id] : 0.f, bn = next_id >= 0 ? g.bias[next_id] : 0.f;
        close = close && !(next_id >= 0 && zs == zn && bs == bn);
        sure = !__ballot(close);
      }
    }
  }
  if (!sure) select64<C>(g, z, lane, keys[wave], id, zs);
  const uint32_t slots = wave_umax(id >= 0 ? logit_key(zs) : 0u);
  const RowWeights w(g, id, zs, slots, all);
  float total = w.part;
  if (!g.sigmoid && !g.renorm) {
    total = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) total += z[c] == -kInf ? 0.f : expf(z[c] - w.peak);
  }
  total = g.sigmoid && !g.renorm ? 1.f : wave_fsum(total);
  if (lane < g.topk) {
    g.ids[row * g.topk + lane] = id;
    g.weights[row * g.topk + lane] = id >= 0 ? w.part / total * g.scale : 0.f;
  }
}

// ---- many rows of up to 256 experts and 16 slots: sixteen lanes a row ----------
// Lane l of a row holds experts C l .. C l + C - 1.  A group is 2^j whole lanes (the
// host checks): its best are found in the lane and merged with DPP moves, its rank
// by rotating the groups' values past each other.  Experts are selected as in the
// softmax top-k's kernel, from sorted lists of keys that no two experts share: the
// choice's key without its last 8 bits, and the expert.  (16-bit logits' own order
// needs no more than the other 24.)  Where two neighbours in a row's slots are too
// close for that, in 4% of rows, its sixteen largest are put in order in 64 bits, a
// lane each; what is left, groups that are too close among them (one row in 10^4),
// goes to the selection in 64 bits, by the whole wave, one row after the other.
// From how many rows: a wave a row until the chip is full of waves (bf16 logits without
// groups, a wave against sixteen lanes a row, of 256 experts: 2048 rows 5.5 and 6.7 us,
// 4096 9.7 and 6.8, 16384 16.6 and 11.3; of 128: 4.5 and 5.6, 6.5 and 5.6, 13.8 and 8.0;
// float32 with groups, of 64: 4.8 and 5.5, 6.0 and 5.6, 13.7 and 7.6; of 256 in 8
// groups, whose selection holds a wave twice as long: 1024 rows 6.0 and 8.0, 2048 10.3
// and 8.1, 16384 23.1 and 14.8).
constexpr int kRouteGroupFrom = 4096, kRouteGroupFromWide = 2048;

template <int kType, int C>
__global__ __launch_bounds__(kRouterThreads) void moe_route_group_kernel(
    const void* __restrict__ logits, int64_t rows, int64_t stride, int wide, int lanes,
    RouteArgs g) {
  using Row = GroupRow<kType, C>;
  constexpr int kC64 = C * kGroup / kWave;
  constexpr uint32_t kLive = (kDeadKey + 1) & ~255u;     // keys of live experts are not below
  __shared__ uint64_t keys[kWaveRows][kC64 * kWave];
  const int lane = threadIdx.x & (kWave - 1), l = lane & (kGroup - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t base = (int64_t)blockIdx.x * kGroupRows + wave * (kWave / kGroup);
  const int64_t own = base + lane / kGroup;
  const int64_t row = own < rows ? own : rows - 1;       // every lane takes part in the maxima
  const typename Row::raw* zrow = static_cast<const typename Row::raw*>(logits) + row * stride;
  const float kInf = __builtin_inff();
  Row x;
  x.load(zrow, l, g.E, wide);
  float z[C], b[C];
  if (g.bias && C * l + C <= g.E) {
    typedef uint32_t vec __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
    for (int c = 0; c < C; c += 4) {
      const vec v = *reinterpret_cast<const vec*>(g.bias + C * l + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) b[c + i] = __uint_as_float(v[i]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c) b[c] = g.bias ? g.bias[min(C * l + c, g.E - 1)] : 0.f;
  }
  uint32_t all = 0u;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    z[c] = C * l + c < g.E ? Row::value(x.r[c]) : -kInf;
    if (!g.sigmoid) all = max(all, logit_key(z[c]));
  }
  if (!g.sigmoid) all = group_max(all);
  const bool sums = g.groups > 1 && g.group_top > 1;
  float score[C];
  float off = 0x1p-22f;
  if (g.bias || sums) {
    if (g.sigmoid) {
#pragma unroll
      for (int c = 0; c < C; ++c) score[c] = fast_sigmoid(z[c]);
    } else {
      const float peak = all > kDeadKey ? key_logit(all) : 0.f;
      float total = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        score[c] = fast_exp(z[c] - peak);
        total += score[c];
      }
      total = __builtin_amdgcn_rcpf(group_sum_last(total, kGroup));
      off = 0x1p-19f * total;
#pragma unroll
      for (int c = 0; c < C; ++c) score[c] *= total;
    }
  }
  uint32_t key[C];
#pragma unroll
  for (int c = 0; c < C; ++c)
    key[c] = z[c] == -kInf ? 0u : logit_key(g.bias ? score[c] + b[c] : z[c]);
  bool doubt = false;
  if (g.groups > 1) {
    uint32_t first = 0u, second = 0u;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t k = sums && !g.bias && key[c] > kDeadKey ? logit_key(score[c]) : key[c];
      second = max(second, min(first, k));
      first = max(first, k);
    }
    if (lanes > 1) two_largest<0xB1>(first, second);
    if (lanes > 2) two_largest<0x4E>(first, second);
    if (lanes > 4) two_largest<0x141>(first, second);
    const GroupValue value(first, second, off, sums);
    const uint32_t mine = value.key;
    int before = 0;                                      // groups ahead of this one
    auto turn = [&](auto by) {
      constexpr int kBy = decltype(by)::value + 1;
      if (kBy & (lanes - 1)) return;                     // uniform
      const uint32_t k =
          (uint32_t)__builtin_amdgcn_update_dpp(0, (int)mine, 0x120 + kBy, 0xF, 0xF, false);
      const int from = __builtin_amdgcn_update_dpp(0, l, 0x120 + kBy, 0xF, 0xF, false);
      before += k > mine || (k == mine && from < l);
    };
    each_of(turn, std::make_integer_sequence<int, kGroup - 1>{});
    const bool in = before < g.topk_groups;
    if (g.bias || sums) {
      // the least open and the largest closed group (lanes past the experts are
      // empty groups behind all others)
      const uint32_t least = ~group_max(in && mine ? ~value.low : 0u);
      const uint32_t most = group_max(!in && mine ? value.high : 0u);
      doubt = most > kDeadKey && least <= most;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) key[c] = in ? key[c] : 0u;
  }
#pragma unroll
  for (int c = 0; c < C; ++c)
    key[c] = key[c] > kDeadKey ? (key[c] & ~255u) | (255u - (uint32_t)(C * l + c)) : 0u;
  sort_down<C>(key);
  uint32_t won = 0u;
  for (int s = 0; s < g.topk; ++s) {
    const uint32_t m = group_max(key[0]);
    won = l == s ? m : won;
    drop_first<C>(key, key[0] == m);
  }
  int id = won >= kLive ? 255 - (int)(won & 255u) : -1;
  float zs = id >= 0 ? Row::value(zrow[id]) : -kInf;
  if (g.bias || kType == GQ_F32) {
    uint32_t left = group_max(key[0]);                   // the largest that was not chosen
    const uint32_t right = (uint32_t)__shfl_down((int)won, 1, kGroup);
    const uint32_t next = l == g.topk - 1 ? left : right;
    bool close = l < g.topk && id >= 0 && next >= kLive;
    if (g.bias) close = close && !clearly(key_logit(won & ~255u), key_logit(next | 255u), off);
    else close = close && (won ^ next) < 256u;
    if (__ballot(close)) {
      // The sixteen largest by these keys in the order of their choices in 64 bits.
      // That settles a row whose last slot then lies clearly above every other expert.
      for (int s = g.topk; s < kGroup; ++s) {
        won = l == s ? left : won;
        drop_first<C>(key, key[0] == left);
        left = group_max(key[0]);
      }
      const int cand = won >= kLive ? 255 - (int)(won & 255u) : -1;
      const float zc = cand >= 0 ? Row::value(zrow[cand]) : -kInf;
      double value = (double)zc;
      if (g.bias) {
        double total = 1.0, peak = 0.0;
        if (!g.sigmoid) {
          peak = all > kDeadKey ? (double)key_logit(all) : 0.0;
          total = 0.0;
#pragma unroll 1
          for (int e = l; e < g.E; e += kGroup) {
            const float v = Row::value(zrow[e]);
            total += v == -kInf ? 0.0 : exp((double)v - peak);
          }
#pragma unroll
          for (int off = kGroup / 2; off > 0; off >>= 1) total += __shfl_xor(total, off, kWave);
        }
        value = cand < 0    ? -(double)kInf
                : g.sigmoid ? 1.0 / (1.0 + exp(-(double)zc)) + (double)g.bias[cand]
                            : exp((double)zc - peak) / total + (double)g.bias[cand];
      }
      const uint64_t mine = cand < 0 ? 0ull : key64(value);
      const int tie = cand < 0 ? 256 + l : cand;
      int rank = 0;
      each_of(
          [&](auto by) {
            constexpr int kCtrl = 0x121 + decltype(by)::value;
            const uint64_t k =
                ((uint64_t)(uint32_t)__builtin_amdgcn_update_dpp(0, (int)(mine >> 32), kCtrl, 0xF,
                                                                 0xF, false) << 32) |
                (uint32_t)__builtin_amdgcn_update_dpp(0, (int)mine, kCtrl, 0xF, 0xF, false);
            const int other = __builtin_amdgcn_update_dpp(0, tie, kCtrl, 0xF, 0xF, false);
            rank += k > mine || (k == mine && other < tie);
          },
          std::make_integer_sequence<int, kGroup - 1>{});
      const bool row_close = (__ballot(close) >> (lane & ~(kGroup - 1)) & 0xFFFFull) != 0;
      close = row_close && rank < g.topk && cand >= 0 && left >= kLive &&
              !clearly((float)value, key_logit(left | 255u), off);
      const int to = 4 * ((lane & ~(kGroup - 1)) + rank);
      const int sent = __builtin_amdgcn_ds_permute(to, cand);
      const int sent_z = __builtin_amdgcn_ds_permute(to, __float_as_int(zc));
      if (row_close) {
        id = l < g.topk ? sent : -1;
        zs = l < g.topk ? __int_as_float(sent_z) : -kInf;
      }
    }
    doubt = doubt || close;
  }
  const uint64_t doubts = __ballot(doubt && own < rows);
  if (doubts) {
    for (int r = 0; r < kWave / kGroup; ++r) {
      if (!((doubts >> (kGroup * r)) & 0xFFFFull)) continue;
      float zr[kC64];
#pragma unroll
      for (int c = 0; c < kC64; ++c) {
        const int e = 64 * c + lane;
        zr[c] = e < g.E ? load1<kType>(logits, (base + r) * stride + e) : -kInf;
      }
      int wid;
      float wz;
      select64<kC64>(g, zr, lane, keys[wave], wid, wz);
      const int tid = __shfl(wid, l, kWave);
      const float tz = __shfl(wz, l, kWave);
      if (lane / kGroup == r) {
        id = tid;
        zs = tz;
      }
    }
  }
  const uint32_t slots = group_max(id >= 0 ? logit_key(zs) : 0u);
  const RowWeights w(g, id, zs, slots, all);
  float total = w.part;
  if (!g.sigmoid && !g.renorm) {
    total = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) total += z[c] == -kInf ? 0.f : expf(z[c] - w.peak);
  }
  total = g.sigmoid && !g.renorm ? 1.f : group_sum_last(total, kGroup);
  if (l < g.topk && own < rows) {
    g.ids[row * g.topk + l] = id;
    g.weights[row * g.topk + l] = id >= 0 ? w.part / total * g.scale : 0.f;
  }
}

// Lanes of a group where C experts a lane make it 1, 2, 4 or 8 whole ones (1 without
// groups), else 0.
static int route_lanes(int E, int groups, int C) {
  if (groups == 1) return 1;
  const int size = E / groups;
  const int lanes = size / C;
  return size % C == 0 && (lanes & (lanes - 1)) == 0 && lanes <= 8 ? lanes : 0;
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
  while (g.share < 4 && groups << (g.share + 1) <= kWave) ++g.share;
  auto go = [&](auto type) {
    constexpr int T = decltype(type)::value;
    bool done = false;
    if (num_experts <= kGroupMaxExperts && topk <= kGroup &&
        rows >= (groups > 1 && num_experts > 128 ? kRouteGroupFromWide : kRouteGroupFrom))
      by_group<kGroupMaxExperts>(num_experts, [&](auto c) {
        constexpr int C = decltype(c)::value;
        const int lanes = route_lanes(num_experts, groups, C);
        if (!lanes) return;
        done = true;
        by_rows(rows, kGroupRows, [&](int64_t at, int64_t n) {
          g.ids = topk_ids + at * topk;
          g.weights = topk_weights + at * topk;
          hipLaunchKernelGGL((moe_route_group_kernel<T, C>),
                             dim3((unsigned)ceil_div64(n, kGroupRows)), dim3(kRouterThreads), 0,
                             stream, row_at<T>(logits, at * stride), n, stride,
                             (int)group_wide<T, C>(logits, num_experts, stride), lanes, g);
        });
      });
    if (done) return;
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
