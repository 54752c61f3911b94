// A whole mixture-of-experts layer for a few tokens (at most 8 tokens and 64
// routed pairs): router product, selection, the experts' gated products and
// the weighted combine, without a host round trip.
//
//   z = x Wr^T + br                                          moe_logits_kernel
//   e_s, w_s = the topk largest logits of a token, softmax   moe_gate_up_kernel
//   a_s = unit(Wgu[e_s] x + bgu[e_s])                        moe_gate_up_kernel
//   y = sum_s w_s (Wd[e_s] a_s + bd[e_s])                    moe_down_kernel
//
// Everything between the bf16 input and the bf16 output is float32 (logits,
// weights, gated products: the workspace holds them).  Bound by the latency
// of the dependent round trips for one token; for eight tokens of NF4 experts
// by VALU time (gate_up 24 us, busy 84%; down 17 us, 62%, LDS 64%), of MXFP4
// experts by the load path (gate_up 50 us, address unit busy 74%; down 38 us).
//
// The launches are the dependencies between workgroups: the logits need
// every hidden element and are spread over the chip (one workgroup per
// expert); the gate_up product needs the selection, the down product whole
// activation rows.  The selection is one wave's work on a token's logits:
// every gate_up workgroup makes it for its own token, as far as its own slot.
// A launch of its own between the two, which wrote all selections, cost more
// than that for any number of tokens (8 NF4 tokens, E = 128: 46.2 us a layer,
// so 44.5; 2 tokens 22.0 and 20.6; 8 MXFP4 tokens of 2880 82.1 and 81.0).
#include <algorithm>
#include <type_traits>

#include "gemv_common.hpp"
#include "topk.hpp"
#include "gq_host.hpp"
#include "../../include/gq.h"

namespace gq {

constexpr int kMoeMaxRows = 8;
constexpr int kMoeMaxPairs = 64;             // a wave's lanes
constexpr int kMoeMaxExperts = 512;          // logits of a token: 8 per lane
constexpr int kMoeMaxHidden = 8192;          // 256 segments of 32 weights
constexpr int kMoeMaxInner = 128 * 32;       // two segments per lane
constexpr int kMoeThreads = 256;
constexpr int kDownWaves = 8;
constexpr int kDownLanes = 8;                // of a row at least: bounds the rows a workgroup keeps

// Place of a pair's activation n in the workspace: the 4-value piece v of
// segment s is piece v S + s, so that the down product's lanes, a segment
// each, read 16 consecutive bytes per lane.  (In the order of n a lane's
// pieces lie 128 bytes apart, 64 lines an instruction: one-token MXFP4 layer
// 21.1 us, so 18.7; eight NF4 tokens 46.2, so 45.3.)
__device__ __forceinline__ int act_place(int n, int S) {
  return ((((n >> 2) & 7) * S + (n >> 5)) << 2) + (n & 3);
}

// ---- logits of one expert for every token -------------------------
// Workgroup e; thread t takes the 16-byte pieces t, t + 256, ... of the
// expert's row and of each token's.  v_dot2_f32_bf16 keeps subnormal operands,
// products and sums; on 80000 random operands its result was off by at most
// 2.6 2^-24 of the sum of its three terms' magnitudes (two fused multiply-adds:
// at most 2), so that the logits have float32 sums' accuracy.
template <int kRows>
__global__ __launch_bounds__(kMoeThreads) void moe_logits_kernel(
    const uint16_t* __restrict__ x, const uint16_t* __restrict__ w, int H, int x_stride, int rows,
    int E, const uint16_t* __restrict__ bias, float* __restrict__ logits) {
  __shared__ float part[kMoeThreads / kWave][kRows];
  const int e = blockIdx.x, tid = threadIdx.x;
  const int wave = tid / kWave, lane = tid & (kWave - 1);
  // raw until it is added, and loaded without a branch (no bias: some weight's
  // bits, not used): converted at once, the load would be waited for here
  const uint32_t braw = (bias ? bias : w)[e];
  float acc[kRows];
#pragma unroll
  for (int t = 0; t < kRows; ++t) acc[t] = 0.f;
  const u32x4* wr = reinterpret_cast<const u32x4*>(w + (int64_t)e * H);
  // (unrolled: ahead of a loop the compiler waits for what is in flight)
#pragma unroll
  for (int it = 0; it < kMoeMaxHidden / 8 / kMoeThreads; ++it) {
    const int c = tid + it * kMoeThreads;
    if (c >= H / 8) break;
    const u32x4 wv = wr[c];
    u32x4 xv[kRows];
#pragma unroll
    for (int t = 0; t < kRows; ++t)
      xv[t] = *reinterpret_cast<const u32x4*>(x + (int64_t)min(t, rows - 1) * x_stride + c * 8);
    // (all loads before the first use: left to itself, the compiler waits for
    // each token's piece before it asks for the next)
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < kRows; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // (scalar copies: a bit_cast of a vector element reads element 0)
        const uint32_t a = wv[i], b = xv[t][i];
        acc[t] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a),
                                                 __builtin_bit_cast(bf16x2, b), acc[t], false);
      }
  }
#pragma unroll
  for (int t = 0; t < kRows; ++t) {
    const float s = group_sum_last(acc[t], kWave);
    if (lane == kWave - 1) part[wave][t] = s;
  }
  lds_barrier();
  if (tid < rows) {
    float s = part[0][tid];
#pragma unroll
    for (int i = 1; i < kMoeThreads / kWave; ++i) s += part[i][tid];
    logits[(int64_t)tid * E + e] = s + (bias ? __uint_as_float(braw << 16) : 0.f);
  }
}

// ---- selection of one token by one wave ----------------------------------------
// The first `slots` slots into id (lane s: slot s); with `write`, all slots'
// ids and softmax weights to memory.
template <int C>
__device__ __forceinline__ int moe_select(const float* __restrict__ logits, int E, int topk,
                                          int slots, int lane, bool write, int renorm,
                                          int32_t* __restrict__ ids, float* __restrict__ w) {
  uint32_t key[C], all[C];
  wave_keys<C>(E, lane, [&](int e) { return logits[e]; }, key);
#pragma unroll
  for (int c = 0; c < C; ++c) all[c] = key[c];
  int id;
  float z;
  wave_topk<C>(key, slots, id, z);
  if (write) {
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
      ids[lane] = id;
      w[lane] = id >= 0 ? part / total : 0.f;
    }
  }
  return id;
}

// ---- gate_up product and gated unit ----------------------------------------------
// Grid (column chunks, pairs), the row layout of the decode GEMV: workgroup
// (x, p) computes the output column chunks x, x + gridDim.x, ... of pair p.
// Pairs that share an expert each read its rows: a workgroup that served all
// of them (as in the decode GEMV) decodes once per pair anyway, and the
// longest such group then sets the time (8 tokens on E = 128 NF4 experts:
// 54.4 us a layer, 8 equal tokens 55.4; one pair a workgroup 50.6 and 45.0,
// the repeated rows coming from the caches).
// NF4: gate row j, up row I + j, SwiGLU; MXFP4: gate row 2j, up row 2j + 1,
// the clamped unit.  The workgroup selects for itself (C logits a lane), as
// far as its own slot (a token's experts are distinct), and the last slot's
// first workgroup writes the token's selection for the down product.  kLoop:
// several chunks a workgroup, the next one's rows loading while this one's
// are decoded, and the NF4 table in 16 copies, so that 16 lanes never meet in
// a bank (8 tokens, E = 128: 44.4 us a layer, so 42.9; where a workgroup has
// one chunk, filling 32 KB costs more than that: one token 14.0, so 16.2; in
// the down product, of a third of the weights, it gains nothing).
constexpr int kCopiesLog = 4;
template <bool kMx, int kIter, bool kWaveRows, int C, bool kLoop>
__global__ __launch_bounds__(kMoeThreads) void moe_gate_up_kernel(
    const float* __restrict__ logits, const uint16_t* __restrict__ x,
    const uint8_t* __restrict__ codes, const void* __restrict__ scl, int H, int I, int E,
    int x_stride, int topk, const uint16_t* __restrict__ bias, float alpha, float limit,
    int renorm, int32_t* __restrict__ ids, float* __restrict__ w, float* __restrict__ act) {
  constexpr int kHalf = kIter / 2;
  constexpr int kLog = !kMx && kLoop ? kCopiesLog : 0;
  __shared__ __attribute__((aligned(4096))) LutT lut_s[kMx ? 1 : kLutN << kLog];
  __shared__ float red[kWaveRows ? 1 : kIter * (kMoeThreads + 32)];
  __shared__ int mine_s;

  const int N = 2 * I;
  const int S = H >> 5;
  int W, G, NT;
  if constexpr (kWaveRows) {
    const int lgW = S > 1 ? 32 - __builtin_clz(S - 1) : 0;
    W = 1 << lgW;
    G = kMoeThreads >> lgW;
    NT = kMoeThreads;
  } else {
    W = S;
    G = S >= kMoeThreads ? 1 : kMoeThreads / S;
    NT = ((S * G + kWave - 1) / kWave) * kWave;
  }
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int p0 = blockIdx.y;
  const int R = G * kIter, Rout = R / 2;
  const int g = tid / W, s = tid - g * W;
  const bool active = kWaveRows ? s < S : tid < S * G;

  // the pair's activations and the table, ahead of the selection
  u32x4 xr[4];
  {
    const u32x4* xp = reinterpret_cast<const u32x4*>(x + (int64_t)(p0 / topk) * x_stride +
                                                      (active ? s : 0) * 32);
#pragma unroll
    for (int v = 0; v < 4; ++v) xr[v] = xp[v];
  }
  if constexpr (!kMx) lut_init_copies<kLog>(lut_s, tid, NT);
  const LutT* lut = lut_s + (lane & ((1 << kLog) - 1));

  if (wave == 0) {
    const int t = p0 / topk, slot = p0 - t * topk;
    const bool write = blockIdx.x == 0 && slot == topk - 1;
    const int id = moe_select<C>(logits + (int64_t)t * E, E, topk, slot + 1, lane, write, renorm,
                                 ids + t * topk, w + t * topk);
    if (lane == slot) mine_s = id;
  }
  lds_barrier();
  const int e = __builtin_amdgcn_readfirstlane(mine_s);
  if (e < 0) return;                                       // no expert (uniform)

  // ---- weight rows: the kIter rows of a thread in the chunk that starts at
  // output column n0; all loads before their first use ----
  auto wrow = [&](int n0, int gg, int i) -> int {
    if constexpr (!kMx) {
      const int j = min(n0 + gg + G * (i % kHalf), I - 1);
      return i < kHalf ? j : I + j;
    } else {
      if constexpr (!kWaveRows) return min(2 * n0 + gg + G * i, N - 1);
      const int j = min(n0 + gg + G * (i % kHalf), I - 1);
      return 2 * j + (i < kHalf ? 0 : 1);
    }
  };
  const uint32_t row_bytes = (uint32_t)H / 2;
  const uint32_t s_cl = active ? s : 0;
  constexpr uint32_t kScaleBytes = kMx ? 1u : 4u;
  const uint32_t spr = kMx ? (uint32_t)(H / 32) : (uint32_t)(H / 64);
  const uint8_t* cbase = codes + (size_t)e * ((size_t)N * row_bytes);
  const uint8_t* sbase =
      static_cast<const uint8_t*>(scl) + (size_t)e * ((size_t)N * spr * kScaleBytes);
  const uint16_t* be = bias ? bias + (size_t)e * N : nullptr;
  struct Rows {
    u32x4 c[kIter];
    float am[kIter];
    uint32_t sb[kIter];
    uint32_t braw[kIter];                    // biases, raw until they are added
  };
  auto load_rows = [&](int n0, Rows& w) {
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const uint32_t r = (uint32_t)wrow(n0, g, i);
      w.c[i] = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4*>(cbase + (__umul24(r, row_bytes) + s_cl * 16u)));
      const uint32_t so = (__umul24(r, spr) + (kMx ? s_cl : s_cl / 2)) * kScaleBytes;
      if constexpr (kMx) {
        w.sb[i] = (uint32_t)sbase[so];
        w.am[i] = 0.f;
      } else {
        w.am[i] = *reinterpret_cast<const float*>(sbase + so);
        w.sb[i] = 0u;
      }
      w.braw[i] = 0u;
    }
    // in-wave rows: each row's bias on its lanes; LDS rows: gate's and up's of
    // output column n0 + tid in the first two
    if (be) {
      if constexpr (kWaveRows) {
#pragma unroll
        for (int i = 0; i < kIter; ++i) w.braw[i] = be[wrow(n0, g, i)];
      } else {
        const int n = min(n0 + tid, I - 1);
        w.braw[0] = be[kMx ? 2 * n : n];
        w.braw[1] = be[kMx ? 2 * n + 1 : I + n];
      }
    }
  };
  auto unit = [&](float gate, float up) {
    if constexpr (kMx) return clamped_unit(gate, up, alpha, limit);
    else return silu_f32(gate) * up;
  };
  auto bias_of = [](uint32_t raw) { return __uint_as_float(raw << 16); };

  float xf[32];
#pragma unroll
  for (int v = 0; v < 4; ++v)
#pragma unroll
    for (int cc = 0; cc < 4; ++cc) {
      xf[8 * v + 2 * cc] = bf16lo_to_f32(xr[v][cc]);
      xf[8 * v + 2 * cc + 1] = bf16hi_to_f32(xr[v][cc]);
    }
  float* arow = act + (int64_t)p0 * I;
  auto compute = [&](int n0, const Rows& w) {
    if constexpr (kWaveRows) {
      float vals[kIter];
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        const float part =
            active ? segment_dot<kMx, kLog>(lut, w.c[i], w.am[i], w.sb[i], xf, xr) : 0.f;
        vals[i] = group_sum_last(part, W) + bias_of(w.braw[i]);     // total on lane s == W - 1
      }
#pragma unroll
      for (int i = 0; i < kHalf; ++i) {
        const int n = n0 + g + G * i;
        if (s == W - 1 && n < I) arow[act_place(n, I >> 5)] = unit(vals[i], vals[i + kHalf]);
      }
    } else {
      constexpr int kStride = kMoeThreads + 32;                // pad: spreads banks
#pragma unroll
      for (int i = 0; i < kIter; ++i)
        red[i * kStride + tid] =
            active ? segment_dot<kMx, kLog>(lut, w.c[i], w.am[i], w.sb[i], xf, xr) : 0.f;
      lds_barrier();
      // each row's segments by L threads (8 where the workgroup has them),
      // then an L-lane sum; the totals go through LDS to the output columns
      const int L = 8 * R <= NT ? 8 : 1;
      const int rr = L == 8 ? tid >> 3 : tid, k = L == 8 ? tid & 7 : 0;
      float v = 0.f;
      if (rr < R) {
        const int gg = rr % G, ii = rr / G;                    // weight row wrow(n0, gg, ii)
        const float* src = red + ii * kStride + gg * S;
        for (int j = k; j < S; j += L) v += src[j];
      }
      if (L == 8) v = group_sum_last(v, 8);                    // in every lane of the group
      lds_barrier();                                           // every partial read
      if (rr < R && k == 0) red[rr] = v;
      lds_barrier();
      if (tid < Rout && n0 + tid < I)
        arow[act_place(n0 + tid, I >> 5)] =
            kMx ? unit(red[2 * tid] + bias_of(w.braw[0]), red[2 * tid + 1] + bias_of(w.braw[1]))
                : unit(red[tid] + bias_of(w.braw[0]), red[tid + Rout] + bias_of(w.braw[1]));
    }
  };
  // (a single token has one chunk a workgroup, and so have rows that meet in
  // LDS: their barriers keep the waves in step, and more workgroups hide them
  // better)
  const int step = gridDim.x * Rout;
  int n0 = blockIdx.x * Rout;
  Rows cur;
  load_rows(n0, cur);
  if constexpr (kLoop) {
    for (; n0 + step < I; n0 += step) {
      Rows next;
      load_rows(n0 + step, next);
      compute(n0, cur);
      cur = next;
    }
  }
  compute(n0, cur);
}

// ---- down product and combine ------------------------------------------------------
// Grid (row ranges, tokens): `steps` times Rb output rows of one token, whose
// products meet in LDS.  Wave w takes slots w, w + waves, ...; its lane
// groups (W lanes, one or two 32-weight segments a lane) take kR rows each
// against the slot's activations, which a lane holds in registers.  kLoop:
// several steps a workgroup, the next step's rows loading while this one's
// are decoded (several tokens, where the chip is full anyway).
template <bool kMx>
__device__ __forceinline__ float segment_dot_f32(const LutT* lut, u32x4 c, float am, uint32_t sb,
                                                 const f32x4 (&xv)[8]) {
  float acc = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t d = c[w];
    float q[8];
    if constexpr (kMx) {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const f32x2 v = e2m1_pair_f32(d, b);
        q[2 * b] = v.x;
        q[2 * b + 1] = v.y;
      }
    } else {
      nf4_pairs8(lut, d, q);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) acc = __builtin_fmaf(q[j], xv[2 * w + j / 4][j % 4], acc);
  }
  if constexpr (kMx) return e8m0_apply(acc, sb);
  else return acc * am;
}

template <bool kMx, int kR, int kSeg, bool kLoop>
__global__ __launch_bounds__(kWave* kDownWaves) void moe_down_kernel(
    const int32_t* __restrict__ ids, const float* __restrict__ act,
    const uint8_t* __restrict__ codes, const void* __restrict__ scl, int I, int H, int topk,
    int steps, const float* __restrict__ weights, const uint16_t* __restrict__ bias,
    uint16_t* __restrict__ y) {
  __shared__ __attribute__((aligned(4096))) LutT lut[kMx ? 1 : kLutN];
  extern __shared__ float ys[];                            // [topk][rows], then topk weights

  const int S = I >> 5;
  const int W = kSeg == 2 ? kWave : max(kDownLanes, S > 1 ? 1 << (32 - __builtin_clz(S - 1)) : 1);
  const int waves = min(topk, kDownWaves);
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int Rb = (kWave / W) * kR;                         // rows a step
  const int Rw = kLoop ? Rb * steps : Rb;                  // rows of the workgroup
  const int n0 = blockIdx.x * Rw;
  const int p0 = blockIdx.y * topk;                        // the token's first pair
  const int g = lane / W, s = lane - g * W;
  bool active[kSeg];
  int s_cl[kSeg];
#pragma unroll
  for (int j = 0; j < kSeg; ++j) {
    active[j] = s + kWave * j < S;
    s_cl[j] = active[j] ? s + kWave * j : 0;
  }
  const float w_own = tid < topk ? weights[p0 + tid] : 0.f;    // used by the combine
  if constexpr (!kMx && kLoop) {
    lut_init(lut, tid, kWave * waves);
    lds_barrier();
  }
  struct Rows {
    u32x4 c[kR][kSeg];
    float am[kR][kSeg];
    uint32_t sb[kR][kSeg];
    uint32_t braw[kR];                       // biases, raw until they are added
  };
  for (int sl = wave; sl < topk; sl += waves) {
    const int e = ids[p0 + sl];                            // uniform
    f32x4 xv[kSeg][8];
#pragma unroll
    for (int j = 0; j < kSeg; ++j) {
      const f32x4* ap =
          reinterpret_cast<const f32x4*>(act + (int64_t)(p0 + sl) * I) + s_cl[j];
#pragma unroll
      for (int v = 0; v < 8; ++v) xv[j][v] = ap[v * S];
    }
    // one step: the table while the expert and the activations are on their way
    if constexpr (!kMx && !kLoop)
      if (sl == wave) {                                    // (every wave's first slot)
        lut_init(lut, tid, kWave * waves);
        lds_barrier();
      }
    if (e < 0) {                                           // no expert: adds nothing
      for (int r = lane; r < Rw; r += kWave) ys[sl * Rw + r] = 0.f;
      continue;
    }
    auto load_rows = [&](int n, Rows& w) {
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        const size_t row = (size_t)e * H + min(n + g * kR + i, H - 1);
#pragma unroll
        for (int j = 0; j < kSeg; ++j) {
          w.c[i][j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(
              codes + row * (size_t)(I / 2) + (size_t)s_cl[j] * 16));
          if constexpr (kMx) {
            w.sb[i][j] =
                (uint32_t)static_cast<const uint8_t*>(scl)[row * (size_t)(I / 32) + s_cl[j]];
            w.am[i][j] = 0.f;
          } else {
            w.am[i][j] = static_cast<const float*>(scl)[row * (size_t)(I / 64) + s_cl[j] / 2];
            w.sb[i][j] = 0u;
          }
        }
        w.braw[i] = 0u;
      }
      if (bias) {
#pragma unroll
        for (int i = 0; i < kR; ++i)
          w.braw[i] = bias[(size_t)e * H + min(n + g * kR + i, H - 1)];
      }
    };
    auto compute = [&](int step, const Rows& w) {
      // MXFP4: idle lanes compute too (the row's first segment) and their sum
      // is dropped: without branches the rows' decodes overlap (8 tokens of
      // 2880 81.0 us a layer, so 79.4).  NF4: idle lanes stay out of the LDS
      // reads (8 tokens, E = 128: 44.2 us, with them 44.9).
      float part[kR];
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        part[i] = 0.f;
#pragma unroll
        for (int j = 0; j < kSeg; ++j) {
          if constexpr (kMx) {
            float d = segment_dot_f32<kMx>(lut, w.c[i][j], w.am[i][j], w.sb[i][j], xv[j]);
            asm volatile("" : "+v"(d));
            part[i] += active[j] ? d : 0.f;
          } else if (active[j]) {
            part[i] += segment_dot_f32<kMx>(lut, w.c[i][j], w.am[i][j], w.sb[i][j], xv[j]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        const float tot = group_sum_last(part[i], W) + __uint_as_float(w.braw[i] << 16);
        if (s == W - 1) ys[sl * Rw + step * Rb + g * kR + i] = tot;
      }
    };
    Rows cur;
    load_rows(n0, cur);
    if constexpr (kLoop) {
      for (int st = 0; st + 1 < steps; ++st) {
        Rows next;
        load_rows(n0 + (st + 1) * Rb, next);
        compute(st, cur);
        cur = next;
      }
      compute(steps - 1, cur);
    } else {
      compute(0, cur);
    }
  }
  float* wts = ys + topk * Rw;
  if (tid < topk) wts[tid] = w_own;
  lds_barrier();
  // thread r sums its row's slots in order
  for (int r = tid; r < Rw; r += kWave * waves) {
    float acc = 0.f;
    for (int sl = 0; sl < topk; ++sl) acc = __builtin_fmaf(wts[sl], ys[sl * Rw + r], acc);
    if (n0 + r < H) y[(int64_t)blockIdx.y * H + n0 + r] = f32_to_bf16_bits(acc);
  }
}

// ---- host -------------------------------------------------------------------------
struct MoeSpace {                            // byte offsets into the workspace
  int64_t logits, ids, weights, act, bytes;
};
static MoeSpace moe_space(const gq_moe_layer& l, int rows) {
  auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
  const int64_t P = (int64_t)rows * l.topk;
  MoeSpace m{};
  m.ids = up((int64_t)rows * l.num_experts * 4);
  m.weights = m.ids + up(P * 4);
  m.act = m.weights + up(P * 4);
  m.bytes = m.act + up(P * l.inner * 4);
  return m;
}

static int layer_checks(const gq_moe_layer* l) {
  if (!l) return kInvalid;
  if (l->format != GQ_NF4 && l->format != GQ_MXFP4) return kInvalid;
  const int blk = l->format == GQ_NF4 ? 64 : 32;
  if (l->num_experts < 1 || l->topk < 1 || l->topk > l->num_experts) return kInvalid;
  if (l->hidden < 1 || l->hidden % blk || l->inner < 1 || l->inner % blk) return kInvalid;
  if (l->format == GQ_MXFP4 &&
      !(l->limit >= 0.f && l->limit < 3.4e38f && l->alpha > -3.4e38f && l->alpha < 3.4e38f))
    return kInvalid;
  if (!l->router_weight || !l->gate_up_codes || !l->gate_up_scales || !l->down_codes ||
      !l->down_scales)
    return kInvalid;
  if (!aligned16(l->router_weight) || !aligned16(l->gate_up_codes) || !aligned16(l->down_codes))
    return kInvalid;
  if (l->format == GQ_NF4 && (!aligned4(l->gate_up_scales) || !aligned4(l->down_scales)))
    return kInvalid;
  for (const uint16_t* b : {l->router_bias, l->gate_up_bias, l->down_bias})
    if (reinterpret_cast<uintptr_t>(b) & 1u) return kInvalid;
  if (l->num_experts > kMoeMaxExperts || l->topk > kMoeMaxPairs || l->hidden > kMoeMaxHidden ||
      l->inner > kMoeMaxInner)
    return kNotSupported;
  return kOk;
}

template <bool kMx, int kIter, bool kWaveRows, int C, bool kLoop>
static void launch_gate_up(int chunks, int NT, hipStream_t stream, const gq_moe_layer& l,
                           const float* logits, const uint16_t* x, int x_stride, int rows,
                           int32_t* ids, float* w, float* act) {
  hipLaunchKernelGGL((moe_gate_up_kernel<kMx, kIter, kWaveRows, C, kLoop>),
                     dim3(chunks, rows * l.topk), dim3(NT), 0, stream, logits, x, l.gate_up_codes, l.gate_up_scales, l.hidden,
                     l.inner, l.num_experts, x_stride, l.topk, l.gate_up_bias, l.alpha,
                     l.limit, l.renormalize, ids, w, act);
}

template <bool kMx, int C>
static void gate_up(hipStream_t stream, const gq_moe_layer& l, const float* logits,
                    const uint16_t* x, int x_stride, int rows, int32_t* ids, float* w,
                    float* act) {
  const int N = 2 * l.inner, P = rows * l.topk;
  int S, W, G, NT;
  segment_layout(l.hidden, S, W, G, NT);
  auto chunks = [&](int iter) { return (N + G * iter - 1) / (G * iter); };
  auto go = [&](auto iter, auto wave_rows, int n, auto loop) {
    launch_gate_up<kMx, decltype(iter)::value, decltype(wave_rows)::value, C,
                   decltype(loop)::value>(n, NT, stream, l, logits, x, x_stride, rows, ids, w,
                                          act);
  };
  using I2 = std::integral_constant<int, 2>;
  using I4 = std::integral_constant<int, 4>;
  using I8 = std::integral_constant<int, 8>;
  if (rows > 1 && S <= kWave) {
    // several tokens: four rows a thread, as many workgroups as the chip
    // holds at once (four a CU), each running on over its chunks
    go(I4{}, std::true_type{}, std::min(chunks(4), std::max(1, 1024 / P)), std::true_type{});
    return;
  }
  // one chunk a workgroup; rows a thread as in the decode GEMV: the largest
  // count that still gives about eight workgroups per CU (two where rows are
  // reduced in LDS)
  const int64_t want = S <= kWave ? 2048 : 512;
  const int iter = chunks(8) * (int64_t)P >= want ? 8 : chunks(4) * (int64_t)P >= want ? 4 : 2;
  auto by_rows = [&](auto wave_rows) {
    if (iter == 8) go(I8{}, wave_rows, chunks(8), std::false_type{});
    else if (iter == 4) go(I4{}, wave_rows, chunks(4), std::false_type{});
    else go(I2{}, wave_rows, chunks(2), std::false_type{});
  };
  if (S > kWave) by_rows(std::false_type{});
  else by_rows(std::true_type{});
}

template <bool kMx, int kSeg>
static void launch_down(hipStream_t stream, const gq_moe_layer& l, int W, int rows,
                        const int32_t* ids, const float* w, const float* act, uint16_t* y) {
  constexpr int kR = 4;
  const int Rb = (kWave / W) * kR;
  // steps a workgroup: while two workgroups a CU remain (and the rows of all
  // slots fit 16 KB of LDS)
  int64_t groups = (l.hidden + Rb - 1) / Rb;
  int steps = 1;
  while (groups / (2 * steps) * rows >= 512 && l.topk * Rb * 2 * steps <= 4096) steps *= 2;
  groups = (groups + steps - 1) / steps;
  const dim3 grid((unsigned)groups, rows), block(kWave * std::min(l.topk, kDownWaves));
  const size_t lds = (size_t)l.topk * (Rb * steps + 1) * 4;
  if (steps > 1)
    hipLaunchKernelGGL((moe_down_kernel<kMx, kR, kSeg, true>), grid, block, lds, stream, ids, act,
                       l.down_codes, l.down_scales, l.inner, l.hidden, l.topk, steps, w,
                       l.down_bias, y);
  else
    hipLaunchKernelGGL((moe_down_kernel<kMx, kR, kSeg, false>), grid, block, lds, stream, ids, act,
                       l.down_codes, l.down_scales, l.inner, l.hidden, l.topk, steps, w,
                       l.down_bias, y);
}

template <bool kMx>
static void moe_decode(hipStream_t stream, const gq_moe_layer& l, const uint16_t* x, int x_stride,
                       int rows, char* ws, uint16_t* y) {
  const MoeSpace m = moe_space(l, rows);
  float* logits = reinterpret_cast<float*>(ws);
  int32_t* ids = reinterpret_cast<int32_t*>(ws + m.ids);
  float* w = reinterpret_cast<float*>(ws + m.weights);
  float* act = reinterpret_cast<float*>(ws + m.act);
  const bool narrow = l.num_experts <= 128;                // two logits a lane, else eight
  if (rows == 1) {
    hipLaunchKernelGGL(moe_logits_kernel<1>, dim3(l.num_experts), dim3(kMoeThreads), 0, stream, x,
                       l.router_weight, l.hidden, x_stride, rows, l.num_experts, l.router_bias,
                       logits);
    if (narrow) gate_up<kMx, 2>(stream, l, logits, x, x_stride, rows, ids, w, act);
    else gate_up<kMx, 8>(stream, l, logits, x, x_stride, rows, ids, w, act);
  } else {
    hipLaunchKernelGGL(moe_logits_kernel<kMoeMaxRows>, dim3(l.num_experts), dim3(kMoeThreads), 0,
                       stream, x, l.router_weight, l.hidden, x_stride, rows, l.num_experts,
                       l.router_bias, logits);
    if (narrow) gate_up<kMx, 2>(stream, l, logits, x, x_stride, rows, ids, w, act);
    else gate_up<kMx, 8>(stream, l, logits, x, x_stride, rows, ids, w, act);
  }
  int S, W, G, NT;
  segment_layout(l.inner, S, W, G, NT);
  if (S > kWave) launch_down<kMx, 2>(stream, l, kWave, rows, ids, w, act, y);
  else launch_down<kMx, 1>(stream, l, std::max(W, kDownLanes), rows, ids, w, act, y);
}

}  // namespace gq

extern "C" int64_t gq_moe_decode_workspace(const gq_moe_layer* layer, int32_t rows) {
  using namespace gq;
  if (layer_checks(layer) != kOk || rows < 0 || rows > kMoeMaxRows ||
      (int64_t)rows * layer->topk > kMoeMaxPairs)
    return -1;
  return moe_space(*layer, rows).bytes;
}

extern "C" int gq_moe_decode(const gq_moe_layer* layer, const uint16_t* x, int32_t rows,
                             int64_t x_stride, void* workspace, int64_t workspace_bytes,
                             uint16_t* y, hipStream_t stream) {
  using namespace gq;
  const int st = layer_checks(layer);
  if (st != kOk) return st;
  if (rows < 0 || x_stride < layer->hidden || x_stride % 8) return kInvalid;
  if (rows > kMoeMaxRows || (int64_t)rows * layer->topk > kMoeMaxPairs || x_stride > INT32_MAX)
    return kNotSupported;
  if (rows == 0) return kOk;
  if (!x || !y || !workspace || !aligned16(x) || !aligned16(workspace) ||
      (reinterpret_cast<uintptr_t>(y) & 1u))
    return kInvalid;
  if (workspace_bytes < moe_space(*layer, rows).bytes) return kInvalid;
  char* ws = static_cast<char*>(workspace);
  if (layer->format == GQ_MXFP4)
    moe_decode<true>(stream, *layer, x, (int)x_stride, rows, ws, y);
  else
    moe_decode<false>(stream, *layer, x, (int)x_stride, rows, ws, y);
  return launch_status();
}
