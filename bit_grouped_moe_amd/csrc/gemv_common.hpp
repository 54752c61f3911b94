// Pieces shared by the decode-time kernels (gemv.hip, moe_decode.hip): the
// dot product of a 32-weight segment and the layout of a row's segments over
// a workgroup's lanes.
#pragma once

#include "gq_device.hpp"

namespace gq {

constexpr int kGemvMaxThreads = 256;

// Partial dot product of one 32-weight segment with the activation slice
// (xf: as float32; xr: the raw bf16 pairs).  NF4: codebook values (float32)
// against xf.  MXFP4: the converter turns each code byte into its two
// weights as a bf16 pair (exact: every e2m1 value is a bf16 value) and
// v_dot2_f32_bf16 multiplies it with the matching activation pair (the
// products are exact in float32; two per instruction, float32 sums): 25%
// fewer VALU instructions than float32 FMAs on converted weights, and no
// activation conversion; one-token gpt-oss gate_up 9.99 -> 9.70 us, down
// 7.34 -> 7.01 us (graph-replayed, same-box A/B).
//
// NF4 values come from a 256-entry table of codebook value pairs indexed by
// the code byte (one 8-byte LDS read per two weights, the table at LDS
// address 0 so its byte offset is one shift).  Against the 16-entry table
// (one 4-byte read per weight) this halves the LDS reads at the end of each
// workgroup, where the decode follows the last weight bytes; same-box A/B
// over three alternations, graph-replayed: one-token gate_up 6.05-6.08 ->
// 5.92-5.97 us, down 4.97-5.05 -> 4.78-4.81 us, decode step 11.1 -> 10.7-10.8
// us, M = 4 down 10.8 -> 10.4 us.
using LutT = f32x2;
constexpr int kLutN = 256;
__device__ __forceinline__ void lut_init(LutT* lut, int tid, int nt) {
  for (int t = tid; t < kLutN; t += nt) nf4_pairs_init(lut, t);
}
// The table in 2^kLog copies side by side, lane l reading copy l mod 2^kLog.
template <int kLog>
__device__ __forceinline__ void lut_init_copies(LutT* lut, int tid, int nt) {
  for (int t = tid; t < kLutN; t += nt) {
    const LutT v = nf4_pair(t);
#pragma unroll
    for (int c = 0; c < 1 << kLog; ++c) lut[(t << kLog) + ((c + t) & ((1 << kLog) - 1))] = v;
  }
}
template <bool kMx, int kLog = 0>
__device__ __forceinline__ float segment_dot(const LutT* lut, u32x4 c, float am, uint32_t sb,
                                             const float (&xf)[32], const u32x4 (&xr)[4]) {
  float acc = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint32_t d = c[w];
    // The decode does not depend on the pair: without this the compiler
    // hoists every row's decoded weights out of the pair loop and needs one
    // register per weight.  (No instruction is emitted.)
    asm volatile("" : "+v"(d));
    if constexpr (kMx) {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const uint32_t wv = e2m1_pair_bf16_scaled(d, b, 1.0f);   // element 2j: low half
        // a scalar copy first: a bit_cast of a vector element reads element 0
        const uint32_t xv = xr[w][b];
        acc = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, wv),
                                              __builtin_bit_cast(bf16x2, xv), acc, false);
      }
    } else {
      float q[8];
      nf4_pairs8<kLog>(lut, d, q);                        // element 2j: high nibble
#pragma unroll
      for (int j = 0; j < 8; ++j) acc = __builtin_fmaf(q[j], xf[8 * w + j], acc);
    }
  }
  if constexpr (kMx) return e8m0_apply(acc, sb);
  else return acc * am;
}

// Segment lanes: S segments of 32 weights per row.  S <= 64: a row's
// segments go to a group of W = S rounded up to a power of two lanes inside
// one wave (lanes s >= S idle); longer rows: S consecutive threads, reduced
// through LDS.
static inline void segment_layout(int K, int& S, int& W, int& G, int& NT) {
  S = K / 32;
  W = S;
  if (S <= kWave)
    while (W & (W - 1)) W += W & -W;
  G = S > kWave ? (S >= kGemvMaxThreads ? 1 : kGemvMaxThreads / S) : kGemvMaxThreads / W;
  NT = S > kWave ? ((S * G + kWave - 1) / kWave) * kWave : kGemvMaxThreads;
}

}  // namespace gq
