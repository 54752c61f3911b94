// Pieces shared by the products of two MX operands (gemm_fp4.hip: MXFP4
// activations; gemm_fp8.hip: MXFP8 activations; the weights MXFP4 in both):
// the mapping of workgroups to tiles, rows of dropped pairs, scale bytes and
// the gated unit's epilogue.
#pragma once

#include "gemm_common.hpp"

namespace gq {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));

constexpr int kRawBuffer = 0x00027000;        // flags of a raw buffer of 32-bit data

// 16 (gate, up) pairs of a transposed block -> 16 outputs, exchanged and
// written as store_block_act does.
__device__ __forceinline__ void store_unit(const float (&v)[16], uint16_t* orow, int lh,
                                           float alpha, float limit) {
  uint32_t o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    o[q] = pack_bf16x2(clamped_unit(v[4 * q], v[4 * q + 1], alpha, limit),
                       clamped_unit(v[4 * q + 2], v[4 * q + 3], alpha, limit));
  const auto a = __builtin_amdgcn_permlane32_swap(o[0], o[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(o[1], o[3], false, false);
  *reinterpret_cast<u32x4*>(orow + 8 * lh) = u32x4{a[0], a[1], b[0], b[1]};
}

// The tile of a workgroup.  Blocks are dealt to the 8 XCDs in turn, each with
// an L2 of its own; kGroup column tiles of a row tile go to one XCD, which so
// fetches the tile's activations for all of them, and row tiles, full and
// short ones, spread evenly (8192 pairs on 32 experts, gate_up / down: all
// column tiles of a row tile on one XCD 162 / 79 us, one column tile at a
// time 154 / 92, four 157 / 81).  Tiles past the last expert tile clear the
// rows of dropped pairs.  A tile entry that cannot come from gq_route_sort is
// rejected.
constexpr int kGroup = 4;
template <int kTNo>
__device__ __forceinline__ bool mx_head(const GemmArgs& g, int tid, TileInfo& t, int& pair) {
  const int bid = blockIdx.x;
  const int q = bid >> 3, xcd = bid & 7;
  const int groups = (g.n_col_tiles + kGroup - 1) / kGroup;
  const int unit = (q / kGroup) * 8 + xcd;
  const int tile = unit / groups;
  const int col = (unit % groups) * kGroup + q % kGroup;
  if (tile >= g.max_tiles || col >= g.n_col_tiles) return false;
  t.n0 = col * kTNo;
  // the tile count and the tile's entry in one round trip (entries past the
  // count hold no expert)
  const int T = *g.num_tiles;
  t.e = g.tiles[2 * tile];
  t.start = g.tiles[2 * tile + 1];
  if (tile >= T) {
    const int dstart = g.offsets[g.E] + (tile - T) * kTM;
    if (dstart >= g.P || dstart < 0) return false;
    const int dvalid = min(kTM, g.P - dstart);
    for (int idx = tid; idx < dvalid * (kTNo / 8); idx += kGemmThreads) {
      const int r = idx / (kTNo / 8), c = t.n0 + idx % (kTNo / 8) * 8;
      const int p = g.sorted_pairs[dstart + r];
      if (c < g.Nout && (unsigned)p < (unsigned)g.P)
        *reinterpret_cast<u32x4*>(g.out + (int64_t)p * g.Nout + c) = u32x4{0u, 0u, 0u, 0u};
    }
    return false;
  }
  if ((unsigned)t.e >= (unsigned)g.E || (unsigned)t.start >= (unsigned)g.P) return false;
  // the segment's end and its pairs in the next
  const int end = g.offsets[t.e + 1];
  const int p = g.sorted_pairs[min(t.start + tid, g.P - 1)];
  t.valid = min(kTM, min(end, g.P) - t.start);
  pair = (unsigned)p < (unsigned)g.P ? p : 0;
  return t.valid > 0;
}

// Host: the workgroups for column tiles of `cols` weight rows.
static inline int64_t mx_grid(GemmArgs& g, int cols) {
  g.n_col_tiles = (g.Nw + cols - 1) / cols;
  return ceil_div64((int64_t)g.max_tiles * ceil_div64(g.n_col_tiles, kGroup), 8) * 8 * kGroup;
}

// Host: the checks of a product's arguments, its argument block and its grid (0:
// nothing to enqueue).  row_bytes: an activation row's codes.
static inline int mx_gemm_args(GemmArgs& g, int64_t& grid, bool unit, const uint8_t* x_codes,
                               const uint8_t* x_scales, int32_t rows, int32_t K,
                               int64_t row_bytes, const uint8_t* blocks, const uint8_t* scales,
                               int32_t num_experts, int32_t N, int32_t topk,
                               const float* pair_scale, float alpha, float limit,
                               const int32_t* expert_offsets, const int32_t* sorted_pairs,
                               const int32_t* tiles, const int32_t* num_tiles,
                               int32_t max_tiles, int32_t tile_m, uint16_t* out) {
  if (rows < 0 || topk < 1 || num_experts < 1 || N < 1 || N % 32 || K <= 0 || K % 32)
    return kInvalid;
  if (unit && !(limit >= 0.f && limit < 3.4e38f && alpha > -3.4e38f && alpha < 3.4e38f))
    return kInvalid;                                       // finite alpha, limit >= 0
  if (tile_m != kTM) return kNotSupported;
  const int64_t P = (int64_t)rows * topk;
  if (P >= INT32_MAX) return kNotSupported;
  if (P == 0) return kOk;                                  // grid 0: nothing to enqueue
  // 32-bit offsets of a row inside the activations and inside one expert
  if ((int64_t)rows * row_bytes >= INT32_MAX || (int64_t)N * (K / 2) >= INT32_MAX)
    return kNotSupported;
  if (!x_codes || !x_scales || !blocks || !scales || !expert_offsets || !sorted_pairs || !tiles ||
      !num_tiles || !out)
    return kInvalid;
  if (!aligned16(x_codes) || !aligned16(blocks) || !aligned16(out)) return kInvalid;
  if (!aligned4(expert_offsets) || !aligned4(sorted_pairs) || !aligned4(tiles) ||
      !aligned4(num_tiles) || (pair_scale && !aligned4(pair_scale)))
    return kInvalid;
  const int64_t need = (P + kTM - 1) / kTM + num_experts + 1;
  if (max_tiles < need) return kInvalid;
  g.x = reinterpret_cast<const uint16_t*>(x_codes);
  g.xs = x_scales;
  g.xs_stride = K / 32;
  g.codes = blocks; g.scl = scales;
  g.Nw = N; g.Kw = K; g.Kc = K; g.Nout = unit ? N / 2 : N;
  g.E = num_experts; g.topk = topk; g.P = (int)P; g.pair_scale = pair_scale;
  g.offsets = expert_offsets; g.sorted_pairs = sorted_pairs; g.tiles = tiles;
  g.num_tiles = num_tiles; g.out = out;
  g.act_alpha = alpha; g.act_limit = limit;
  g.max_tiles = max_tiles;
  grid = mx_grid(g, kXN);
  return grid > most_groups(kGemmThreads) ? kNotSupported : kOk;
}

}  // namespace gq
