// MXFP4 x MXFP4 prefill grouped GEMM: activations and weights both as e2m1
// codes with e8m0 scales, fed as stored to the block-scaled matrix
// instruction (v_mfma_scale_f32_32x32x64_f8f6f4, both operands e2m1).
//
//   out[p, n] = bf16(ps[p] sum_k xq[p / topk, k] W_{ids[p]}[n, k])
//
// The instruction multiplies the codes exactly, applies both blocks' scales
// and adds in float32: the only rounding besides the float32 sums is the
// output's.  At the e2m1 x e2m1 rate (5.3 PF/s measured on random operands,
// 3.5 times the bf16 rate) a tile's bytes, not its arithmetic, are what has
// to be kept small: a 256 x 256 tile moves 16 KB per 64 k for 8.4 MFLOP.
//
// Operand layout (measured on the device, as in gemm_mx8.hip): lane (c, h) =
// (lane % 32, lane / 32) holds column c's 32-element K block h of the
// instruction's 64 k: one stored 16-byte block, its e8m0 byte as the scale.
//
// Stage of 256 k (four instructions deep): a row is 128 bytes of codes and 8
// scale bytes.  Codes of both operands go from memory straight into LDS
// (double-buffered; 16-byte chunks XOR-swizzled by (row >> 1) & 7, so reads
// of 32 rows' same chunk touch every bank once), scales through registers
// (their rows start at any byte).  One barrier per stage.
#include <type_traits>

#include "gemm_mx.hpp"
#include "../../include/gq.h"

namespace gq {

constexpr int kF4K = 256;                     // k per stage
constexpr int kF4RowBytes = kF4K / 2;
// Tiles of up to this many rows: waves side by side, each over all of the rows
// (the most that it can be: a wave holds four sub-tiles).  Inputs in turn, never
// / up to 64 / up to 128 rows, us: 2048 tokens x 4 of 32, [5760, 2880] 154.3 /
// 149.5 / 150.0; 512 tokens x 4 (64 rows an expert) 91.5 / 90.0 / 84.3; 64 x 4 of
// 16, [2400, 2880] 20.7 / 18.6 / 18.8; 20 x 2 of 4, [1024, 2880] 18.3 / 16.1 /
// 16.3; balanced routing, whose tiles are full, 116 each.
constexpr int kF4Small = 128;

// kWide: waves 2 x 2, a wave takes every second 32-row sub-tile (so that the
// row halves stay balanced when the tile is not full) and 128 columns; else
// (tiles of at most 128 rows) four waves side by side, 64 columns each.
template <bool kWide, bool kUnit>
__device__ __forceinline__ void fp4_tile(const GemmArgs& g, const TileInfo& t, int tid,
                                         uint8_t* A0, uint8_t* A1, uint8_t* B0, uint8_t* B1,
                                         u32x2* SA0, u32x2* SA1, u32x2* SB0, u32x2* SB1,
                                         int* pair_s, int* row_s, float* scale_s, int pair) {
  constexpr int kC = kWide ? 4 : 2;                       // column blocks of a wave
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int lr = lane & 31, lh = lane >> 5;
  const int nb = g.Kw / 32;                               // K blocks
  const int nstages = (nb + 7) / 8;
  const int xrow = pair / g.topk;                         // (rows past the tile: some other pair's)
  pair_s[tid] = pair;
  row_s[tid] = xrow;
  const int wn0 = kUnit ? 2 * t.n0 : t.n0;                // first weight row of the tile
  const uint8_t* as_row = g.xs + (size_t)xrow * g.xs_stride;
  const uint8_t* bs_row = static_cast<const uint8_t*>(g.scl) +
                          ((size_t)t.e * g.Nw + min(wn0 + tid, g.Nw - 1)) * (size_t)nb;
  // raw buffers over the activations and the expert's weights.  (Buffer loads
  // into LDS, not global ones: after a global one the compiler waits for
  // everything in flight where it needs one earlier load or LDS read.  Global ->
  // buffer, inputs in turn, least and most of nine: 8192 random pairs on 32
  // experts, gate_up 152.6-153.4 -> 149.9-152.2 us, down 93.6-94.0 -> 92.8-93.1;
  // 512 tokens x 4, gate_up 85.5-86.5 -> 84.2-84.9; one set of inputs 149.4-149.8
  // -> 146.7-147.3.)
  const __amdgpu_buffer_rsrc_t arsrc = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t*>(g.x), 0, g.P / g.topk * (g.Kw / 2), kRawBuffer);
  const __amdgpu_buffer_rsrc_t brsrc = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(g.codes) + (size_t)t.e * g.Nw * (size_t)(g.Kw / 2), 0,
      g.Nw * (g.Kw / 2), kRawBuffer);
  // ---- loads: 8 rows of 128 bytes per instruction, rows 8 (4 j + wave) + ..;
  // lane L fills the 16-byte slot L % 8 of row L / 8 with the chunk that the
  // swizzle puts there ((row >> 1) & 7 = 4 (wave & 1) + (L >> 4)).  Rows past
  // the tile re-read its last one, chunks past a row's end that row's last
  // (in bounds, never used): no branch, so that the loads can be placed
  // between the matrix instructions
  const uint32_t row_bytes = (uint32_t)(g.Kw / 2);
  const uint32_t chunk = (uint32_t)((lane & 7) ^ (4 * (wave & 1) + (lane >> 4)));
  constexpr int kJA = kWide ? 8 : 4;                      // 8-row groups of activations a wave loads
  uint32_t aoff[kJA], boff[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    boff[j] = (uint32_t)min(wn0 + 8 * (4 * j + wave) + (lane >> 3), g.Nw - 1) * row_bytes;
  auto next_chunk = [&](int ks) { return 16u * min((uint32_t)ks * 8 + chunk, (uint32_t)(nb - 1)); };
  // load v of a stage: 0 to 7 weight rows, then activation rows
  auto load_rows = [&](int v, uint32_t c, uint8_t* A, uint8_t* B) {
    const int j = v & 7, r0 = 8 * (4 * j + wave);
    if (v < 8)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(brsrc, (lds_void_t*)(B + r0 * kF4RowBytes), 16,
                                               (int)(boff[j] + c), 0, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(arsrc, (lds_void_t*)(A + r0 * kF4RowBytes), 16,
                                               (int)(aoff[j] + c), 0, 0, 0);
  };
  // 8 scale bytes of a row at stage ks.  The first stage of a short row takes
  // them one by one (past its end the last again); a later stage, whose row
  // has more than 8, reads the 8 bytes that end inside the row and shifts,
  // with no branch (the codes past the end are skipped or zeroed).
  auto first_scales = [&](const uint8_t* row) -> u32x2 {
    u32x2 v{0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t s = row[min(i, nb - 1)];
      v[i / 4] |= s << (8 * (i % 4));
    }
    return v;
  };
  auto load_scales = [&](const uint8_t* row, int ks) -> u32x2 {
    return *reinterpret_cast<const u32x2_a1*>(row + min(ks * 8, nb - 8));
  };
  auto align_scales = [&](u32x2 v, int ks) -> u32x2 {
    return __builtin_bit_cast(u32x2, __builtin_bit_cast(uint64_t, v) >>
                                         (8 * max(ks * 8 - (nb - 8), 0)));
  };

  // sub-tile i of this wave / its column block c, as rows of the LDS tiles
  auto arow = [&](int i) { return 32 * (kWide ? 2 * i + (wave >> 1) : i) + lr; };
  auto bcol = [&](int c) { return (kWide ? 128 * (wave & 1) : 64 * wave) + 32 * c + lr; };
  const int swz = (lr >> 1) & 7;                          // of every row of a lane
  auto frag = [&](const uint8_t* buf, int row, int u) -> u32x4 {
    return *reinterpret_cast<const u32x4*>(buf + row * kF4RowBytes + 16 * ((2 * u + lh) ^ swz));
  };
  auto wide = [](u32x4 v) {
    return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
  };

  f32x16 acc[4][kC];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][c][r] = 0.f;

  // first stage: the weight rows need no routing and go first
#pragma unroll
  for (int v = 0; v < 8; ++v) load_rows(v, next_chunk(0), A0, B0);
  const u32x2 sa_first = first_scales(as_row), sb_first = first_scales(bs_row);
  lds_barrier();                                          // row_s
#pragma unroll
  for (int j = 0; j < kJA; ++j)
    aoff[j] =
        (uint32_t)row_s[min(8 * (4 * j + wave) + (lane >> 3), t.valid - 1)] * row_bytes;
#pragma unroll
  for (int v = 8; v < kJA + 8; ++v) load_rows(v, next_chunk(0), A0, B0);
  // the pairs' weights arrive with the first stage; added after the loop
  const float own_scale = !kUnit && g.pair_scale ? g.pair_scale[pair] : 1.f;
  SA0[tid] = sa_first;
  SB0[tid] = sb_first;
  __builtin_amdgcn_s_waitcnt(0);
  scale_s[tid] = own_scale;
  lds_barrier();

  auto run_loop = [&](auto rows_c) {
    constexpr int kA = decltype(rows_c)::value;           // active sub-tiles of the wave
    // One stage, as 4 kA groups of kC matrix instructions that the scheduler
    // keeps in order: the next depth's fragment reads and, in the first three
    // depths, the next stage's loads stand between the groups.  (Issued in
    // one run, the loads hold the wave's instruction stream up for as long as
    // the address unit takes to accept them.)
    auto compute = [&](int ks, const uint8_t* A, const uint8_t* B, const u32x2* SA,
                       const u32x2* SB, uint8_t* An, uint8_t* Bn) {
      constexpr int kR = kA + kC, kV = kJA + 8, kG = 3 * kA;
      const uint32_t chunk_off = next_chunk(ks + 1);
      u32x2 sa[kA], sb[kC];
      u32x4 fa[2][kA], fb[2][kC];
      auto read = [&](int u, int r) {
        if (r < kC) fb[u & 1][r] = frag(B, bcol(r), u);
        else fa[u & 1][r - kC] = frag(A, arow(r - kC), u);
      };
#pragma unroll
      for (int r = 0; r < kR; ++r) read(0, r);
#pragma unroll
      for (int i = 0; i < kA; ++i) sa[i] = SA[arow(i)] >> (uint32_t)(8 * lh);
#pragma unroll
      for (int c = 0; c < kC; ++c) sb[c] = SB[bcol(c)] >> (uint32_t)(8 * lh);
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int i = 0; i < kA; ++i) {
          __builtin_amdgcn_sched_barrier(0);
          if (u < 3) {
            const int gi = u * kA + i;
#pragma unroll
            for (int v = kV * gi / kG; v < kV * (gi + 1) / kG; ++v)
              load_rows(v, chunk_off, An, Bn);
#pragma unroll
            for (int r = kR * i / kA; r < kR * (i + 1) / kA; ++r) read(u + 1, r);
          }
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            if (u & 1)
              acc[i][c] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                  wide(fb[1][c]), wide(fa[1][i]), acc[i][c], 4, 4, 2, (int)sb[c][u >> 1], 2,
                  (int)sa[i][u >> 1]);
            else
              acc[i][c] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                  wide(fb[0][c]), wide(fa[0][i]), acc[i][c], 4, 4, 0, (int)sb[c][u >> 1], 0,
                  (int)sa[i][u >> 1]);
          }
        }
    };
    // the last stage, one instruction depth at a time: it may hold 1 to 8 K
    // blocks; where K ends inside an instruction (K % 64 == 32) the upper
    // lane half holds no block and takes zero activations
    auto compute_last = [&](const uint8_t* A, const uint8_t* B, const u32x2* SA, const u32x2* SB,
                            int left) {
      for (int u = 0; 2 * u < left; ++u) {
        const bool live = 2 * u + lh < left;
        const int sh = 8 * (2 * u + lh) & 31, half = u >> 1;
        u32x4 fa[kA], fb[kC];
        uint32_t sa[kA], sb[kC];
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          fb[c] = frag(B, bcol(c), u);
          sb[c] = reinterpret_cast<const uint32_t*>(SB + bcol(c))[half] >> sh;
        }
#pragma unroll
        for (int i = 0; i < kA; ++i) {
          fa[i] = frag(A, arow(i), u);
          if (!live) fa[i] = u32x4{0u, 0u, 0u, 0u};
          sa[i] = reinterpret_cast<const uint32_t*>(SA + arow(i))[half] >> sh;
        }
#pragma unroll
        for (int i = 0; i < kA; ++i)
#pragma unroll
          for (int c = 0; c < kC; ++c)
            acc[i][c] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                wide(fb[c]), wide(fa[i]), acc[i][c], 4, 4, 0, (int)sb[c], 0, (int)sa[i]);
      }
    };
    auto stage = [&](int ks, const uint8_t* Ac, const uint8_t* Bc, const u32x2* SAc,
                     const u32x2* SBc, uint8_t* An, uint8_t* Bn, u32x2* SAn, u32x2* SBn) {
      __builtin_amdgcn_sched_barrier(0);
      const u32x2 na = load_scales(as_row, ks + 1), nbs = load_scales(bs_row, ks + 1);
      compute(ks, Ac, Bc, SAc, SBc, An, Bn);
      __builtin_amdgcn_sched_barrier(0);
      SAn[tid] = align_scales(na, ks + 1);
      SBn[tid] = align_scales(nbs, ks + 1);
      // the next stage is in LDS for this wave, then for all; and every wave
      // has read this stage before it is refilled
      __builtin_amdgcn_s_waitcnt(0);
      lds_barrier();
    };
    int ks = 0;
    for (; ks + 2 < nstages; ks += 2) {
      stage(ks, A0, B0, SA0, SB0, A1, B1, SA1, SB1);
      stage(ks + 1, A1, B1, SA1, SB1, A0, B0, SA0, SB0);
    }
    const bool odd = ks + 1 < nstages;
    if (odd) stage(ks, A0, B0, SA0, SB0, A1, B1, SA1, SB1);
    compute_last(odd ? A1 : A0, odd ? B1 : B0, odd ? SA1 : SA0, odd ? SB1 : SB0,
                 nb - (nstages - 1) * 8);
  };
  const int nsub = (t.valid + 31) / 32;                   // sub-tiles of the tile
  // (a wave without rows or columns runs along on one sub-tile, unstored)
  const int mine = __builtin_amdgcn_readfirstlane(kWide ? (nsub + 1 - (wave >> 1)) / 2 : nsub);
  if (mine == 4) run_loop(std::integral_constant<int, 4>{});
  else if (mine == 3) run_loop(std::integral_constant<int, 3>{});
  else if (mine == 2) run_loop(std::integral_constant<int, 2>{});
  else run_loop(std::integral_constant<int, 1>{});

  // ---- epilogue: transposed blocks, a lane holds its row's 32 columns ----
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i >= mine) continue;
    const int m = arow(i);
    const int pr = pair_s[m];
    const float sc = scale_s[m];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int wcol = wn0 + bcol(c) - lr;                // first weight row of the block
      if (m < t.valid && wcol < g.Nw) {
        float v[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = kUnit ? acc[i][c][r] : acc[i][c][r] * sc;
        if constexpr (kUnit)
          store_unit(v, g.out + (int64_t)pr * g.Nout + wcol / 2, lh, g.act_alpha, g.act_limit);
        else
          store_block_t(v, g.out + (int64_t)pr * g.Nout + wcol, lh);
      }
    }
  }
}

template <bool kUnit>
__global__ __launch_bounds__(kGemmThreads, 1) void grouped_gemm_fp4_kernel(GemmArgs g) {
  // separate arrays: a load into one buffer does not alias reads of the other
  __shared__ __attribute__((aligned(16))) uint8_t A0[kTM * kF4RowBytes];
  __shared__ __attribute__((aligned(16))) uint8_t A1[kTM * kF4RowBytes];
  __shared__ __attribute__((aligned(16))) uint8_t B0[kXN * kF4RowBytes];
  __shared__ __attribute__((aligned(16))) uint8_t B1[kXN * kF4RowBytes];
  __shared__ u32x2 SA0[kTM];
  __shared__ u32x2 SA1[kTM];
  __shared__ u32x2 SB0[kXN];
  __shared__ u32x2 SB1[kXN];
  __shared__ int pair_s[kTM];
  __shared__ int row_s[kTM];
  __shared__ float scale_s[kTM];
  const int tid = threadIdx.x;
  TileInfo t;
  int pair = 0;
  if (!mx_head<kUnit ? kXN / 2 : kXN>(g, tid, t, pair)) return;
  if (t.valid <= kF4Small)
    fp4_tile<false, kUnit>(g, t, tid, A0, A1, B0, B1, SA0, SA1, SB0, SB1, pair_s, row_s, scale_s,
                           pair);
  else
    fp4_tile<true, kUnit>(g, t, tid, A0, A1, B0, B1, SA0, SA1, SB0, SB1, pair_s, row_s, scale_s,
                           pair);
}

template <bool kUnit>
static int fp4_entry(const uint8_t* x_blocks, const uint8_t* x_scales, int32_t rows, int32_t K,
                     const uint8_t* blocks, const uint8_t* scales, int32_t num_experts, int32_t N,
                     int32_t topk, const float* pair_scale, float alpha, float limit,
                     const int32_t* expert_offsets, const int32_t* sorted_pairs,
                     const int32_t* tiles, const int32_t* num_tiles, int32_t max_tiles,
                     int32_t tile_m, uint16_t* out, hipStream_t stream) {
  GemmArgs g{};
  int64_t grid = 0;
  const int st = mx_gemm_args(g, grid, kUnit, x_blocks, x_scales, rows, K, K / 2, blocks, scales,
                              num_experts, N, topk, pair_scale, alpha, limit, expert_offsets,
                              sorted_pairs, tiles, num_tiles, max_tiles, tile_m, out);
  if (st != kOk || grid == 0) return st;
  hipLaunchKernelGGL(grouped_gemm_fp4_kernel<kUnit>, dim3((unsigned)grid), dim3(kGemmThreads), 0,
                     stream, g);
  return launch_status();
}

}  // namespace gq

extern "C" int gq_mxfp4_grouped_gemm_fp4(const uint8_t* x_blocks, const uint8_t* x_scales,
                                         int32_t rows, int32_t K, const uint8_t* blocks,
                                         const uint8_t* scales, int32_t num_experts, int32_t N,
                                         int32_t topk, const float* pair_scale,
                                         const int32_t* expert_offsets,
                                         const int32_t* sorted_pairs, const int32_t* tiles,
                                         const int32_t* num_tiles, int32_t max_tiles,
                                         int32_t tile_m, uint16_t* out, hipStream_t stream) {
  return gq::fp4_entry<false>(x_blocks, x_scales, rows, K, blocks, scales, num_experts, N, topk,
                              pair_scale, 0.f, 0.f, expert_offsets, sorted_pairs, tiles, num_tiles,
                              max_tiles, tile_m, out, stream);
}

extern "C" int gq_mxfp4_grouped_gemm_fp4_swiglu(
    const uint8_t* x_blocks, const uint8_t* x_scales, int32_t rows, int32_t K,
    const uint8_t* blocks, const uint8_t* scales, int32_t num_experts, int32_t N, int32_t topk,
    float alpha, float limit, const int32_t* expert_offsets, const int32_t* sorted_pairs,
    const int32_t* tiles, const int32_t* num_tiles, int32_t max_tiles, int32_t tile_m,
    uint16_t* act, hipStream_t stream) {
  return gq::fp4_entry<true>(x_blocks, x_scales, rows, K, blocks, scales, num_experts, N, topk,
                             nullptr, alpha, limit, expert_offsets, sorted_pairs, tiles, num_tiles,
                             max_tiles, tile_m, act, stream);
}
