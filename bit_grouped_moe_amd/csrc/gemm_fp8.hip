// MXFP8 x MXFP4 prefill grouped GEMM: activations as e4m3 codes, weights as
// e2m1 codes, both with e8m0 scales, fed as stored to the block-scaled matrix
// instruction (v_mfma_scale_f32_32x32x64_f8f6f4).
//
//   out[p, n] = bf16(ps[p] sum_k xq[p / topk, k] W_{ids[p]}[n, k])
//
// The instruction multiplies the codes exactly.  It adds eight neighbouring k at
// once, and there cuts each product toward zero to a multiple of 2^(e - 13), 2^e
// the largest of the eight products' powers of two (the codes' exponents added,
// e2m1's 0.5 with the exponent of 1; zeros do not count).  Behind that it works in
// float32, rounded to nearest: a group's sum, both blocks' scales, the sum of the
// groups.  A group so loses at most 7 2^-12 of its largest product: less than
// half a bf16 step of the sum of magnitudes, and nothing where its products lie
// within 2^9.  That is the price of the instruction's rate: a 6-bit product has
// bits below the cut only where it is under 2^-9 of a neighbour, one whose e4m3
// rounding alone is up to 2^-4 of it.  (Normal activations, K 2880: 4 10^-6 of the
// results, whose rounding to bf16 is 1.7 10^-3; one result in 270 rounds to the
// other bf16 neighbour.)  Two of e2m1 lose nothing (gemm_fp4.hip), nor does the
// single-token form, which multiplies as bf16.
// An 8-bit operand sets the instruction's rate, half of e2m1 x e2m1's, and a
// 256 x 256 tile moves 24 KB per 64 k, one and a half times as much.
//
// Operand layout (as in gemm_mx8.hip and gemm_fp4.hip): of the instruction's 64
// k, lane (c, h) = (lane % 32, lane / 32) holds column c's block h of 32 weights,
// and row c's activations 16 h + [0, 16) of both blocks, and the scale bytes of
// column c's and row c's block h.  Codes in element order so are two 16-byte
// chunks, 2 b + h of a row for block b.
//
// LDS holds 128 k of activations (128 bytes a row) and 256 k of weights (128
// bytes a row too: pieces of 64 bytes would cost the load path as much as
// these), each twice.  A step is 128 k, two instructions deep: while it runs,
// the next 128 k of activations and half of the next weights' rows go from
// memory straight into the other buffers.  16-byte chunks lie XOR-swizzled by
// (row >> 1) & 7, so that reads of 32 rows' same chunk touch every bank once.
// Scale bytes go through registers, 256 k at a time.  One barrier per step.
#include <type_traits>

#include "gemm_mx.hpp"
#include "../../include/gq.h"

namespace gq {

constexpr int kF8RowBytes = 128;
// Tiles of up to this many rows: waves side by side, each over all of the rows (32
// experts of 5760 rows of K 2880 with 32, 64 and 128 pairs each: 88, 95 and 103 us; as
// larger tiles 100, 102 and 112).
constexpr int kF8Small = 128;
// Column tiles of 128 instead of 256 where all of a call's tiles then still run at
// once, on a compute unit each: a tile's time is what counts there (us, 256 and 128
// columns: 4096 pairs of 8 experts, [1024, 2048] 28.9 and 22.7, 8192 of 8, [512, 768]
// 16.9 and 12.0, 1024 of 4, [2880, 2880] 36.5 and 30.2, 666 of 6, [544, 1056] 11.4 and
// 9.6).  Tiles that need more rounds read the activations twice as often (256 of 16,
// [2400, 2880] 23.6 and 38.9), and where an expert has few rows the waves side by side
// of the wide tile make up for it (32 of 8, [1536, 2048] 11.5 and 12.2).
constexpr int kF8Narrow = 128, kF8Units = 256, kF8FewRows = 32;
static bool narrow_tiles(int64_t P, int E, int N) {
  return P > (int64_t)kF8FewRows * E &&
         (P / kTM + E) * ceil_div64(N, kF8Narrow) <= kF8Units;
}


// kWide: waves 2 x 2, a wave takes every second 32-row sub-tile (so that the
// row halves stay balanced when the tile is not full) and half of the tile's kCols
// columns; else (tiles of 256 columns and at most 128 rows) four waves side by
// side, 64 columns each.
template <bool kWide, bool kUnit, int kCols>
__device__ __forceinline__ void fp8_tile(const GemmArgs& g, const TileInfo& t, int tid,
                                         uint8_t* A0, uint8_t* A1, uint8_t* B0, uint8_t* B1,
                                         u32x2* SA0, u32x2* SA1, u32x2* SB0, u32x2* SB1,
                                         int* pair_s, int* row_s, float* scale_s, int pair) {
  constexpr int kC = kWide ? kCols / 64 : 2;              // column blocks of a wave
  constexpr int kJB = kCols / 32;                         // 8-row groups of weights a wave loads
  static_assert(kWide || kCols == kXN);
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int lr = lane & 31, lh = lane >> 5;
  const int nb = g.Kw / 32;                               // K blocks
  const int nsteps = (nb + 3) / 4;
  const int xrow = pair / g.topk;                         // (rows past the tile: some other pair's)
  pair_s[tid] = pair;
  row_s[tid] = xrow;
  const int wn0 = kUnit ? 2 * t.n0 : t.n0;                // first weight row of the tile
  const uint8_t* as_row = g.xs + (size_t)xrow * g.xs_stride;
  const uint8_t* bs_row = static_cast<const uint8_t*>(g.scl) +
                          ((size_t)t.e * g.Nw + min(wn0 + tid, g.Nw - 1)) * (size_t)nb;
  const __amdgpu_buffer_rsrc_t arsrc = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t*>(g.x), 0, g.P / g.topk * g.Kw, kRawBuffer);
  const __amdgpu_buffer_rsrc_t brsrc = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(g.codes) + (size_t)t.e * g.Nw * (size_t)(g.Kw / 2), 0,
      g.Nw * (g.Kw / 2), kRawBuffer);
  // ---- loads: 8 rows of 128 bytes per instruction, rows 8 (4 j + wave) + ..;
  // lane L fills the 16-byte slot L % 8 of row L / 8 with the chunk that the
  // swizzle puts there ((row >> 1) & 7 = 4 (wave & 1) + (L >> 4)).  Rows past
  // the tile re-read its last one; chunks past a row's end are the next row's, or
  // past the buffer, which its range check answers with zeros, and are never
  // used.  (The check takes the lane's offset against the buffer's length less the
  // scalar one, which is below the length: a step of the activations starts inside
  // a row, a piece of the weights at most 64 bytes past a row's length, of which an
  // expert has 32 or more.)  So a lane's offsets stay as they are and the step is a
  // scalar: an address that is formed for each load holds the wave up until the load
  // before has read its own from the same register (8192 pairs evenly on 32 experts,
  // gate_up with clamped chunks 156 us, so 148)
  const uint32_t chunk = (uint32_t)((lane & 7) ^ (4 * (wave & 1) + (lane >> 4)));
  constexpr int kJA = kWide ? 8 : 4;                      // 8-row groups of activations a wave loads
  uint32_t aoff[kJA], boff[kJB];
#pragma unroll
  for (int j = 0; j < kJB; ++j)
    boff[j] = (uint32_t)min(wn0 + 8 * (4 * j + wave) + (lane >> 3), g.Nw - 1) *
                  (uint32_t)(g.Kw / 2) +
              16 * chunk;
  // s: of a, the step; of b, half of it (a buffer holds two steps' weights)
  auto load_a = [&](int j, int s, uint8_t* A) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        arsrc, (lds_void_t*)(A + 8 * (4 * j + wave) * kF8RowBytes), 16, (int)aoff[j],
        s * kF8RowBytes, 0, 0);
  };
  auto load_b = [&](int j, int s, uint8_t* B) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        brsrc, (lds_void_t*)(B + 8 * (4 * j + wave) * kF8RowBytes), 16, (int)boff[j],
        s * kF8RowBytes, 0, 0);
  };
  // 8 scale bytes of a row for steps 2 s and 2 s + 1.  The first ones of a short
  // row are taken one by one (past its end the last again); later ones, whose
  // row has more than 8, as the 8 bytes that end inside the row, shifted.
  auto first_scales = [&](const uint8_t* row) -> u32x2 {
    u32x2 v{0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t s = row[min(i, nb - 1)];
      v[i / 4] |= s << (8 * (i % 4));
    }
    return v;
  };
  auto load_scales = [&](const uint8_t* row, int s) -> u32x2 {
    return *reinterpret_cast<const u32x2_a1*>(row + min(s * 8, nb - 8));
  };
  auto align_scales = [&](u32x2 v, int s) -> u32x2 {
    return __builtin_bit_cast(u32x2, __builtin_bit_cast(uint64_t, v) >>
                                         (8 * max(s * 8 - (nb - 8), 0)));
  };

  // sub-tile i of this wave / its column block c, as rows of the LDS tiles
  auto arow = [&](int i) { return 32 * (kWide ? 2 * i + (wave >> 1) : i) + lr; };
  auto bcol = [&](int c) { return (kWide ? kCols / 2 * (wave & 1) : 64 * wave) + 32 * c + lr; };
  const int swz = (lr >> 1) & 7;                          // of every row of a lane
  auto piece = [&](const uint8_t* buf, int row, int c) -> u32x4 {
    return *reinterpret_cast<const u32x4*>(buf + row * kF8RowBytes + 16 * (c ^ swz));
  };
  // the weights' operand takes 16 bytes; the activations' the lane's half of
  // two blocks
  auto b_operand = [](u32x4 v) {
    return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
  };
  auto a_operand = [](u32x4 v, u32x4 w) {
    return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3],
                 (int)w[0], (int)w[1], (int)w[2], (int)w[3]};
  };

  f32x16 acc[4][kC];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < kC; ++c)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][c][r] = 0.f;

  // first step: the weight rows need no routing and go first
#pragma unroll
  for (int j = 0; j < kJB; ++j) load_b(j, 0, B0);
  const u32x2 sa_first = first_scales(as_row), sb_first = first_scales(bs_row);
  lds_barrier();                                          // row_s
#pragma unroll
  for (int j = 0; j < kJA; ++j)
    aoff[j] =
        (uint32_t)row_s[min(8 * (4 * j + wave) + (lane >> 3), t.valid - 1)] * (uint32_t)g.Kw +
        16 * chunk;
#pragma unroll
  for (int j = 0; j < kJA; ++j) load_a(j, 0, A0);
  // the pairs' weights arrive with the first step; added after the loop
  const float own_scale = !kUnit && g.pair_scale ? g.pair_scale[pair] : 1.f;
  SA0[tid] = sa_first;
  SB0[tid] = sb_first;
  __builtin_amdgcn_s_waitcnt(0);
  scale_s[tid] = own_scale;
  lds_barrier();

  auto run_loop = [&](auto rows_c) {
    constexpr int kA = decltype(rows_c)::value;           // active sub-tiles of the wave
    // One step, as 2 kA groups of kC matrix instructions that the scheduler keeps
    // in order: the second depth's fragment reads stand between the first half of
    // the groups, the next loads between three quarters of them, so that the last
    // ones have a quarter of the step's time to arrive (8192 pairs on 32 experts of
    // K 2880, gate_up 192 us with the loads over all groups, 193 over half, so 189.5;
    // down 109, 107, 105).  kOdd: the step's weights are its buffer's second half.
    auto step = [&](auto odd_c, int s, const uint8_t* A, const uint8_t* B, const u32x2* SA,
                    const u32x2* SB, uint8_t* An, uint8_t* Bn, u32x2* SAn, u32x2* SBn) {
      constexpr int kOdd = decltype(odd_c)::value;
      constexpr int kR = 2 * kA + kC, kV = kJA + kJB / 2, kG = (3 * kA + 1) / 2;
      __builtin_amdgcn_sched_barrier(0);
      u32x2 na, nbs;
      if constexpr (kOdd) {
        na = load_scales(as_row, s / 2 + 1);
        nbs = load_scales(bs_row, s / 2 + 1);
      }
      uint32_t sa[kA], sb[kC];
      u32x4 fa[2][kA][2], fb[2][kC];
      auto read = [&](int u, int r) {
        if (r < kC) fb[u][r] = piece(B, bcol(r), 4 * kOdd + 2 * u + lh);
        else fa[u][(r - kC) / 2][(r - kC) % 2] =
            piece(A, arow((r - kC) / 2), 4 * u + 2 * ((r - kC) % 2) + lh);
      };
#pragma unroll
      for (int r = 0; r < kR; ++r) read(0, r);
#pragma unroll
      for (int i = 0; i < kA; ++i)
        sa[i] = reinterpret_cast<const uint32_t*>(SA + arow(i))[kOdd] >> (uint32_t)(8 * lh);
#pragma unroll
      for (int c = 0; c < kC; ++c)
        sb[c] = reinterpret_cast<const uint32_t*>(SB + bcol(c))[kOdd] >> (uint32_t)(8 * lh);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < kA; ++i) {
          __builtin_amdgcn_sched_barrier(0);
          const int gi = u * kA + i;
#pragma unroll
          for (int v = kV * gi / kG; v < (gi < kG ? kV * (gi + 1) / kG : 0); ++v) {
            if (v < kJB / 2) load_b(kJB / 2 * kOdd + v, s / 2 + 1, Bn);
            else load_a(v - kJB / 2, s + 1, An);
          }
          if (u == 0) {
#pragma unroll
            for (int r = kR * i / kA; r < kR * (i + 1) / kA; ++r) read(1, r);
          }
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            if (u)
              acc[i][c] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                  b_operand(fb[1][c]), a_operand(fa[1][i][0], fa[1][i][1]), acc[i][c], 4, 0, 2,
                  (int)sb[c], 2, (int)sa[i]);
            else
              acc[i][c] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                  b_operand(fb[0][c]), a_operand(fa[0][i][0], fa[0][i][1]), acc[i][c], 4, 0, 0,
                  (int)sb[c], 0, (int)sa[i]);
          }
        }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (kOdd) {
        SAn[tid] = align_scales(na, s / 2 + 1);
        SBn[tid] = align_scales(nbs, s / 2 + 1);
      }
      // the next step is in LDS for this wave, then for all; and every wave has
      // read this step before it is refilled
      __builtin_amdgcn_s_waitcnt(0);
      lds_barrier();
    };
    // the last step, one instruction depth at a time: it holds 1 to 4 K blocks;
    // where K ends inside an instruction (K % 64 == 32) its upper block takes
    // zero activations
    auto last_step = [&](int s, const uint8_t* A, const uint8_t* B, const u32x2* SA,
                         const u32x2* SB) {
      const int odd = s & 1, left = nb - 4 * s;
      for (int u = 0; 2 * u < left; ++u) {
        const bool both = 2 * u + 1 < left;
        const int sh = 8 * (2 * u + lh);
        u32x4 fa[kA][2], fb[kC];
        uint32_t sa[kA], sb[kC];
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          fb[c] = piece(B, bcol(c), 4 * odd + 2 * u + lh);
          sb[c] = reinterpret_cast<const uint32_t*>(SB + bcol(c))[odd] >> sh;
        }
#pragma unroll
        for (int i = 0; i < kA; ++i) {
          fa[i][0] = piece(A, arow(i), 4 * u + lh);
          fa[i][1] = piece(A, arow(i), 4 * u + 2 + lh);
          if (!both) fa[i][1] = u32x4{0u, 0u, 0u, 0u};
          sa[i] = reinterpret_cast<const uint32_t*>(SA + arow(i))[odd] >> sh;
        }
#pragma unroll
        for (int i = 0; i < kA; ++i)
#pragma unroll
          for (int c = 0; c < kC; ++c)
            acc[i][c] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                b_operand(fb[c]), a_operand(fa[i][0], fa[i][1]), acc[i][c], 4, 0, 0, (int)sb[c], 0,
                (int)sa[i]);
      }
    };
    using Even = std::integral_constant<int, 0>;
    using Odd = std::integral_constant<int, 1>;
    int s = 0;
    for (; s + 4 < nsteps; s += 4) {
      step(Even{}, s, A0, B0, SA0, SB0, A1, B1, SA1, SB1);
      step(Odd{}, s + 1, A1, B0, SA0, SB0, A0, B1, SA1, SB1);
      step(Even{}, s + 2, A0, B1, SA1, SB1, A1, B0, SA0, SB0);
      step(Odd{}, s + 3, A1, B1, SA1, SB1, A0, B0, SA0, SB0);
    }
    const int rest = nsteps - s;                          // 1 to 4, the last apart
    if (rest > 1) step(Even{}, s, A0, B0, SA0, SB0, A1, B1, SA1, SB1);
    if (rest > 2) step(Odd{}, s + 1, A1, B0, SA0, SB0, A0, B1, SA1, SB1);
    if (rest > 3) step(Even{}, s + 2, A0, B1, SA1, SB1, A1, B0, SA0, SB0);
    last_step(nsteps - 1, rest & 1 ? A0 : A1, rest > 2 ? B1 : B0, rest > 2 ? SA1 : SA0,
              rest > 2 ? SB1 : SB0);
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

template <bool kUnit, int kCols>
__global__ __launch_bounds__(kGemmThreads, 1) void grouped_gemm_fp8_kernel(GemmArgs g) {
  // separate arrays: a load into one buffer does not alias reads of the other
  __shared__ __attribute__((aligned(16))) uint8_t A0[kTM * kF8RowBytes];
  __shared__ __attribute__((aligned(16))) uint8_t A1[kTM * kF8RowBytes];
  __shared__ __attribute__((aligned(16))) uint8_t B0[kCols * kF8RowBytes];
  __shared__ __attribute__((aligned(16))) uint8_t B1[kCols * kF8RowBytes];
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
  if (!mx_head<kUnit ? kCols / 2 : kCols>(g, tid, t, pair)) return;
  if constexpr (kCols == kXN)
    if (t.valid <= kF8Small) {
      fp8_tile<false, kUnit, kCols>(g, t, tid, A0, A1, B0, B1, SA0, SA1, SB0, SB1, pair_s, row_s,
                                    scale_s, pair);
      return;
    }
  fp8_tile<true, kUnit, kCols>(g, t, tid, A0, A1, B0, B1, SA0, SA1, SB0, SB1, pair_s, row_s,
                               scale_s, pair);
}

template <bool kUnit>
static int fp8_entry(const uint8_t* x_codes, const uint8_t* x_scales, int32_t rows, int32_t K,
                     const uint8_t* blocks, const uint8_t* scales, int32_t num_experts, int32_t N,
                     int32_t topk, const float* pair_scale, float alpha, float limit,
                     const int32_t* expert_offsets, const int32_t* sorted_pairs,
                     const int32_t* tiles, const int32_t* num_tiles, int32_t max_tiles,
                     int32_t tile_m, uint16_t* out, hipStream_t stream) {
  GemmArgs g{};
  int64_t grid = 0;
  const int st = mx_gemm_args(g, grid, kUnit, x_codes, x_scales, rows, K, K, blocks, scales,
                              num_experts, N, topk, pair_scale, alpha, limit, expert_offsets,
                              sorted_pairs, tiles, num_tiles, max_tiles, tile_m, out);
  if (st != kOk || grid == 0) return st;
  GemmArgs n = g;
  const int64_t narrow = mx_grid(n, kF8Narrow);
  if (narrow_tiles(g.P, num_experts, N) && narrow <= most_groups(kGemmThreads))
    hipLaunchKernelGGL((grouped_gemm_fp8_kernel<kUnit, kF8Narrow>), dim3((unsigned)narrow),
                       dim3(kGemmThreads), 0, stream, n);
  else
    hipLaunchKernelGGL((grouped_gemm_fp8_kernel<kUnit, kXN>), dim3((unsigned)grid),
                       dim3(kGemmThreads), 0, stream, g);
  return launch_status();
}

}  // namespace gq

extern "C" int gq_mxfp4_grouped_gemm_fp8(const uint8_t* x_codes, const uint8_t* x_scales,
                                         int32_t rows, int32_t K, const uint8_t* blocks,
                                         const uint8_t* scales, int32_t num_experts, int32_t N,
                                         int32_t topk, const float* pair_scale,
                                         const int32_t* expert_offsets,
                                         const int32_t* sorted_pairs, const int32_t* tiles,
                                         const int32_t* num_tiles, int32_t max_tiles,
                                         int32_t tile_m, uint16_t* out, hipStream_t stream) {
  return gq::fp8_entry<false>(x_codes, x_scales, rows, K, blocks, scales, num_experts, N, topk,
                              pair_scale, 0.f, 0.f, expert_offsets, sorted_pairs, tiles, num_tiles,
                              max_tiles, tile_m, out, stream);
}

extern "C" int gq_mxfp4_grouped_gemm_fp8_swiglu(
    const uint8_t* x_codes, const uint8_t* x_scales, int32_t rows, int32_t K,
    const uint8_t* blocks, const uint8_t* scales, int32_t num_experts, int32_t N, int32_t topk,
    float alpha, float limit, const int32_t* expert_offsets, const int32_t* sorted_pairs,
    const int32_t* tiles, const int32_t* num_tiles, int32_t max_tiles, int32_t tile_m,
    uint16_t* act, hipStream_t stream) {
  return gq::fp8_entry<true>(x_codes, x_scales, rows, K, blocks, scales, num_experts, N, topk,
                             nullptr, alpha, limit, expert_offsets, sorted_pairs, tiles, num_tiles,
                             max_tiles, tile_m, act, stream);
}
