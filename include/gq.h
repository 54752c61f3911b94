/*
 * gq.h -- C ABI of libgq: grouped mixture-of-experts matmul on 4-bit packed
 * expert weights (NF4 and MXFP4) for AMD MI355X (gfx950).
 *
 * What the library computes follows these web pages:
 *   [P1] "grouped-nf4-gemm 0.43.0" (PyPI project page): section "Which
 *        entry point?" (grouped NF4 forward and backward, the single-row
 *        decode bandwidth route, native MXFP4 expert math) and the page
 *        header (one GPU launch for the active experts, no full-size bf16
 *        weight copies); section "Try the packers and byte checks on CPU"
 *        (packed shapes).
 *   [P2] "Receipts-driven engineering": opening summary (codebook decoded
 *        in registers inside the GEMM mainloop; NF4 in the bitsandbytes
 *        packed layout; MXFP4 as OCP e2m1 on released bytes; the NF4 path
 *        is differentiable).
 *   [P4] "flashrt/grouped-moe-gemv": section "Functions" (routing tensor
 *        [M, top_k] of expert ids, output [M, top_k, N], flatten to
 *        M = routed pairs and top_k = 1 when each pair has its own input;
 *        no atomics, no host synchronisation, caller-owned buffers).
 *   [P5] GPTQModel wiki "NF12": malformed arguments to native C-ABI calls
 *        return hipErrorInvalidValue; launches beyond supported limits
 *        return hipErrorNotSupported before launch.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Every buffer pointer is DEVICE memory on the current HIP device and is
 *   owned by the caller; the library never allocates, frees or keeps a
 *   pointer after the call returns.
 * - Work is enqueued asynchronously on `stream` (NULL = default stream);
 *   nothing synchronises the host.  Results are ready when the stream is.
 * - bf16 values travel as raw uint16_t bit patterns.
 * - Packed weights (all experts stacked, contiguous):
 *     NF4   codes  uint8 [E, N, K/2]  element 2j of a row in the HIGH nibble
 *                                     of byte j (bitsandbytes layout)
 *           absmax float [E, N, K/64] one scale per 64 consecutive k
 *           weight = float32(nf4_codebook[code] * absmax)
 *     MXFP4 blocks uint8 [E, N, K/32, 16] element 2j of a 32-block in the LOW
 *                                     nibble of byte j (released gpt-oss layout)
 *           scales uint8 [E, N, K/32] e8m0: factor 2^(s-127); 255 = NaN
 *           weight = e2m1(code) * 2^(s-127)
 * - Routing: topk_ids int32 [rows, topk], pair index p = t*topk + s.  A pair
 *   routed to an id outside [0, E) is dropped and its output row is zeros.
 *   Gather mode (topk > 1): pair p reads activation row p / topk.  Flatten
 *   mode (per-pair inputs, e.g. a down projection): pass rows = pairs and
 *   topk = 1.
 * - Outputs are bf16, rounded to nearest even from an fp32 accumulator,
 *   optionally multiplied by pair_scale[p] (fp32, one per pair; NULL = 1).
 *   No atomics: each output element is written by exactly one thread, so
 *   results are bitwise reproducible run to run.
 * - Return value: 0 on success; hipErrorInvalidValue (1) for a malformed
 *   argument (checked on the host before anything is enqueued; nothing is
 *   truncated or clamped); hipErrorNotSupported (801) for a well-formed
 *   request outside what the kernels support (stated per function);
 *   otherwise the HIP error reported by the launch.
 * - Expert ids are data on the device; the kernels treat any id outside
 *   [0, E) as dropped, so no id can make a kernel read outside the banks.
 */
#ifndef GQ_H
#define GQ_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Name of a status code returned by this library (static string). */
const char* gq_status_string(int status);

/* ------------------------------------------------------------------------
 * Token-to-expert grouping.  [P1] header and [P2] summary: all active
 * experts run in one launch, which needs the pairs grouped by expert on the
 * device without a host round trip ([P4] "Functions": no host sync).
 *
 * Upper bound on the number of tiles gq_route_sort can emit, including the
 * tiles the grouped GEMM uses to clear dropped rows:
 *     ceil(rows*topk / tile_m) + E + 1.
 * Returns -1 if an argument is negative, tile_m < 1 or E < 1.
 */
int32_t gq_route_max_tiles(int32_t rows, int32_t topk, int32_t num_experts, int32_t tile_m);

/*
 * Stable counting sort of the rows*topk (token, slot) pairs by expert.
 *   topk_ids       int32 [rows, topk]       in
 *   expert_offsets int32 [E + 1]            out: offsets[e] = #valid pairs with
 *                                                expert < e; offsets[E] = #valid pairs
 *   sorted_pairs   int32 [rows*topk]        out: expert by expert, ascending pair
 *                                                index within an expert; dropped
 *                                                pairs last, ascending
 *   tiles          int32 [max_tiles, 2]     out: (expert, start in sorted_pairs) of
 *                                                every tile_m-row slice of each
 *                                                expert's segment, experts
 *                                                ascending; unused entries = -1
 *   num_tiles      int32 [1]                out: number of valid tiles
 * Deterministic: the output is the unique answer to the definition above.
 * InvalidValue: null pointer, rows/topk < 0, E < 1, tile_m < 1,
 *               max_tiles < gq_route_max_tiles(...).
 * NotSupported: E > 1024, rows*topk >= 2^31.
 * rows*topk == 0 is valid (offsets all 0, num_tiles 0, tiles all -1).
 */
int gq_route_sort(const int32_t* topk_ids, int32_t rows, int32_t topk, int32_t num_experts,
                  int32_t tile_m, int32_t* expert_offsets, int32_t* sorted_pairs,
                  int32_t* tiles, int32_t max_tiles, int32_t* num_tiles, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Decode probes.  [P1] "Try the packers and byte checks on CPU" (packed
 * shapes) and [P2] summary (codes decoded in registers).  They write the
 * decoded weights with the same device decode routines the matmul kernels
 * use, so decoding can be compared bit for bit.  Not on the hot path.
 *   NF4:   codes [n_rows, K/2], absmax [n_rows, K/64]; K % 64 == 0
 *   MXFP4: blocks [n_rows, K/32, 16], scales [n_rows, K/32]; K % 32 == 0
 *   out_f32 float [n_rows, K] (may be NULL), out_bf16 uint16 [n_rows, K]
 *   (may be NULL; bf16 = RNE of the float32 weight).  At least one output.
 * InvalidValue: null inputs, both outputs NULL, n_rows < 0, K <= 0 or not a
 * multiple of the block.
 */
int gq_nf4_decode(const uint8_t* codes, const float* absmax, int64_t n_rows, int32_t K,
                  float* out_f32, uint16_t* out_bf16, hipStream_t stream);
int gq_mxfp4_decode(const uint8_t* blocks, const uint8_t* scales, int64_t n_rows, int32_t K,
                    float* out_f32, uint16_t* out_bf16, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Decode-time GEMV: 1..8 tokens in gather mode, or their routed pairs in
 * flatten mode (at most 256 pairs).  [P1] header, "Which entry point?"
 * (single-row decode bandwidth route), [P4] "Functions" (one product per
 * routed slot, [M, top_k] -> [M, top_k, N]).
 *
 *   out[p, n] = bf16( pair_scale[p] * sum_k x[p/topk, k] * W_{ids[p]}[n, k] )
 *
 *   x          uint16 bf16 [rows, K] with row stride x_stride elements
 *              (x_stride >= K, x_stride % 8 == 0, x 16-byte aligned)
 *   codes/absmax (NF4) or blocks/scales (MXFP4) for E experts of shape [N, K]
 *   topk_ids   int32 [rows, topk]; pair_scale float [rows*topk] or NULL
 *   out        uint16 bf16 [rows*topk, N]
 * Each distinct active expert's bytes are read once, whichever tokens use
 * it; no sort is needed (the kernel reads topk_ids directly).  Arithmetic,
 * float32 throughout with no bf16 rounding of the weights: each group of 32
 * consecutive k is summed as sum(codebook_value * x) (NF4) or
 * sum(e2m1_value * x) (MXFP4; exact products, two per bf16-pair dot
 * instruction, float32 sums), then multiplied once by the group's factor
 * (the NF4 absmax of its 64-block; the MXFP4 2^(s-127), exact); the group
 * partials are added in a fixed order.  A one-hot x therefore returns
 * bf16(float32(value * factor)), the decoded weight, bit for bit.
 * InvalidValue: null pointer (pair_scale may be NULL), rows < 1,
 *   topk < 1, E < 1, N < 1, K not a positive multiple of 64 (NF4) / 32
 *   (MXFP4), bad stride or alignment.
 * A pair whose id lies outside [0, E) is dropped: its output row is zero.
 * NotSupported: rows*topk > 256, K > 8192, N >= 2^24, N*K/2 >= 2^31 (one
 *   expert's codes), x_stride > 2^31 - 1.
 */
int gq_nf4_grouped_gemv(const uint16_t* x, int32_t rows, int32_t K, int64_t x_stride,
                        const uint8_t* codes, const float* absmax, int32_t num_experts,
                        int32_t N, const int32_t* topk_ids, int32_t topk,
                        const float* pair_scale, uint16_t* out, hipStream_t stream);
int gq_mxfp4_grouped_gemv(const uint16_t* x, int32_t rows, int32_t K, int64_t x_stride,
                          const uint8_t* blocks, const uint8_t* scales, int32_t num_experts,
                          int32_t N, const int32_t* topk_ids, int32_t topk,
                          const float* pair_scale, uint16_t* out, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Experts streamed from host memory.  [P1] page header (streaming expert
 * weights from RAM or SSD) and section "Which entry point?" (the row for
 * streaming experts from RAM or NVMe); [P2] "What the discipline caught" (the fused
 * kernel as the only expert compute while experts stream over the host
 * link, against the link's ceiling) and "The numbers" (t ~ c + bytes/link).
 *
 * gq_nf4_grouped_gemv_host / gq_mxfp4_grouped_gemv_host: gq_nf4_grouped_gemv
 * / gq_mxfp4_grouped_gemv with the expert bank (codes and absmax, or blocks
 * and scales) in pinned, device-mapped host memory (hipHostMalloc, or a
 * pinned torch tensor), passed as HOST pointers.  The kernel reads the
 * routed experts' bytes straight over the host link as it decodes them: no
 * staging copy, each active expert's bytes cross the link once per launch.
 * x, topk_ids, pair_scale and out are device pointers as before; same
 * arithmetic, results bit-identical to the device-resident call.
 * InvalidValue also when a bank pointer is not pinned, mapped host memory
 * (checked before anything is enqueued).
 */
int gq_nf4_grouped_gemv_host(const uint16_t* x, int32_t rows, int32_t K, int64_t x_stride,
                             const uint8_t* codes, const float* absmax, int32_t num_experts,
                             int32_t N, const int32_t* topk_ids, int32_t topk,
                             const float* pair_scale, uint16_t* out, hipStream_t stream);
int gq_mxfp4_grouped_gemv_host(const uint16_t* x, int32_t rows, int32_t K, int64_t x_stride,
                               const uint8_t* blocks, const uint8_t* scales, int32_t num_experts,
                               int32_t N, const int32_t* topk_ids, int32_t topk,
                               const float* pair_scale, uint16_t* out, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Prefill grouped GEMM.  [P1] "Which entry point?" (grouped NF4 forward,
 * native MXFP4 expert math) and header (one launch for the active experts,
 * no full-size bf16 weight copies); [P2] summary (codebook decoded in
 * registers inside the mainloop).
 *
 *   out[p, n] = bf16( pair_scale[p] * sum_k x[p/topk, k] * W_{ids[p]}[n, k] )
 *
 * Same x / weights / pair_scale / out conventions as the GEMV.  The
 * grouping comes from gq_route_sort(topk_ids, rows, topk, E, tile_m, ...)
 * called with the same tile_m: expert_offsets, sorted_pairs, tiles,
 * num_tiles and max_tiles are passed through unchanged.  Dropped pairs'
 * rows are written as zeros by the same launch.  Arithmetic: decoded weight
 * rounded to bf16 (NF4: RNE of the float32 weight; MXFP4: exact), bf16
 * matrix-core products, float32 accumulation.
 * InvalidValue: null pointer (pair_scale may be NULL), rows < 0, topk < 1,
 *   E < 1, N < 1 or N % 32, K not a positive multiple of 64 (NF4) / 32
 *   (MXFP4), bad stride or alignment, max_tiles below the bound.
 * NotSupported: tile_m != 256, rows*topk >= 2^31, grid beyond 2^31 blocks.
 * rows == 0 enqueues nothing.
 */
int gq_nf4_grouped_gemm(const uint16_t* x, int32_t rows, int32_t K, int64_t x_stride,
                        const uint8_t* codes, const float* absmax, int32_t num_experts,
                        int32_t N, int32_t topk, const float* pair_scale,
                        const int32_t* expert_offsets, const int32_t* sorted_pairs,
                        const int32_t* tiles, const int32_t* num_tiles, int32_t max_tiles,
                        int32_t tile_m, uint16_t* out, hipStream_t stream);
int gq_mxfp4_grouped_gemm(const uint16_t* x, int32_t rows, int32_t K, int64_t x_stride,
                          const uint8_t* blocks, const uint8_t* scales, int32_t num_experts,
                          int32_t N, int32_t topk, const float* pair_scale,
                          const int32_t* expert_offsets, const int32_t* sorted_pairs,
                          const int32_t* tiles, const int32_t* num_tiles, int32_t max_tiles,
                          int32_t tile_m, uint16_t* out, hipStream_t stream);

/* ------------------------------------------------------------------------
 * MXFP4 prefill on the block-scaled fp4 matrix instruction.  [P2] summary
 * (MXFP4 as OCP e2m1 on the checkpoint's released bytes, decoded inside the
 * mainloop); [P3] summary (native MXFP4 expert inference); [P1] "Which
 * entry point?" (native MXFP4 expert math).  The weights' e2m1 codes and
 * e8m0 scales are fed to the gfx950 instruction as stored, with no decode.
 * The pages keep activations in bf16; the instruction's other operand must
 * be an MX format too, so the activations are first written as two e4m3
 * terms (the reading of this library):
 *
 *   x[t, k] ~= hi[t, k] * 2^(s_hi[t, k/32] - 127) + lo[t, k] * 2^(s_lo[t, k/32] - 127)
 *
 * per 32 consecutive k: X = the smallest integer with amax * 2^-X <= 448
 * (the largest e4m3 magnitude; -127 for an all-zero block), hi = e4m3 of
 * x * 2^-Xh rounded to nearest even, lo the same for the exact residual
 * x - hi * 2^Xh with its own exponent.  The two terms hold every bf16 value
 * of a block exactly unless its magnitudes span 2^12 or more; in any case
 * |x - split| <= 2^-8 |x| + 2^-16 amax.  Results are then within the same
 * tolerance of the float64 W4A16 product as the bf16 path.
 *
 * gq_act_split_e4m3: x uint16 bf16 [rows, K] (row stride x_stride elements,
 * a multiple of 8; K a multiple of 32) -> with Kp = K rounded up to 64:
 *   codes  uint8 [rows, 2*Kp]: per row and 64-k step s, 128 bytes: hi codes
 *          then lo codes, 64 bytes each; in each, bytes [32h, 32h+32) hold
 *          elements 16h + [0, 16) of k block 2s, then of block 2s+1 (the
 *          order the instruction's e4m3 operand takes them in)
 *   scales uint8 [rows, Kp/16]: per step s_hi(2s), s_lo(2s), s_hi(2s+1),
 *          s_lo(2s+1)
 * A block past K (K % 64 == 32) is written as zeros with scale byte 0.
 * codes 16-byte aligned, scales 4-byte aligned.
 * InvalidValue: null pointer, rows < 0, K not a positive multiple of 32,
 *   bad stride or alignment.  NotSupported: grid beyond 2^31 blocks.
 *
 * gq_mxfp4_grouped_gemm_scaled: as gq_mxfp4_grouped_gemm with the
 * activations given as gq_act_split_e4m3's output for x [rows, K]:
 *
 *   out[p, n] = bf16( pair_scale[p] * sum_k split(x)[p/topk, k] * W_{ids[p]}[n, k] )
 *
 * float32 accumulation of groups of 8 neighbouring k, whose products of codes
 * are cut as gq_mxfp4_grouped_gemm_fp8 says.  Same grouping, pair_scale and out
 * conventions.
 * InvalidValue: null pointer (pair_scale may be NULL), rows < 0, topk < 1,
 *   E < 1, N < 1 or N % 32, K not a positive multiple of 32, bad alignment,
 *   max_tiles below the bound.
 * NotSupported: tile_m != 256, rows*topk >= 2^31, rows*2*Kp >= 2^31, grid
 *   beyond 2^31 blocks.  rows == 0 enqueues nothing.
 *
 * gq_mxfp4_grouped_gemm_scaled_swiglu: the gate_up product of gpt-oss's
 * experts with their gated unit applied in the epilogue.  The pages run
 * gpt-oss MXFP4 experts ("Receipts-driven engineering", "The numbers") but
 * do not define the activation; the reading of this library is gpt-oss's
 * published expert MLP, whose fused gate_up weight interleaves gate row j
 * (row 2j) and up row j (row 2j + 1):
 *
 *   g = sum_k split(x)[p/topk, k] * W[2j, k],  u = ... W[2j + 1, k]
 *   act[p, j] = bf16( gc * sigmoid(alpha * gc) * (uc + 1) ),
 *   gc = min(g, limit),  uc = min(max(u, -limit), limit)
 *
 * in float32, sigmoid(z) = 1 / (1 + 2^(-z log2 e)) from the hardware
 * exponential and reciprocal (a few float32 ulp; gpt-oss: alpha = 1.702,
 * limit = 7).  blocks/scales [E, N, K]
 * with N = 2I; act uint16 bf16 [rows*topk, I], rows of dropped pairs zero.
 * No pair_scale.  Errors as gq_mxfp4_grouped_gemm_scaled, plus
 * InvalidValue for a non-finite alpha or limit, or limit < 0.
 *
 * gq_mxfp4_grouped_gemm_scaled_swiglu_split: the same product and gated
 * unit, the bf16 result written as its two-term e4m3 split (the layout of
 * gq_act_split_e4m3 for [rows*topk, I]) instead of as bf16, so that it
 * feeds the down product directly:
 *
 *   act_codes, act_scales = gq_act_split_e4m3(act)   (bytes identical)
 *
 * act_codes uint8 [rows*topk, 2I] (16-byte aligned), act_scales uint8
 * [rows*topk, I/16] (4-byte aligned); rows of dropped pairs get zero codes
 * and zero scale bytes (the split of a zero row).  Errors as
 * gq_mxfp4_grouped_gemm_scaled_swiglu; NotSupported also when N % 128 != 0
 * (I a multiple of 64: whole 64-column split steps).
 */
int gq_act_split_e4m3(const uint16_t* x, int32_t rows, int32_t K, int64_t x_stride,
                      uint8_t* codes, uint8_t* scales, hipStream_t stream);
int gq_mxfp4_grouped_gemm_scaled(const uint8_t* x_codes, const uint8_t* x_scales, int32_t rows,
                                 int32_t K, const uint8_t* blocks, const uint8_t* scales,
                                 int32_t num_experts, int32_t N, int32_t topk,
                                 const float* pair_scale, const int32_t* expert_offsets,
                                 const int32_t* sorted_pairs, const int32_t* tiles,
                                 const int32_t* num_tiles, int32_t max_tiles, int32_t tile_m,
                                 uint16_t* out, hipStream_t stream);
int gq_mxfp4_grouped_gemm_scaled_swiglu(const uint8_t* x_codes, const uint8_t* x_scales,
                                        int32_t rows, int32_t K, const uint8_t* blocks,
                                        const uint8_t* scales, int32_t num_experts, int32_t N,
                                        int32_t topk, float alpha, float limit,
                                        const int32_t* expert_offsets,
                                        const int32_t* sorted_pairs, const int32_t* tiles,
                                        const int32_t* num_tiles, int32_t max_tiles,
                                        int32_t tile_m, uint16_t* act, hipStream_t stream);
int gq_mxfp4_grouped_gemm_scaled_swiglu_split(
    const uint8_t* x_codes, const uint8_t* x_scales, int32_t rows, int32_t K,
    const uint8_t* blocks, const uint8_t* scales, int32_t num_experts, int32_t N, int32_t topk,
    float alpha, float limit, const int32_t* expert_offsets, const int32_t* sorted_pairs,
    const int32_t* tiles, const int32_t* num_tiles, int32_t max_tiles, int32_t tile_m,
    uint8_t* act_codes, uint8_t* act_scales, hipStream_t stream);

/* ------------------------------------------------------------------------
 * NF4 input gradient.  [P1] "Which entry point?" (grouped NF4 backward);
 * [P2] summary (the NF4 path is differentiable, fine-tuning stays packed).
 *
 *   dx[p, k] = bf16( sum_n dy[p, n] * W_{e(p)}[n, k] )
 *
 *   dy   uint16 bf16 [P, N] with row stride dy_stride elements (per pair)
 *   dx   uint16 bf16 [P, K]
 * The grouping comes from gq_route_sort(pair_expert, P, 1, E, tile_m, ...);
 * pairs with an expert outside [0, E) get dx rows of zeros.  Same decode
 * and arithmetic as the NF4 GEMM, contraction over N.
 * InvalidValue: null pointer, P < 0, E < 1, N < 1 or N % 64, K not a
 *   positive multiple of 64, bad stride or alignment, max_tiles too small.
 * NotSupported: tile_m != 256, grid beyond 2^31 blocks.
 */
int gq_nf4_grouped_dgrad(const uint16_t* dy, int32_t P, int32_t N, int64_t dy_stride,
                         const uint8_t* codes, const float* absmax, int32_t num_experts,
                         int32_t K, const int32_t* expert_offsets, const int32_t* sorted_pairs,
                         const int32_t* tiles, const int32_t* num_tiles, int32_t max_tiles,
                         int32_t tile_m, uint16_t* dx, hipStream_t stream);

/* ------------------------------------------------------------------------
 * MXFP4 input gradient.  [P1] "Which entry point?" (native MXFP4 expert
 * math next to the grouped NF4 backward).  The pages name no MXFP4
 * backward entry point; this is the NF4 one with the MXFP4 decode:
 *
 *   dx[p, k] = bf16( sum_n dy[p, n] * W_{e(p)}[n, k] )
 *
 *   blocks  uint8 [E, N, K/32, 16] e2m1 codes (element 2j: low nibble)
 *   scales  uint8 [E, N, K/32] e8m0 (255 = NaN)
 * Decoded weights are exact in bf16; bf16 matrix-core products, float32
 * accumulation.  dy, dx and the grouping as for gq_nf4_grouped_dgrad.
 * InvalidValue: null pointer, P < 0, E < 1, N < 1 or N % 64, K not a
 *   positive multiple of 32, bad stride or alignment, max_tiles too small.
 * NotSupported: tile_m != 256, grid beyond 2^31 blocks.
 */
int gq_mxfp4_grouped_dgrad(const uint16_t* dy, int32_t P, int32_t N, int64_t dy_stride,
                           const uint8_t* blocks, const uint8_t* scales, int32_t num_experts,
                           int32_t K, const int32_t* expert_offsets, const int32_t* sorted_pairs,
                           const int32_t* tiles, const int32_t* num_tiles, int32_t max_tiles,
                           int32_t tile_m, uint16_t* dx, hipStream_t stream);

/* ------------------------------------------------------------------------
 * MoE-layer epilogues.  The pages benchmark the grouped products on the
 * Qwen3-30B-A3B expert shapes, whose experts are SwiGLU MLPs; [P1] header
 * (one launch for the active experts) and [P4] "Functions" ([M, top_k]
 * routing, per-slot [M, top_k, N] outputs that the caller reduces over
 * top_k).  The pages leave the activation and the reduction to the caller;
 * these entry points fuse them (readings: gate rows [0, I) then up rows
 * [I, 2I) in a fused gate_up weight; SwiGLU act = silu(gate) * up with
 * silu(z) = z / (1 + exp(-z)); combine = router-weighted sum over a
 * token's slots, in slot order).  All arithmetic float32, one bf16
 * rounding per output; sigmoid (in silu and in gpt-oss's gated unit) is
 * 1 / (1 + 2^(-z log2 e)) from the hardware exponential and reciprocal, a
 * few float32 ulp from the correctly rounded value.
 *
 * gq_nf4_grouped_gemv_swiglu / gq_nf4_grouped_gemm_swiglu:
 *   act[p, j] = bf16( silu(g) * u ),  g = sum_k x[p/topk, k] * W[j, k],
 *                                     u = sum_k x[p/topk, k] * W[I + j, k]
 *   codes/absmax [E, N, K] with N = 2I; act uint16 bf16 [rows*topk, I].
 *   Arguments, grouping and errors as gq_nf4_grouped_gemv / _gemm without
 *   pair_scale; InvalidValue also for N odd (GEMV) or N % 64 (GEMM).
 *
 * gq_mxfp4_grouped_gemv_swiglu: the decode gate_up GEMV of gpt-oss's
 * experts with their gated unit (the gq_mxfp4_grouped_gemm_scaled_swiglu
 * reading: gate row 2j, up row 2j + 1, act = gc * sigmoid(alpha * gc) *
 * (uc + 1), gc = min(g, limit), uc = min(max(u, -limit), limit)), on the
 * exact float32 products of gq_mxfp4_grouped_gemv.  blocks/scales
 * [E, N, K] with N = 2I; act uint16 bf16 [rows*topk, I].  Errors as
 * gq_mxfp4_grouped_gemv without pair_scale, plus InvalidValue for N odd, a
 * non-finite alpha or limit, or limit < 0.
 *
 * gq_nf4_grouped_gemv_down_combine (decode, rows*topk <= 64):
 *   y[t, n] = bf16( sum_s w[t, s] * sum_i act[t*topk + s, i] * W_{ids[t, s]}[n, i] )
 *   act   uint16 bf16 [rows*topk, I], row stride act_stride elements
 *   codes/absmax [E, H, I] NF4 (I % 64 == 0); topk_weights float [rows, topk]
 *   or NULL (weights 1); y uint16 bf16 [rows, H].  A slot whose expert is
 *   outside [0, E) contributes 0.
 *   InvalidValue: null pointer (topk_weights may be NULL), rows < 1,
 *     topk < 1, E < 1, H < 1, I not a positive multiple of 64, bad stride
 *     or alignment.  NotSupported: rows*topk > 64, I > 4096, I > 2048 with
 *     rows*topk > 32, H >= 2^24, act_stride > 2^31 - 1.
 *
 * gq_mxfp4_grouped_gemv_down_combine: the same on MXFP4 experts
 *   (blocks/scales [E, H, I], I a positive multiple of 32), float32 exact
 *   decode as gq_mxfp4_grouped_gemv; same errors with I % 32 for I % 64.
 *
 * gq_moe_combine (prefill):
 *   y[t, :] = bf16( sum_s w[t, s] * y_pairs[t*topk + s, :] )
 *   y_pairs uint16 bf16 [rows*topk, H] (row stride `stride` elements);
 *   topk_weights float [rows, topk] or NULL (plain sum, e.g. when the
 *   router weight was applied as pair_scale); y uint16 bf16 [rows, H].
 *   InvalidValue: rows < 0, topk < 1, H < 1 or H % 8, stride < H or
 *   stride % 8, null or misaligned pointers.  rows == 0 enqueues nothing.
 */
int gq_nf4_grouped_gemv_swiglu(const uint16_t* x, int32_t rows, int32_t K, int64_t x_stride,
                               const uint8_t* codes, const float* absmax, int32_t num_experts,
                               int32_t N, const int32_t* topk_ids, int32_t topk, uint16_t* act,
                               hipStream_t stream);
int gq_nf4_grouped_gemm_swiglu(const uint16_t* x, int32_t rows, int32_t K, int64_t x_stride,
                               const uint8_t* codes, const float* absmax, int32_t num_experts,
                               int32_t N, int32_t topk, const int32_t* expert_offsets,
                               const int32_t* sorted_pairs, const int32_t* tiles,
                               const int32_t* num_tiles, int32_t max_tiles, int32_t tile_m,
                               uint16_t* act, hipStream_t stream);
int gq_mxfp4_grouped_gemv_swiglu(const uint16_t* x, int32_t rows, int32_t K, int64_t x_stride,
                                 const uint8_t* blocks, const uint8_t* scales,
                                 int32_t num_experts, int32_t N, const int32_t* topk_ids,
                                 int32_t topk, float alpha, float limit, uint16_t* act,
                                 hipStream_t stream);
int gq_nf4_grouped_gemv_down_combine(const uint16_t* act, int32_t rows, int32_t I,
                                     int64_t act_stride, const uint8_t* codes,
                                     const float* absmax, int32_t num_experts, int32_t H,
                                     const int32_t* topk_ids, int32_t topk,
                                     const float* topk_weights, uint16_t* y,
                                     hipStream_t stream);
int gq_mxfp4_grouped_gemv_down_combine(const uint16_t* act, int32_t rows, int32_t I,
                                       int64_t act_stride, const uint8_t* blocks,
                                       const uint8_t* scales, int32_t num_experts, int32_t H,
                                       const int32_t* topk_ids, int32_t topk,
                                       const float* topk_weights, uint16_t* y,
                                       hipStream_t stream);
int gq_moe_combine(const uint16_t* y_pairs, int32_t rows, int32_t topk, int32_t H,
                   int64_t stride, const float* topk_weights, uint16_t* y, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Element types of entry points that take more than one.
 */
enum { GQ_F32 = 0, GQ_BF16 = 1, GQ_F16 = 2 };

/* ------------------------------------------------------------------------
 * MXFP4 quantisation on the device: the bytes that every MXFP4 entry point
 * reads, from rows of values.  [P1] "Try the packers and byte checks on CPU"
 * (packed shapes, round trip), [P2] summary (OCP e2m1 codes, e8m0 scales).
 *   x       x_dtype [rows, K], row stride x_stride elements (any >= K, any
 *           alignment of one element)
 *   blocks  uint8 [rows, K/32, 16], scales uint8 [rows, K/32]         out
 *   values  uint16 bf16 [rows, K] or NULL: the values that the codes stand
 *           for (exact), the forward value of quantisation-aware training
 *           (whose gradient passes straight through)                   out
 * Per block of 32: X = clamp(floor(log2 amax) - 2, -127, 127), -127 for a
 * zero block; code = sign and the nearest e2m1 magnitude of |v| 2^-X, ties
 * to the even code, above 6 becomes 6; scale byte X + 127.  A block with an
 * infinity or NaN stores scale 255 and codes 0: it decodes to NaN.
 * Re-quantising decoded values reproduces the bytes.
 * InvalidValue: null pointer (values may be NULL), unknown x_dtype, rows < 0,
 *   K not a positive multiple of 32, x_stride < K, x not aligned to its
 *   element, blocks or values not 16-byte aligned.
 * NotSupported: rows*x_stride >= 2^60.  rows == 0 enqueues nothing.
 */
int gq_mxfp4_quantize(const void* x, int32_t x_dtype, int64_t rows, int32_t K, int64_t x_stride,
                      uint8_t* blocks, uint8_t* scales, uint16_t* values, hipStream_t stream);

/* ------------------------------------------------------------------------
 * MXFP8 quantisation on the device: what gq_mxfp4_quantize is to MXFP4, for
 * the entry points that take 8-bit activations.
 *   codes   uint8 [rows, K]: OCP e4m3 (NaN at 0x7F and 0xFF), in element order;
 *           scales uint8 [rows, K/32] e8m0, 255 = NaN                  out
 *   values  uint16 bf16 [rows, K] or NULL: the values that the codes stand for
 *           (exact; magnitudes below 2^-133 rounded to bf16's steps, and
 *           float32 values that round up to 2^128 infinite)           out
 * A decoded block, quantised again, decodes to the same values.
 * Per block of 32: X = the smallest integer in [-127, 127] with
 * amax 2^-X <= 448, the largest e4m3 magnitude (so that no code saturates;
 * the rule of the first term of gq_act_split_e4m3), -127 for a zero block;
 * code = e4m3 of v 2^-X, ties to even, sign kept; scale byte X + 127.  A block
 * with an infinity or NaN stores scale 255 and codes 0: it decodes to NaN.
 * Arguments and errors as gq_mxfp4_quantize.
 */
int gq_mxfp8_quantize(const void* x, int32_t x_dtype, int64_t rows, int32_t K, int64_t x_stride,
                      uint8_t* codes, uint8_t* scales, uint16_t* values, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Root-mean-square norm of rows before the experts: the residual's addition,
 * the norm, and its result in 8 bits, in one pass.
 *
 *   h = x + residual, rounded to the rows' type (h = x without a residual)
 *   y_i = h_i weight_i / sqrt(mean(h^2) + eps)
 *
 *   x         dtype [rows, H], row stride x_stride elements (any >= H, any
 *             alignment of one element); residual the same, or NULL
 *   weight    weight_dtype [H]: the rows' type or GQ_F32
 *   sum       dtype [rows, H] or NULL: h (only with a residual)        out
 *   y         dtype [rows, H] or NULL                                  out
 *   codes, scales, values  or NULL: y in MXFP8, as gq_mxfp8_quantize would
 *             write it for a float32 y (H a multiple of 32)            out
 * float32 throughout; h and y are rounded once each, the codes are made of
 * the unrounded y.  The norm is the norm of the rounded h.  A finite row whose
 * squares' sum passes float32's largest value gives zeros; with eps = 0 one whose
 * squares vanish in float32 (a zero row among them) gives infinities or NaN.
 * sum and y may each be x or residual where that is contiguous (they must not
 * both be the same one); no other output may overlap an input.
 * InvalidValue: null x or weight, no output, sum without a residual, codes
 *   without scales or the reverse, values without codes, codes with H % 32,
 *   unknown dtype, a weight_dtype that is neither, rows < 0, H < 1, a stride
 *   < H, eps < 0 or not finite, a pointer not aligned to its element, codes or
 *   values not 16-byte aligned, sum and y at one address, or one of them in place
 *   of an input that is not contiguous.
 * NotSupported: H > 32768, rows*stride >= 2^60.  rows == 0 enqueues nothing.
 *
 * gq_rms_norm_backward: gradients of y to x (and residual, the same) and to
 * the weight.  With rstd = 1 / sqrt(mean(h^2) + eps), n = h rstd, g = d_y weight:
 *   d_x_i = rstd (g_i - n_i mean(g n)) + d_h_i,  d_weight_i = sum_rows d_y_i n_i
 *   h         dtype [rows, H]: forward's sum (x, where there was no residual)
 *   d_h       dtype [rows, H] or NULL: the gradient of forward's sum
 *   d_x       dtype [rows, H]                                          out
 *   d_weight  weight_dtype [H] or NULL: not wanted                     out
 *   workspace 16-byte aligned device memory of at least
 *             gq_rms_norm_backward_workspace(rows, H) bytes (with d_weight),
 *             which never falls as rows grow: one made for the most rows
 *             serves any number of them; carries nothing from one call to the
 *             next; two calls that may run at the same time need one each
 * float32 sums in a fixed order; rows == 0 writes d_weight = 0.  The gradient
 * of codes is taken as y's (straight through).  d_x may be d_y, h or d_h where
 * that is contiguous.
 * Errors as gq_rms_norm; InvalidValue also for a workspace that is too small.
 * gq_rms_norm_backward_workspace returns -1 for rows < 0 or an H outside
 * [1, 32768].
 */
int gq_rms_norm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                int32_t dtype, int64_t rows, int32_t H, const void* weight, int32_t weight_dtype,
                float eps, void* sum, void* y, uint8_t* codes, uint8_t* scales, uint16_t* values,
                hipStream_t stream);
int64_t gq_rms_norm_backward_workspace(int64_t rows, int32_t H);
int gq_rms_norm_backward(const void* d_y, int64_t d_y_stride, const void* h, int64_t h_stride,
                         const void* d_h, int64_t d_h_stride, int32_t dtype, int64_t rows,
                         int32_t H, const void* weight, int32_t weight_dtype, float eps, void* d_x,
                         void* d_weight, void* workspace, int64_t workspace_bytes,
                         hipStream_t stream);

/* ------------------------------------------------------------------------
 * MXFP4 activations times MXFP4 experts, on the e2m1 x e2m1 block-scaled
 * matrix instruction ([P1] "Which entry point?": native MXFP4 expert math).
 *
 *   out[p, n] = bf16( pair_scale[p] * sum_k xq[p/topk, k] * W_{ids[p]}[n, k] )
 *
 * x_blocks uint8 [rows, K/32, 16] and x_scales uint8 [rows, K/32] are what
 * gq_mxfp4_quantize writes; everything else is as for gq_mxfp4_grouped_gemm
 * (routing from gq_route_sort, dropped pairs' rows zero) and
 * gq_mxfp4_grouped_gemv (1..8 tokens, topk_ids read directly).  Products of
 * codes are exact, sums float32, one rounding to bf16.  Scale byte 255 on
 * either side makes every output that its block enters NaN.
 * The _swiglu forms apply the clamped gated unit of
 * gq_mxfp4_grouped_gemv_swiglu (weight rows 2j gate, 2j + 1 up) and write
 * [rows*topk, N/2]; a NaN passes through the unit.  No form takes expert
 * biases, as none of the other products does: a model whose gate_up has one,
 * which enters before the unit, takes the plain form and applies both itself,
 * or gq_moe_decode.
 * InvalidValue / NotSupported: as for the named entry points; K % 32, and
 *   NotSupported: rows*K/2 or N*K/2 >= 2^31, or 2^24 workgroups or more
 *   (max_tiles * 4 * ceil(N / 1024), rounded up to 32) (GEMM), rows*topk > 256
 *   or K > 8192 (GEMV).
 */
int gq_mxfp4_grouped_gemm_fp4(const uint8_t* x_blocks, const uint8_t* x_scales, int32_t rows,
                              int32_t K, const uint8_t* blocks, const uint8_t* scales,
                              int32_t num_experts, int32_t N, int32_t topk,
                              const float* pair_scale, const int32_t* expert_offsets,
                              const int32_t* sorted_pairs, const int32_t* tiles,
                              const int32_t* num_tiles, int32_t max_tiles, int32_t tile_m,
                              uint16_t* out, hipStream_t stream);
int gq_mxfp4_grouped_gemm_fp4_swiglu(const uint8_t* x_blocks, const uint8_t* x_scales,
                                     int32_t rows, int32_t K, const uint8_t* blocks,
                                     const uint8_t* scales, int32_t num_experts, int32_t N,
                                     int32_t topk, float alpha, float limit,
                                     const int32_t* expert_offsets, const int32_t* sorted_pairs,
                                     const int32_t* tiles, const int32_t* num_tiles,
                                     int32_t max_tiles, int32_t tile_m, uint16_t* act,
                                     hipStream_t stream);
int gq_mxfp4_grouped_gemv_fp4(const uint8_t* x_blocks, const uint8_t* x_scales, int32_t rows,
                              int32_t K, const uint8_t* blocks, const uint8_t* scales,
                              int32_t num_experts, int32_t N, const int32_t* topk_ids,
                              int32_t topk, const float* pair_scale, uint16_t* out,
                              hipStream_t stream);
int gq_mxfp4_grouped_gemv_fp4_swiglu(const uint8_t* x_blocks, const uint8_t* x_scales,
                                     int32_t rows, int32_t K, const uint8_t* blocks,
                                     const uint8_t* scales, int32_t num_experts, int32_t N,
                                     const int32_t* topk_ids, int32_t topk, float alpha,
                                     float limit, uint16_t* act, hipStream_t stream);

/* ------------------------------------------------------------------------
 * MXFP8 activations times MXFP4 experts, on the e4m3 x e2m1 block-scaled
 * matrix instruction: half the matrix work of the two-term split of
 * gq_mxfp4_grouped_gemm_scaled, with the activations' rounding of 8 bits.
 *
 *   out[p, n] = bf16( pair_scale[p] * sum_k xq[p/topk, k] * W_{ids[p]}[n, k] )
 *
 * x_codes uint8 [rows, K] and x_scales uint8 [rows, K/32] are what
 * gq_mxfp8_quantize and gq_rms_norm write; everything else, the errors
 * included, is as for the _fp4 entry points of the same name (x_codes 16-byte
 * aligned; NotSupported: rows*K >= 2^31 in the GEMM).  An e4m3 NaN code makes
 * every output that it enters NaN, as scale byte 255 does.
 * Sums: the matrix instruction of the GEMM forms adds 8 neighbouring k (8 i ..
 * 8 i + 7) at once and cuts each product of codes there toward zero to a
 * multiple of 2^(e - 13), e the largest sum of two codes' exponents among them
 * (a subnormal code's is the least normal one's; products of a zero do not
 * count): at most 7 2^-12 of the largest of them is lost, less than half a bf16
 * step of the sum of magnitudes.  Groups are added in float32, as everything is
 * in the GEMV forms.
 */
int gq_mxfp4_grouped_gemm_fp8(const uint8_t* x_codes, const uint8_t* x_scales, int32_t rows,
                              int32_t K, const uint8_t* blocks, const uint8_t* scales,
                              int32_t num_experts, int32_t N, int32_t topk,
                              const float* pair_scale, const int32_t* expert_offsets,
                              const int32_t* sorted_pairs, const int32_t* tiles,
                              const int32_t* num_tiles, int32_t max_tiles, int32_t tile_m,
                              uint16_t* out, hipStream_t stream);
int gq_mxfp4_grouped_gemm_fp8_swiglu(const uint8_t* x_codes, const uint8_t* x_scales,
                                     int32_t rows, int32_t K, const uint8_t* blocks,
                                     const uint8_t* scales, int32_t num_experts, int32_t N,
                                     int32_t topk, float alpha, float limit,
                                     const int32_t* expert_offsets, const int32_t* sorted_pairs,
                                     const int32_t* tiles, const int32_t* num_tiles,
                                     int32_t max_tiles, int32_t tile_m, uint16_t* act,
                                     hipStream_t stream);
int gq_mxfp4_grouped_gemv_fp8(const uint8_t* x_codes, const uint8_t* x_scales, int32_t rows,
                              int32_t K, const uint8_t* blocks, const uint8_t* scales,
                              int32_t num_experts, int32_t N, const int32_t* topk_ids,
                              int32_t topk, const float* pair_scale, uint16_t* out,
                              hipStream_t stream);
int gq_mxfp4_grouped_gemv_fp8_swiglu(const uint8_t* x_codes, const uint8_t* x_scales,
                                     int32_t rows, int32_t K, const uint8_t* blocks,
                                     const uint8_t* scales, int32_t num_experts, int32_t N,
                                     const int32_t* topk_ids, int32_t topk, float alpha,
                                     float limit, uint16_t* act, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Expert routing ([P4] "Functions": the routing tensor [M, top_k] and its
 * weights, which the other entry points take).
 *
 * gq_moe_topk: the topk largest logits of each row, largest first, equal
 * ones by lower index, with float32 softmax weights
 *   w_s = exp(z_s - peak) / sum exp(z - peak)
 * where the sum runs over the chosen logits (renormalize != 0) or over all
 * of the row's.  A logit of -inf is a masked expert: it is never chosen, and
 * a slot that only masked experts are left for gets id -1 and weight 0 (a
 * dropped pair for every other entry point).  A NaN or +inf logit is chosen
 * first and makes its row's weights NaN.
 *   logits       dtype [rows, E], row stride `stride` elements
 *   topk_ids     int32 [rows, topk], topk_weights float [rows, topk]   out
 *
 * gq_moe_topk_backward: gradient of the weights to the logits, through the
 * same softmax, the selection held fixed:
 *   d_logits[j] = p_j (G_j - sum_i p_i G_i),   G_j = sum of d_weights over
 * the slots that name expert j; p the softmax over the chosen logits (0 for
 * the others) or over all.  Ids outside [0, E) and masked experts take no
 * gradient; an id that stands in several slots counts once per slot (so
 * topk may exceed E here).
 *   d_weights    float [rows, topk]
 *   d_logits     dtype [rows, E], contiguous                           out
 * InvalidValue: null pointer, unknown dtype, rows < 0, E < 1, topk < 1,
 *   forward: topk > E, stride < E, misaligned pointers.
 * NotSupported: E > 1024, topk > 64, rows > 2^33, rows*stride >= 2^61.
 * rows == 0 enqueues nothing.
 */
int gq_moe_topk(const void* logits, int32_t dtype, int64_t rows, int32_t num_experts,
                int64_t stride, int32_t topk, int32_t renormalize, int32_t* topk_ids,
                float* topk_weights, hipStream_t stream);
int gq_moe_topk_backward(const float* d_weights, const void* logits, int32_t dtype, int64_t rows,
                         int32_t num_experts, int64_t stride, const int32_t* topk_ids,
                         int32_t topk, int32_t renormalize, void* d_logits, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Expert routing as models with many experts do it: scores of either kind, a
 * bias that balances the experts' load, and groups of experts.
 *
 *   s_e = softmax(z)_e or sigmoid(z_e);   c_e = s_e + bias_e
 * gq_moe_route: the experts lie in `groups` groups of E / groups neighbours.  A
 * group counts as the sum of its group_top (1 or 2) largest c; the topk_groups
 * largest groups are open, equal ones by lower index.  topk_ids are the topk
 * largest c of the open groups, largest first, equal ones by lower index.
 * Weights are of the scores without the bias:
 *   w_s = scale s_s   or   scale s_s / sum of the chosen s   (renormalize != 0)
 * c and the groups' sums are compared in float64.  Without a bias the experts are
 * in the order of their logits (and so are groups of group_top 1), of which the
 * scores are increasing functions.  groups = 1 leaves groups out.  The bias
 * takes no gradient.
 * A logit of -inf, or a c of -inf, is a masked expert: it is never chosen, a group
 * counts without it, a group of masked experts is never open, and a slot that
 * only masked experts are left for gets id -1 and weight 0.  A NaN counts above
 * every number; a sigmoid's NaN makes its own weight NaN and, renormalised, its
 * row's; a NaN or +inf logit makes a softmax row's weights NaN.  Renormalised
 * weights are right also where every chosen score is too small for a float32.
 *   logits   dtype [rows, E], row stride `stride` elements; bias float [E] or NULL
 *   topk_ids int32 [rows, topk], topk_weights float [rows, topk]      out
 *
 * gq_moe_route_backward: gradient of the weights to the logits, the selection
 * held fixed.  For each slot s of expert j, with G = scale d_weights:
 *   sigmoid  d_z_j += G_s s_j (1 - s_j), or renormalised, with n = s / sum s,
 *            d_z_j += n_s (1 - s_j) (G_s - sum_i n_i G_i)
 *   softmax  as gq_moe_topk_backward of G
 * ids outside [0, E) and masked logits take none; an id in several slots counts
 * once per slot.
 * InvalidValue: as gq_moe_topk / gq_moe_topk_backward; unknown score, groups < 1
 *   or not a divisor of E, topk_groups outside [1, groups], group_top not 1 or
 *   2, topk > topk_groups * E / groups, scale not finite, bias misaligned.
 * NotSupported: as there; groups > 64.
 */
enum { GQ_SOFTMAX = 0, GQ_SIGMOID = 1 };
int gq_moe_route(const void* logits, int32_t dtype, int64_t rows, int32_t num_experts,
                 int64_t stride, const float* bias, int32_t topk, int32_t score, int32_t groups,
                 int32_t topk_groups, int32_t group_top, int32_t renormalize, float scale,
                 int32_t* topk_ids, float* topk_weights, hipStream_t stream);
int gq_moe_route_backward(const float* d_weights, const void* logits, int32_t dtype, int64_t rows,
                          int32_t num_experts, int64_t stride, const int32_t* topk_ids,
                          int32_t topk, int32_t score, int32_t renormalize, float scale,
                          void* d_logits, hipStream_t stream);

/* ------------------------------------------------------------------------
 * A whole mixture-of-experts layer for a few tokens: router product,
 * selection, the experts' gated products and the weighted combine.
 *
 *   z = x Wr^T + br;   e_s, w_s as gq_moe_topk(z, topk, renormalize)
 *   a_s = unit(Wgu[e_s] x + bgu[e_s]);   y = bf16(sum_s w_s (Wd[e_s] a_s + bd[e_s]))
 *
 * unit: GQ_NF4 SwiGLU (gate rows [0, I), up rows [I, 2I)), GQ_MXFP4 the
 * clamped gated unit (gate row 2j, up row 2j + 1; alpha, limit), as in
 * gq_nf4_grouped_gemv_swiglu and gq_mxfp4_grouped_gemv_swiglu.  float32
 * throughout between the bf16 input and the bf16 output, the gated products
 * included.  A NaN of a token reaches that token's output (and no other).
 */
enum { GQ_NF4 = 0, GQ_MXFP4 = 1 };

typedef struct gq_moe_layer {
  int32_t format;                 /* GQ_NF4 or GQ_MXFP4 */
  int32_t num_experts;            /* E */
  int32_t topk;
  int32_t hidden;                 /* H */
  int32_t inner;                  /* I */
  int32_t renormalize;            /* weights: softmax over the chosen logits, else over all */
  float alpha, limit;             /* GQ_MXFP4's unit */
  const uint16_t* router_weight;  /* bf16 [E, H] */
  const uint16_t* router_bias;    /* bf16 [E] or NULL */
  const uint8_t* gate_up_codes;   /* the E experts' [2I, H] as the other entry points take them */
  const void* gate_up_scales;
  const uint16_t* gate_up_bias;   /* bf16 [E, 2I] or NULL */
  const uint8_t* down_codes;      /* [H, I] */
  const void* down_scales;
  const uint16_t* down_bias;      /* bf16 [E, H] or NULL */
} gq_moe_layer;

/*
 * gq_moe_decode_workspace: bytes of device memory that gq_moe_decode needs
 * for `rows` tokens (16-byte aligned); -1 if the layer or rows are not ones
 * that gq_moe_decode takes.  The workspace carries nothing from one call to
 * the next and needs no clearing; two calls that may run at the same time
 * need one each.
 *
 * gq_moe_decode:
 *   layer      read during the call only (the arrays it names stay the caller's)
 *   x          uint16 bf16 [rows, H], row stride x_stride elements
 *   y          uint16 bf16 [rows, H]
 * InvalidValue: null layer or array (biases may be NULL), unknown format,
 *   topk outside [1, E], H or I not a positive multiple of 64 (GQ_NF4) / 32
 *   (GQ_MXFP4), alpha or limit not finite or limit < 0 (GQ_MXFP4), rows < 0,
 *   x_stride < H or % 8, workspace too small, misaligned pointers.
 * NotSupported: rows > 8, rows*topk > 64, E > 512, H > 8192, I > 4096,
 *   x_stride > 2^31 - 1.
 * rows == 0 enqueues nothing.
 */
int64_t gq_moe_decode_workspace(const gq_moe_layer* layer, int32_t rows);
int gq_moe_decode(const gq_moe_layer* layer, const uint16_t* x, int32_t rows, int64_t x_stride,
                  void* workspace, int64_t workspace_bytes, uint16_t* y, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GQ_H */
