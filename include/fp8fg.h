/*
 * fp8fg.h -- fine-grained FP8 quantization and block-scaled FP8 GEMM on AMD
 * Instinct MI355X (gfx950).  C ABI of libfp8fg.so.
 *
 * The method (DeepSeek-V3's FP8 recipe, as retold by the pages this library
 * follows):
 *   - "The Insider Secrets Of Deepseek Discovered", passage on Figure 7(a):
 *     activations are scaled per 1x128 tile (one token, 128 channels) and
 *     weights per 128x128 block; passage on Figure 7(b): partial GEMM sums are
 *     promoted to FP32 at a fixed K interval and the scales are applied there;
 *     passage on Figure 6: Fprop, Dgrad and Wgrad of a Linear all run in FP8.
 *   - DeepSeek-V3 FP8 knowledge-base page (codingmall.com), sections on
 *     fine-grained quantization, online quantization (scales from the current
 *     tile's max-abs), increased accumulation precision and unified E4M3.
 *   - DeepGEMM launch article (itstec.com.br), "Principais caracteristicas":
 *     dense GEMMs plus two MoE grouped layouts, contiguous and masked.
 *
 * Conventions shared by every entry point
 *   - Every pointer is a DEVICE pointer owned by the caller, 16-byte aligned.
 *     The library allocates, frees and synchronizes nothing; it keeps no state
 *     between calls and is reentrant.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).  Work
 *     is enqueued asynchronously on it; the call returns before it runs.
 *   - Codes are OCP E4M3 bytes ("E4M3FN": bias 7, max 448, NaN = 0x7F/0xFF,
 *     no infinities).  Scales are FP32 DEQUANTIZATION multipliers:
 *     value ~= decode(code) * scale, with scale = RN32(amax / 448) and the
 *     code = E4M3 round-to-nearest-even-saturating of RN32(x / scale), IEEE
 *     division throughout.  A group whose amax is 0 gets scale 0 and signed
 *     zero codes.  Inputs must be finite (NaN/Inf: unspecified output).
 *   - Return value: FP8FG_OK, or a negative fp8fg_status.  Argument errors are
 *     detected on the host BEFORE anything is enqueued (no partial work);
 *     FP8FG_ERR_HIP means the kernel launch itself failed.  A zero-sized
 *     problem (M == 0, G == 0, ...) is a successful no-op.  The quantizers
 *     also accept NULL for the pointers of an operand with no elements.
 *   - Scale layouts.  A 1x128-scaled operand of logical shape [R][K] (K = the
 *     axis the 128-element groups run along) stores codes u8 [R][K] row-major
 *     and scales f32 [K/128][R] ("kb-major").  A 128x128-scaled [N][K] operand
 *     stores codes u8 [N][K] and scales f32 [N/128][K/128].
 *   - Partial groups.  The grouped axis (K, or the token axis of the
 *     token-wise layout) need only be a multiple of 16: the last group then
 *     holds fewer than 128 elements and is quantized as that group padded
 *     with zeros (its max-abs runs over the elements that exist).  Every
 *     count "K/128" in this header means ceil(K/128).  Likewise N, the
 *     output channels (rows of B), need only be a multiple of 16 where stated:
 *     "N/128" then means ceil(N/128).
 *   - GEMM: C[M][N] = A[M][K] . B[N][K]^T, both operands K-major (a Linear
 *     layer y = x . W^T with W [out][in]).  C is the sum over k of
 *     decode(a) * sA * decode(b) * sB, the scales of each 128-wide K-block
 *     applied once per block in FP32 (promotion at a fixed K interval).
 *     Output row-major [M][N], BF16 (round-to-nearest-even) or FP32.
 *     Accuracy contract, element by element, against the exact real-number
 *     result C*:  |C - C*| <= 2^-14 * S  (FP32 out), with
 *     S = sum_k |decode(a) sA decode(b) sB|, plus one BF16 rounding of C*
 *     for BF16 out.  The codes are widened exactly to BF16 and multiplied on
 *     the BF16 matrix cores (exact products, FP32 sums).  One call,
 *     fp8_gemm_blockscaled_fp8mfma, runs the FP8 matrix cores instead and
 *     has its own, looser contract (see there).  Results are deterministic
 *     (no atomics, no split-K).  The library reads no environment variables.
 *   - The 2^-14 * S contract is a worst-case bound: it counts at most 1024
 *     FP32 roundings of quantities no larger than S.  The calls that take any
 *     K keep it for K <= 114688 (896 K-blocks: fresh FP32 sums per K-block,
 *     one rounding per promotion); beyond that it holds for the typical
 *     (random-sign) accumulation, not in the worst case.
 */
#ifndef FP8FG_H
#define FP8FG_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FP8FG_ABI_VERSION 15

enum fp8fg_status {
    FP8FG_OK = 0,
    FP8FG_ERR_NULL = -1,         /* a required pointer is NULL                 */
    FP8FG_ERR_SHAPE = -2,        /* negative size, or a size rule of the call  */
    FP8FG_ERR_ALIGN = -3,        /* a pointer is not 16-byte aligned           */
    FP8FG_ERR_UNSUPPORTED = -4,  /* unknown enum value or size beyond limits   */
    FP8FG_ERR_HIP = -5           /* the HIP runtime refused the launch         */
};

enum fp8fg_out { FP8FG_OUT_BF16 = 0, FP8FG_OUT_FP32 = 1 };

enum fp8fg_bscale {
    FP8FG_BSCALE_128x128 = 0,    /* sb f32 [N/128][K/128]   (weights: Fprop, Dgrad) */
    FP8FG_BSCALE_1x128 = 1       /* sb f32 [K/128][N]       (token-wise operand: Wgrad) */
};

enum fp8fg_score { FP8FG_SCORE_SOFTMAX = 0, FP8FG_SCORE_SIGMOID = 1 };

/*
 * Online 1x128 activation quantization.
 * x: f32 [M][K] row-major (M tokens, K channels).
 * transpose_out = 0: tiles run along K (one token x 128 channels).
 *     q: u8 [M][K], s: f32 [K/128][M].          Requires K % 16 == 0.
 * transpose_out = 1: tiles run along M (128 tokens x one channel), the
 *     operand layout of the Wgrad GEMM, whose contraction runs over tokens.
 *     q: u8 [K][M] (transposed), s: f32 [M/128][K].  Requires M % 16 == 0.
 * Sizes: M, K >= 0 and M * K < 2^40.
 */
int fp8_quant_act_1x128(const float* x, int64_t M, int64_t K, int transpose_out,
                        uint8_t* q, float* s, void* stream);

/*
 * Online 128x128 weight quantization.
 * w: f32 [N][K] row-major (N output channels, K input channels).
 * transpose_out = 0: q u8 [N][K], s f32 [N/128][K/128].
 * transpose_out = 1: q u8 [K][N] = the codes of w, transposed, with
 *     s f32 [K/128][N/128]: the B operand of the Dgrad GEMM.  Square blocks
 *     make this identical to quantizing w^T.
 * Requires N % 16 == 0 and K % 16 == 0 (partial blocks at either end);
 * N * K < 2^40.
 */
int fp8_quant_weight_128x128(const float* w, int64_t N, int64_t K, int transpose_out,
                             uint8_t* q, float* s, void* stream);

/*
 * The same two quantizations with BF16 inputs: x / w hold bf16 bit patterns
 * (u16, same shapes and layouts as above).  The tensors around the FP8 GEMMs
 * stay in a wider format (DeepSeek-V3 FP8 knowledge-base page, section on
 * the mixed-precision framework), and BF16 is the one named beside FP8 ("The
 * Insider Secrets Of Deepseek Discovered", passage on FP8 and BF16 modes).
 * Each bf16 value widens to fp32 exactly, so codes and scales are identical to
 * those of the fp32 entry points on the widened tensor; the reads are half as
 * many bytes.  Sizes, alignment (16 bytes for every pointer), errors and
 * layouts as for the fp32 calls.
 */
int fp8_quant_act_1x128_bf16(const uint16_t* x, int64_t M, int64_t K, int transpose_out,
                             uint8_t* q, float* s, void* stream);
int fp8_quant_weight_128x128_bf16(const uint16_t* w, int64_t N, int64_t K, int transpose_out,
                                  uint8_t* q, float* s, void* stream);

/*
 * Both operands of a Linear layer's Fprop GEMM in one launch (both are
 * quantized online each step: "The Insider Secrets Of Deepseek Discovered",
 * passages on Figure 7(a) and on online quantization): exactly
 *   fp8_quant_act_1x128(x, M, K, 0, qa, sa)        (or _bf16 when x_bf16 = 1)
 *   fp8_quant_weight_128x128(w, N, K, 0, qb, sb)   (or _bf16 when w_bf16 = 1)
 * byte for byte, with the same layouts (qa u8 [M][K], sa f32 [K/128][M],
 * qb u8 [N][K], sb f32 [N/128][K/128]).  x / w are f32, or bf16 bit patterns
 * when x_bf16 / w_bf16 is 1.  The two small grids share one launch, so they
 * overlap instead of each paying its own ramp-up and drain.  Requires
 * K % 16 == 0, N % 16 == 0, M, N, K >= 0, M * K < 2^40 and N * K < 2^40;
 * 16-byte aligned pointers; x_bf16 and w_bf16 in {0, 1}.  M = 0 or N = 0
 * skips that operand only, as the separate call would, and that operand's
 * pointers may then be NULL; K = 0, or M = N = 0, is a successful no-op.
 * Errors as for the separate calls.
 */
int fp8_quant_fprop_operands(const void* x, int x_bf16, int64_t M, const void* w, int w_bf16, int64_t N,
                             int64_t K, uint8_t* qa, float* sa, uint8_t* qb, float* sb, void* stream);

/*
 * FP8 activation cache for backward ("The Insider Secrets Of Deepseek
 * Discovered", passage on Figure 6: with Wgrad in FP8, the input of a Linear
 * can be kept in FP8 for the backward pass).  Builds the Wgrad operand from
 * the cached Fprop operand without its fp32 source:
 *   q: u8 [M][K] with s: f32 [K/128][M]  -- 1x128 codes along K (the output
 *      of fp8_quant_act_1x128 with transpose_out = 0);
 *   x'[m][k] = RN32(decode(q[m][k]) * s[k/128][m])  (fp32, one rounding);
 *   qt: u8 [K][M], st: f32 [M/128][K]  -- 1x128 codes of x' along tokens,
 *      transposed: exactly fp8_quant_act_1x128(x', transpose_out = 1).
 * Requires M % 16 == 0 and K % 16 == 0; M * K < 2^40.  Codes 0x7F / 0xFF
 * (NaN) in q give unspecified output.
 */
int fp8_requant_act_tokenwise(const uint8_t* q, const float* s, int64_t M, int64_t K,
                              uint8_t* qt, float* st, void* stream);

/*
 * MX variant (microscaling).  "The Insider Secrets Of Deepseek Discovered",
 * passage after Figure 7: the method is consistent with microscaling
 * formats.  Reading (the pages define no MX rule): the OCP MX rule for E4M3
 * elements, one power-of-two scale per block of 32 consecutive K, stored as
 * an E8M0 byte.  This is a different numeric contract from the calls above
 * (power-of-two scales, 32-element blocks, no FP32 scale), offered beside
 * them for comparison; gfx950 applies these scales inside the MFMA.
 *
 * fp8_quant_mx_1x32: x f32 [R][K] -> codes q u8 [R][K] and scale bytes
 *   e u8 [K/32][R]:  s = clamp(floor(log2(amax)) - 8, -127, 127) per block
 *   (amax = 0 gives -127), code = E4M3_RNE_SAT(RN32(x * 2^-s)), e = s + 127.
 *   Requires K % 32 == 0; R * K < 2^40.
 * fp8_quant_mx_1x32_transposed: the same rule on blocks of 32 consecutive
 *   rows (tokens) of one column, codes written transposed -- exactly
 *   fp8_quant_mx_1x32 applied to x^T: x f32 [M][K] -> q u8 [K][M], e u8
 *   [M/32][K].  The operands of the MX Wgrad (X and dY, contraction over
 *   tokens) and the MX Dgrad weight (W [N][K] -> W^T blocked along N; "The
 *   Insider Secrets Of Deepseek Discovered", Figure 6: all three GEMMs of a
 *   Linear in FP8).  Requires M % 32 == 0 (any K); M * K < 2^40,
 *   ceil(K / 64) <= 65535.  Empty arrays may be NULL.
 * fp8_gemm_mx: C[M][N] = sum_k decode(a) 2^(ea-127) decode(b) 2^(eb-127) with
 *   a u8 [M][K], ea u8 [K/32][M], b u8 [N][K], eb u8 [K/32][N]; c BF16 or FP32
 *   [M][N].  Accuracy: |C - C*| <= 2^-9 * S (S = sum_k |a_k b_k| of the
 *   dequantized operands) plus the BF16 rounding: gfx950's FP8 MFMA sums its
 *   products with limited width.  Requires M % 4 == 0, N % 256 == 0,
 *   K % 64 == 0, K > 0 when M * N > 0, K < 2^24, (K / 32) * max(M, N) < 2^32.
 */
int fp8_quant_mx_1x32(const float* x, int64_t R, int64_t K, uint8_t* q, uint8_t* e, void* stream);
int fp8_quant_mx_1x32_transposed(const float* x, int64_t M, int64_t K, uint8_t* q, uint8_t* e, void* stream);
int fp8_gemm_mx(const uint8_t* a, const uint8_t* ea, const uint8_t* b, const uint8_t* eb,
                void* c, int out_dtype, int64_t M, int64_t N, int64_t K, void* stream);

/*
 * The MX GEMM in the two MoE layouts ("Deepgemm lançado no dia 4 da semana de
 * código aberto Deepseek", section "Principais características": dense plus a
 * contiguous and a masked grouped layout), with fp8_gemm_mx's arithmetic and
 * accuracy contract for each expert's rows:
 *   b u8 [G][N][K] with eb u8 [G][K/32][N] (each expert's weight quantized by
 *   fp8_quant_mx_1x32).
 * fp8_grouped_gemm_contiguous_mx: a u8 [M_total][K] with ea u8 [K/32][M_total]
 *   (all rows quantized together), group_offsets as for
 *   fp8_grouped_gemm_contiguous (DEVICE int32 [G+1], non-decreasing, from 0 to
 *   M_total, multiples of 128); c [M_total][N].  Rows in no expert's range are
 *   not written.  Requires M_total % 128 == 0, N % 256 == 0, K % 64 == 0,
 *   K > 0 when there is work, K < 2^24, (K / 32) * max(M_total, N) < 2^32.
 * fp8_grouped_gemm_masked_mx: a u8 [G][M_max][K] with ea u8 [G][K/32][M_max],
 *   masked_m as for fp8_grouped_gemm_masked (DEVICE int32 [G], clamped to
 *   [0, M_max] on the device); c [G][M_max][N], rows at or beyond masked_m[g]
 *   NOT written.  Requires M_max % 4 == 0, N % 256 == 0, K % 64 == 0, K > 0
 *   when there is work, K < 2^24, (K / 32) * max(M_max, N) < 2^32.
 * Each expert's rows come out bit for bit as fp8_gemm_mx gives them for that
 * expert's operands.
 */
int fp8_grouped_gemm_contiguous_mx(const uint8_t* a, const uint8_t* ea, const uint8_t* b, const uint8_t* eb,
                                   const int32_t* group_offsets, int64_t G, int64_t M_total,
                                   int64_t N, int64_t K, void* c, int out_dtype, void* stream);
int fp8_grouped_gemm_masked_mx(const uint8_t* a, const uint8_t* ea, const uint8_t* b, const uint8_t* eb,
                               const int32_t* masked_m, int64_t G, int64_t M_max,
                               int64_t N, int64_t K, void* c, int out_dtype, void* stream);

/*
 * Dense block-scaled FP8 GEMM: C[M][N] = A[M][K] . B[N][K]^T.
 * a: u8 [M][K] with sa f32 [K/128][M] (1x128 along K).
 * b: u8 [N][K] with sb laid out per bscale_kind (fp8fg_bscale).
 * c: [M][N], BF16 (uint16 bit patterns) or FP32 per out_dtype (fp8fg_out).
 * Requires M >= 0 (any value, ragged tails allowed), N % 16 == 0,
 * K % 16 == 0 (a last partial K-block is allowed), K > 0 when M*N > 0;
 * M, N, K < 2^31.
 */
int fp8_gemm_blockscaled(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb,
                         int bscale_kind, void* c, int out_dtype,
                         int64_t M, int64_t N, int64_t K, void* stream);

/*
 * fp8_gemm_blockscaled on the FP8 matrix cores: the same arguments, layouts,
 * rules and errors, and the same per-K-block promotion with the scale
 * product applied at it ("The Insider Secrets Of Deepseek Discovered",
 * passage on Figure 7(b)), but each K-block's partial sum P_kb comes from
 * gfx950's FP8 MFMA (two 64-deep instructions per block) on the codes
 * themselves, at twice the rate of the BF16 matrix cores.  That instruction
 * adds its products in groups of eight consecutive K and keeps about 14
 * significant bits of each group (every product truncated toward zero to
 * 13 fractional bits below the group's largest exponent): the limited
 * accumulation the same passage measures on H800 Tensor Cores, here inside
 * one instruction, so promoting every 128 cannot remove it.
 * Accuracy contract: |C - C*| <= 2^-9 * S (FP32 out), plus one BF16
 * rounding of C* for BF16 out; the 2^-14 contract of every other call does
 * not hold here.  Deterministic.
 */
int fp8_gemm_blockscaled_fp8mfma(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb,
                                 int bscale_kind, void* c, int out_dtype,
                                 int64_t M, int64_t N, int64_t K, void* stream);

/*
 * Dense GEMM with the next layer's quantization fused into the epilogue
 * ("The Insider Secrets Of Deepseek Discovered", passage on Figure 6: with
 * every Linear in FP8, a layer's output is quantized again before it feeds
 * the next one).  Computes the FP32 C of fp8_gemm_blockscaled (128x128 B
 * scales) and writes, instead of C, its 1x128 quantization along N:
 *   q: u8 [M][N], s: f32 [N/128][M] -- exactly fp8_quant_act_1x128 applied to
 *   the FP32 C that out_dtype = FP8FG_OUT_FP32 would write (same values, bit
 *   for bit), i.e. the A operand layout of a following GEMM with K = N.
 * Requires N % 256 == 0, K % 16 == 0, K > 0 when M * N > 0, K <= 11776
 * (92 K-blocks: this kernel keeps one FP32 accumulator over all of K, about
 * eleven roundings per K-block, within the 2^-14 contract up to there; else
 * FP8FG_ERR_UNSUPPORTED), ceil(K/128) * M * 4 < 2^32.
 */
int fp8_gemm_blockscaled_fp8out(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb,
                                uint8_t* q, float* s, int64_t M, int64_t N, int64_t K, void* stream);

/*
 * MoE grouped GEMM, contiguous layout (training / prefill).
 * The rows of all G local experts are concatenated: expert g owns rows
 * [group_offsets[g], group_offsets[g+1]) of a / c.
 * group_offsets: DEVICE int32 [G+1], non-decreasing, group_offsets[0] = 0,
 *     group_offsets[G] = M_total, every entry a multiple of 128 (each expert's
 *     rows padded to whole 128-row tiles).  Read only on the device, so the
 *     host never waits for routing results.  A 128-row tile of a that lies
 *     outside [0, group_offsets[G]) is not computed and its rows of c are not
 *     written.  Padding rows are computed like any other row.
 * a: u8 [M_total][K], sa f32 [K/128][M_total];
 * b: u8 [G][N][K], sb f32 [G][N/128][K/128] (128x128 blocks per expert);
 * c: [M_total][N] BF16 or FP32.
 * Requires M_total % 128 == 0, N % 16 == 0, K % 16 == 0, K > 0, G >= 0.
 */
int fp8_grouped_gemm_contiguous(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb,
                                const int32_t* group_offsets, int64_t G, int64_t M_total,
                                int64_t N, int64_t K, void* c, int out_dtype, void* stream);

/*
 * fp8_grouped_gemm_contiguous with the next layer's quantization fused into
 * the epilogue ("The Insider Secrets Of Deepseek Discovered", passage on
 * Figure 6: with every Linear in FP8, a layer's output is quantized again
 * before it feeds the next one -- for a MoE layer, the gate+up output that
 * feeds the down projection).  Computes the FP32 C of
 * fp8_grouped_gemm_contiguous and writes, instead of C, its 1x128
 * quantization along N:
 *   q: u8 [M_total][N], s: f32 [N/128][M_total] -- exactly
 *   fp8_quant_act_1x128 applied to the FP32 C that out_dtype = FP8FG_OUT_FP32
 *   would write (same values, bit for bit); rows in no expert's range are not
 *   written (neither q nor s).
 * Same arguments and rules as fp8_grouped_gemm_contiguous, and in addition
 * N % 256 == 0, K <= 11776 (92 K-blocks, as for fp8_gemm_blockscaled_fp8out:
 * else FP8FG_ERR_UNSUPPORTED), ceil(K/128) * M_total * 4 < 2^32.
 */
int fp8_grouped_gemm_contiguous_fp8out(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb,
                                       const int32_t* group_offsets, int64_t G, int64_t M_total,
                                       int64_t N, int64_t K, uint8_t* q, float* s, void* stream);

/*
 * MoE grouped GEMM, masked layout (decode).
 * Expert g has a padded buffer of M_max rows of which the first masked_m[g]
 * are valid.
 * masked_m: DEVICE int32 [G]; each value is clamped to [0, M_max] on the
 *     device.  Rows at or beyond masked_m[g] of c are NOT written.
 * a: u8 [G][M_max][K], sa f32 [G][K/128][M_max];
 * b: u8 [G][N][K], sb f32 [G][N/128][K/128];
 * c: [G][M_max][N] BF16 or FP32.
 * Requires M_max >= 0, N % 16 == 0, K % 16 == 0, K > 0, G >= 0.
 */
int fp8_grouped_gemm_masked(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb,
                            const int32_t* masked_m, int64_t G, int64_t M_max,
                            int64_t N, int64_t K, void* c, int out_dtype, void* stream);

/*
 * Decode-tiled weight layout for the masked GEMM (this library's own format;
 * the pages define the masked layout's operation -- "Deepgemm lançado no dia 4
 * da semana de código aberto Deepseek", section "Principais características"
 * -- not a storage order).  Decode streams every expert's weights once per
 * step, so a storage order in which each step of the kernel reads one
 * contiguous block raises the HBM rate; weights are static, so the
 * rearrangement is made once, when they are loaded.
 * q: u8 [G][N][K] codes, as written by fp8_quant_weight_128x128 per expert.
 * q_tiled: u8, G*N*K bytes (caller-owned, must not overlap q).  Block
 *   blk = (g * N/256 + t) * (K/64) + h (16384 bytes at offset 16384 * blk)
 *   holds rows 256 t .. 256 t + 255 of expert g, K bytes 64 h .. 64 h + 63,
 *   as sixteen 1024-byte units u = 4 w + 2 n + j (w 0..3, n 0..1, j 0..1):
 *   bytes 16 l .. 16 l + 15 of unit u (l = 0..63) are K bytes
 *   64 h + 32 j + 16 (l / 32) .. + 15 of row 256 t + 64 w + 32 n + l % 32 --
 *   the 16-byte MFMA fragments of the decode kernel in the order its lanes
 *   load them.  A pure byte permutation; the scales are not touched (sb stays
 *   [G][N/128][K/128]).
 * Requires N % 256 == 0, K % 64 == 0, K < 2^24, G >= 0 (empty arrays may be
 * NULL).
 */
int fp8_tile_weights_decode(const uint8_t* q, int64_t G, int64_t N, int64_t K, uint8_t* q_tiled, void* stream);

/*
 * fp8_grouped_gemm_masked on decode-tiled weights: the same operation, the
 * same arguments and the same result bit for bit, except that b_tiled holds
 * the experts' codes in the layout written by fp8_tile_weights_decode.
 * Requires M_max <= 128, N % 256 == 0, K % 64 == 0, K > 0, K <= 11776 (92
 * K-blocks, as for fp8_gemm_blockscaled_fp8out), G >= 0, and
 * G * ceil(M_max / 64) <= 4096 (FP8FG_ERR_UNSUPPORTED beyond).
 */
int fp8_grouped_gemm_masked_tiled(const uint8_t* a, const float* sa, const uint8_t* b_tiled, const float* sb,
                                  const int32_t* masked_m, int64_t G, int64_t M_max,
                                  int64_t N, int64_t K, void* c, int out_dtype, void* stream);

/*
 * fp8_grouped_gemm_masked_mx on decode-tiled weights: the same operation,
 * arguments and result bit for bit (each expert's valid rows as
 * fp8_gemm_mx gives them), with the experts' codes in the layout written by
 * fp8_tile_weights_decode (which the scaled FP8 MFMA reads as it stands: a
 * lane's two 16-byte pieces of a 64-K step are one operand).
 * a u8 [G][M_max][K], ea u8 [G][K/32][M_max], b_tiled (decode-tiled [G][N][K]
 * codes), eb u8 [G][K/32][N], masked_m DEVICE int32 [G] (clamped to
 * [0, M_max]); c [G][M_max][N] BF16 or FP32, rows past masked_m[g] NOT
 * written.  Requires M_max <= 128, M_max % 4 == 0, N % 256 == 0, K % 64 == 0,
 * K > 0 when there is work, K < 2^24, (K / 32) * N < 2^32,
 * G * ceil(M_max / 64) <= 4096 (FP8FG_ERR_UNSUPPORTED beyond).
 */
int fp8_grouped_gemm_masked_tiled_mx(const uint8_t* a, const uint8_t* ea, const uint8_t* b_tiled, const uint8_t* eb,
                                     const int32_t* masked_m, int64_t G, int64_t M_max,
                                     int64_t N, int64_t K, void* c, int out_dtype, void* stream);

/*
 * fp8_grouped_gemm_masked_tiled with the next layer's quantization fused into
 * the epilogue ("The Insider Secrets Of Deepseek Discovered", passage on
 * Figure 6: every Linear runs in FP8, so a layer's output is quantized again
 * before the next GEMM reads it), the decode counterpart of
 * fp8_grouped_gemm_contiguous_fp8out.  Computes the FP32 C of
 * fp8_grouped_gemm_masked_tiled and writes, instead of C, its 1x128
 * quantization along N, in the masked A operand's own layout:
 *   q: u8 [G][M_max][N], s: f32 [G][N/128][M_max] -- for every valid row,
 *   exactly fp8_quant_act_1x128 applied to the FP32 C that out_dtype =
 *   FP8FG_OUT_FP32 would write (same values, bit for bit); rows at or beyond
 *   masked_m[g] are not written (neither q nor s).
 * Same arguments and rules as fp8_grouped_gemm_masked_tiled.
 */
int fp8_grouped_gemm_masked_tiled_fp8out(const uint8_t* a, const float* sa, const uint8_t* b_tiled, const float* sb,
                                         const int32_t* masked_m, int64_t G, int64_t M_max,
                                         int64_t N, int64_t K, uint8_t* q, float* s, void* stream);

/* ------------------------------------------------------------------------
 * The operators around the grouped GEMMs of a mixture-of-experts layer.
 *   forward:   moe_route -> fp8_moe_dispatch_contiguous (or _masked: decode)
 *              -> grouped GEMM (gate+up) -> fp8_swiglu -> grouped GEMM (down)
 *              -> moe_combine
 *   backward:  fp8_moe_combine_backward -> grouped GEMM (down, transposed
 *              weights) -> fp8_swiglu_backward -> grouped GEMM (gate+up,
 *              transposed weights) -> moe_combine without weights (the
 *              gradient of the tokens) and moe_route_backward; the weight
 *              gradients by fp8_grouped_gemm_wgrad.
 * All of them are deterministic: no atomics on results, sums in a fixed
 * order, FP32 throughout.  Type flags (x_bf16, ...) are 0 for f32, 1 for bf16
 * bit patterns (u16).
 * ------------------------------------------------------------------------ */

/*
 * Routing.  logits: [T][E], f32 or bf16, rows ld elements apart (ld >= E).
 *   s = sigmoid(x) or softmax(x) over the row (score: fp8fg_score),
 *   c = s + bias      (bias f32 [E], NULL for none: the correction that
 *                      balances the experts' load; it only steers the choice).
 * The E experts form n_groups equal groups of consecutive ones.  A group
 * scores the sum of its group_top (1 or 2) largest c; the topk_groups best
 * groups stay in (all of them when topk_groups = n_groups), and the topk
 * largest c among their experts are chosen, in decreasing order.  Equal
 * scores go to the lowest index, for groups and experts alike; scores are
 * compared in FP32, subnormals included.  An expert whose logit, or c, is -inf is
 * never chosen and adds nothing to its group's score; where fewer than topk experts can be
 * chosen the index is -1 and the weight 0 (a row of -inf, a padding token,
 * chooses nothing).  A NaN or +inf logit gives unspecified weights and an
 * unspecified choice, with every index still in [-1, E).
 *   idx: int32 [T][topk];  w: f32 [T][topk] = scale * s_idx, divided by the
 *   sum of the chosen s when renormalize = 1 (weights whose scores are all too
 *   small for FP32 keep their ratios).
 * Requires 1 <= topk <= 16, topk <= topk_groups * (E / n_groups),
 * E % n_groups == 0, 1 <= topk_groups <= n_groups <= 16, and
 * (E / n_groups) * P <= 1024, P the power of two from n_groups on.
 */
int moe_route(const void* logits, int logits_bf16, int64_t ld, const float* bias, int64_t T, int64_t E, int64_t topk,
              int64_t n_groups, int64_t topk_groups, int group_top, int score, int renormalize, float scale,
              int32_t* idx, float* w, void* stream);

/*
 * The gradient of the logits from dw (f32 [T][topk], the gradient of w), for
 * the choice idx (entries outside [0, E) contribute nothing; the choice itself
 * and the bias have no gradient).  With g_i = scale * dw_i, S the chosen
 * experts, p_i = s_i / sum_S s and d_i = sum_j (g_i - g_j) p_j:
 *   renormalize = 1: softmax dx_i = p_i d_i, sigmoid dx_i = p_i (1 - s_i) d_i
 *     for i in S, 0 elsewhere;
 *   renormalize = 0: sigmoid dx_i = g_i s_i (1 - s_i) for i in S, 0 elsewhere;
 *     softmax dx_e = s_e ((g_e if e in S) - sum_S g_j s_j) for every expert.
 * dlogits: [T][E] in the logits' type, rows E apart.  Requires E <= 1024,
 * 1 <= topk <= 16 and topk <= E.
 */
int moe_route_backward(const void* logits, int logits_bf16, int64_t ld, const int32_t* idx, const float* dw, int64_t T,
                       int64_t E, int64_t topk, int score, int renormalize, float scale, void* dlogits, void* stream);

/*
 * The tokens' rows in the contiguous layout, quantized.
 * x: [T][H], f32 or bf16;  idx: int32 [T][topk], experts of each token (as
 * moe_route gives them).  The local experts are first .. first + G - 1;
 * entries outside (experts elsewhere, -1) have no row.
 *   counts: int32 [G], entries per expert;
 *   group_offsets: int32 [G+1], the experts' first rows: every count rounded
 *     up to a multiple of 128 (as fp8_grouped_gemm_contiguous reads them; its
 *     last entry, at most M_total, is the number of rows in use);
 *   row_of: int32 [T][topk], the row of each entry, or -1.  An expert's rows
 *     are its entries in their order in idx.
 *   q: u8 [M_total][H], s: f32 [H/128][M_total]: row row_of[t][j] holds the
 *     1x128 quantization of x[t] (exactly fp8_quant_act_1x128's; each token
 *     is quantized once, whatever its number of rows).  Rows from an expert's
 *     count to the next offset are zero (codes and scales); rows from
 *     group_offsets[G] on are not written.
 * Requires H % 16 == 0, 1 <= topk <= 16, 1 <= G <= 256 (G = 0: a no-op, for any
 * M_total),
 * M_total % 128 == 0 and M_total >= the bound that holds any choice:
 * (n + 127 * min(G, n)) / 128 * 128 with n = T * topk; M_total < 2^31.
 * T = 0 writes the (zero) counts and offsets.
 */
int fp8_moe_dispatch_contiguous(const void* x, int x_bf16, int64_t T, int64_t H, const int32_t* idx, int64_t topk,
                                int64_t first, int64_t G, int64_t M_total, uint8_t* q, float* s, int32_t* row_of,
                                int32_t* group_offsets, int32_t* counts, void* stream);

/*
 * The same in the masked layout (decode): expert first + g owns rows
 * g * M_max .. of q u8 [G][M_max][H] and s f32 [G][H/128][M_max];
 * masked_m: int32 [G], its entries, at most M_max (as fp8_grouped_gemm_masked
 * reads them).  row_of holds g * M_max + r, r the entry's place among the
 * expert's; entries beyond M_max have no row (-1).  Rows at or beyond
 * masked_m[g] are not written.  Requires H % 16 == 0, 1 <= topk <= 16,
 * G <= 256 (G = 0: a no-op), M_max >= 1, G * M_max < 2^31.
 */
int fp8_moe_dispatch_masked(const void* x, int x_bf16, int64_t T, int64_t H, const int32_t* idx, int64_t topk,
                            int64_t first, int64_t G, int64_t M_max, uint8_t* q, float* s, int32_t* row_of,
                            int32_t* masked_m, void* stream);

/*
 * The experts' rows back to their tokens:
 *   out[t] = sum_j w[t][j] * y[row_of[t][j]]   over the entries that have a
 * row (row_of outside [0, R) has none; a token without rows gets 0), in the
 * order of j, FP32 sums.  y: [R][H] f32 or bf16 (R = M_total, or G * M_max of
 * the masked layout); w: f32 [T][topk], or NULL for weights of 1 (the
 * backward pass of the dispatch); out: [T][H] per out_dtype (fp8fg_out).
 * Requires H % 8 == 0, 1 <= topk <= 16.
 */
int moe_combine(const void* y, int y_bf16, int64_t R, int64_t H, const int32_t* row_of, const float* w, int64_t T,
                int64_t topk, void* out, int out_dtype, void* stream);

/*
 * The backward pass of moe_combine in the contiguous layout.
 * dout: [T][H], y: [R][H] (f32 or bf16 each); row_of, w, group_offsets,
 * counts as the forward pass had them.
 *   dw: f32 [T][topk] = <dout[t], y[row_of[t][j]]> (0 without a row);
 *   q: u8 [R][H], s: f32 [H/128][R]: the gradient w[t][j] * dout[t] of the
 *     rows as a grouped GEMM's A operand: row row_of[t][j] holds the 1x128 codes
 *     of dout[t] (sign-flipped where w < 0) with the scales RN32(|w| * scale),
 *     so a token is quantized once.  Padding rows are zero and rows from
 *     group_offsets[G] on are not written, as in the dispatch.
 * Requires H % 16 == 0, 1 <= topk <= 16, G <= 256.
 */
int fp8_moe_combine_backward(const void* dout, int dout_bf16, int64_t T, int64_t H, const void* y, int y_bf16,
                             int64_t R, const int32_t* row_of, const float* w, int64_t topk,
                             const int32_t* group_offsets, const int32_t* counts, int64_t G, uint8_t* q, float* s,
                             float* dw, void* stream);

/*
 * The gate between an expert's two products, with its 8-bit checkpoint.
 * gu: [G][M][2 I], f32 or bf16: gate g = columns [0, I), up u = [I, 2 I).
 *   q: u8 [G][M][I], s: f32 [G][I/128][M]: the 1x128 quantization of
 *     h = g * sigmoid(g) * u (FP32), the A operand of the second product;
 *   qc: u8 [G][M][2 I], sc: f32 [G][2 I/128][M]: the 1x128 quantization of gu
 *     itself (exactly fp8_quant_act_1x128's), the checkpoint that
 *     fp8_swiglu_backward starts from; both NULL to leave it out (inference).
 * rows: int32 [G] (4-byte aligned), or NULL for all rows: only rows
 * r < rows[g] of buffer g are read and written.  The contiguous layout is G = 1 with
 * rows = &group_offsets[G]; the masked one rows = masked_m.
 * A sigmoid(g) below FP32's smallest normal (g < -87.3) counts as 0.  Requires
 * I % 128 == 0, I <= 2^23, G <= 65535; h must be finite.
 */
int fp8_swiglu(const void* gu, int gu_bf16, int64_t G, int64_t M, int64_t I, const int32_t* rows, uint8_t* q, float* s,
               uint8_t* qc, float* sc, void* stream);

/*
 * Its backward pass from the checkpoint (qc u8 [M][2 I], sc f32 [2 I/128][M],
 * contiguous layout) and dh ([M][I], f32 or bf16).  With g, u the decoded
 * checkpoint and sg = sigmoid(g):
 *   du = dh * g * sg,  dg = dh * u * sg * (1 + g * (1 - sg)),  h = g * sg * u,
 * formed in FP32 (sg below FP32's smallest normal counts as 0) and quantized 1x128
 * once in each layout that the products read:
 *   q:  u8 [M][2 I],  s:  f32 [2 I/128][M]   (dg, du) along the channels
 *   qt: u8 [2 I][M],  st: f32 [M/128][2 I]   (dg, du) along the rows, transposed
 *   qh: u8 [I][M],    sh: f32 [M/128][I]     h along the rows, transposed
 * -- the A operand of the gate+up product's Dgrad, and the operands of
 * the gate+up and down products' weight gradients.
 * rows: int32 [1], or NULL: rows from rows[0] on count as zero; their rows of
 * q and s, and the 128-row groups of qt and qh that lie wholly past them, are
 * not written.  Requires I % 128 == 0, I <= 2^23, M % 16 == 0,
 * M <= 128 * 65535.
 */
int fp8_swiglu_backward(const uint8_t* qc, const float* sc, const void* dh, int dh_bf16, int64_t M, int64_t I,
                        const int32_t* rows, uint8_t* q, float* s, uint8_t* qt, float* st, uint8_t* qh, float* sh,
                        void* stream);

/*
 * The experts' weight gradients:
 *   c[g][M][N] (+)= sum over rows r of expert g of a[:, r] b[:, r]^T,
 * a: u8 [M][R], sa f32 [R/128][M];  b: u8 [N][R], sb f32 [R/128][N]: operands
 * quantized 1x128 along the rows, transposed (fp8_requant_act_tokenwise of a
 * checkpoint, fp8_swiglu_backward's qt and qh, fp8_quant_act_1x128 with
 * transpose_out = 1); R all experts' rows, M the output and N the input
 * channels of the weight.
 * group_offsets: DEVICE int32 [G+1] as for fp8_grouped_gemm_contiguous (entries
 * are clamped to [0, R] and rounded down to multiples of 128).  An expert
 * without rows gets zeros.  c: FP32 [G][M][N]; accumulate = 1 adds to it
 * (gradient accumulation) instead of writing it.  The accuracy contract and
 * engine are fp8_gemm_blockscaled's (2^-14 * S; in the worst case for experts of up
 * to 114688 rows, as for K there); each addition to c, one per 8192 rows at the most,
 * rounds once more, by up to 2^-24 of the sum there.
 * Requires R % 128 == 0, N % 16 == 0; M, N, R < 2^31.
 */
int fp8_grouped_gemm_wgrad(const uint8_t* a, const float* sa, const uint8_t* b, const float* sb,
                           const int32_t* group_offsets, int64_t G, int64_t M, int64_t N, int64_t R, float* c,
                           int accumulate, void* stream);

/* Human-readable name of a status code (static string, never NULL). */
const char* fp8fg_status_string(int status);

/* FP8FG_ABI_VERSION of the loaded library. */
int fp8fg_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FP8FG_H */
