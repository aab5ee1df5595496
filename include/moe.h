/*
 * libmoe -- routed-token scatter -> grouped GEMM MoE expert path for MI355X
 * (gfx950), as a C ABI.
 *
 * Sources ("the pages"): three sglang pull-request reports --
 *   [P1] "Support DeepGEMM for standard MoE dispatch" (PR #33128)
 *   [P2] "Add BF16 support to EP-MoE for DeepGEMM" (PR #17392)
 *   [P3] "[Feature] Support BF16 and batch-invariant inference with DeepEP v2"
 *        (PR #38160)
 *
 * General contract
 *   - Every pointer named "device" is a device pointer on the current HIP
 *     device; the caller owns all memory.  The library never allocates: scratch
 *     comes in through ws/ws_bytes (size from moe_scatter_ws_bytes); the one
 *     exception is moe_scatter_compact_noalloc, whose scratch is a static
 *     device array of fixed size.
 *   - Every compute call validates its arguments on the host first and returns
 *     a status without launching anything when they are wrong; otherwise it
 *     enqueues its kernels on `stream` (a hipStream_t; NULL = default stream)
 *     and returns without synchronising.  No call reads device data back to the
 *     host, so all sizes are fixed by the host arguments (static shapes, P1
 *     implementation breakdown item 2: buffers usable under graph capture).
 *   - Buffers may be uninitialised on entry (P1 implementation breakdown item 4):
 *     every valid row is written before it is read.  Rows marked -1 in
 *     m_indices, and masked rows at or past masked_m, hold unspecified values in
 *     every output.
 *   - Sizes and byte offsets are 64-bit inside the library.
 *   - bf16 tensors are raw 16-bit patterns; e4m3 is OCP float8 e4m3fn (bias 7,
 *     max 448); a UE8M0 scale byte s stands for 2^(s-127).
 *   - Activation scale layout ("K-block major"): compact rows use
 *     scale[b * M + r] for row r of M and 128-channel block b; masked rows use
 *     scale[(g * (K/128) + b) * max_m + r] for row r of group g.  Weight scales
 *     are [G][N/128][K/128].
 */
#ifndef LIBMOE_MOE_H
#define LIBMOE_MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* status codes */
#define MOE_OK 0
#define MOE_EINVAL 1          /* null pointer, negative or inconsistent size */
#define MOE_EUNSUPPORTED 2    /* dtype / alignment the kernels do not cover */
#define MOE_ECAPACITY 3       /* a static buffer is below the required bound */
#define MOE_EDEVICE 4         /* a HIP launch or copy failed */

/* element types */
#define MOE_DTYPE_BF16 0
#define MOE_DTYPE_FP8_E4M3_UE8M0 1
/* GEMM operand dtype: activations as MOE_DTYPE_FP8_E4M3_UE8M0, weights e4m3
 * with MX scales (one UE8M0 exponent per 32 k of a weight row) in the tiled
 * layout of moe_quant_weight_mx. */
#define MOE_DTYPE_FP8_E4M3_MXFP8 2
/* GEMM operand dtype: activations as MOE_DTYPE_FP8_E4M3_UE8M0, weights e2m1
 * [G][N][K/2] (moe_quant_weight_mx with MOE_MX_E2M1) with the same tiled MX
 * scales. */
#define MOE_DTYPE_FP8_MXFP4 3
/* fp32 tensors of the training calls (weight gradients, parameters). */
#define MOE_DTYPE_FP32 16

/* Activations of the products with an epilogue (moe_linear, grouped_gemm_*_act)
 * and of moe_act_bwd.  sigma(x) = 1 / (1 + e^-x), Phi the normal distribution.
 *   one for each column:
 *     MOE_ACT_NONE       x
 *     MOE_ACT_SILU       x sigma(x)
 *     MOE_ACT_GELU       x Phi(x)
 *     MOE_ACT_GELU_TANH  x (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))) / 2
 *     MOE_ACT_RELU2      max(x, 0)^2
 *   of the two halves of a row, gate g = columns [0, N/2) and up u = [N/2, N):
 *     MOE_ACT_SILU_MUL, MOE_ACT_GELU_MUL, MOE_ACT_GELU_TANH_MUL   act(g) u
 *     MOE_ACT_SWIGLU_CLAMP   g' sigma(alpha g') (u' + 1) with g' = min(g, limit) and
 *                            u' = u cut to [-limit, limit]; 1e-3 <= alpha <= 1e3,
 *                            limit > 0 (infinity: not cut).  The others ignore both.
 * All in fp32.  A NaN stays one; of -infinity, SILU and both GELUs give NaN. */
#define MOE_ACT_NONE 0
#define MOE_ACT_SILU 1
#define MOE_ACT_GELU 2
#define MOE_ACT_GELU_TANH 3
#define MOE_ACT_RELU2 4
#define MOE_ACT_SILU_MUL 9
#define MOE_ACT_GELU_MUL 10
#define MOE_ACT_GELU_TANH_MUL 11
#define MOE_ACT_SWIGLU_CLAMP 12

/* device error word bits (see moe_get_device_error) */
#define MOE_DEVERR_MASKED_OVERFLOW 1  /* an expert received more than max_m rows */

/* ---------------------------------------------------------------------------
 * Host helpers (no device work)
 * ------------------------------------------------------------------------- */

/* Static row bound of the compact layout, P1 key source excerpt of
 * _get_compact_all_tokens: block_e * (min(A, E) + (A - min(A, E)) / block_e)
 * with A = num_assignments and E = num_local_experts.  No routing of A
 * assignments over E experts can need more rows when every non-empty expert is
 * padded to a multiple of block_e.  Returns -1 for negative or zero sizes. */
int64_t moe_compact_rows_bound(int64_t num_assignments, int32_t num_local_experts,
                               int32_t block_e);

/* Layout rule, P1 key source excerpt of _should_use_masked_standard_layout:
 * 1 (masked) when num_experts > num_local_experts and num_local_experts <= 32,
 * else 0 (compact). */
int32_t moe_use_masked_layout(int32_t num_experts, int32_t num_local_experts);

/* Layout policy measured on MI355X in place of the rule above, which the pages
 * leave open ("Support DeepGEMM for standard MoE dispatch", comments section:
 * compact slower than masked up to a crossover in token count).  Timing the
 * whole path in both layouts over 16 .. 16384 tokens (DeepSeek-V3 with 256 and
 * 32 local experts, BF16 with 128 and 8) put the masked layout ahead while the
 * experts hold few rows (up to about 64 per expert on average) and the
 * compact layout level or ahead beyond, while the masked buffers grow as
 * num_local_experts * max_tokens rows.  Returns 1 (masked) when
 *   max_tokens * top_k <= 64 * num_experts            (mean rows per expert)
 *   and num_local_experts * max_tokens <= 4 * moe_compact_rows_bound(
 *       max_tokens * top_k, num_local_experts, block_e)   (memory cap),
 * else 0 (compact); -1 for a zero or negative argument, more local experts
 * than experts, or top_k above num_experts. */
int32_t moe_choose_layout(int64_t max_tokens, int32_t top_k, int32_t num_experts,
                          int32_t num_local_experts, int32_t block_e);

/* Scratch bytes moe_scatter_compact / moe_scatter_masked need for T tokens,
 * top-k, num_local_experts local experts and H hidden channels (per-chunk
 * expert counts, per-expert starts and totals, the assignment of each valid
 * row, and FP8 scale bytes staged per token).  0 on a negative size. */
size_t moe_scatter_ws_bytes(int32_t T, int32_t k, int32_t num_local_experts, int32_t H);

/* Static text for a status code. */
const char* moe_status_str(int32_t status);

/* Copies the device error word kept at the start of a scatter workspace to
 * *host_err after waiting for `stream`; 0 means no data-dependent error was
 * seen by the last scatter call that used this workspace.  Synchronises: this
 * is the one call that blocks the host (it waits for `stream` itself), unlike
 * the enqueue-only contract of every other call, where synchronising is left
 * to the caller. */
int32_t moe_get_device_error(const void* ws, int32_t* host_err, void* stream);

/* ---------------------------------------------------------------------------
 * Routing
 * ------------------------------------------------------------------------- */

/* Top-k routing: softmax over E experts, the k most probable kept and their
 * probabilities renormalised to sum to 1 (the router output the pages feed
 * into dispatch as topk_output; P3 related-PR note keeps the router in fp32).
 *   logits        device fp32 [T][E]
 *   topk_ids      device int32 [T][k], out: slot j holds the j-th most
 *                 probable expert; equal logits go to the lower index.
 *   topk_weights  device fp32 [T][k], out.
 * Limits: 1 <= E <= 1024, 1 <= k <= min(E, 32), T >= 0. */
int32_t moe_route_topk(const float* logits, int32_t T, int32_t E, int32_t k,
                       int32_t* topk_ids, float* topk_weights, void* stream);

/* ---------------------------------------------------------------------------
 * Scatter into the expert layouts
 * ------------------------------------------------------------------------- */

/* Compact ("contiguous") layout, P1 implementation breakdown items 2-4 and the
 * key source excerpt of _fwd_kernel_ep_scatter_1.  Assignment (t, j) is local
 * when e = topk_ids[t][j] - expert_start lies in [0, num_local_experts)
 * (P3 implementation breakdown item 1).  Local rows are grouped by expert e in
 * increasing e; inside an expert they follow increasing (t, j).  Each
 * non-empty expert is padded to a multiple of block_e rows.
 *   x                 device bf16 [T][H]
 *   rows_capacity     rows of every per-row output; must be at least
 *                     moe_compact_rows_bound(T*k, num_local_experts, block_e)
 *                     (else MOE_ECAPACITY)
 *   out_dtype         MOE_DTYPE_BF16: x_out bf16 [rows_capacity][H] copies;
 *                     MOE_DTYPE_FP8_E4M3_UE8M0: x_out e4m3 [rows_capacity][H]
 *                     with scale_out [H/128][rows_capacity] (the token's own
 *                     per-128-channel UE8M0 quantisation, see
 *                     moe_quant_fp8_ue8m0)
 *   m_indices         device int32 [rows_capacity], out: e on valid rows, -1 on
 *                     padding rows and on every row past the last expert block
 *   expert_start_loc  device int32 [num_local_experts], out: first row of e
 *   num_valid         device int32 [num_local_experts], out: rows of e
 *   src2dst           device int32 [T][k], out: row of (t, j), -1 if not local
 *   ws, ws_bytes      scratch, at least moe_scatter_ws_bytes(T, k, El, H)
 * Limits: H % 128 == 0, block_e a positive multiple of 128 (the grouped GEMM
 * tiles never straddle experts), 1 <= num_local_experts <= 1024,
 * rows_capacity < 2^31. */
int32_t moe_scatter_compact(const void* x, int32_t T, int32_t H, const int32_t* topk_ids,
                            int32_t k, int32_t expert_start, int32_t num_local_experts,
                            int32_t block_e, int64_t rows_capacity, int32_t out_dtype,
                            void* x_out, uint8_t* scale_out, int32_t* m_indices,
                            int32_t* expert_start_loc, int32_t* num_valid, int32_t* src2dst,
                            void* ws, size_t ws_bytes, void* stream);

/* Largest scratch (bytes, as moe_scatter_ws_bytes counts it) that
 * moe_scatter_compact_noalloc serves: 4 MiB, e.g. T = 32768 tokens, top-8,
 * H = 7168 with 256 local experts (about 3.75 MiB). */
#define MOE_SCATTER_NOALLOC_MAX_BYTES (4u << 20)

/* moe_scatter_compact without the ws/ws_bytes arguments, for callers that
 * cannot allocate device memory (code under HIP graph capture, tight serving
 * loops, harnesses that forbid hipMalloc).  Same arguments, outputs, limits
 * and status codes as moe_scatter_compact; the scratch is a static device
 * array of MOE_SCATTER_NOALLOC_MAX_BYTES per device, held until the process
 * ends.  The call allocates nothing.
 *   Returns MOE_ECAPACITY when moe_scatter_ws_bytes(T, k, num_local_experts, H)
 *   exceeds MOE_SCATTER_NOALLOC_MAX_BYTES, and MOE_EDEVICE when the scratch's
 *   device address cannot be obtained.
 * Every call on one device shares that device's scratch: calls that may run
 * at the same time on one device (different streams without ordering, other
 * threads) race and give undefined results; calls in one stream are fine.
 * The compact scatter sets no device error bits, so there is no error word to
 * read back. */
int32_t moe_scatter_compact_noalloc(const void* x, int32_t T, int32_t H, const int32_t* topk_ids,
                                    int32_t k, int32_t expert_start, int32_t num_local_experts,
                                    int32_t block_e, int64_t rows_capacity, int32_t out_dtype,
                                    void* x_out, uint8_t* scale_out, int32_t* m_indices,
                                    int32_t* expert_start_loc, int32_t* num_valid,
                                    int32_t* src2dst, void* stream);

/* Masked layout, P1 implementation breakdown item 2 (masked branch) and P2 key
 * source excerpt of _BF16GroupedMaskedWarmupExecutor: expert e's rows are
 * x_out[e][0 .. masked_m[e]) in increasing (t, j); src2dst holds the flat row
 * e*max_m + rank so moe_combine serves both layouts.
 *   x_out      [num_local_experts][max_m][H] bf16 or e4m3
 *   scale_out  FP8 only: [num_local_experts][H/128][max_m]
 *   masked_m   device int32 [num_local_experts], out
 * max_m must be >= T (a token contributes at most one row per expert when its
 * k ids are distinct), else MOE_ECAPACITY.  Repeated ids inside one token that
 * push an expert past max_m set MOE_DEVERR_MASKED_OVERFLOW in the device error
 * word; the overflowing rows are dropped (src2dst = -1) and masked_m is
 * clamped to max_m. */
int32_t moe_scatter_masked(const void* x, int32_t T, int32_t H, const int32_t* topk_ids,
                           int32_t k, int32_t expert_start, int32_t num_local_experts,
                           int32_t max_m, int32_t out_dtype, void* x_out, uint8_t* scale_out,
                           int32_t* masked_m, int32_t* src2dst, void* ws, size_t ws_bytes,
                           void* stream);

/* ---------------------------------------------------------------------------
 * Quantisation
 * ------------------------------------------------------------------------- */

/* Per-token, per-128-channel FP8 e4m3 with UE8M0 scales computed directly
 * (P1 implementation breakdown item 3; P3 key source excerpt of the dispatch
 * path calling per-token-group quantisation with ue8m0): for each group the
 * exponent e is the smallest integer in [-126, 127] with amax <= 448 * 2^e, then
 * each value is x * 2^-e rounded to nearest-even e4m3.
 *   x          device bf16, row r at x + r*ld_x (elements)
 *   m_indices  optional device int32 [M]; rows with a negative entry are skipped
 *   q          device e4m3 [M][K]
 *   scale      device u8 [K/128][M]
 * Limits: K % 128 == 0, ld_x >= K. */
int32_t moe_quant_fp8_ue8m0(const void* x, int64_t M, int32_t K, int64_t ld_x,
                            const int32_t* m_indices, uint8_t* q, uint8_t* scale,
                            void* stream);

/* Expert weights to 128x128 block-scaled e4m3 with UE8M0 block scales (the same
 * rule over each block; P1 implementation breakdown item 1 expresses both w13
 * and w2 with power-of-two block scales).
 *   w      device bf16 [G][N][K];  q  device e4m3 [G][N][K]
 *   scale  device u8 [G][N/128][K/128]
 * Limits: N % 128 == 0, K % 128 == 0. */
int32_t moe_quant_weight_fp8_ue8m0(const void* w, int32_t G, int32_t N, int32_t K,
                                   uint8_t* q, uint8_t* scale, void* stream);

/* MX expert weights (OCP microscaling: every 32 consecutive k of a weight row
 * share one power-of-two scale), the weight format the pages flag as not yet
 * covered ("Support DeepGEMM for standard MoE dispatch", comments section on
 * FP4 and MX weights).  The exponent follows the pages' direct UE8M0 rule
 * (implementation breakdown item 3) over each 32-value block: the smallest e in
 * [-126, 127] with max|w| <= fmax * 2^e, fmax = 448 (e4m3) or 6 (e2m1); each
 * value w * 2^-e is then rounded to nearest, ties to even.
 *   w            device bf16 [G][N][K]
 *   fmt          MOE_MX_E4M3: q e4m3 [G][N][K];
 *                MOE_MX_E2M1: q e2m1 [G][N][K/2], two codes per byte, even k in
 *                the low nibble (OCP FP4: sign, 2 exponent bits with bias 1,
 *                1 mantissa bit)
 *   scale_tiled  device u8 exponents + 127, tiled for the GEMM:
 *                [G][N/64][K/128][4][16][4], the byte of (row n, 32-block b) at
 *                ((g*(N/64) + n/64)*(K/128) + b/4)*256 + (b%4)*64 + (n%16)*4 + (n%64)/16
 * Limits: N % 64 == 0, K % 128 == 0.  Non-finite weights: unspecified codes. */
#define MOE_MX_E4M3 0
#define MOE_MX_E2M1 1
int32_t moe_quant_weight_mx(const void* w, int32_t G, int32_t N, int32_t K, int32_t fmt,
                            uint8_t* q, uint8_t* scale_tiled, void* stream);
/* Plain MX scales [G][N][K/32] (one byte per row and 32-block, as a checkpoint
 * stores them) -> the tiled layout above. */
int32_t moe_mx_scales_tile(const uint8_t* scale_plain, int32_t G, int32_t N, int32_t K,
                           uint8_t* scale_tiled, void* stream);

/* Requantise block-FP8 expert weights (a checkpoint's e4m3 codes with one
 * fp32 scale per 128x128 block) to the UE8M0 block format, through a bf16
 * intermediate ("Support DeepGEMM for standard MoE dispatch", implementation
 * breakdown item 1: both w13 and w2 of the standard layer are requantised with
 * bf16 as the output dtype): w = bf16(decode(q) * s) in fp32, then exactly
 * moe_quant_weight_fp8_ue8m0 of w.
 *   q_in   device e4m3 [G][N][K];  s_in  device fp32 [G][N/128][K/128]
 *   q_out  device e4m3 [G][N][K] (may be q_in);  s_out  device u8 [G][N/128][K/128]
 *   Non-finite codes or products give unspecified results.
 * Limits: N % 128 == 0, K % 128 == 0. */
int32_t moe_requant_weight_fp8_ue8m0(const uint8_t* q_in, const float* s_in, int32_t G, int32_t N,
                                     int32_t K, uint8_t* q_out, uint8_t* s_out, void* stream);

/* Rows on which a grouped GEMM call runs its MFMAs (whole 16-row blocks of
 * its tiles, padding included), for throughput accounting: the tile choice of
 * grouped_gemm_masked(_silu) with this expected_m (masked != 0), or of
 * grouped_gemm_contig(_silu) on a layout with M rows in which each of the G
 * experts is one run of counts[g] valid rows (what moe_scatter_compact
 * writes).  counts: host int32 [G].  N is the GEMM's output width (2I for
 * the SiLU variants).  Returns -1 on a null pointer or negative size. */
int64_t grouped_gemm_rows_executed(int32_t dtype, int32_t masked, const int32_t* counts, int32_t G,
                                   int32_t expected_m, int64_t M, int32_t N, int32_t K);

/* ---------------------------------------------------------------------------
 * Grouped GEMMs ("NT": C = A . B[g]^T), fp32 accumulation, bf16 output
 * ------------------------------------------------------------------------- */

/* Contiguous layout, P2 key source excerpts of _BF16GroupedContWarmupExecutor
 * and _run_bf16_contiguous_gemm: C[r, :] = A[r, :] . B[m_indices[r]]^T.
 *   dtype     MOE_DTYPE_BF16 (A bf16 [M][K], B bf16 [G][N][K]; scales NULL),
 *             MOE_DTYPE_FP8_E4M3_UE8M0 (A e4m3 [M][K] with A_scale [K/128][M],
 *             B e4m3 [G][N][K] with B_scale [G][N/128][K/128]) or
 *             MOE_DTYPE_FP8_E4M3_MXFP8 (A as before, B e4m3 [G][N][K] with MX
 *             B_scale tiled as moe_quant_weight_mx writes it) or
 *             MOE_DTYPE_FP8_MXFP4 (A as before, B e2m1 [G][N][K/2], MX scales)
 *   C         device bf16 [M][N].  Rows of an aligned 128-row block whose
 *             first row is -1 are not written; other rows with m_indices < 0
 *             (the padding at the end of an expert) receive unspecified values.
 *   m_indices device int32 [M]; layout contract: every aligned 128-row block
 *             holds one expert id on its valid rows, valid rows come first
 *             (what moe_scatter_compact produces with block_e % 128 == 0)
 * Limits: N % 128 == 0, K % 128 == 0, K <= 4194304, 0 <= m_indices < G,
 * ceil(M / 128) <= 8176 (about one million rows) -> else MOE_EUNSUPPORTED.
 * FP8 without scales -> MOE_EUNSUPPORTED (the dtype follows the weights and a
 * contradiction is an error, P3 implementation breakdown item 2). */
int32_t grouped_gemm_contig(int32_t dtype, const void* A, const uint8_t* A_scale,
                            const void* B, const uint8_t* B_scale, void* C,
                            const int32_t* m_indices, int64_t M, int32_t N, int32_t K,
                            int32_t G, void* stream);

/* Masked layout, P2 key source excerpt of _BF16GroupedMaskedWarmupExecutor:
 * C[g, r, :] = A[g, r, :] . B[g]^T for r < masked_m[g].
 *   A [G][max_m][K], C [G][max_m][N]; FP8 A_scale [G][K/128][max_m].
 *   expected_m  a hint of typical masked_m (sizes tiles: 16 or 32 rows when
 *               1 <= expected_m <= 16 or <= 32 and N % 256 == 0, 64 rows when
 *               1 <= expected_m <= 64, else 128); it never changes a result.
 *               0 = no hint.
 *   Rows at or past masked_m[g] receive unspecified values, except that rows
 *   at or past masked_m[g] rounded up to 128 are never written.
 * Limits: N, K as grouped_gemm_contig; G <= 1024; the tile count, at most
 * G * ceil(max_m / 64) * N / 128, below 2^31 -> else MOE_EUNSUPPORTED. */
int32_t grouped_gemm_masked(int32_t dtype, const void* A, const uint8_t* A_scale,
                            const void* B, const uint8_t* B_scale, void* C,
                            const int32_t* masked_m, int32_t expected_m, int32_t max_m,
                            int32_t N, int32_t K, int32_t G, void* stream);

/* The w13 GEMM with SiLU-and-mul in its epilogue (the two steps of P2 key
 * source excerpt _run_bf16_contiguous_gemm, w13 then silu_and_mul, in one
 * pass): B is w13 [G][2I][K] (gate rows [0, I), up rows [I, 2I)) and the
 * result is the activation act[r][i] = silu(C[r][i]) * C[r][I + i] with
 * C = A . B[g]^T rounded to bf16 first, exactly as grouped_gemm_* followed by
 * silu_and_mul computes it (bit for bit).
 *   out_dtype  MOE_DTYPE_BF16: out bf16 [rows][I];
 *              MOE_DTYPE_FP8_E4M3_UE8M0: out e4m3 [rows][I] with out_scale
 *              laid out as silu_and_mul's (compact [I/128][M], masked
 *              [G][I/128][max_m]).
 *   Rows follow the underlying GEMM: rows of blocks whose first row is -1
 *   (compact) or at or past masked_m rounded up to 128 (masked) are not
 *   written; other rows past an expert's valid rows receive unspecified values.
 * Limits: I % 128 == 0, (I + 256) * K * 2 < 2^32; the rest as the underlying
 * GEMM. */
int32_t grouped_gemm_contig_silu(int32_t dtype, const void* A, const uint8_t* A_scale,
                                 const void* B, const uint8_t* B_scale, int32_t out_dtype,
                                 void* out, uint8_t* out_scale, const int32_t* m_indices,
                                 int64_t M, int32_t I, int32_t K, int32_t G, void* stream);
int32_t grouped_gemm_masked_silu(int32_t dtype, const void* A, const uint8_t* A_scale,
                                 const void* B, const uint8_t* B_scale, int32_t out_dtype,
                                 void* out, uint8_t* out_scale, const int32_t* masked_m,
                                 int32_t expected_m, int32_t max_m, int32_t I, int32_t K,
                                 int32_t G, void* stream);

/* ---------------------------------------------------------------------------
 * Activation and combine
 * ------------------------------------------------------------------------- */

/* SiLU-and-mul, P2 key source excerpt of _run_bf16_contiguous_gemm (the w13
 * output [M][2I] is halved): out[r][i] = silu(gateup[r][i]) * gateup[r][I+i],
 * computed in fp32 (silu(g) = g * 1/(1 + 2^(-g log2 e)) with the hardware
 * exp2 and reciprocal, each within about one fp32 ulp) and rounded to bf16;
 * for FP8 output that bf16 row is then quantised as moe_quant_fp8_ue8m0 does.
 *   Row selection: m_indices (compact; rows with -1 skipped) or masked_m with
 *   max_m (masked; M = G*max_m, rows r % max_m >= masked_m[r / max_m] skipped);
 *   both NULL = every row.
 *   out_scale  FP8 only: compact [I/128][M], masked [G][I/128][max_m].
 * Limits: I % 128 == 0. */
int32_t silu_and_mul(const void* gateup, int64_t M, int32_t I, const int32_t* m_indices,
                     const int32_t* masked_m, int32_t max_m, int32_t out_dtype, void* out,
                     uint8_t* out_scale, void* stream);

/* Weighted combine back to token order (P1 risks item 2: the post-permute
 * reads src2dst; P3 review notes: combine follows per-slot pointers):
 * out[t][h] = sum over j = 0..k-1 with src2dst[t][j] >= 0 of
 * topk_weights[t][j] * Y[src2dst[t][j]][h], each product and partial sum
 * rounded to fp32 in slot order, then one rounding to bf16; tokens with no
 * local slot get 0.
 *   Y bf16 [num_rows][H]; out bf16 [T][H].  A src2dst entry >= num_rows is
 *   treated as -1 (never read).  Limits: H % 8 == 0, 1 <= k <= 32. */
int32_t moe_combine(const void* Y, int64_t num_rows, const int32_t* src2dst,
                    const float* topk_weights, int32_t T, int32_t k, int32_t H, void* out,
                    void* stream);

/* ---------------------------------------------------------------------------
 * Products with an epilogue.  The product is summed in fp32 over ascending k (with
 * quantised weights the products of 128 of k by the matrix core, to about 2^-15 of the
 * largest, and these sums in fp32), and bias, activation and residual follow in fp32
 * before the one rounding to the output's type.  A row's result depends on its own row
 * and its weights alone: it is the same for any number of rows, and in both layouts.
 * ------------------------------------------------------------------------- */

/* Dense product: with p[m][n] = sum over k of A[m][k] * B[n][k] + bias[n],
 *   out[m][:] = act(p[m][:]) + residual[m][:]
 * (the router's logits; a shared expert, whose second product takes what the
 * routed experts gave as its residual).
 *   A            device bf16, row m at A + m*lda (elements)
 *   B            device bf16 [N][K]
 *   bias         device bf16 or fp32 [N] (bias_dtype MOE_DTYPE_BF16 or
 *                MOE_DTYPE_FP32), or NULL
 *   act, alpha, limit   see MOE_ACT_*; the output has N columns, N/2 with a gated one
 *   residual     device, of out's type, row m at residual + m*ld_residual, or NULL.
 *                May be out itself with ld_out, not otherwise overlap it, and holds no
 *                element of pre
 *   out          device, out_dtype MOE_DTYPE_BF16 or MOE_DTYPE_FP32, row m at
 *                out + m*ld_out
 *   pre          device bf16 [M][N], out: p for moe_act_bwd, or NULL
 * out and pre hold no element of A, B, bias or each other.
 * Limits: K % 8 == 0, lda % 8 == 0 and >= K, A and B 16-byte aligned, ld_out and
 * ld_residual at least the output's columns, N even with a gated activation, and then
 * (N/2 + 256) * K * 2 < 2^32; lda < 2^22, M < 2^31, ceil(M / 128) * ceil(N / 128) < 2^24. */
int32_t moe_linear(const void* A, int64_t lda, const void* B, const void* bias, int32_t bias_dtype,
                   int32_t act, float alpha, float limit, const void* residual, int64_t ld_residual,
                   int32_t out_dtype, void* out, int64_t ld_out, void* pre, int64_t M, int32_t N,
                   int32_t K, void* stream);

/* grouped_gemm_contig with each expert's bias and an activation: for row r of
 * expert g = m_indices[r], p[r][:] = A[r, :] . B[g]^T + bias[g][:],
 *   out[r][:] = act(p[r][:]).
 *   dtype, A, A_scale, B, B_scale, m_indices   as grouped_gemm_contig
 *   bias         device bf16 or fp32 [G][N] (bias_dtype), or NULL
 *   out          out_dtype MOE_DTYPE_BF16: bf16 [M][N], [M][N/2] with a gated
 *                activation; gated also MOE_DTYPE_FP8_E4M3_UE8M0: e4m3 [M][N/2] with
 *                out_scale [N/256][M], quantised from the fp32 values
 *   pre          dtype MOE_DTYPE_BF16 only: device bf16 [M][N], out: p for
 *                moe_act_bwd, or NULL
 * Rows with m_indices < 0 are left as they were in every output.
 * Limits as grouped_gemm_contig; N % 256 == 0 with a gated activation, and then
 * (N/2 + 256) * K * 2 < 2^32; pointers of tensors 16-byte aligned. */
int32_t grouped_gemm_contig_act(int32_t dtype, const void* A, const uint8_t* A_scale, const void* B,
                                const uint8_t* B_scale, const void* bias, int32_t bias_dtype,
                                int32_t act, float alpha, float limit, int32_t out_dtype, void* out,
                                uint8_t* out_scale, void* pre, const int32_t* m_indices, int64_t M,
                                int32_t N, int32_t K, int32_t G, void* stream);

/* The same for the masked layout: rows r < masked_m[g] of group g.
 *   out [G][max_m][N or N/2]; out_scale [G][N/256][max_m]; pre [G][max_m][N];
 *   expected_m   as grouped_gemm_masked
 * Rows at or past masked_m[g] are left as they were in every output. */
int32_t grouped_gemm_masked_act(int32_t dtype, const void* A, const uint8_t* A_scale, const void* B,
                                const uint8_t* B_scale, const void* bias, int32_t bias_dtype,
                                int32_t act, float alpha, float limit, int32_t out_dtype, void* out,
                                uint8_t* out_scale, void* pre, const int32_t* masked_m,
                                int32_t expected_m, int32_t max_m, int32_t N, int32_t K, int32_t G,
                                void* stream);

/* ---------------------------------------------------------------------------
 * Training: gradients of the calls above and the AdamW step.  All BF16 (weights
 * held in FP8 or MX formats have no gradient here).  Device pointers of tensors
 * must be 16-byte aligned -> else MOE_EUNSUPPORTED.  Every gradient is the same
 * from run to run: no sum depends on the order in which workgroups finish.
 * ------------------------------------------------------------------------- */

/* Gradient of moe_combine.  For every slot with r = src2dst[t][j] in
 * [0, num_rows):
 *   dY[r][h] = topk_weights[t][j] * dout[t][h]            (rounded to bf16)
 *   dtopk_weights[t][j] = sum over h of dout[t][h] * Y[r][h]  (fp32)
 * and dtopk_weights[t][j] = 0 for the other slots.  Serves both layouts.
 *   dout bf16 [T][H]; Y, dY bf16 [num_rows][H]; src2dst int32 [T][k];
 *   topk_weights, dtopk_weights fp32 [T][k].
 *   Rows of dY that no slot names (padding) are left as they were.  The rows
 *   named must be distinct (as the scatter leaves them); a row named twice gets
 *   one of its two values.  dY must not overlap the inputs.
 * Limits: H % 8 == 0, H <= 2^30, 1 <= k <= 32, T times the lesser of H / 8 (rounded
 * up to 64) and 1024 below 2^32. */
int32_t moe_combine_bwd(const void* dout, const void* Y, int64_t num_rows, const int32_t* src2dst,
                        const float* topk_weights, int32_t T, int32_t k, int32_t H, void* dY,
                        float* dtopk_weights, void* stream);

/* Gradient of moe_route_topk: the weights are the softmax of the kept logits, so
 *   dlogits[t][topk_ids[t][j]] = w_j * (dw_j - sum over i of w_i * dw_i)
 * with w = topk_weights[t], dw = dtopk_weights[t], and 0 for every other expert
 * (all fp32; an id named twice gets the sum of its terms, ids outside [0, E)
 * are skipped).  Linear in dw: where the experts are shared out, the shares'
 * results add up to the whole gradient.
 *   dlogits fp32 [T][E].  Limits as moe_route_topk, T < 2^26. */
int32_t moe_route_topk_bwd(const int32_t* topk_ids, const float* topk_weights,
                           const float* dtopk_weights, int32_t T, int32_t E, int32_t k,
                           float* dlogits, void* stream);

/* Gradient of the scatter: dx[t][h] = sum over j with src2dst[t][j] in
 * [0, num_rows) of dX[src2dst[t][j]][h], added in fp32 in slot order and
 * rounded once to bf16; 0 for a token without such a slot.  Serves both layouts.
 *   dX bf16 [num_rows][H]; dx bf16 [T][H].
 * Limits as moe_combine_bwd. */
int32_t moe_scatter_bwd(const void* dX, int64_t num_rows, const int32_t* src2dst, int32_t T,
                        int32_t k, int32_t H, void* dx, void* stream);

/* Gradient of silu_and_mul (bf16 output).  With g, u the halves of a row and
 * s = 1 / (1 + e^-g), in fp32:
 *   dgateup[r][i] = dact * u * s * (1 + g * (1 - s)),  dgateup[r][I+i] = dact * g * s,
 *   act[r][i] = silu(g) * u  (only if act is not NULL: the forward's activation
 *   again, bit for bit),
 * each rounded once to bf16.  Rows are chosen as in silu_and_mul; skipped rows
 * are left as they were.
 *   gateup, dgateup bf16 [M][2I] (may be one buffer); dact, act bf16 [M][I].
 * Limits: I % 128 == 0, I <= 67107840, M < 2^26 - 3. */
int32_t silu_and_mul_bwd(const void* gateup, const void* dact, int64_t M, int32_t I,
                         const int32_t* m_indices, const int32_t* masked_m, int32_t max_m,
                         void* dgateup, void* act, void* stream);

/* Scratch bytes moe_act_bwd needs for dbias (G = 1 without a layout): sums of
 * blocks of rows.  0 where it needs none (few rows), and on a negative or zero size. */
size_t moe_act_bwd_ws_bytes(int64_t M, int32_t N, int32_t G);

/* Gradient of the epilogue of moe_linear and grouped_gemm_*_act (the residual's
 * gradient is dout itself).  With p = pre[r],
 *   dpre[r][:] = dout[r][:] * act'(p)          rounded once to bf16
 *   dbias[g][n] = sum over g's rows of dpre[r][n] as it was before that rounding
 *                 (fp32), added to what dbias holds if accumulate is not 0, and
 *                 rounded once to its type
 * At a gate or up part that equals its limit the cut passes the gradient on, past
 * it the part's gradient is 0.
 * act' of a NaN is a NaN; at the infinities it is its limit (0 below, 1 above, where
 * RELU2's is infinite).
 *   Rows: m_indices (compact), masked_m with max_m (masked; M = G*max_m) or, both
 *   NULL, every row (then G = 1).  Other rows of dpre are left as they were and are
 *   part of no sum.
 *   pre, dpre    bf16 [M][N]; dpre may be pre, and may be a bf16 dout where the
 *                activation is not gated.  With MOE_ACT_NONE pre is not read, and dpre may be
 *                NULL: the bias gradient alone.  dpre and dbias share memory with
 *                nothing else
 *   dout         dout_dtype MOE_DTYPE_BF16 or MOE_DTYPE_FP32 (as the output was): [M][N],
 *                [M][N/2] with a gated activation
 *   expert_start_loc, num_valid   device int32 [G] as moe_scatter_compact writes them,
 *                needed with m_indices and dbias
 *   dbias        dbias_dtype MOE_DTYPE_BF16 or MOE_DTYPE_FP32 [G][N], or NULL.  An
 *                expert without rows gets 0 (or keeps what it holds)
 *   ws, ws_bytes scratch for dbias, at least moe_act_bwd_ws_bytes(M, N, G); calls that
 *                may run at the same time need one each
 * Limits: N % 8 == 0 (16 with a gated activation), N <= 2^27, M < 2^26, G <= 65535;
 * pointers of tensors 16-byte aligned. */
int32_t moe_act_bwd(const void* pre, int32_t dout_dtype, const void* dout, int64_t M, int32_t N,
                    int32_t act, float alpha, float limit, const int32_t* m_indices, const int32_t* masked_m,
                    int32_t max_m, const int32_t* expert_start_loc, const int32_t* num_valid,
                    int32_t G, void* dpre, int32_t dbias_dtype, int32_t accumulate, void* dbias,
                    void* ws, size_t ws_bytes, void* stream);

/* Gradient of grouped_gemm_contig with respect to A:
 *   dA[r][:] = dC[r][:] . B[m_indices[r]]   (the sum runs over N, in fp32)
 * rounded to bf16.
 *   dC bf16 [M][N]; B bf16 [G][N][K]; dA bf16 [M][K]; m_indices as
 *   grouped_gemm_contig.  Rows with m_indices < 0 are left as they were.
 *   A row's result depends on its own dC row and its expert's weights alone.
 * Limits: N % 128 == 0, K % 128 == 0, N, K <= 4194304, G <= 1024,
 * ceil(M / 128) <= 8160, tile positions G * ceil(N / 256) * ceil(K / 256) / 8 and
 * ceil(M / 128) * ceil(K / 256) below 2^30 -> else MOE_EUNSUPPORTED. */
int32_t grouped_gemm_contig_dgrad(const void* dC, const void* B, void* dA,
                                  const int32_t* m_indices, int64_t M, int32_t N, int32_t K,
                                  int32_t G, void* stream);

/* Gradient of grouped_gemm_contig with respect to B:
 *   dB[g][n][k] = sum over r in [expert_start_loc[g], expert_start_loc[g] +
 *   num_valid[g]) of dC[r][n] * A[r][k]   (fp32), added to what dB holds if
 * accumulate is not 0, and rounded once to dB's type.  Experts without rows get
 * 0 (or keep what they hold).  Rows outside the experts' ranges are not part of
 * any sum, whatever they hold; ranges are cut at M.
 *   dC bf16 [M][N]; A bf16 [M][K]; dB [G][N][K], out_dtype MOE_DTYPE_BF16 or
 *   MOE_DTYPE_FP32; expert_start_loc, num_valid as moe_scatter_compact writes
 *   them.
 * Limits as grouped_gemm_contig_dgrad. */
int32_t grouped_gemm_contig_wgrad(const void* dC, const void* A, const int32_t* expert_start_loc,
                                  const int32_t* num_valid, int32_t out_dtype, int32_t accumulate,
                                  void* dB, int64_t M, int32_t N, int32_t K, int32_t G,
                                  void* stream);

/* One tensor of an AdamW step.
 *   param         device bf16 or fp32 [numel] (param_dtype MOE_DTYPE_BF16 or
 *                 MOE_DTYPE_FP32)
 *   master        device fp32 [numel]: the weight itself where param is bf16
 *                 (param is its rounding); NULL where param is fp32
 *   grad          device bf16 or fp32 [numel] (grad_dtype)
 *   m, v          state_bits 32: device fp32 [numel], the running means of the
 *                 gradient and of its square.  state_bits 8: device u8, numel
 *                 rounded up to 128: the e4m3 codes of m and of the root of v
 *   m_scale, v_scale  state_bits 8: device u8 [ceil(numel / 128)], the UE8M0
 *                 scale of each 128 elements; else NULL
 *   weight_decay  of this tensor
 * No param, master, m, v or scale may overlap another tensor of the plan or a
 * gradient; gradients may overlap each other. */
typedef struct {
  void* param;
  float* master;
  const void* grad;
  void* m;
  void* v;
  uint8_t* m_scale;
  uint8_t* v_scale;
  int64_t numel;
  float weight_decay;
  int32_t param_dtype;
  int32_t grad_dtype;
  int32_t state_bits;
} moe_adamw_tensor;

/* Host: bytes of the plan for n tensors, 0 where they are invalid.  Limit: fewer
 * than 2^31 pieces of 2048 elements over all tensors. */
size_t moe_adamw_plan_bytes(const moe_adamw_tensor* tensors, int32_t n);

/* Host: writes the plan of n tensors to host_plan.  The caller copies its
 * plan_bytes bytes to the device once and keeps them there for as long as the
 * tensors stay where they are.  Fewer than moe_adamw_plan_bytes -> MOE_ECAPACITY. */
int32_t moe_adamw_plan(const moe_adamw_tensor* tensors, int32_t n, void* host_plan,
                       size_t plan_bytes);

/* One AdamW step over the plan's tensors, in one launch.  With t = counter[0] + 1
 * and g the gradient times *grad_scale, in fp32:
 *   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2,
 *   w = w (1 - lr wd) - lr / (1 - beta1^t) m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * (1 - beta^t in double).  The step uses m and v before they are rounded to 8
 * bits.  8-bit states: for each 128 elements e is the smallest integer in
 * [-126, 127] with amax <= 448 * 2^e; x * 2^-e (the power within one fp32 place)
 * is cut to e4m3 after adding 16 random bits below its last place, so its
 * expectation is x (a positive root of v never becomes 0).  v, the root's square,
 * is higher than its formula by the variance of that: it settles 2% above at beta2
 * = 0.95 and 4% at 0.999 with normally distributed gradients (7% with sparse ones),
 * and the steps come out half as much short.  The bits are a hash of (seed, t,
 * tensor's place in the plan, element): the same call on the same state gives the
 * same result.
 *   plan       device copy of the plan, plan_bytes its size, 16-byte aligned; with
 *              a plan that is cut short the call does nothing: tensors and
 *              counter stay as they are
 *   lr         device fp32 [1], grad_scale device fp32 [1] or NULL (1): read by
 *              the kernel, so a captured step follows them
 *   counter    device int64 [2]: the number of steps taken (>= 0), and 0.  The
 *              call counts its step; two steps on one counter must not overlap
 * Non-finite gradients make their weight NaN and leave their group's 8-bit
 * states unspecified.
 * Limits: 0 <= beta < 1, eps > 0 -> else MOE_EINVAL. */
int32_t moe_adamw_step(const void* plan, size_t plan_bytes, const float* lr,
                       const float* grad_scale, int64_t* counter, double beta1, double beta2,
                       float eps, uint32_t seed, void* stream);

#ifdef __cplusplus
}
#endif
#endif
