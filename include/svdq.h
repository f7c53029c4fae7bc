/*
 * svdq.h -- C ABI of the SVDQuant W4A4 linear layer for AMD Instinct MI355X
 * (gfx950).
 *
 * The layer computes
 *
 *     Y = X^ L1 L2 + dequant( Q4(X^) Q4(R)^T ) + b,
 *     X^ = X diag(lambda)^-1,   W^ = diag(lambda) W = L1 L2 + R
 *
 * (model card "svdq-int4-flux.1-dev", "Overview of SVDQuant" caption:
 * stage 2 migrates activation outliers into the weights, stage 3 splits the
 * weights by SVD into a 16-bit low-rank branch and a 4-bit residual; the
 * SVDQuant abstract: W4A4 with a high-precision low-rank branch).
 *
 * It runs as two fused kernels (same card, Nunchaku engine caption (b)):
 *   svdq_quantize_act_lora_down  smoothing + 4-bit activation quantization +
 *                                down projection X^ L1, reading X once;
 *   svdq_gemm_w4a4_lora_up       4-bit GEMM + per-group dequant + up
 *                                projection + bias, writing Y once.
 * The weights are packed offline on the CPU by svdq_pack_weights.
 *
 * Conventions shared by every call
 * --------------------------------
 *  - All buffers are allocated and owned by the caller.  The library keeps
 *    no per-call state and allocates nothing on the two hot calls.  Host
 *    pointers are marked (host), device pointers (dev).
 *  - Matrices are dense, row-major, contiguous.  bf16 and fp16 values are
 *    passed as their 16-bit patterns.
 *  - W is given in nn.Linear layout [N][K] (out x in); the blog "Nunchaku
 *    4-bit inference in Diffusers" ("Introducing Nunchaku Lite") replaces
 *    nn.Linear modules with the quantized layer.  The low-rank factors are
 *    stored the same way: lora_down = L1^T as [rank][K] and lora_up = L2^T
 *    as [N][rank], i.e. the weights of the two small linears K->rank and
 *    rank->N.
 *  - INT4 codes, q in [-7, 7]: 4 bits each, rows of K/2 bytes, in units of
 *    16 consecutive k stored as two little-endian 32-bit words I0, I1.
 *    Code q has the 6-bit image 32 [q < 0] + |q| (sign in bit 5, |q| in
 *    bits 0-2, bits 3-4 zero: the FP6 E2M3 pattern of q/8); image j of a
 *    unit sits at bits 6j..6j+5 of the 96-bit string D0 | D1<<32 | D2<<64,
 *    and I0 = D0 | (D2 & 0x18618618), I1 = D1 | (D2 & 0x86186186) (the
 *    masks are the zero bits 3-4 of the images in D0 and D1, which together
 *    are the data bits of D2).  Zero carries no sign.
 *    INT4 scales: fp16, one per 64 consecutive k of a row, group-major
 *    [K/64][rows].  MXFP4 codes: E2M1 nibbles (sign in bit 3), code k in
 *    the low nibble of byte k/2 when k is even;
 *    MXFP4 scales: E8M0 bytes, one per 32 k, group-major [K/32][rows].
 *  - Shapes: M, N >= 1 (any value); K >= 64 and K % 64 == 0 for INT4,
 *    K % 128 == 0 for MXFP4; rank == 0 (no low-rank branch) or a multiple of
 *    16, at most 256 and at most min(K, N).  The GEMM calls address each
 *    4-bit operand and its scale array with 32-bit byte offsets: rows * K/2
 *    code bytes and the scale bytes of X (rows = M) and of W (rows = N)
 *    must each stay below 2^31, else SVDQ_ERR_SHAPE (M or N up to ~349,000
 *    at K = 12288).
 *  - Device pointers must be 16-byte aligned.
 *  - Errors: arguments and the device are checked before anything is
 *    launched and reported as a status code; nothing is thrown across the
 *    ABI.  A launch failure returns SVDQ_ERR_HIP.  A device that is not
 *    gfx950 (or no device) gives SVDQ_ERR_UNSUPPORTED_DEVICE, never a wrong
 *    result: the blog's "Hardware support" section has the loader check the
 *    GPU generation and raise a clear error instead of producing wrong
 *    outputs.
 *  - The hot calls enqueue on `stream` (a hipStream_t; NULL = the default
 *    stream of the current device) and never synchronize.
 */
#ifndef SVDQ_H
#define SVDQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__) || defined(__clang__)
#define SVDQ_API __attribute__((visibility("default")))
#else
#define SVDQ_API
#endif

#define SVDQ_OK                       0
#define SVDQ_ERR_INVALID_ARG         -1   /* NULL or misaligned pointer, bad enum */
#define SVDQ_ERR_SHAPE               -2   /* M, N, K or rank outside the rules above */
#define SVDQ_ERR_UNSUPPORTED_DEVICE  -3   /* no gfx950 device */
#define SVDQ_ERR_HIP                 -4   /* a HIP runtime call or launch failed */

#define SVDQ_INT4   0   /* int4 codes, groups of 64 along K, fp16 scales */
#define SVDQ_MXFP4  1   /* FP4 E2M1 codes, blocks of 32 along K, E8M0 scales */

/* Library version, major*10000 + minor*100 + patch. */
SVDQ_API int svdq_version(void);

/* Static text for a status code (never NULL). */
SVDQ_API const char* svdq_status_string(int status);

/* SVDQ_OK if HIP device `device` exists and is a gfx950, else
 * SVDQ_ERR_UNSUPPORTED_DEVICE.  The answer is cached per device. */
SVDQ_API int svdq_device_check(int device);

/* Byte sizes of the packed weight buffers for (K, N, rank, precision):
 * out_bytes[0] smooth_inv, [1] lora_down, [2] lora_up, [3] wq, [4] ws.
 * (host) out_bytes must hold 5 entries. */
SVDQ_API int svdq_packed_sizes(int K, int N, int rank, int precision, size_t* out_bytes);

/* Byte sizes of the activation buffers for (M, K, rank, precision):
 * out_bytes[0] xq, [1] xs, [2] lora_act.  (host) out_bytes holds 3 entries. */
SVDQ_API int svdq_act_sizes(int M, int K, int rank, int precision, size_t* out_bytes);

/* Offline pack, on the CPU (all pointers host).
 *
 * Stage 2 (smoothing): lambda_j = sqrt(max(act_absmax_j, 1e-5)) /
 * sqrt(max(max_n |W[n][j]|, 1e-5)) in fp64 (migration strength 0.5; the
 * pages give no formula) and smooth_inv_j = fp32(1/lambda_j).
 * W^ = W / smooth_inv in fp64.  Stage 3: top-`rank` SVD of W^ =
 * U S V^T by subspace iteration on the Gram matrix of the smaller side;
 * L1 = bf16(fp32(U_r S_r)), L2 = bf16(fp32(V_r^T)); residual
 * R = fp32(W^ - L1 L2) with the rounded factors; R quantized per output
 * channel with the layer's 4-bit rule.
 *
 *   w_bf16      [N][K] bf16 bits        nn.Linear weight
 *   act_absmax  [K] fp32                max |X[:, j]| of calibration data
 *   smooth_inv  [K] fp32                out
 *   lora_down   [rank][K] bf16          out (L1^T); may be NULL if rank == 0
 *   lora_up     [N][rank] bf16          out (L2^T); may be NULL if rank == 0
 *   wq          [N][K/2] uint8          out, packed codes of R
 *   ws          [K/64][N] fp16 (INT4) or [K/32][N] uint8 E8M0 (MXFP4), out
 *   r_out       [K][N] fp32             out, the unquantized residual; may be NULL
 * Threads: SVDQ_NUM_THREADS, else OMP_NUM_THREADS, else the host's cores
 * (at most 64). */
SVDQ_API int svdq_pack_weights(const uint16_t* w_bf16, const float* act_absmax,
                      int K, int N, int rank, int precision,
                      float* smooth_inv, uint16_t* lora_down, uint16_t* lora_up,
                      uint8_t* wq, void* ws, float* r_out);

/* Merge an off-the-shelf LoRA (Y += X A B) into the packed 16-bit branch,
 * on the CPU, without touching the 4-bit residual (SVDQuant abstract: the
 * engine supports low-rank adapters without re-quantization).  The branch
 * reads X^ = X diag(smooth_inv), so A is folded with 1/smooth_inv:
 * L1' = [L1 | A diag(1/smooth_inv)], L2' = [L2 ; B]; each folded element is
 * a[k][j] / smooth_inv[k] in fp64, rounded to fp32, then to bf16 (RNE).
 *
 *   lora_down      [rank][K] bf16        from svdq_pack_weights; NULL if rank == 0
 *   lora_up        [N][rank] bf16        from svdq_pack_weights; NULL if rank == 0
 *   smooth_inv     [K] fp32              from svdq_pack_weights
 *   a              [K][lora_rank] bf16   adapter down factor
 *   b              [lora_rank][N] bf16   adapter up factor
 *   lora_down_out  [rank+lora_rank][K] bf16, out (caller-allocated)
 *   lora_up_out    [N][rank+lora_rank] bf16, out (caller-allocated)
 * rank + lora_rank must meet the hot calls' rank rule (a multiple of 16, at
 * most 256 and at most min(K, N)), else SVDQ_ERR_SHAPE.  All pointers host;
 * the outputs must not overlap the inputs. */
SVDQ_API int svdq_merge_lora(const uint16_t* lora_down, const uint16_t* lora_up, int rank,
                             const float* smooth_inv, const uint16_t* a, const uint16_t* b,
                             int lora_rank, int K, int N,
                             uint16_t* lora_down_out, uint16_t* lora_up_out);

/* Fused kernel 1 (Nunchaku engine caption (b): the down projection and the
 * quantizer share their input, so X is read once).
 *
 *   x          (dev) [M][K] bf16        activations
 *   smooth_inv (dev) [K] fp32           from svdq_pack_weights
 *   lora_down  (dev) [rank][K] bf16     L1^T; ignored if rank == 0
 *   xq         (dev) [M][K/2] uint8     out, 4-bit codes of X^
 *   xs         (dev) [K/64][M] fp16 (INT4) | [K/32][M] E8M0 (MXFP4), out
 *   lora_act   (dev) [M][rank] fp32     out, X^ L1 (fp32 accumulation);
 *                                       ignored if rank == 0
 * X^ = bf16(fp32(x * smooth_inv)) is rounded once and feeds both branches.
 * INT4 rule per 64-group of a row: s = fp16(fp32(amax/7)) (round to
 * nearest even, saturating at 65504), s == 0 -> codes 0, else
 * q = clamp(rint(fp32(x^ * fp32(1/s))), -7, 7), ties to even.
 * MXFP4 rule per 32-block (OCP Microscaling v1.0): amax == 0 -> byte 0 and
 * codes 0; else e = clamp(floor(log2 amax) - 2, -127, 127) from the fp32
 * exponent field, byte e + 127, code = E2M1(x^ / 2^e) rounded to nearest
 * (ties to the even code, saturating at 6); zero magnitudes carry no sign.
 * lora_act partials of several workgroups may be summed with fp32 atomics,
 * so its last bits can differ between calls. */
SVDQ_API int svdq_quantize_act_lora_down(const void* x, int M, int K,
                                const float* smooth_inv, const void* lora_down,
                                int rank, int precision,
                                uint8_t* xq, void* xs, float* lora_act,
                                void* stream);

/* Fused kernel 2 (Nunchaku engine caption (b): the up projection and the
 * 4-bit compute share their output, so Y is written once).
 *
 *   xq, xs     (dev) from svdq_quantize_act_lora_down
 *   wq, ws     (dev) from svdq_pack_weights
 *   lora_act   (dev) [M][rank] fp32; ignored if rank == 0
 *   lora_up    (dev) [N][rank] bf16 (L2^T); ignored if rank == 0
 *   bias       (dev) [N] bf16, or NULL for no bias
 *   y          (dev) [M][N] bf16        out
 * INT4: for every 64-group g the exact integer partial
 * P = sum_k qx qw is scaled by s_x[m,g] s_w[n,g] into fp32 accumulators;
 * the up projection bf16(lora_act) L2 and the bias are added in fp32 and Y
 * is rounded to bf16 once.  MXFP4: the E2M1 codes with their E8M0 block
 * scales go to the matrix core as they are (fp32 accumulation); up
 * projection, bias and rounding as for INT4. */
SVDQ_API int svdq_gemm_w4a4_lora_up(const uint8_t* xq, const void* xs,
                           const uint8_t* wq, const void* ws,
                           const float* lora_act, const void* lora_up,
                           const void* bias, void* y,
                           int M, int N, int K, int rank, int precision,
                           void* stream);

/* svdq_gemm_w4a4_lora_up with a caller workspace, for grids that leave the
 * device mostly idle (the token rows one of several GPUs holds when a batch
 * is split by rows).  Same operation and arguments as above (the Nunchaku
 * engine caption (b) of the "svdq-int4-flux.1-dev" card), plus:
 *   workspace (dev) workspace_bytes bytes, 16-byte aligned, owned by the
 *             caller; its contents on entry do not matter; it must not be
 *             used by another call that may run at the same time.
 * svdq_gemm_workspace_size gives the bytes this call can use for the
 * shape on the current device: 0 when the single-pass schedule runs
 * anyway.  With a workspace of that size an INT4 grid whose tiles fill
 * under half the workgroup slots (two per CU) and whose K loop has at
 * least 16 stages of 128 k is cut along K: each part writes fp32 tile
 * partials into the workspace, and a second kernel adds them in a fixed
 * order and applies the up projection, the bias and the single rounding to
 * bf16.  The result is deterministic, and within the same bounds as the
 * single-pass schedule: its fp32 sums run in a different order.  A NULL
 * or smaller workspace runs the single-pass schedule.  MXFP4 always runs
 * the single-pass schedule. */
SVDQ_API int svdq_gemm_workspace_size(int M, int N, int K, int precision, size_t* out_bytes);
SVDQ_API int svdq_gemm_w4a4_lora_up_ws(const uint8_t* xq, const void* xs,
                              const uint8_t* wq, const void* ws,
                              const float* lora_act, const void* lora_up,
                              const void* bias, void* y,
                              int M, int N, int K, int rank, int precision,
                              void* workspace, size_t workspace_bytes,
                              void* stream);

/* First layer of an MLP pair with its activation fused: the original
 * engine's model-specific paths include a fused GELU/MLP kernel (blog
 * "Nunchaku 4-bit inference in Diffusers", "Introducing Nunchaku Lite").
 * The activation is the tanh-form GELU of FLUX's MLP (a reading; the pages
 * do not name the form).  INT4 only.
 *
 * svdq_gemm_w4a4_lora_up_gelu: as svdq_gemm_w4a4_lora_up, but y receives
 * bf16(GELU(Y)) with Y the layer's bf16 output (rounded first, as the next
 * layer would read it) and GELU(y) = 0.5 y (1 + tanh(sqrt(2/pi) (y +
 * 0.044715 y^3))) evaluated in fp32.
 *
 * svdq_mlp_gemm_gelu_quant: writes no Y at all.  The tile of X2 =
 * bf16(GELU(Y)) goes straight into the second layer's first kernel
 * (svdq_quantize_act_lora_down's rule with smooth_inv2 and lora_down2):
 *   smooth_inv2 (dev) [N] fp32            second layer's smoothing
 *   lora_down2  (dev) [rank2][N] bf16     second layer's L1^T; ignored if rank2 == 0
 *   xq2         (dev) [M][N/2] uint8      out, 4-bit codes of X2^
 *   xs2         (dev) [N/64][M] fp16      out
 *   lora_act2   (dev) [M][rank2] fp32     out (cleared, then summed over the
 *                                         output tiles with fp32 atomics)
 * N % 128 == 0 (a 64-column group lies inside one 128-column tile), else
 * SVDQ_ERR_SHAPE; rank2 follows the rank rule with K = N.  Other arguments
 * as for svdq_gemm_w4a4_lora_up. */
SVDQ_API int svdq_gemm_w4a4_lora_up_gelu(const uint8_t* xq, const void* xs,
                           const uint8_t* wq, const void* ws,
                           const float* lora_act, const void* lora_up,
                           const void* bias, void* y,
                           int M, int N, int K, int rank, int precision,
                           void* stream);
SVDQ_API int svdq_mlp_gemm_gelu_quant(const uint8_t* xq, const void* xs,
                           const uint8_t* wq, const void* ws,
                           const float* lora_act, const void* lora_up,
                           const void* bias, int M, int N, int K, int rank,
                           const float* smooth_inv2, const void* lora_down2, int rank2,
                           int precision, uint8_t* xq2, void* xs2, float* lora_act2,
                           void* stream);

/* W4A16 comparison layer: 4-bit weights, bf16 activations (the 4-bit
 * weight-only baseline that the SVDQuant abstract measures W4A4 against:
 * 3.0x with INT4, 3.1x with NVFP4, whole model).  The weights carry the
 * layer's INT4 rule per output channel in groups of 64 along K, with no
 * smoothing and no low-rank branch.
 *
 * svdq_pack_w4a16 (host): w_bf16 [N][K] -> wq [N][K/2] (same code layout as
 *   the W4A4 codes), ws [K/64][N] fp16.  K % 64 == 0.
 * svdq_gemm_w4a16 (device): y [M][N] bf16 = bf16(x . (q s)^T + bias); x
 *   bf16 [M][K], bias bf16 [N] or NULL.  Each weight q*s is rounded to bf16
 *   once, the products accumulate in fp32. */
SVDQ_API int svdq_pack_w4a16(const uint16_t* w_bf16, int K, int N, uint8_t* wq, void* ws);
SVDQ_API int svdq_gemm_w4a16(const void* x, const uint8_t* wq, const void* ws,
                             const void* bias, void* y, int M, int N, int K, void* stream);

/* Unfused baseline of the same layer, for measuring what the two fusions
 * save (model card "svdq-int4-flux.1-dev", Nunchaku engine caption (a): a
 * naive low-rank branch as separate kernels costs an extra 16-bit read of
 * X in the down projection and an extra 16-bit write of Y in the up
 * projection).  Four kernels on `stream`: quantize (writes xq, xs),
 * down projection (reads X again, writes lora_act), 4-bit GEMM (writes Y
 * in bf16) and up projection (reads Y, adds bf16(lora_act) L2 and the
 * bias, writes Y).  Arguments, layouts and errors as for the two fused
 * calls; xq, xs and lora_act are caller-owned intermediates.  Results equal
 * the fused path's up to the second bf16 rounding of Y.  INT4 only. */
SVDQ_API int svdq_unfused_linear(const void* x, int M, int K,
                        const float* smooth_inv, const void* lora_down, int rank,
                        const uint8_t* wq, const void* ws,
                        const void* lora_up, const void* bias, int N, int precision,
                        uint8_t* xq, void* xs, float* lora_act, void* y,
                        void* stream);

/* svdq_unfused_linear for callers that cannot allocate (code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc): the
 * same four kernels and the same result, without the xq, xs and lora_act
 * workspace arguments.  Those intermediates live in one device array of
 * 32 MiB (SVDQ_NOALLOC_SCRATCH_BYTES) that the library holds on every GPU
 * it runs on until the process ends; the call itself allocates nothing.
 * The array needs M*K/2 + (K/64)*M*2 + M*rank*4 bytes, each part rounded up
 * to 256 bytes (FLUX.1's 12288 -> 3072 MLP layer at M = 4608, rank 32:
 * ~30.7 MB); a larger call returns SVDQ_ERR_SHAPE.  Every call on a GPU
 * shares that GPU's array and leaves its contents behind, so calls that
 * overlap on one GPU (two streams, two threads) race and must be
 * serialized by the caller.  INT4 only; other arguments and errors as for
 * svdq_unfused_linear. */
#define SVDQ_NOALLOC_SCRATCH_BYTES (32u << 20)
SVDQ_API int svdq_unfused_linear_noalloc(const void* x, int M, int K,
                        const float* smooth_inv, const void* lora_down, int rank,
                        const uint8_t* wq, const void* ws,
                        const void* lora_up, const void* bias, int N, int precision,
                        void* y, void* stream);

/* ---------------------------------------------------------------------
 * 16-bit operators that stand between the quantized linears of a
 * transformer block.  Values are bf16 or fp16 (dtype), held in fp32 between
 * load and the one rounding to nearest even at the end.  They allocate
 * nothing; conventions, errors and streams are those of the hot calls.
 * --------------------------------------------------------------------- */
#define SVDQ_BF16  0
#define SVDQ_F16   1

/* Attention over packed sequences with grouped heads.
 *
 *   s_ij = scale q_i . k_j over the keys j of query i's sequence,
 *   o_i = sum_j softmax_j(s_ij) v_j,   lse_i = log sum_j exp(s_ij)
 *
 *   q, o   (dev) [total_q][heads_q][head_dim]   token and head strides below
 *   k, v   (dev) [total_k][heads_k][head_dim]
 *   lse    (dev) [total_q][heads_q] fp32, out, or NULL
 *   cu_seqlens_q, cu_seqlens_k (dev) [batch+1] int32 each: sequence b holds
 *          queries cu_q[b] .. cu_q[b+1]-1 and keys cu_k[b] .. cu_k[b+1]-1.
 *          They lie in [0, total] and do not fall; sequences may be empty on
 *          either side.  Tokens of q before the first start or past the last
 *          (padding) belong to no sequence: o = 0, lse = -inf.  With starts
 *          that break this, o and lse are unspecified, but values outside
 *          are cut to [0, total], so no access leaves the tensors.  NULL
 *          (both, batch == 1): one sequence of all tokens.
 *   strides (host) 8 strides in elements: q token, q head, k token, k head,
 *          v token, v head, o token, o head.  Multiples of 8, not negative;
 *          k and v token strides in [head_dim, 2^23] when total_k > 1.  The last dimension
 *          is dense.  Q, K and V can so be read out of one fused projection.
 * Query head h reads key head h / (heads_q / heads_k).
 * causal != 0: counted from the sequences' ends, query i sees keys
 * j <= i + len_k - len_q (the last query sees the last key; with one query
 * all keys).  A query that sees no key gives o = 0 and lse = -inf.  Keys
 * that no query of a row's sequence can see, and what lies past a
 * sequence's end, may hold anything; a NaN or infinity in v at a key hidden
 * from a query only by the causal rule can reach that query's o (0 * NaN).
 * o overlaps none of q, k and v.
 * head_dim: a multiple of 8, 8 to 128.  total_q, total_k >= 0; total_k and
 * rows = total_q (heads_q / heads_k) at most 2^31 - 2^16, and
 * (rows / 32 + batch) heads_k below 2^24.  0 < scale < 2^127.  Scores lie
 * within 2^26 of 0: past that their maximum is rounded by more than the 16
 * bits of a weight hold.
 * workspace (dev, 16-byte aligned): with the bytes that
 * svdq_attention_workspace_size names, calls with few queries (single
 * tokens against long caches) cut the keys into parts whose results a second
 * kernel joins in a fixed order; with NULL or fewer bytes one workgroup runs
 * through all keys of its queries.  Results are deterministic; the schedule
 * goes by the sizes passed here, not by the lengths on the device. */
SVDQ_API int svdq_attention_workspace_size(int total_q, int total_k, int batch, int heads_q,
                              int heads_k, int head_dim, size_t* out_bytes);
SVDQ_API int svdq_attention(const void* q, const void* k, const void* v, void* o, float* lse,
                              const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                              int batch, int total_q, int total_k, int heads_q, int heads_k,
                              int head_dim, const int64_t* strides, float scale, int causal,
                              int dtype, void* workspace, size_t workspace_bytes, void* stream);

/* 16-bit linear with its epilogue, for the layers that stay in 16 bits
 * (embedders, modulation, output projections):
 *
 *   y = residual + gate_g * act(x W^T + bias),   g = row / group_rows
 *
 *   x        (dev) [M][K], row stride ldx
 *   w        (dev) [N][K] (nn.Linear layout), row stride ldw
 *   bias     (dev) [N], or NULL
 *   gate     (dev) [ceil(M / group_rows)][N], row stride ld_gate, or NULL
 *   residual (dev) [M][N], row stride ldr, or NULL; may be y itself
 *   y        (dev) [M][N], row stride ldy, out
 * Products accumulate in fp32; bias, activation, gate and residual are
 * applied in fp32 and y is rounded once.  activation: SVDQ_ACT_NONE,
 * SVDQ_ACT_GELU (the tanh form, as in svdq_gemm_w4a4_lora_up_gelu) or
 * SVDQ_ACT_SILU (z / (1 + exp(-z))).
 * M, N, K >= 1, M at most 2^31 - 2^16, N at most 2^29 - 32, fewer than 2^24
 * tiles of 64 x 64 in the result; strides in elements, at least
 * the row's length; those of x and w at most 2^22 with 255 ld + K < 2^30;
 * group_rows >= 1.  y overlaps neither x nor w.  Pointers need 2-byte
 * alignment only; rows of x and w that are 16-byte aligned with
 * K % 8 == 0 take the faster loads.
 * workspace (dev, 16-byte aligned): with the bytes that
 * svdq_linear16_workspace_size names (at any alignment), or those that
 * svdq_linear16_workspace_size_for names for these operands (their addresses
 * and strides alone are looked at), grids that would leave the device idle
 * are cut along K into fp32 parts that a second kernel adds in a fixed
 * order; with NULL or fewer bytes than the latter they run in one piece.
 * Results are deterministic. */
#define SVDQ_ACT_NONE  0
#define SVDQ_ACT_GELU  1
#define SVDQ_ACT_SILU  2
SVDQ_API int svdq_linear16_workspace_size(int M, int N, int K, size_t* out_bytes);
SVDQ_API int svdq_linear16_workspace_size_for(const void* x, int64_t ldx, const void* w, int64_t ldw,
                              int M, int N, int K, size_t* out_bytes);
SVDQ_API int svdq_linear16(const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias,
                              const void* gate, int64_t ld_gate, int group_rows,
                              const void* residual, int64_t ldr, void* y, int64_t ldy,
                              int M, int N, int K, int activation, int dtype,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Adaptive layer norm, the input of a block's projections:
 *
 *   y = (x - mean) rstd [* weight + bias] [* (1 + scale_g) + shift_g],
 *   rstd = 1 / sqrt(var + eps),   g = row / group_rows
 *
 * with mean and (biased) variance of the row's K values in fp32, the
 * variance taken from the deviations; y is rounded once.
 *   x, y           (dev) [M][K], row strides ldx, ldy >= K; y may be x
 *   weight, bias   (dev) [K], each or both NULL
 *   scale, shift   (dev) [ceil(M / group_rows)][K], row stride ld_mod >= K,
 *                  each or both NULL
 * 1 <= M <= 2^31 - 2^16; K from 1 to 65536; group_rows >= 1; eps >= 0 and finite.  Pointers
 * need 2-byte alignment only. */
SVDQ_API int svdq_layer_norm(const void* x, int64_t ldx, const void* weight, const void* bias,
                              const void* scale, const void* shift, int64_t ld_mod, int group_rows,
                              void* y, int64_t ldy, int M, int K, float eps, int dtype,
                              void* stream);

/* ---------------------------------------------------------------------
 * 8-bit operators of a block that is served in 8 bits.  Codes are OCP e4m3
 * (largest value 448, no infinity), a byte each; arithmetic is fp32 between
 * load and the one rounding at the end.  They allocate nothing; conventions,
 * errors and streams are those of the hot calls.
 *
 * Matrices of codes are dense [rows][K], 16-byte aligned, K % 16 == 0, with a
 * scale for each block of 128 values along K (the last may be shorter):
 *   activations  scales fp32 [ceil(K / 128)][rows], group-major
 *   weights      scales fp32 [ceil(N / 128)][ceil(K / 128)], one for
 *                128 x 128 values
 * Rule: s = max(amax, 2^-100) / 448, code = e4m3(fp32(v * fp32(1 / s))) to
 * nearest even.  amax passes over NaN; a NaN's code is NaN; an infinity makes
 * s infinite and the block's codes 0 and NaN, so that it is not lost.
 * --------------------------------------------------------------------- */
#define SVDQ_FP8_BLOCK 128

/* Root-mean-square norm with the residual's addition:
 *
 *   h = x [+ residual],   y = h rstd [* weight],   rstd = 1 / sqrt(mean(h^2) + eps)
 *
 *   x         (dev) [M][K], row stride ldx
 *   residual  (dev) [M][K], row stride ldr, or NULL
 *   weight    (dev) [K], or NULL
 *   sum       (dev) [M][K], row stride ld_sum, out: h rounded once, or NULL;
 *             may be x or residual
 *   y         (dev) [M][K], row stride ldy, out, or NULL; may be x or residual
 *   yq, ys    (dev) codes and scales of y, out, or both NULL; taken from the
 *             fp32 y (rounded once)
 * Either y or yq and ys is given.  y is taken from h in fp32, not from its
 * rounding, at any size that fp32 holds: where the squares' sum leaves its
 * range it is taken at another scale.  sum and y do not overlap.
 * 1 <= M <= 2^31 - 2^16; K from 1 to 65536, K % 16 == 0 for codes; eps >= 0
 * and finite.  16-bit pointers need 2-byte alignment only. */
SVDQ_API int svdq_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                              void* sum, int64_t ld_sum, void* y, int64_t ldy, uint8_t* yq, float* ys,
                              int M, int K, float eps, int dtype, void* stream);

/* Codes and scales of activations x (dev) [M][K], row stride ldx, bf16 or
 * fp16: xq (dev) [M][K], xs (dev) [ceil(K / 128)][M], out.
 * 1 <= M <= 2^31 - 2^16; K a multiple of 16 to 2^22. */
SVDQ_API int svdq_quantize_fp8(const void* x, int64_t ldx, uint8_t* xq, float* xs, int M, int K, int dtype,
                              void* stream);

/* Offline pack of a weight, on the CPU (all pointers host): w [N][K] bf16 or
 * fp16 bits -> wq [N][K] codes, ws [ceil(N / 128)][ceil(K / 128)]. */
SVDQ_API int svdq_pack_fp8(const uint16_t* w, int K, int N, int dtype, uint8_t* wq, float* ws);

/* 8-bit linear with the epilogue of svdq_linear16:
 *
 *   z[m][n] = sum_g xs[g][m] ws[n / 128][g] sum_(k in block g) xq[m][k] wq[n][k]
 *   y = residual + gate_r * act(z + bias),   r = row / group_rows
 *
 * xq, xs, wq, ws (dev) as above, xs and ws 4-byte aligned; bias, gate,
 * residual, y, activation and dtype (theirs) as for svdq_linear16.  Sums are
 * fp32, the blocks' in a fixed order (a block's two scales are multiplied
 * first: their product has to lie in fp32's range), but that the matrix core
 * takes the 8-bit products of 8 consecutive k to the largest one's exponent E
 * and cuts what lies below 2^(E - 13) (about 1e-4 of a result of 4096
 * products); y is rounded once and overlaps no operand but residual.
 * M, N >= 1, M at most 2^31 - 2^16, N at most 2^28 - 32, fewer than 2^23 tiles
 * of 64 x 64 in the result; K a multiple of 16 to 2^22.
 * Results are deterministic. */
SVDQ_API int svdq_gemm_fp8(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws, const void* bias,
                              const void* gate, int64_t ld_gate, int group_rows, const void* residual, int64_t ldr,
                              void* y, int64_t ldy, int M, int N, int K, int activation, int dtype, void* stream);

/* Keys and values of packed sequences in a paged cache of 8-bit codes.
 *
 *   k_cache     (dev) [pages][heads_k][64][head_dim] codes, by place
 *   v_cache     (dev) [pages][heads_k][4][head_dim][16] codes: place p of the
 *               page at [p / 4 % 4][d][4 (p / 16) + p % 4]
 *   exponents   (dev) [pages][heads_k][2] int8: value = code * 2^e, of keys
 *               and of values; taken as cut to [-40, 40]
 *   block_table (dev) [batch][table_width] int32: the page of positions 64 i
 *               to 64 i + 63 of each sequence
 *   lengths     (dev) [batch] int32: tokens of each sequence in the cache, the
 *               new ones (of this call's q, k and v) included
 *   cu_seqlens  (dev) [batch+1] int32: sequence b has tokens cu[b] .. cu[b+1]-1
 *               of the pack, the last of its positions; NULL: one token each
 *               (batch == total)
 * Entries of the table that name no page (below 0, or pages and more) have
 * none: nothing is written there, and their keys are hidden.  Positions past
 * the table, and tokens before position 0, are passed over in the same way.
 * Whatever these arrays hold, no access leaves the tensors.
 *
 * svdq_cache_append writes the new tokens' keys and values, and rotates q:
 *
 *   q         (dev) [total][heads_q][head_dim] and q_out, its rotation; or both
 *             NULL.  q_out may be q itself (with its strides) and overlaps
 *             nothing else.
 *   k, v      (dev) [total][heads_k][head_dim]
 *   rope      (dev) fp32 [rope_rows][rotary]: rotary / 2 cosines and as many
 *             sines for each position (those past the last row take it); or
 *             NULL with rotary == 0: nothing is rotated
 *   strides   (host) 8 strides in elements: q token, q head, k token, k head,
 *             v token, v head, q_out token, q_out head; not negative, the last
 *             dimension is dense, 2-byte alignment suffices
 * Of the first `rotary` values of a head (a multiple of 16, at most head_dim)
 * the pairs are i and i + rotary / 2, or (interleaved != 0) 2 i and 2 i + 1:
 * (a, b) -> (a cos - b sin, b cos + a sin).  q is rounded once to its type, k
 * and v once to their codes.  A page's exponent (of each head, keys and values
 * apart) is the least e with amax <= 448 * 2^e over the finite values that
 * enter it, cut to [-40, 40], and not below the one it has if it holds earlier
 * tokens of the sequence; those codes are then rescaled (rounded to nearest
 * even, exact but for codes below 2^-6).  Values past 448 * 2^40 become that;
 * what is not finite becomes NaN.  Other places of a page stay as they are.
 * Tokens of no sequence are not appended, and their q is not rotated.  Two
 * sequences may share pages that no call appends to; a page that is written
 * for two places at once holds either's.
 *
 * svdq_attention_paged lets q's tokens attend to their sequences in the cache:
 *
 *   q, o      (dev) [total][heads_q][head_dim], 16-byte aligned
 *   lse       (dev) [total][heads_q] fp32, out, or NULL: log sum_j exp(s_ij)
 *   strides   (host) 4 strides in elements: q token, q head, o token, o head;
 *             multiples of 8, not negative
 * Query head h reads key head h / (heads_q / heads_k).  causal != 0: query i of
 * n sees keys j <= i + length - n, else all of its sequence's.  A query that
 * sees no key, or belongs to no sequence, gives o = 0 and lse = -inf, whatever
 * the pages hold.  Pages' places past a sequence's length may hold anything;
 * a NaN at a key that only causal masking hides can reach a query that sees
 * others.  The codes are taken exactly; P is rounded to 16 bits for the matrix
 * core; softmax statistics and sums are fp32.  Scores may have any size that
 * fp32 holds (times log2 e); one past it is an infinity, and below it counts as
 * hidden.  o overlaps no operand.  2^-80 <= scale < 2^80.
 * workspace (dev, 16-byte aligned): with the bytes that
 * svdq_attention_paged_workspace_size names, calls with few queries a sequence
 * cut the keys into equal shares, which a second kernel joins in a fixed
 * order; with NULL or fewer bytes a workgroup runs through all keys of its
 * queries.  Results are deterministic; the schedule goes by sizes alone.
 *
 * Both: head_dim a multiple of 16 from 16 to 128; heads_q a multiple of
 * heads_k; batch, pages >= 1; table_width from 1 to 2^24; total >= 0; caches
 * 16-byte aligned; (total (heads_q / heads_k) / 16 + batch) heads_k
 * (table_width + 4) below 2^31, and (total (heads_q / heads_k) / 16 + 2 batch + total) heads_k below 2^24. */
#define SVDQ_PAGE 64
SVDQ_API int svdq_cache_append(const void* q, const void* k, const void* v, void* q_out, const int64_t* strides,
                              uint8_t* k_cache, uint8_t* v_cache, int8_t* exponents, int pages,
                              const int32_t* block_table, int table_width, const int32_t* lengths,
                              const int32_t* cu_seqlens, int batch, int total, int heads_q, int heads_k, int head_dim,
                              const float* rope, int rope_rows, int rotary, int interleaved, int dtype, void* stream);
SVDQ_API int svdq_attention_paged_workspace_size(int total, int batch, int table_width, int heads_q, int heads_k,
                              int head_dim, size_t* out_bytes);
SVDQ_API int svdq_attention_paged(const void* q, void* o, float* lse, const int64_t* strides, const uint8_t* k_cache,
                              const uint8_t* v_cache, const int8_t* exponents, int pages, const int32_t* block_table,
                              int table_width, const int32_t* lengths, const int32_t* cu_seqlens, int batch, int total,
                              int heads_q, int heads_k, int head_dim, float scale, int causal, int dtype,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Measurement hook: the dense matrix-core rate this GPU sustains.  Each of
 * `blocks` workgroups (4 waves; launch two per CU) issues 8 * iters
 * independent v_mfma_scale_f32_32x32x64_f8f6f4 per wave, with FP8 operands
 * (precision SVDQ_INT4: 16 passes per instruction, the matrix time the INT4
 * GEMM spends per K-group and 32x32 tile as one 8-pass FP6 product plus one
 * 8-pass rank-1 scale product) or FP4 operands (SVDQ_MXFP4).
 * Ops per launch = blocks * 4 * 8 * iters * 131072;
 * the caller times it.  out (dev) [blocks] fp32 receives one checksum per
 * workgroup.  blocks, iters >= 1. */
SVDQ_API int svdq_bench_mfma_ceiling(int precision, int blocks, int iters, float* out, void* stream);

/* Test hook: the exact per-group integer partials of the INT4 GEMM for the
 * output window rows [m0, m0+mt) x columns [n0, n0+nt).  It runs the INT4
 * GEMM kernel of svdq_gemm_w4a4_lora_up in a test mode that shares its code
 * loader, the conversion of the codes for the matrix core, the LDS layout
 * and the matrix instruction that forms each group's partial; the scale
 * handling (the per-group dequant into the accumulators), the up
 * projection and the epilogue are replaced by a store of the partials.
 *   out (dev) [mt][nt][K/64] int32.  mt, nt >= 1; the window must lie
 *   inside [0, M) x [0, N). */
SVDQ_API int svdq_debug_group_partials(const uint8_t* xq, const uint8_t* wq,
                              int M, int N, int K,
                              int m0, int n0, int mt, int nt,
                              int32_t* out, void* stream);

/* Test hooks (host): the schedule that these operators take for these sizes, given the workspace that they name for them.
 *   attention: plan[0] rows of a tile, [1] parts of its keys within a
 *   workgroup, [2] splits of them over workgroups, [3] workgroups that take
 *   equal shares of all keys (0: a tile's keys are one workgroup's)
 *   linear16: plan[0] rows and [1] channels of a tile, [2] waves of a
 *   workgroup, [3] splits along K; aligned != 0: rows of x and w are 16-byte
 *   aligned, which takes K % 8 == 0
 *   gemm_fp8: plan[0] to [2] as for linear16
 *   attention_paged: plan[0] rows of a tile, [1] workgroups that take equal
 *   shares of all keys (0: a tile's keys are one workgroup's) */
SVDQ_API int svdq_debug_attention_plan(int total_q, int total_k, int batch, int heads_q,
                              int heads_k, int head_dim, int causal, int32_t* plan);
SVDQ_API int svdq_debug_linear16_plan(int M, int N, int K, int aligned, int32_t* plan);
SVDQ_API int svdq_debug_gemm_fp8_plan(int M, int N, int K, int32_t* plan);
SVDQ_API int svdq_debug_attention_paged_plan(int total, int batch, int table_width, int heads_q, int heads_k,
                              int head_dim, int32_t* plan);

#ifdef __cplusplus
}
#endif

#endif /* SVDQ_H */
