/*
 * svq.h -- C ABI of the weight-only quantized linear layer for decode and
 * speculative-verify shapes on AMD Instinct MI355X (gfx950).
 *
 *   y[M][N] = x[M][K] . deq(W)^T     (bf16 x, fp32 accumulation, bf16 y)
 *
 * Two weight formats:
 *  - W4A16: symmetric INT4 with zero point 8, one fp16 scale per group of G
 *    K-rows (G = 32, 64 or 128), GPTQ words packed 8 per int32 along K, no
 *    group reordering. GPTQ INT4 card "Qwen3.8-27B-GPTQ-Int4-sym-G128-MTP-BF16",
 *    section "Quantization contract"; Eole recipe "Qwen3.8-27B and native MTP
 *    speculative decoding", section "Compressed-tensors INT4 layout".
 *  - MXFP8: OCP E4M3FN elements with one E8M0 scale per 32 K-elements. MXFP8
 *    card "Qwen3.8-27B-MXFP8-CT-AutoRound-mtp", opening summary, sections
 *    "2. Precision plan" (N >= 128, K % 32 == 0) and "8. License and
 *    attribution" (OCP MX, E8M0 scale per 32-element block).
 *  - W8A16, the quantized vocabulary head: symmetric int8 codes with one fp16
 *    scale per group of G K-rows, produced at load time from the dense bf16
 *    projection by svq_rtn_quantize (which also produces W4A16 weights). Eole
 *    recipe, section "Optional vocabulary-head quantization".
 *
 * M is the number of tokens verified per call: streams x (1 + draft tokens)
 * (Eole recipe, opening paragraph: the main model verifies a chunk of drafted
 * tokens). Packed INT4 weights are repacked once at setup, as the Eole recipe's
 * section "Pack inference projections" does before its own GEMM kernel runs.
 *
 * Conventions for every entry point:
 *  - All buffer pointers are DEVICE pointers to memory the caller owns. The
 *    library keeps no pointer after returning and allocates, frees and
 *    synchronizes nothing.
 *  - `stream` is a hipStream_t passed as void* (NULL = the null stream). Work
 *    is enqueued asynchronously on it; buffers must stay alive until it runs.
 *  - Every argument is checked on the host BEFORE anything is enqueued. On any
 *    error nothing is launched and outputs are left untouched. Unsupported
 *    formats (asymmetric weights, zero points, group reordering, activation
 *    quantization) cannot be expressed: there are no such parameters.
 *  - Row-major everywhere; bf16 and fp16 values are passed as their 16-bit
 *    patterns.
 *  - GEMM operands stay below 2 GiB each (M*K*2, N*K, M*N*2 < 2^31 bytes;
 *    the kernels use 32-bit buffer offsets); larger shapes return
 *    SVQ_ERR_DIM.
 *  - Results are deterministic: repeated calls with equal inputs give equal
 *    bits (all reductions run in a fixed order).
 */
#ifndef SVQ_H
#define SVQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SVQ_ABI_VERSION 1

typedef enum svq_status {
    SVQ_OK = 0,
    SVQ_ERR_NULL = 1,          /* a required pointer is NULL */
    SVQ_ERR_DIM = 2,           /* M, N or K out of range (<= 0 or too large) */
    SVQ_ERR_GROUP = 3,         /* group size not supported for this format */
    SVQ_ERR_DIVISIBILITY = 4,  /* N % 16 != 0, K % 128 != 0 or K % G != 0 */
    SVQ_ERR_MXFP8_SHAPE = 5,   /* MXFP8 needs N >= 128 and K % 32 == 0 */
    SVQ_ERR_ALIGN = 6,         /* a pointer is not suitably aligned */
    SVQ_ERR_OVERLAP = 7,       /* output overlaps an input */
    SVQ_ERR_WORKSPACE = 8,     /* workspace missing, too small or misaligned */
    SVQ_ERR_HIP = 9,           /* the HIP runtime refused the launch */
    SVQ_ERR_UNSUPPORTED = 10   /* the requested kernel cannot run this shape */
} svq_status;

/* Kernel selectors for the *_with entry points (diagnostics and benchmarks).
 * SVQ_KERNEL_AUTO is what svq_w4a16_gemm / svq_mxfp8_gemm use. */
typedef enum svq_kernel {
    SVQ_KERNEL_AUTO = 0,
    SVQ_KERNEL_DOT2 = 1,        /* VALU bf16 dot2, M <= 8: 16-column blocks with row
                                   broadcast of x; for M <= 2 and fewer 16-column
                                   blocks than CUs, 4-column units with x in LDS */
    SVQ_KERNEL_MFMA_SKINNY = 2, /* one 16-row MFMA tile, waves split K, M <= 16 */
    SVQ_KERNEL_MFMA_WIDE = 3    /* LDS-staged x, 64/128-row MFMA tiles, split-K, any M */
} svq_kernel;

/* Operations, for the format-generic queries svq_workspace_bytes and
 * svq_kernel_name. */
typedef enum svq_op {
    SVQ_OP_W4A16 = 1,  /* svq_w4a16_gemm */
    SVQ_OP_MXFP8 = 2,  /* svq_mxfp8_gemm (group_size must be 32) */
    SVQ_OP_W8A16 = 3   /* svq_w8a16_gemm */
} svq_op;

int svq_abi_version(void);

/* Static text for a status code; never NULL. */
const char *svq_status_string(int status);

/* ---- W4A16 ------------------------------------------------------------------ */

/* Bytes of the repacked weight buffer: K*N/2 (the same as the GPTQ input). */
size_t svq_q4_repacked_bytes(int64_t N, int64_t K);

/*
 * One-time repack of GPTQ INT4 words into the device tile layout read by the
 * W4A16 kernels (a pure bit permutation; reads and writes K*N/2 bytes once).
 *   qweight_gptq  int32 [K/8][N]; nibble i (bits 4i..4i+3) of word [j][n] is
 *                 the code of row 8j+i, column n. 16-byte aligned.
 *   qweight_tiled int32, svq_q4_repacked_bytes(N, K) bytes, 16-byte aligned,
 *                 must not overlap qweight_gptq. Layout: tiles of 16 columns x
 *                 128 rows (1 KiB), column-block-major with the K-tiles of a
 *                 column block consecutive; lane l of a tile owns 16 bytes:
 *                 column 16*nb + l%16, word j = rows 128*kt + 32*(l/16) + 8*j
 *                 + e (e = 0..7) with row e in nibble slot p, e = (0,2,4,6,
 *                 1,3,5,7)[p].
 * Requires N % 16 == 0, K % 128 == 0.
 */
int svq_q4_repack(const int32_t *qweight_gptq, int32_t *qweight_tiled, int64_t N,
                  int64_t K, void *stream);

/* Most projections svq_fuse_projections takes in one call. */
#define SVQ_MAX_FUSED_PARTS 16

/*
 * Setup-time projection fusion: `parts` quantized projections that read the
 * same x (same K, same format, same group size) become one projection whose
 * output columns are the parts' columns in the order given, so a single GEMM
 * call replaces `parts` calls and y_fused = [y_0 | y_1 | ...] (Eole recipe
 * "Qwen3.8-27B and native MTP speculative decoding", section "Pack inference
 * projections": K/V/Q and gate/up are packed at setup, before the repack, with
 * no requantization; projections that do not fit stay separate -- here the
 * call returns an error and changes nothing, and the caller keeps them).
 *   bits 4: weights[p]   GPTQ int32 words [K/8][widths[p]], 4-byte aligned;
 *           weight_fused the REPACKED fused weight (the svq_q4_repack layout of
 *                        the concatenated words), K*N/2 bytes, 16-byte aligned,
 *                        ready for svq_w4a16_gemm with N = sum of widths
 *   bits 8: weights[p]   int8 codes [widths[p]][K], 16-byte aligned;
 *           weight_fused int8 [N][K], 16-byte aligned (svq_w8a16_gemm input)
 *   scales[p]     fp16 [K/G][widths[p]], 2-byte aligned
 *   scales_fused  fp16 [K/G][N]; 4-byte aligned if it feeds a GEMM
 *   weights, scales, widths: host arrays of `parts` entries (device pointers
 *   and column counts), 1 <= parts <= SVQ_MAX_FUSED_PARTS, read during the
 *   call only. Requires every width % 16 == 0, K % 128 == 0, G in {32, 64,
 *   128}, K % G == 0. The outputs must not overlap any input or each other
 *   (inputs may overlap one another). Reads and writes every byte once, in one
 *   launch.
 */
int svq_fuse_projections(int32_t bits, const void *const *weights, const void *const *scales,
                         const int64_t *widths, int32_t parts, int64_t K, int32_t group_size,
                         void *weight_fused, void *scales_fused, void *stream);

/*
 * Compressed-tensors W4A16 ingest: words [N][K/8] and scales [N][K/G] become
 * the GPTQ layout [K/8][N] and [K/G][N] by transposition, every word and scale
 * unchanged (Eole recipe, section "Compressed-tensors INT4 layout": the
 * converter transposes packed words and scales and does not requantize). The
 * nibble order is the GPTQ one: nibble i of word [n][j] is the code of row
 * 8j + i of column n.
 *   weight_packed int32 [N][K/8], 4-byte aligned
 *   weight_scale  fp16 [N][K/G], 2-byte aligned
 *   qweight       int32 [K/8][N], 4-byte aligned (the svq_q4_repack input)
 *   scales        fp16 [K/G][N], 2-byte aligned
 *   group_size    G in {32, 64, 128}; K % G == 0 (any N >= 1)
 * Outputs must not overlap the inputs or each other. Words and scales are
 * transposed in one launch.
 */
int svq_ct_to_gptq(const int32_t *weight_packed, const void *weight_scale, int32_t *qweight,
                   void *scales, int64_t N, int64_t K, int32_t group_size, void *stream);

/* Workspace bytes needed by svq_w4a16_gemm (kernel = SVQ_KERNEL_AUTO) or by
 * svq_w4a16_gemm_with for the given kernel; 0 if none. (size_t)-1 if the
 * arguments are invalid or the kernel cannot run the shape. */
size_t svq_w4a16_workspace_bytes(int kernel, int64_t M, int64_t N, int64_t K,
                                 int32_t group_size);

/*
 * y = x . ((q - 8) * s)^T, the W4A16 linear layer: symmetric INT4 with zero
 * point 8, one fp16 scale per group of G K-rows, no group reordering (GPTQ
 * INT4 card "Qwen3.8-27B-GPTQ-Int4-sym-G128-MTP-BF16", section "Quantization
 * contract": INT4, symmetric, group 128, desc_act off, packed int32; Eole
 * recipe, section "Compressed-tensors INT4 layout": groups of 32, 64 or 128).
 * Products are accumulated in fp32 and y is rounded to bf16 (nearest even).
 *   x             bf16 [M][K], 16-byte aligned
 *   qweight_tiled output of svq_q4_repack, 16-byte aligned
 *   scales        fp16 [K/G][N], 4-byte aligned (read as aligned 32-bit words)
 *   out           bf16 [M][N], 4-byte aligned, fully overwritten, must not
 *                 overlap any input or the workspace
 *   group_size    G in {32, 64, 128}; K % 128 == 0, N % 16 == 0
 *   workspace     device buffer of at least svq_w4a16_workspace_bytes(...)
 *                 bytes, 256-byte aligned, ZERO-FILLED before its first use;
 *                 the kernels leave it zero-filled again where it matters
 *                 (split-K arrival counters). NULL/0 when 0 bytes are needed.
 *                 Calls that share a workspace must be stream-ordered.
 */
int svq_w4a16_gemm(const void *x, const int32_t *qweight_tiled, const void *scales,
                   void *out, int64_t M, int64_t N, int64_t K, int32_t group_size,
                   void *workspace, size_t workspace_bytes, void *stream);

/* Same, with an explicit kernel choice; SVQ_ERR_UNSUPPORTED if that kernel
 * cannot run M (SVQ_KERNEL_DOT2: M <= 8; SVQ_KERNEL_MFMA_SKINNY: M <= 16). */
int svq_w4a16_gemm_with(int kernel, const void *x, const int32_t *qweight_tiled,
                        const void *scales, void *out, int64_t M, int64_t N, int64_t K,
                        int32_t group_size, void *workspace, size_t workspace_bytes,
                        void *stream);

/* Name of the kernel the call would launch (static text), or NULL if invalid. */
const char *svq_w4a16_kernel_name(int kernel, int64_t M, int64_t N, int64_t K,
                                  int32_t group_size);

/* Size of the device scratch array svq_w4a16_gemm_noalloc uses on each device:
 * the 256 KiB counter region plus 32 MiB of fp32 partials. */
#define SVQ_NOALLOC_SCRATCH_BYTES ((size_t)(32u << 20) + (size_t)(256u << 10))

/*
 * svq_w4a16_gemm without a workspace argument, for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation. Same arguments, results and errors as
 * svq_w4a16_gemm with the automatic kernel choice (identical bits: the same
 * kernels run); the cross-workgroup reductions use a file-scope device array
 * of SVQ_NOALLOC_SCRATCH_BYTES that each device holds until the process ends.
 * It allocates nothing (no hipMalloc, hipFree or allocating library call).
 * Shapes whose workspace (svq_w4a16_workspace_bytes) exceeds the array return
 * SVQ_ERR_WORKSPACE before anything is enqueued. The first call on a device
 * looks the array up and enqueues one small fill kernel on `stream` that
 * clears its counter region. All calls on one device share the array and each
 * call leaves it as the last call wrote it: calls that overlap in time on one
 * device race and must be ordered by the caller (one stream, or events).
 */
int svq_w4a16_gemm_noalloc(const void *x, const int32_t *qweight_tiled, const void *scales,
                           void *out, int64_t M, int64_t N, int64_t K, int32_t group_size,
                           void *stream);

/* ---- MXFP8 ------------------------------------------------------------------ */

/*
 * One-time repack of E4M3 codes into the device tile layout read by the MXFP8
 * GEMM kernels (a byte permutation; reads and writes N*K bytes once; the
 * pages repack weights once at setup, Eole recipe "Qwen3.8-27B and native MTP
 * speculative decoding", section "Pack inference projections").
 *   w        E4M3FN codes [N][K] (row n holds the K elements of output column
 *            n), 16-byte aligned
 *   w_tiled  N*K bytes, 16-byte aligned, must not overlap w. Layout: tiles of
 *            16 columns x 128 K-elements (2 KiB), column-block-major with the
 *            K-tiles of a block consecutive (tile (nb, kt) at byte
 *            2048*(nb*K/128 + kt)); byte 1024*h + 16*l + b of a tile holds
 *            column 16*nb + l%16, K-element 128*kt + 32*(l/16) + 16*h + b.
 * Requires N % 16 == 0, K % 128 == 0. The E8M0 scales keep their [N][K/32]
 * layout.
 */
int svq_mxfp8_repack(const uint8_t *w, uint8_t *w_tiled, int64_t N, int64_t K, void *stream);

size_t svq_mxfp8_workspace_bytes(int kernel, int64_t M, int64_t N, int64_t K);

/*
 * y = x . (e4m3(w) * 2^(e8m0(s) - 127))^T, the MXFP8 linear layer: OCP E4M3FN
 * elements with one E8M0 power-of-two scale per 32 consecutive K-elements
 * (MXFP8 card "Qwen3.8-27B-MXFP8-CT-AutoRound-mtp", opening summary and
 * section "8. License and attribution"); the kernel constraints N >= 128 and
 * K % 32 == 0 of its section "2. Precision plan" are checked and reported as
 * SVQ_ERR_MXFP8_SHAPE (its section "7. Known issues and caveats" records a
 * crash at N = 96). fp32 accumulation, bf16 (nearest even) output.
 *   x       bf16 [M][K], 16-byte aligned
 *   w       E4M3FN codes in the svq_mxfp8_repack tile layout (N*K bytes),
 *           16-byte aligned
 *   scales  E8M0 codes [N][K/32], one per 32 consecutive K-elements of a row,
 *           4-byte aligned (read as aligned 32-bit words)
 *   out     bf16 [M][N], 4-byte aligned, fully overwritten, no overlap
 *   group_size must be 32. Requires N >= 128, N % 16 == 0, K % 128 == 0.
 *   workspace as for svq_w4a16_gemm.
 * Element code 0x7F/0xFF (NaN) and scale code 255 (NaN) are not supported
 * inputs: the result for them is unspecified.
 */
int svq_mxfp8_gemm(const void *x, const uint8_t *w, const uint8_t *scales, void *out,
                   int64_t M, int64_t N, int64_t K, int32_t group_size, void *workspace,
                   size_t workspace_bytes, void *stream);

int svq_mxfp8_gemm_with(int kernel, const void *x, const uint8_t *w, const uint8_t *scales,
                        void *out, int64_t M, int64_t N, int64_t K, int32_t group_size,
                        void *workspace, size_t workspace_bytes, void *stream);

const char *svq_mxfp8_kernel_name(int kernel, int64_t M, int64_t N, int64_t K);

/*
 * MXFP8 quantization of a dense bf16 projection into the svq_mxfp8_gemm input,
 * as a model is quantized (MXFP8 card "Qwen3.8-27B-MXFP8-CT-AutoRound-mtp":
 * plain round-to-nearest, opening summary; the optimized round-to-nearest of
 * its notes on the quantizer, which evaluates the baseline block scale with
 * the scales twice and half as large and keeps the best). Per block of 32
 * consecutive K-elements of row n:
 *   baseline  X0 = floor(log2 amax) - 8, b0 = clamp(X0 + 127, 0, 254); an
 *             all-zero block takes b0 = 127
 *   candidate b: codes E4M3_RNE(|v| / 2^(b-127)) with the sign of v (-0 and
 *             negatives that round to zero give 0x80), saturating at 448;
 *             score = sum over the block, in ascending order, of fp32
 *             (v - decoded)^2 with round-to-nearest subtract, multiply, add
 *   optimized = 1: candidates b0, b0 + 1, b0 - 1 (those in 0..254); a later
 *             one is kept only with a strictly smaller score. optimized = 0:
 *             b0 (plain round-to-nearest).
 *   w       bf16 [N][K] (row n = output column n), 16-byte aligned, finite
 *   codes   E4M3FN [N][K], 16-byte aligned
 *   scales  E8M0 [N][K/32]
 * Requires K % 32 == 0 (svq_mxfp8_gemm further needs N >= 128, K % 128 == 0).
 * Outputs must not overlap w or each other. optimized outside {0, 1} returns
 * SVQ_ERR_UNSUPPORTED.
 */
int svq_mxfp8_quantize(const void *w, int32_t optimized, uint8_t *codes, uint8_t *scales, int64_t N,
                       int64_t K, void *stream);

/* ---- quantized vocabulary head (W8A16) and the load-time quantizer --------- */

/*
 * Symmetric group-wise round-to-nearest quantization of a dense projection,
 * done once when the model loads (Eole recipe, section "Optional
 * vocabulary-head quantization": int8 or int4, groups of 32, 64 or 128 along
 * K, symmetric, round to nearest). Per group of G consecutive K-elements of
 * row n, in fp32 with IEEE division:
 *     amax = max |w|,  s = fp16_rne(amax / qmax),  qmax = 127 (int8) or 7 (int4)
 *     q    = clamp(rint(w / s), -qmax - 1, qmax)   (rint: nearest, ties to even)
 * with s used as stored; a group whose stored s is 0 gets q = 0.
 *   w           bf16 [N][K] (row n = output column n), 16-byte aligned; finite values
 *   bits        8: codes = int8 [N][K] (two's complement), 16-byte aligned
 *               4: codes = GPTQ int32 words [K/8][N] holding q + 8, the W4A16
 *                  input of svq_q4_repack; 4-byte aligned
 *   scales      fp16 [K/G][N], 2-byte aligned
 *   group_size  G in {32, 64, 128}; K % G == 0
 * codes and scales must not overlap w or each other. Errors as for the GEMMs.
 */
int svq_rtn_quantize(const void *w, int32_t bits, int32_t group_size, void *codes, void *scales,
                     int64_t N, int64_t K, void *stream);

/* Workspace bytes needed by svq_w8a16_gemm; 0 if none, (size_t)-1 if invalid. */
size_t svq_w8a16_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t group_size);

/*
 * y = x . (q * s)^T for the int8 codes of svq_rtn_quantize, M <= 16
 * (SVQ_ERR_UNSUPPORTED above): the quantized vocabulary head (Eole recipe,
 * section "Optional vocabulary-head quantization"; the AWQ card
 * "Qwen3.8-27B-AWQ-INT4-MTP-LowLatency" measures the decode-latency gain of
 * a quantized head in its head-precision section). fp32 accumulation, bf16
 * (nearest even) output.
 *   x       bf16 [M][K], 16-byte aligned
 *   w       int8 codes [N][K], 16-byte aligned
 *   scales  fp16 [K/G][N], 4-byte aligned (read as aligned 32-bit words)
 *   out     bf16 [M][N], 4-byte aligned, fully overwritten, no overlap
 *   group_size G in {32, 64, 128}; K % 128 == 0, N % 16 == 0
 *   workspace as for svq_w4a16_gemm.
 */
int svq_w8a16_gemm(const void *x, const int8_t *w, const void *scales, void *out, int64_t M,
                   int64_t N, int64_t K, int32_t group_size, void *workspace,
                   size_t workspace_bytes, void *stream);

/* Name of the kernel svq_w8a16_gemm would launch (static text), or NULL. */
const char *svq_w8a16_kernel_name(int64_t M, int64_t N, int64_t K, int32_t group_size);

/* ---- per-request operators of a verify chunk ------------------------------------ */

/* Largest rank of svq_adapter_add. */
#define SVQ_MAX_ADAPTER_RANK 256

/* Workspace bytes needed by svq_adapter_add (never 0); (size_t)-1 if the
 * arguments are invalid. */
size_t svq_adapter_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t R, int32_t slots);

/*
 * Low-rank adapters of many requests at once, beside a projection that they
 * share: y = base is the output of any of the GEMMs above for the same x, and
 * every row adds its own adapter's product,
 *     out[m] = base[m] + scales[s] * B_s (A_s x[m]),   s = rows[m].
 * A row whose index is outside [0, slots) has no adapter: out[m] = base[m].
 * Products and sums are fp32, the rank-R intermediate too (all 24 bits of it enter
 * the second product), out is rounded to bf16 (nearest even) once. Rows are
 * independent: no row's result depends on another row or on an adapter that is
 * not its own.
 *   base     bf16 [M][ld_base], the first N columns of each row; 16-byte aligned
 *   x        bf16 [M][K], 16-byte aligned
 *   a        bf16 [slots][R][K], 16-byte aligned, finite (any size: 64-bit offsets)
 *   b        bf16 [slots][N][R], 16-byte aligned, finite
 *   rows     int32 [M], the adapter of each row
 *   scales   fp32 [slots]
 *   out      bf16 [M][ld_out], 16-byte aligned; its first N columns are written,
 *            the rest of each row is left as it was. May be base itself (same
 *            pointer, ld_out == ld_base) or other columns of the same matrix
 *            (ld_out == ld_base); otherwise the memory from the first to the last
 *            element of the one must not overlap the other's.
 *   ld_base, ld_out >= N, multiples of 8: the columns of one projection inside a
 *            fused output are addressed by their first column and the fused width
 * Requires N % 16 == 0, K % 128 == 0, R % 8 == 0, R <= SVQ_MAX_ADAPTER_RANK.
 * An adapter of a smaller rank is padded with zero rows of A and zero columns of B.
 *   workspace  at least svq_adapter_workspace_bytes(...) bytes, 256-byte aligned;
 *              it need not be cleared, and a workspace of the GEMMs may be passed
 *              (its arrival counters are left alone). Calls that share a workspace
 *              must be stream-ordered.
 */
int svq_adapter_add(const void *base, int64_t ld_base, const void *x, const void *a, const void *b,
                    const int32_t *rows, const float *scales, void *out, int64_t ld_out, int64_t M, int64_t N,
                    int64_t K, int32_t R, int32_t slots, void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes needed by svq_sample; 0 if none, (size_t)-1 if invalid. */
size_t svq_sample_workspace_bytes(int64_t M, int64_t V);

/*
 * One token per row of logits, as a vocabulary head writes them, from given
 * random numbers. A row's tokens stand in order of descending logit, equal ones
 * by ascending index (-0 equals +0). With w(i) = exp((l_i - max) / T) and W(n)
 * the sum of the first n:
 *     n1 = top_k tokens (all if top_k <= 0)
 *     n2 = the fewest tokens with W(n2) >= top_p W(n1)   (no limit if top_p >= 1)
 *     n3 = the tokens with w >= min_p                    (no limit if min_p <= 0)
 *     n  = the least of these, at least 1
 *     token = the first whose W, itself included, exceeds u W(n)
 *     logprob = ln of the probability of that token among the n
 * Weights and sums are fp64. temperature <= 0 (or NaN) takes the first token,
 * with logprob 0, whatever the other parameters. Logits that are NaN or -inf are
 * never drawn; among +inf ones the draw is uniform. A row with nothing to draw
 * gives token -1 and logprob -inf. u is clamped to [0, 1), NaN to 0.
 *   logits       bf16 [M][ld], the first V of each row; 2-byte aligned (rows of
 *                any alignment; 16-byte aligned rows are not faster)
 *   u            fp32 [M]
 *   temperature  fp32 [M], or NULL for 1
 *   top_k        int32 [M], or NULL for no limit
 *   top_p, min_p fp32 [M], or NULL for no limit
 *   tokens       int32 [M]
 *   logprobs     fp32 [M], or NULL
 * Requires ld >= V; the logits may pass 2 GiB. Outputs must not overlap each
 * other, the inputs or the workspace (svq_sample_workspace_bytes(...) bytes,
 * 256-byte aligned, as for svq_adapter_add; NULL/0 when 0 bytes are needed).
 */
int svq_sample(const void *logits, int64_t ld, const float *u, const float *temperature, const int32_t *top_k,
               const float *top_p, const float *min_p, int32_t *tokens, float *logprobs, int64_t M, int64_t V,
               void *workspace, size_t workspace_bytes, void *stream);

/*
 * Acceptance of drafted tokens (Eole recipe, opening paragraph: the main model
 * verifies a chunk of drafted tokens). Sequence s owns rows starts[s] ..
 * starts[s+1] - 1 of the chunk: the first row's input is its last committed
 * token, the others' inputs are its drafts. tokens are what the main model
 * sampled at each row (svq_sample). A draft is accepted if it and all drafts
 * before it equal the token sampled one row earlier:
 *     n    = number of leading rows i with tokens[i] == inputs[i + 1]
 *     next = tokens[starts[s] + n], the token that follows the accepted drafts
 * For drafts that are given tokens this is speculative sampling: drawing t from
 * p and accepting a draft d when t == d accepts with probability p(d), and
 * otherwise t is distributed as p without d.
 *   tokens, inputs  int32 [M]; a negative token (nothing to draw) accepts nothing
 *   starts          int32 [S + 1], ascending, in [0, M] (values outside are clamped
 *                   to it); a sequence may be empty
 *   accepted, next  int32 [S]; an empty sequence gets 0 and -1
 *   committed       int32 [M]: the accepted drafts and then next at the first
 *                   n + 1 rows of each sequence, -1 at its other rows and at rows
 *                   outside every sequence
 * Outputs must not overlap the inputs or each other.
 */
int svq_accept_drafts(const int32_t *tokens, const int32_t *inputs, const int32_t *starts, int32_t *accepted,
                      int32_t *next, int32_t *committed, int64_t M, int64_t S, void *stream);

/* ---- a tree of drafted tokens over a cache ---------------------------------------- */

/*
 * A verify chunk may branch: the rows of a sequence are the nodes of a tree. Its first
 * row is the root (the last committed token) and every other row's input is a draft
 * that follows its parent. The operators below share these arguments:
 *   starts   int32 [S + 1], ascending, in [0, M] (values outside are clamped to it):
 *            sequence s owns rows starts[s] .. starts[s+1] - 1; it may be empty
 *   parents  int32 [M]: the parent of each row, counted from the sequence's first row
 *            and smaller than the row's own number; anything else is no parent. NULL
 *            (where allowed): a chain, every row's parent is the row before it
 *   lengths  int32 [S]: committed tokens before the sequence's first row
 * The path of a row is its ancestors and itself; its depth is the number of ancestors,
 * its position lengths[s] + depth.
 */

/* Types of cached keys and values. */
#define SVQ_CACHE_BF16 0
#define SVQ_CACHE_E4M3 1 /* OCP E4M3FN codes */

/* Keys and values of committed tokens, in pages that sequences hold by table. */
typedef struct svq_kv_cache {
    const void *k, *v;     /* token t, head h of page p at element
                              p*strides[0] + t*strides[1] + h*strides[2]; D contiguous
                              elements, 16-byte aligned (pointers and strides) */
    int64_t k_strides[3];  /* page, token, head; in elements. Pages and tokens lie less than
                              4 GiB apart; of a single one the stride is not used */
    int64_t v_strides[3];
    int64_t pages;         /* pages in the pool; with none k and v may be NULL */
    int32_t page_size;     /* tokens in a page, 1 .. 2^20 */
    int32_t type;          /* SVQ_CACHE_* */
    const float *k_scale;  /* E4M3: fp32 [KVH], positive; a cached value is code * scale; */
    const float *v_scale;  /* NULL for 1. BF16: both NULL */
    const int32_t *page_table; /* int32 [S][ld_table], the first max_pages of each row: the
                              pages of a sequence in order. Tokens of an entry outside
                              [0, pages) are not seen */
    int64_t ld_table;
    int32_t max_pages;     /* with none page_table may be NULL */
    const int32_t *lengths; /* int32 [S], clamped to [0, max_pages * page_size] */
} svq_kv_cache;

/* Workspace bytes needed by svq_tree_attention (never 0); (size_t)-1 if the arguments
 * are invalid. */
size_t svq_tree_attention_workspace_bytes(int64_t M, int64_t S, int32_t H, int32_t KVH, int32_t D);

/*
 * Attention of every row of a chunk to its sequence's cache and to its own path:
 *     out[m][h] = sum_j w_j v_j / sum_j w_j,   w_j = exp(scale * q[m][h] . k_j)
 * over the tokens j that row m sees, heads h of group h / (H / KVH) sharing one key and
 * value head. A row at position p sees of the cache and of its path the tokens at
 * positions > p - window and those < sinks; window <= 0 is no limit. The chunk's own
 * keys and values are rows beside q, not in the cache: what is accepted is written to
 * the cache afterwards. A score of -inf has weight zero; a row that sees nothing, or
 * only such scores, is zero. Rows outside every sequence are left as they were. What a
 * row does not see, infinities and NaN too, does not change its result. What it sees does,
 * whatever its weight: a value that is infinite or NaN leaves its column of the row infinite
 * or NaN. (Which of the two follows IEEE sums where its weight is in fp32's range; where it is
 * smaller, or 0, it may be either.) With starts that do not ascend nothing is written.
 * Scores, weights' sums and products are fp32; weights enter the second product as bf16;
 * out is rounded to bf16 (nearest even).
 *   q        bf16 [M][ld_q], the first H*D of each row: H heads of D elements
 *   k, v     bf16 [M][ld_k], [M][ld_v], the first KVH*D of each row
 *   cache    host struct, read during the call only
 *   starts, parents (or NULL): above
 *   out      bf16 [M][ld_out], the first H*D of each row are written
 *   q, k, v, out 16-byte aligned, their row strides multiples of 8 and at least the
 *   columns used. D is 64, 128 or 256, H a multiple of KVH, H <= 65536.
 *   workspace  at least svq_tree_attention_workspace_bytes(...) bytes, 256-byte aligned,
 *              not cleared; as for svq_adapter_add.
 * out and the workspace must not overlap any input or each other (out, q, k and v may be
 * different columns of one matrix). KVH times the tiles of 64 tokens that a sequence may have
 * (max_pages * page_size and M) times the blocks of 16 (row, head of a group) pairs must stay
 * below 2^31 (SVQ_ERR_DIM).
 */
int svq_tree_attention(const void *q, int64_t ld_q, const void *k, int64_t ld_k, const void *v, int64_t ld_v,
                       const svq_kv_cache *cache, const int32_t *starts, const int32_t *parents, float scale,
                       int32_t window, int32_t sinks, void *out, int64_t ld_out, int64_t M, int64_t S, int32_t H,
                       int32_t KVH, int32_t D, void *workspace, size_t workspace_bytes, void *stream);

/* What svq_adjust_logits changes; a NULL pointer leaves its part out. */
typedef struct svq_adjustments {
    const int32_t *history;        /* int32 [S][ld_history]: committed tokens before a chunk */
    int64_t ld_history;
    int32_t max_history;           /* lengths are clamped to [0, max_history] */
    const int32_t *lengths;        /* int32 [S] */
    const int32_t *prompt_lengths; /* int32 [S]: that many of them are the prompt's; NULL for 0 */
    const int32_t *inputs;         /* int32 [M]: the input of each row */
    const int32_t *parents;        /* int32 [M], or NULL for chains */
    const float *repetition;       /* fp32 [S], positive; NULL for 1 */
    const float *presence;         /* fp32 [S]; NULL for 0 */
    const float *frequency;        /* fp32 [S]; NULL for 0 */
    const int32_t *bias_starts;    /* int32 [S + 1], ascending, clamped to [0, biases] */
    const int32_t *bias_tokens;    /* int32 [biases] */
    const float *bias_values;      /* fp32 [biases] */
    int64_t biases;
    const int32_t *allowed;        /* int32 [masks][ld_allowed], at least one mask: bit v % 32 of word
                                      v / 32 is 1 if token v may follow */
    int64_t ld_allowed, masks;
    const int32_t *mask_rows;      /* int32 [M]: the mask of each row; outside [0, masks): none */
} svq_adjustments;

/*
 * Logits as the sampler takes them, from those of the vocabulary head, by what stands
 * before each row: the sequence's history and the inputs of the row's path. For token v
 * of row m of sequence s, with c its number of occurrences in the history after the
 * prompt and on the path:
 *     x = logit;  if v occurs in the history or on the path: x = x > 0 ? x / r : x * r
 *     x = x - frequency * c - (c > 0 ? presence : 0)
 *     x = x + the biases of v in s, in their order
 *     x = -inf if the row's mask has v's bit clear
 * in fp32, rounded to bf16 (nearest even) once; r is applied as a product with r or with
 * 1 / r, rounded to fp32. A logit that nothing applies to keeps its bits. Tokens outside
 * [0, V) are passed over. Rows outside every sequence are left as they were.
 *   logits   bf16 [M][ld], the first V of each row; 2-byte aligned
 *   out      bf16 [M][ld_out]; may be logits itself (same pointer and stride) or other columns
 *            of the same matrix, and must otherwise not overlap any input
 */
int svq_adjust_logits(const void *logits, int64_t ld, const int32_t *starts, const svq_adjustments *adjustments,
                      void *out, int64_t ld_out, int64_t M, int64_t S, int64_t V, void *stream);

/*
 * Acceptance along a tree (svq_accept_drafts for chunks that branch): from the
 * sequence's first row on, while a child's input is the token sampled at the current
 * node, the first such child (the lowest row) is accepted and becomes the current node.
 *   tokens, inputs  int32 [M]: the sample and the input of each row; a negative token
 *                   accepts nothing
 *   parents, starts as above
 *   accepted, next  int32 [S]: the number n of accepted drafts and the token sampled at
 *                   the last of them; an empty sequence gets 0 and -1
 *   committed       int32 [M]: the accepted drafts and then next at the first n + 1 rows
 *                   of each sequence, -1 elsewhere
 *   path            int32 [M]: at the same places the nodes whose samples these are,
 *                   counted from the sequence's first row (0 first), -1 elsewhere: the
 *                   rows whose keys and values belong into the cache
 * Outputs must not overlap the inputs or each other.
 */
int svq_accept_tree(const int32_t *tokens, const int32_t *inputs, const int32_t *parents, const int32_t *starts,
                    int32_t *accepted, int32_t *next, int32_t *committed, int32_t *path, int64_t M, int64_t S,
                    void *stream);

/* ---- format-generic queries ---------------------------------------------------- */

/* Workspace bytes the GEMM of `op` (an svq_op) needs with its automatic kernel
 * choice: svq_w4a16_workspace_bytes(SVQ_KERNEL_AUTO, ...),
 * svq_mxfp8_workspace_bytes(SVQ_KERNEL_AUTO, ...) (group_size must be 32) or
 * svq_w8a16_workspace_bytes(...). (size_t)-1 for an unknown op or invalid
 * arguments. */
size_t svq_workspace_bytes(int op, int64_t M, int64_t N, int64_t K, int32_t group_size);

/* Name of the kernel the GEMM of `op` would launch for this shape (static
 * text), or NULL for an unknown op or invalid arguments. */
const char *svq_kernel_name(int op, int64_t M, int64_t N, int64_t K, int32_t group_size);

/* ---- measurement ---------------------------------------------------------------- */

/*
 * Launch shape of a GEMM call: the grid (workgroups), workgroup size (threads)
 * and dynamic LDS bytes the call would launch with, for op (an svq_op) and
 * kernel (an svq_kernel; SVQ_KERNEL_AUTO only for SVQ_OP_W8A16). Nothing is
 * launched. Returns the status the call would return for valid buffers.
 */
int svq_launch_geometry(int op, int kernel, int64_t M, int64_t N, int64_t K, int32_t group_size,
                        uint64_t *grid, uint32_t *threads, size_t *lds_bytes);

/*
 * Streaming probe: reads `bytes` (a non-zero multiple of 16) from src (16-byte
 * aligned) in `grid` workgroups of `threads` threads (a multiple of 64, at most
 * 1024), each workgroup one contiguous share, and does nothing with them. It
 * measures the bandwidth a plain read of that many bytes reaches in that
 * launch shape: the ceiling of a GEMM's weight stream. sink (grid words, 4-byte
 * aligned) may be written with data-dependent values; nothing else is.
 */
int svq_stream_probe(const void *src, size_t bytes, uint32_t grid, uint32_t threads, uint32_t *sink,
                     void *stream);

/*
 * Matrix-core probe: every wave of `grid` workgroups of `threads` threads (a
 * multiple of 64, at most 1024) issues `per_wave` bf16 16x16x32 MFMAs (a
 * non-zero multiple of 8, at most 2^24) as eight independent chains on
 * register operands, with no memory traffic: the floor that MFMA issue sets
 * for a kernel doing that many MFMAs per wave in that launch shape (the
 * compute-bound batched-verify case of the autobench page "Qwen3.8-27B · vLLM ·
 * FP8 + MTP"). operands: 0 = constant (one small value in every register: the
 * issue floor at the clock the chip holds when the multipliers' inputs never
 * change), 1 = random (per chain: A random bf16 like activations, B the bf16 of
 * 128 + q for random nibbles q, the W4A16 weight operand; the matrix cores'
 * power draw then lowers the shader clock as real data does); anything else
 * is SVQ_ERR_DIM. sink (grid floats, 4-byte aligned) may be written with
 * data-dependent values; nothing else is.
 */
int svq_mfma_probe(uint32_t grid, uint32_t threads, uint32_t per_wave, int32_t operands, float *sink,
                   void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SVQ_H */
