/*
 * w4a16.h -- C ABI of the GB300 (sm_103a) W4A16 weight-only INT4 library.
 *
 * The library computes y = x * W^T for fp16 activations x [M, K] and weights
 * W [N, K] stored as symmetric INT4 in groups of 128 along K with one fp16
 * scale per group: the dequantize-on-the-fly product that dominates
 * memory-bound single-batch LLM decode ("W4A16 量化算子解码性能基准跑分与端侧大模型
 * 推理显存实测报告", mhpq.cn, §二 and §五), together with the group-wise
 * round-to-nearest quantizer that produces the packed weights ("LLM
 * quantization from IEEE 754 to GPTQ/AWQ/GGUF" tutorial, qaqbuyan.com
 * article 126, chapter "量化的数学基石" §2 formula and §3
 * per_group_symmetric_quantize / per_group_symmetric_dequantize).  Around the
 * linear layers it has the operators that a decoding program needs between
 * them: a paged key-value cache, the attention of a new token over it, the
 * care of its pages, and the scores of sampled tokens.
 *
 * Conventions for every entry point
 *  - Pointers are DEVICE pointers owned by the caller (for example a torch
 *    tensor's data_ptr()); the library never allocates, frees or keeps them.
 *    Every pointer must be 16-byte aligned.  Tensors are dense and row-major.
 *  - `stream` is a cudaStream_t passed as void*; NULL means the legacy
 *    default stream.  Work is enqueued asynchronously on it; the call returns
 *    without synchronising.  Calls on one stream execute in order.
 *  - Argument errors are reported synchronously, before anything is
 *    launched, as a w4a16_status code; nothing is written in that case.
 *  - A device-side failure (a bounded wait inside a kernel that gave up) is
 *    recorded in a device status word, readable with w4a16_device_status().
 *  - All kernels are built for sm_103a only; on another device the calls
 *    return W4A16_ERR_DEVICE.
 *  - The library keeps no state across calls other than the device status
 *    word and per-device launch attributes set on first use (first use on a
 *    device should happen before any CUDA graph capture).
 */
#ifndef W4A16_H
#define W4A16_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum w4a16_status {
    W4A16_OK = 0,
    W4A16_ERR_NULL = 1,      /* a required pointer is NULL                    */
    W4A16_ERR_SHAPE = 2,     /* unsupported M, N, K or group size             */
    W4A16_ERR_ALIGN = 3,     /* a pointer is not 16-byte aligned              */
    W4A16_ERR_CUDA = 4,      /* a CUDA runtime call or launch failed          */
    W4A16_ERR_TIMEOUT = 5,   /* a kernel's bounded wait gave up (device)      */
    W4A16_ERR_DEVICE = 6     /* current device is not an sm_103 GPU           */
} w4a16_status;

/* Group size along K: one fp16 scale per 128 consecutive weights of a row. */
#define W4A16_GROUP 128

/* Human-readable name of a status code (static string, never NULL). */
const char *w4a16_status_string(int status);

/* Library ABI version (major * 100 + minor). */
int w4a16_version(void);

/*
 * w4a16_quantize -- group-wise symmetric round-to-nearest INT4 quantizer.
 *
 * Source: qaqbuyan.com tutorial, "量化的数学基石" §2 (x_q = clamp(round(x / s),
 * -8, 7), s = max|x| / 7) and §3 per_group_symmetric_quantize (groups along
 * in_features, clamp(min = 1e-8) on the scale, two nibbles per byte with the
 * even index in the low nibble, each stored as q + 8, scales cast to fp16).
 *
 * For each row n and group g of 128 weights, in IEEE binary32 on the exactly
 * upcast fp16 inputs:
 *     s32 = max(max_k |W[n,k]| / 7, 1e-8)             (correctly rounded /)
 *     q   = clamp(round_half_even(W[n,k] / s32), -8, 7)
 *     scales[n, g] = fp16_round_nearest_even(s32)
 *     qweight[n, k/2] = (q[k+1] + 8) << 4 | (q[k] + 8)   for even k
 *
 *   W_f16      [N, K] fp16, row-major (rows are output features).  Finite.
 *   N, K       N >= 1; K >= 128 and K % 128 == 0.
 *   group      must be 128 (W4A16_GROUP).
 *   qweight    [N, K/2] bytes, written (the canonical packed layout).
 *   scales_f16 [N, K/128] fp16, written.
 * The result is bit-identical to the library's CPU reference definition.
 * Errors: NULL -> W4A16_ERR_NULL; bad N, K or group -> W4A16_ERR_SHAPE;
 *         misaligned pointer -> W4A16_ERR_ALIGN.
 */
int w4a16_quantize(const void *W_f16, int64_t N, int64_t K, int32_t group, void *qweight,
                   void *scales_f16, void *stream);

/* group argument of the format variants: one group spanning each row. */
#define W4A16_GROUP_PER_CHANNEL (-1)

/*
 * w4a16_quantize_ex -- format variants of the quantizer: other group sizes
 * and asymmetric INT4 with a zero point per group.
 *
 * Source: the same tutorial chapter, §3 granularity (per-channel, per-group
 * 128 and 32) and §2 asymmetric formula x_q = clamp(round(x / s) + z, 0, 15),
 * s = (max - min) / 15, z = -round(min / s).
 *
 * Per row n and group g, in IEEE binary32 on the exactly upcast inputs:
 *   symmetric   as w4a16_quantize with the given group; the nibble holds q + 8.
 *   asymmetric  lo = min(0, min_k W), hi = max(0, max_k W) over the group
 *               (0 is kept in range so that z, the code of 0.0, is a 4-bit
 *               code); s32 = max((hi - lo) / 15, 1e-8);
 *               z = -round_half_even(lo / s32), in [0, 15];
 *               q = clamp(round_half_even(W / s32) + z, 0, 15);
 *               the nibble holds q; zeros_u8[n, g] = z.
 *   scales_f16[n, g] = fp16_round_nearest_even(s32).
 *
 *   group      32, 64, 128, or W4A16_GROUP_PER_CHANNEL (one group of K).
 *   asymmetric 0 (symmetric) or 1.
 *   qweight    [N, K/2] bytes (low nibble = even k), written.
 *   scales_f16 [N, K/group] fp16, written.
 *   zeros_u8   [N, K/group] bytes, written when asymmetric (may be NULL
 *              otherwise).
 * Group 128 symmetric is exactly w4a16_quantize.  The results are
 * bit-identical to the library's CPU reference definition.
 * Errors: as w4a16_quantize; a group other than the above -> W4A16_ERR_SHAPE.
 */
int w4a16_quantize_ex(const void *W_f16, int64_t N, int64_t K, int32_t group, int32_t asymmetric,
                      void *qweight, void *scales_f16, void *zeros_u8, void *stream);

/*
 * Bytes of the kernel layout produced by w4a16_repack for an [N, K] weight:
 * N rounded up to a multiple of 128, times K/2.  Returns -1 on a bad shape.
 */
int64_t w4a16_repacked_bytes(int64_t N, int64_t K);

/*
 * w4a16_repack -- one-time re-layout of canonical packed weights into the
 * kernel layout read by w4a16_gemm (a pure permutation of nibbles; rows
 * beyond N are padded with nibble 8, i.e. q = 0).
 *
 * The tutorial's packed layout is row-major [N, K/2]; its "block-major"
 * cache-friendly re-layout advice (qaqbuyan.com, llama.cpp tuning section)
 * motivates this step, but the exact layout is the library's own:
 *   block b = n / 128 (128 rows), chunk c = k / 64, tile i = (n % 128) / 16;
 *   512 bytes per (b, c, i), 16 bytes per lane L = 4 * g + t of a warp,
 *   holding rows 16 i + g and 16 i + g + 8 at k = 64 c + 16 t ... + 15.
 *   byte offset = ((b * (K/64) + c) * 8 + i) * 512 + 16 * L.
 *   Within the lane's 16 bytes, 32-bit word s covers k' = 64c + 16t + 4s
 *   .. k' + 3; its nibble positions 0..7 hold (row, k) =
 *   (r0,k'), (r1,k'), (r0,k'+2), (r1,k'+2), (r0,k'+1), (r1,k'+1),
 *   (r0,k'+3), (r1,k'+3) with r0 = 16 i + g and r1 = r0 + 8,
 *   so one lop3 per nibble pair yields the f16 MMA fragment directly.
 *
 *   qweight   [N, K/2] canonical bytes (from w4a16_quantize).
 *   repacked  w4a16_repacked_bytes(N, K) bytes, written.
 * Errors: as w4a16_quantize.  unrepack(repack(P)) == P byte for byte.
 */
int w4a16_repack(const void *qweight, int64_t N, int64_t K, void *repacked, void *stream);

/* Inverse of w4a16_repack: kernel layout -> canonical [N, K/2] bytes. */
int w4a16_unrepack(const void *repacked, int64_t N, int64_t K, void *qweight, void *stream);

/*
 * w4a16_gemm -- y[M, N] = x[M, K] * dequant(W)[N, K]^T.
 *
 * Source: mhpq.cn report §二/§五 (dequantize in registers on the fly, never
 * materialise the fp16 weights; the decode step is memory-bound) and the
 * qaqbuyan.com tutorial §3 dequantizer: W[n, k] = (nibble - 8) * scale[n, k/128].
 *
 *   x_f16      [M, K] fp16 activations.
 *   repacked   weights in the kernel layout (w4a16_repack).
 *   scales_f16 [N, K/128] fp16 scales (canonical layout, as quantized).
 *   y_f16      [M, N] fp16 output, written (FP32 accumulation, rounded to
 *              nearest-even fp16 once at the end).
 *   M          1..16 runs the decode GEMV (warp MMAs fed by a bulk-copy
 *              shared-memory ring); M > 16 runs the tcgen05 tensor-core GEMM
 *              (fp16 q*scale staged in shared memory, FP32 accumulators in
 *              tensor memory).
 *   N, K       N >= 1; K >= 128 and K % 128 == 0.
 * Accuracy against the exact result: max|y - y_ref| <= 2e-3 * max|y_ref|
 * and ||y - y_ref||_2 <= 1e-3 * ||y_ref||_2 for the library's test inputs.
 * The call is graph-capturable and uses programmatic dependent launch.
 * Weights and scales are read as constants of the call: their first tiles
 * may be loaded while the kernel enqueued before it on the stream is still
 * running (x is read and y written only after that kernel completes).  So
 * the weights and scales must not be written by work that is still pending
 * on the stream when w4a16_gemm is enqueued -- synchronise (or wait on an
 * event) after writing them -- except by w4a16_quantize and w4a16_repack,
 * which make their results visible before they finish.
 * Errors: NULL -> W4A16_ERR_NULL; bad M, N, K -> W4A16_ERR_SHAPE;
 *         misaligned pointer -> W4A16_ERR_ALIGN; launch failure ->
 *         W4A16_ERR_CUDA.
 */
int w4a16_gemm(const void *x_f16, const void *repacked, const void *scales_f16, void *y_f16,
               int64_t M, int64_t N, int64_t K, void *stream);

/*
 * w4a16_gemm_ex -- w4a16_gemm for the format variants of w4a16_quantize_ex,
 * with an optional AWQ activation scale:
 *   y[m, n] = sum_k x~[m, k] * (nib[n, k] - z[n, k/g]) * scale[n, k/g],
 * z = zeros_u8[n, k/g] for asymmetric codes, z = 8 for symmetric codes
 * (zeros_u8 NULL); x~ = x, or x~[m, k] = fp16_rne(x[m, k] * alpha[k]) when
 * alpha_f16 is given.  Source: tutorial §2 symmetric / asymmetric formulas,
 * §3 granularity and its AWQ section (x~_j = x_j alpha_j against weights
 * quantized from W_{:,j} / alpha_j; the alpha search is the caller's);
 * report §二/§五 for the decode product.
 *
 *   alpha_f16  [K] fp16 per-input-channel scale, or NULL.
 *   repacked   w4a16_repack of the variant's packed codes (the layout does
 *              not depend on the format).
 *   scales_f16 [N, K/g] fp16; zeros_u8 [N, K/g] bytes or NULL.
 *   group      32, 64, 128 or W4A16_GROUP_PER_CHANNEL (g = K).
 *   M          1 .. 2^22.  M <= 16 runs the variant decode GEMV while
 *              x[M, K] fits in its shared memory beside the weight ring
 *              (about 2 * M * K <= 200 KB: M = 1 any K up to 32768, M = 16
 *              K up to 6144); larger M, or a shape that does not fit, runs
 *              the tcgen05 tensor-core GEMM of w4a16_gemm with the variant's
 *              dequantisers.  There alpha multiplies the fp16 dequantised
 *              weight instead of x: y[m, n] = sum_k x[m, k] *
 *              fp16(fp16((nib - z) * scale) * alpha[k]), the same product
 *              with its rounding on the weight operand.
 * Group 128 with symmetric codes and no alpha runs w4a16_gemm's kernels
 * (exact q * x products, one FP32 rescale per group).  The other calls dequantise
 * (nib - z) * scale once to fp16 per weight (the tutorial's own fp16
 * dequantised weight) and accumulate in FP32; the accuracy bar is the same.
 * Errors: as w4a16_gemm; a group other than the above -> W4A16_ERR_SHAPE.
 */
int w4a16_gemm_ex(const void *x_f16, const void *alpha_f16, const void *repacked,
                  const void *scales_f16, const void *zeros_u8, void *y_f16, int64_t M,
                  int64_t N, int64_t K, int32_t group, void *stream);

/*
 * w4a16_quantize_q4_0 -- weights in GGUF Q4_0 blocks.
 *
 * Source: tutorial GGUF section (a Q4_0 block: 32 weights in 18 bytes, d as
 * little-endian fp16, then 16 bytes whose byte i holds element 2i in its low
 * nibble and 2i + 1 in its high nibble, decoded as (nibble - 8) * d); the
 * codes are the §2 / §3 symmetric quantizer with groups of 32 (the pages
 * give the block's decoder, not a separate quantizer), i.e. exactly
 * w4a16_quantize_ex(group 32, symmetric) laid out block after block.
 *
 *   W_f16      [N, K] fp16.  N >= 1; K >= 256, K % 256 == 0 (rows of whole
 *              16-byte lines for the GEMV's copies).
 *   blocks_u8  [N, K/32 * 18] bytes, written; block b of row n at byte
 *              (n * K/32 + b) * 18.
 * Bit-identical to the library's CPU reference definition.
 * Errors: NULL -> W4A16_ERR_NULL; bad N, K -> W4A16_ERR_SHAPE; misaligned
 *         pointer -> W4A16_ERR_ALIGN.
 */
int w4a16_quantize_q4_0(const void *W_f16, int64_t N, int64_t K, void *blocks_u8, void *stream);

/*
 * w4a16_gemm_q4_0 -- decode GEMV on Q4_0 blocks:
 *   y[m, n] = sum_b d[n, b] * sum_{i<32} x[m, 32 b + i] * (nib[n, 32 b + i] - 8),
 * exact q * x products, one FP32 rescale per block, y rounded once to fp16.
 * M = 1..16; K % 256 == 0; x[M, K] held in shared memory whole (as
 * w4a16_gemm_w8).  Errors: as w4a16_gemm_w8.
 */
int w4a16_gemm_q4_0(const void *x_f16, const void *blocks_u8, void *y_f16, int64_t M, int64_t N,
                    int64_t K, void *stream);

/*
 * w4a16_quantize_w8 -- W8A16 weights: per-channel symmetric INT8.
 *
 * Source: tutorial "量化的数学基石" §2 formula with b = 8 and its INT8
 * section ("per-channel, 对称").  Per row n, in IEEE binary32 on the exactly
 * upcast inputs:
 *     s32 = max(max_k |W[n, k]| / 127, 1e-8)          (correctly rounded /)
 *     q   = clamp(round_half_even(W[n, k] / s32), -128, 127)
 *     codes[n, k] = q + 128;  scales_f16[n] = fp16_round_nearest_even(s32)
 *
 *   W_f16      [N, K] fp16.  N >= 1; K >= 128, K % 128 == 0.
 *   codes_u8   [N, K] bytes, written (row-major; no repack step).
 *   scales_f16 [N] fp16, written.
 * Bit-identical to the library's CPU reference definition.
 * Errors: NULL -> W4A16_ERR_NULL; bad N, K -> W4A16_ERR_SHAPE; misaligned
 *         pointer -> W4A16_ERR_ALIGN.
 */
int w4a16_quantize_w8(const void *W_f16, int64_t N, int64_t K, void *codes_u8, void *scales_f16,
                      void *stream);

/*
 * w4a16_gemm_w8 -- W8A16 decode GEMV:
 *   y[m, n] = scale[n] * sum_k x[m, k] * (codes[n, k] - 128),
 * exact q * x products accumulated in FP32, the per-row scale applied once,
 * y rounded once to fp16.  M = 1..16; x[M, K] is held in shared memory whole
 * beside the ring (as w4a16_gemm_ex: about 2 * M * K <= 200 KB), a shape
 * that does not fit -> W4A16_ERR_SHAPE.  Graph-capturable, programmatic
 * dependent launch; codes and scales are constants of the call as in
 * w4a16_gemm.
 * Errors: as w4a16_gemm.
 */
int w4a16_gemm_w8(const void *x_f16, const void *codes_u8, const void *scales_f16, void *y_f16,
                  int64_t M, int64_t N, int64_t K, void *stream);

/* Paths reported by w4a16_gemm_plan. */
enum { W4A16_PATH_GEMV = 1, W4A16_PATH_TENSOR_CORE = 2 };

/*
 * w4a16_gemm_plan -- the launch w4a16_gemm makes for (M, N, K) on the current
 * device, without launching anything (introspection for tests and tuning).
 *
 *   *path            W4A16_PATH_GEMV (M <= 16) or W4A16_PATH_TENSOR_CORE.
 *   *splits          the thread-block cluster size: for the GEMV, the CTAs
 *                    sharing the K range of one 128-row block (1 = no
 *                    split); for the tensor-core GEMM, 1 (a CTA per
 *                    128 x 128 tile), 2 (CTA pairs with 2-CTA MMAs) or 4, 6, 8
 *                    (CTA pairs splitting K 2, 3, 4 ways, reduced through the
 *                    cluster's shared memory).
 *   *ctas            CTAs launched.
 *   *blocks_per_cta  most 128-row blocks one CTA walks (> 1: persistent).
 *   *rows_per_cta    weight rows one CTA computes of each block it handles:
 *                    128 (a whole block), or for the GEMV 16, 32 or 64 (1, 2
 *                    or 4 of a block's 16-row tiles over the whole K range,
 *                    the CTA's warps splitting K and reducing in its own
 *                    shared memory), or for the tensor-core GEMM's CTA pairs
 *                    with two x tiles 96 (six 16-row tiles; a pair covers 192
 *                    weight rows).
 * Errors: NULL output -> W4A16_ERR_NULL; bad M, N, K -> W4A16_ERR_SHAPE;
 *         no supported device -> W4A16_ERR_DEVICE / W4A16_ERR_CUDA.
 */
int w4a16_gemm_plan(int64_t M, int64_t N, int64_t K, int *path, int *splits, int *ctas,
                    int *blocks_per_cta, int *rows_per_cta);

/*
 * w4a16_gemm_plan_tail -- the last round of a persistent GEMV launch (more
 * 128-row blocks than CTAs, each CTA walking blocks y, y + ctas, ...).  When
 * the blocks do not divide evenly, the R blocks of the partial last round run
 * as R * 128 / tail_rows units of tail_rows weight rows (16, 32 or 64) over
 * the whole K range, one per CTA, so that round costs tail_rows / 128 of a
 * block instead of a whole one on a few CTAs.
 *
 *   *tail_rows   rows of each tail unit, 0 when the launch has no such round
 *                (not persistent, blocks divide evenly, or more than half a
 *                round left over) or M > 16.
 *   *tail_units  number of tail units (0 with tail_rows = 0).
 * Errors: as w4a16_gemm_plan.
 */
int w4a16_gemm_plan_tail(int64_t M, int64_t N, int64_t K, int *tail_rows, int *tail_units);

/*
 * w4a16_gemm_ex_plan -- the launch w4a16_gemm_ex makes for (M, N, K) with
 * the given group (32, 64, 128 or W4A16_GROUP_PER_CHANNEL), zero points
 * (nonzero: asymmetric codes) and AWQ scale (nonzero: alpha given), without
 * launching anything.
 *
 *   *path         W4A16_PATH_GEMV (M <= 16 with x[M, K] fitting in the
 *                 variant GEMV's shared memory) or W4A16_PATH_TENSOR_CORE.
 *   *splits       as w4a16_gemm_plan (1 for the variant GEMV).
 *   *ctas         CTAs launched.
 *   *rows_per_cta weight rows per CTA: 16, 32 or 64 for the variant GEMV,
 *                 128 for the tensor-core GEMM.
 * Group 128 with symmetric codes and no alpha reports w4a16_gemm_plan's
 * launch (the call runs w4a16_gemm).
 * Errors: NULL output -> W4A16_ERR_NULL; bad M, N, K or group ->
 *         W4A16_ERR_SHAPE; no supported device -> W4A16_ERR_DEVICE /
 *         W4A16_ERR_CUDA.
 */
int w4a16_gemm_ex_plan(int64_t M, int64_t N, int64_t K, int32_t group, int32_t zero_points,
                       int32_t alpha, int *path, int *splits, int *ctas, int *rows_per_cta);

/* ------------------------------------------------------------------------
 * Serving operators: the paged key-value cache between the quantized linear
 * layers, rotary positions, the attention of a new token or of chunks of them
 * over the cache, the care of its pages, the adjustment of logits and the
 * scores of sampled tokens.
 *
 * The conventions above hold, with these differences.  Tensors may be
 * strided where a stride is an argument (in elements, or in bytes where the
 * argument says so); the innermost dimension is always dense, and the stride
 * of a dimension of size 1 is not looked at.  Integer
 * tensors (int32) need 4-byte alignment only.  What an integer tensor holds
 * is device data that the call cannot see: kernels check every page and row
 * number against its range before they use it, and what each does with one
 * that is outside is said below.
 * ------------------------------------------------------------------------ */

/* Element types. */
enum { W4A16_F16 = 0, W4A16_BF16 = 1, W4A16_F32 = 2 };

/*
 * A cache: two pools of `pages` pages of `page_size` positions, and `batch`
 * rows of page numbers.  Position p of row b lies in page
 * tables[b * table_stride + p / page_size] at slot p % page_size; its head h
 * starts at page * page_stride + slot * slot_stride + h * head_stride
 * elements from the pool's start, head_dim elements long.  Both pools have
 * the same strides, so token-major, head-major and interleaved pools are all
 * of this form.
 *   pages >= 1; page_size 1 .. 65536; kv_heads 1 .. 1024; head_dim 8 .. 256,
 *   a multiple of 8; type W4A16_F16 or W4A16_BF16; the three strides
 *   multiples of 8 elements and >= 0; batch 1 .. 65535; table_width 1 .. 2^24,
 *   table_width * page_size < 2^31; pages < 2^31.
 */
typedef struct w4a16_cache_shape {
    int64_t pages, page_size, kv_heads, head_dim, type;
    int64_t page_stride, slot_stride, head_stride;
    int64_t batch, table_width, table_stride;
} w4a16_cache_shape;

/*
 * w4a16_paged_append -- new tokens' keys and values into their pages.
 *   token t of row b (offsets[b] <= t < offsets[b + 1]; one token a row,
 *   t = b, when offsets is NULL) goes to position starts[b] + t - offsets[b].
 *
 *   k, v       [tokens, kv_heads, head_dim]; strides in elements, multiples
 *              of 8 (a slice of a wider product is such a tensor).
 *   tables     [batch, table_width] int32; starts [batch]; offsets
 *              [batch + 1], not descending, or NULL.
 * A token whose position is negative or past table_width * page_size, or
 * whose page number is outside [0, pages), and one that no row claims, is
 * left out.
 * Errors: NULL -> W4A16_ERR_NULL; a size or stride outside the ranges above,
 * tokens < 0, or offsets NULL with tokens != batch -> W4A16_ERR_SHAPE; k, v
 * or a pool not 16-byte aligned -> W4A16_ERR_ALIGN.
 */
int w4a16_paged_append(const void *k, const void *v, void *k_pool, void *v_pool,
                       const int32_t *tables, const int32_t *starts, const int32_t *offsets,
                       const w4a16_cache_shape *cache, int64_t tokens, int64_t k_token_stride,
                       int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                       void *stream);

/* The queries and outputs of w4a16_paged_attention: q_heads a multiple of
 * kv_heads (at most 1024), batch * table_width * page_size * q_heads at most
 * 2^43; strides in elements, multiples of 8. */
typedef struct w4a16_query_shape {
    int64_t q_heads;
    int64_t q_row_stride, q_head_stride, out_row_stride, out_head_stride;
    double scale;
} w4a16_query_shape;

/*
 * w4a16_paged_attention -- one new token's attention over a paged cache:
 *   out[b, h] = sum_p w[p] V[b, p, h / g],  w = softmax_p(scale * q[b, h] . K[b, p, h / g])
 * over positions p < lengths[b], g = q_heads / kv_heads.  Scores, statistics
 * and sums are held in FP32; out is rounded once.
 *
 *   q          [batch, q_heads, head_dim] of the cache's type.
 *   lengths    [batch] int32; a length below 0 counts as 0, one past
 *              table_width * page_size as that.
 *   out        [batch, q_heads, head_dim], written.  A row of length 0 gets
 *              zeros.
 *   lse        NULL, or [batch, q_heads] float, written: the natural
 *              logarithm of sum_p exp(scale * q . K), -infinity for a row of
 *              length 0.
 *   workspace  w4a16_paged_attention_workspace(cache, q_heads) bytes, 16-byte
 *              aligned, of any content; not read after the call's work is
 *              done, and not to be shared by calls that may run at once.  Where
 *              that is 0 bytes, any aligned pointer other than NULL.
 * Positions whose page number is outside [0, pages) are left out, as if
 * masked, and so are those whose score is -infinity; a head that has no other
 * position gets what a row of length 0 gets.  A head with a score that is NaN
 * or +infinity gets NaN, in out and in lse.  A value of +-infinity gives the
 * infinity in its dimension of out, NaN beside a NaN or the opposite one, and
 * also where its weight is below 2^-36 (fp16) or 2^-126 (bf16) of the head's
 * largest, which may count as 0.  How the work is split, which goes by the
 * sizes and the device, changes the order of the FP32 sums and the maximum that
 * the weights are held against: they keep 22 bits in fp16 and 16 in bf16.  Two
 * calls on the same inputs and sizes give the same bits.
 * Errors: NULL -> W4A16_ERR_NULL; sizes outside the ranges above ->
 * W4A16_ERR_SHAPE; q, out, a pool or the workspace not 16-byte aligned ->
 * W4A16_ERR_ALIGN.
 */
int w4a16_paged_attention(const void *q, const void *k_pool, const void *v_pool,
                          const int32_t *tables, const int32_t *lengths, void *out, float *lse,
                          void *workspace, const w4a16_cache_shape *cache,
                          const w4a16_query_shape *query, void *stream);

/* Bytes of workspace of w4a16_paged_attention on the current device, 0 for
 * tables of few positions that need none (-1 on a bad shape or device). */
int64_t w4a16_paged_attention_workspace(const w4a16_cache_shape *cache, int64_t q_heads);

/*
 * A rotation: the first `dims` of a head's dimensions are turned in pairs,
 * (2 i, 2 i + 1) where interleaved = 1, (i, i + dims / 2) where it is 0; the
 * others stay as they are.  At position p the pair (a, b) becomes
 *   magnitude * (a cos(p w[i]) - b sin(p w[i])),  magnitude * (a sin(p w[i]) + b cos(p w[i])).
 * The rates come as `turns` [dims / 2] uint64: w[i] / (2 pi) * 2^64, modulo
 * 2^64.  The angle is reduced exactly, so far positions lose nothing; sums are
 * FP32, rounded once.
 *   dims 2 .. head_dim, even.
 */
typedef struct w4a16_rotary_shape {
    int64_t dims, interleaved;
    double magnitude;
} w4a16_rotary_shape;

/* Heads [tokens, heads, head_dim] that are read and heads of the same sizes
 * that are written: tokens 0 .. 2^31, heads 1 .. 1024, head_dim 8 .. 256, a
 * multiple of 8; strides in elements, multiples of 8; no two heads that are
 * written share a value (W4A16_ERR_SHAPE). */
typedef struct w4a16_heads_shape {
    int64_t tokens, heads, head_dim, type;
    int64_t token_stride, head_stride, out_token_stride, out_head_stride;
} w4a16_heads_shape;

/*
 * w4a16_rotate -- rotary positions: out[t] is x[t] rotated to positions[t].
 *   x, out     heads of `type` (W4A16_F16, _BF16, _F32), 16-byte aligned; out
 *              is x (with the same strides) or overlaps none of it.
 *   positions  [tokens] int32, of either sign: a rotation to -p is the gradient of
 *              one to p, and after it gives the values times the magnitude's
 *              square (so it undoes a rotation of magnitude 1).
 * Errors: NULL -> W4A16_ERR_NULL; sizes outside the ranges above, a magnitude
 * that is not finite -> W4A16_ERR_SHAPE; x or out not 16-byte aligned ->
 * W4A16_ERR_ALIGN.
 */
int w4a16_rotate(const void *x, const int32_t *positions, const uint64_t *turns, void *out,
                 const w4a16_rotary_shape *rotary, const w4a16_heads_shape *heads, void *stream);

/*
 * w4a16_paged_append_rotary -- w4a16_paged_append with the keys rotated to
 * their positions in the cache, and queries of the same tokens rotated to
 * theirs.
 *   q, out     [tokens, heads, head_dim] of the cache's type, described by
 *              `queries` (whose head_dim and type are the cache's); out is q
 *              (with the same strides) or overlaps none of it.  Both NULL: keys
 *              and values only (of `queries`, tokens alone is looked at).
 * A token whose position has no page has its queries rotated all the same; the
 * queries of one that no row claims become zeros.
 * Errors: as w4a16_paged_append and w4a16_rotate.
 */
int w4a16_paged_append_rotary(const void *k, const void *v, const uint64_t *turns, void *k_pool,
                              void *v_pool, const int32_t *tables, const int32_t *starts,
                              const int32_t *offsets, const void *q, void *out,
                              const w4a16_cache_shape *cache, const w4a16_rotary_shape *rotary,
                              const w4a16_heads_shape *queries, int64_t k_token_stride,
                              int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                              void *stream);

/*
 * w4a16_paged_chunk_attention -- attention of each row's last tokens over a
 * paged cache: row b's tokens offsets[b] <= t < offsets[b + 1] are its last
 * positions, token t at position lengths[b] - offsets[b + 1] + t, and each sees
 * the positions up to its own:
 *   out[t, h] = sum_p w[p] V[b, p, h / g],  w = softmax_p(scale * q[t, h] . K[b, p, h / g])
 * over p <= that position, g = q_heads / kv_heads.  Scores, statistics and sums
 * are held in FP32; weights enter the products with V in the cache's type.
 *
 *   q          [tokens, q_heads, head_dim] of the cache's type; the strides of
 *              `query` for rows are those of tokens here.
 *   lengths    [batch] int32, the new tokens among them, clamped as
 *              w4a16_paged_attention does.
 *   offsets    [batch + 1] int32, not descending, within 0 .. tokens.  A row
 *              may have no tokens.
 *   out        [tokens, q_heads, head_dim], written; no two heads share a value
 *              (W4A16_ERR_SHAPE) and out overlaps no input.  A token with a position
 *              below 0 (a row with more tokens than positions) and one that no row
 *              claims get zeros.
 *   lse        NULL, or [tokens, q_heads] float, written: the natural logarithm
 *              of sum_p exp(scale * q . K), -infinity for tokens as above.
 *   workspace  w4a16_paged_chunk_workspace(cache, q_heads, tokens) bytes,
 *              16-byte aligned, of any content; not to be shared by calls that
 *              may run at once.
 *   tokens     0 .. 2^24, tokens * q_heads at most 2^30; q_heads as for
 *              w4a16_paged_attention.
 * Positions without a valid page are left out, as if masked, and so are those
 * whose score is -infinity; a head that has no other position gets zeros and
 * -infinity.  A score that is NaN or +infinity gives NaN.  A value that is not
 * finite makes its dimension of out not finite (an infinity may come out as
 * NaN) for the tokens that see it, and for no other; at a position left out for
 * its score alone it may do so or not.  Two calls on the same
 * inputs and sizes give the same bits.
 * A weight keeps 11 bits in fp16 and 8 in bf16, and what divides is the sum of
 * the weights before that rounding: out is off by up to 2^-11 (2^-8) of the
 * weighted average of |V|, its own rounding aside.  w4a16_paged_attention keeps
 * 22 (16) bits for single tokens.
 * Errors: as w4a16_paged_attention.
 */
int w4a16_paged_chunk_attention(const void *q, const void *k_pool, const void *v_pool,
                                const int32_t *tables, const int32_t *lengths,
                                const int32_t *offsets, void *out, float *lse, void *workspace,
                                const w4a16_cache_shape *cache, const w4a16_query_shape *query,
                                int64_t tokens, void *stream);

/* Bytes of workspace of w4a16_paged_chunk_attention on the current device (-1
 * on a bad shape or device). */
int64_t w4a16_paged_chunk_workspace(const w4a16_cache_shape *cache, int64_t q_heads,
                                    int64_t tokens);

/*
 * The books of a cache's pages: how many rows hold each page (`refs`, <= 0 is
 * free), each row's page numbers (`tables`, -1 past its pages) and each row's
 * positions (`lengths`).  Row r of length n holds ceil(n / page_size) pages.
 *   pages 1 .. 2^31 - 1; rows 1 .. 2^24; width 1 .. 2^24, rows * width at
 *   most 2^40, width * page_size < 2^31; strides in elements.  Every call reads the `in` books and writes
 *   the `out` ones whole; each `out` tensor is its `in` tensor (with the same
 *   stride) or overlaps none.
 */
typedef struct w4a16_books_shape {
    int64_t pages, rows, width, in_stride, out_stride, page_size;
} w4a16_books_shape;

/* The pages themselves: `planes` pools (keys and values of every layer),
 * page p of plane l at l * plane_stride + p * page_stride bytes, page_bytes
 * long, all three multiples of 16. */
typedef struct w4a16_pool_shape {
    int64_t planes, plane_stride, page_stride, page_bytes;
} w4a16_pool_shape;

/* Bytes of workspace of w4a16_pages_extend for `count` requests, and of
 * w4a16_pages_fork and w4a16_pages_compact, where small pools need none (0)
 * if every `out` tensor is apart from its `in` tensor (apart = 1).  16-byte
 * aligned, of any content, as the attention's; -1 on a bad shape. */
int64_t w4a16_pages_workspace(const w4a16_books_shape *books, int64_t count);
int64_t w4a16_pages_fork_workspace(const w4a16_books_shape *books, const w4a16_pool_shape *shape,
                                   int64_t count, int32_t apart);
int64_t w4a16_pages_compact_workspace(const w4a16_books_shape *books,
                                      const w4a16_pool_shape *shape, int32_t apart);

/*
 * w4a16_pages_rows -- the listed rows of the books, for calls on some rows:
 * tables_out [count, width], dense, and lengths_out [count], if it is not
 * NULL, get those of row listed[i]; of a row outside [0, rows) they get -1 and
 * 0, so that such a row has no position and takes no token.  pages, page_size
 * and out_stride of the books are checked only.  Neither output overlaps an
 * input.
 */
int w4a16_pages_rows(const int32_t *tables_in, const int32_t *lengths_in, const int32_t *listed,
                     int64_t count, int32_t *tables_out, int32_t *lengths_out,
                     const w4a16_books_shape *books, void *stream);

/*
 * w4a16_pages_free -- gives back every page of the `count` rows listed: one
 * holder fewer for each, the row's page numbers -1 and its length 0.  A row
 * listed twice is given back once; one outside [0, rows) is passed over.
 */
int w4a16_pages_free(const int32_t *refs_in, const int32_t *tables_in, const int32_t *lengths_in,
                     const int32_t *listed, int64_t count, int32_t *refs_out, int32_t *tables_out,
                     int32_t *lengths_out, const w4a16_books_shape *books, void *stream);

/*
 * w4a16_pages_extend -- makes row listed[i] longer by counts[i] positions,
 * giving it the free pages it then needs: the lowest numbers first, in the
 * order of the list.  done[i] is 1, or 0 with the row unchanged: the row is
 * outside [0, rows) or was listed before, the count is negative, the row
 * would pass width * page_size, or it or one listed before it would need
 * more free pages than there are.
 */
int w4a16_pages_extend(const int32_t *refs_in, const int32_t *tables_in,
                       const int32_t *lengths_in, const int32_t *listed, const int32_t *counts,
                       int64_t count, int32_t *refs_out, int32_t *tables_out,
                       int32_t *lengths_out, int32_t *done, void *workspace,
                       const w4a16_books_shape *books, void *stream);

/*
 * w4a16_pages_fork -- makes the empty row children[i] a copy of row
 * parents[i]: full pages are shared (one holder more), a last page that is
 * partly filled is copied in every plane to the lowest free page, in the
 * order of the list.  done[i] is 1, or 0 with the child unchanged: a row is
 * outside [0, rows), the child's length is not 0 or it was listed before, the
 * parent's last page is none, or this child or one listed before it would
 * need more free pages than there are.
 */
int w4a16_pages_fork(void *pool, const int32_t *refs_in, const int32_t *tables_in,
                     const int32_t *lengths_in, const int32_t *parents, const int32_t *children,
                     int64_t count, int32_t *refs_out, int32_t *tables_out, int32_t *lengths_out,
                     int32_t *done, void *workspace, const w4a16_books_shape *books,
                     const w4a16_pool_shape *shape, void *stream);

/*
 * w4a16_pages_compact -- moves the pages that are held to the lowest
 * numbers: with n held pages in all, those numbered n or above move, in
 * ascending order, to the free ones below n, in ascending order.  Their
 * numbers in the tables follow.  used[0] = n.  Pages left behind keep their
 * old content.
 */
int w4a16_pages_compact(void *pool, const int32_t *refs_in, const int32_t *tables_in,
                        int32_t *refs_out, int32_t *tables_out, int32_t *used, void *workspace,
                        const w4a16_books_shape *books, const w4a16_pool_shape *shape,
                        void *stream);

/*
 * w4a16_pages_copy -- page from[i] to page to[i] in every plane, for i <
 * count.  A pair with a number outside [0, pages) is passed over.  No page
 * may be the target of two pairs, or both a target and a source.
 *
 * Errors of the w4a16_pages_* calls: NULL -> W4A16_ERR_NULL; sizes outside
 * the ranges above or count < 0 (count > 2^24) -> W4A16_ERR_SHAPE; pool or
 * workspace not 16-byte aligned -> W4A16_ERR_ALIGN.
 */
int w4a16_pages_copy(void *pool, const int32_t *from, const int32_t *to, int64_t count,
                     int64_t pages, const w4a16_pool_shape *shape, void *stream);

/* Most alternatives w4a16_token_logprobs gives. */
#define W4A16_MAX_TOP 32

/*
 * w4a16_token_logprobs -- the scores of given tokens under rows of logits:
 *   lse = ln sum_j exp(x[j]),  logprob = x[token] - lse,
 *   entropy = lse - sum_j p[j] x[j] with p[j] = exp(x[j] - lse) (p x = 0 where p = 0),
 *   and the `top` largest x[j], of equal ones the lowest j first, with x[j] - lse.
 * Statistics are held in FP32.
 *
 *   logits     [rows, vocabulary] of `type` (W4A16_F16, _BF16, _F32), rows
 *              row_stride elements apart, aligned to their element only.
 *   tokens     [rows], int64 (wide = 1) or int32 (wide = 0).  A token outside
 *              [0, vocabulary) has the logprob NaN.
 *   logprob, entropy  [rows] float; top_ids [rows, top] int32, top_logprobs
 *              [rows, top] float (both may be NULL when top = 0).
 *   rows       1 .. 2^24; vocabulary 1 .. 2^30; top 0 .. min(32, vocabulary).
 * -infinity masks a logit.  A row with nothing but -infinity has lse =
 * -infinity, every logprob -infinity and the entropy 0.  A row with a NaN or
 * +infinity has NaN for every number; its ids count NaN as the largest.
 * Errors: NULL -> W4A16_ERR_NULL; sizes or type outside the ranges above ->
 * W4A16_ERR_SHAPE; logits not aligned to their element -> W4A16_ERR_ALIGN.
 */
int w4a16_token_logprobs(const void *logits, const void *tokens, float *logprob, float *entropy,
                         int32_t *top_ids, float *top_logprobs, int64_t rows, int64_t vocabulary,
                         int64_t row_stride, int32_t type, int32_t wide, int32_t top,
                         void *stream);

/* Most biases a row of w4a16_adjust_logits. */
#define W4A16_MAX_BIASES 1024

/* The tensors of w4a16_adjust_logits; all but logits and out may be NULL. */
typedef struct w4a16_adjust_tensors {
    const void *logits, *tokens;
    const int32_t *lengths, *prompts;
    const float *repetition, *presence, *frequency;
    const int32_t *bias_ids;
    const float *biases;
    const uint32_t *mask;
    void *out;
} w4a16_adjust_tensors;

/* Its sizes: rows 1 .. 2^24, vocabulary 1 .. 2^30, type W4A16_F16, _BF16 or
 * _F32; strides in elements of rows; wide = 1 where tokens are int64; width of
 * the rows of tokens, below 2^30; biases of a row (0 .. 1024); and the penalties of every
 * row where the tensor of that name is NULL. */
typedef struct w4a16_adjust_shape {
    int64_t rows, vocabulary, type, logits_stride, out_stride;
    int64_t wide, width, token_stride, biases, bias_stride, mask_stride;
    double repetition, presence, frequency;
} w4a16_adjust_shape;

/*
 * w4a16_adjust_logits -- penalties, biases and masks on logits, in this order.
 * Of row r the first lengths[r] of tokens[r] (all of them where lengths is NULL;
 * clamped to 0 .. width) have been said, the first prompts[r] of those (none
 * where prompts is NULL) by the prompt.  With c[j] the times that token j is
 * among the others:
 *   x[j] / repetition where x[j] > 0, else x[j] * repetition, if j was said at all;
 *   - frequency * c[j], and - presence where c[j] > 0;
 *   + every biases[r, i] with bias_ids[r, i] = j, in the order of the list;
 *   -infinity where bit j % 32 of mask[r, j / 32] is 0.
 * In FP32, rounded once; a logit that nothing applies to keeps its bits.
 *
 *   logits, out    [rows, vocabulary] of `type`, aligned to their element; out
 *                  is logits (with the same stride) or overlaps none of it, and its
 *                  rows overlap one another nowhere.
 *   tokens         [rows, width] int32 or int64; one outside [0, vocabulary) is
 *                  passed over, as is such a bias_ids entry ([rows, biases] int32,
 *                  with biases [rows, biases] float, in rows of the same stride).
 *   repetition, presence, frequency  [rows] float, or NULL.
 *   mask           [rows, (vocabulary + 31) / 32] int32.
 * Errors: logits or out NULL, or bias_ids without biases -> W4A16_ERR_NULL; sizes
 * outside the ranges above -> W4A16_ERR_SHAPE; logits or out not aligned to
 * their element -> W4A16_ERR_ALIGN.
 */
int w4a16_adjust_logits(const w4a16_adjust_tensors *tensors, const w4a16_adjust_shape *shape,
                        void *stream);

/*
 * w4a16_device_status -- synchronises the current device, returns in
 * *status the OR of the W4A16_ERR_* conditions recorded by kernels since
 * the last call (W4A16_OK if none: W4A16_ERR_TIMEOUT when a bounded wait
 * gave up) and clears the record.  Returns W4A16_ERR_CUDA if the device
 * cannot be read.
 */
int w4a16_device_status(int *status);

/*
 * Upper bound, in nanoseconds, of every wait inside the library's kernels
 * (default 2e9, i.e. two seconds; 0 is taken as 1).  Applies to launches made
 * after the call.  A wait that gives up records W4A16_ERR_TIMEOUT (see
 * w4a16_device_status); the kernel then issues no more copies and waits for
 * those in flight before it exits.  That last wait is bounded by the larger
 * of this value and 100 ms, so a short limit cannot let a block exit while a
 * copy still writes into its shared memory.  Safe to call from any thread.
 */
void w4a16_set_wait_timeout_ns(uint64_t timeout_ns);

/*
 * w4a16_selftest_wait_timeout -- diagnostic: launches one block that waits
 * on an mbarrier nothing will ever arrive on, with a wait bound of
 * `timeout_ns`.  The kernel gives up after that time, records
 * W4A16_ERR_TIMEOUT in the device status word and exits normally, leaving
 * the context usable.  Used by the tests of the failure path.
 */
int w4a16_selftest_wait_timeout(uint64_t timeout_ns, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A16_H */
