/*
 * w4a8.h -- C ABI of the MI355X (gfx950) W4A8 linear / MoE-expert library.
 *
 * W4A8: weights stored as 4-bit integers in groups along K with one float32
 * scale (and, in asymmetric mode, one integer zero point) per group and output
 * column; activations quantized per token to INT8 at run time; an INT8 x INT8
 * -> INT32 GEMM whose weight nibbles are unpacked inside the kernel, with the
 * weight and activation scales applied in a float32 epilogue.
 *
 * Sources (cited as P1..P5 with the page's own section names):
 *   P1 "Kimi 2.7 MoE: from 4-bit storage to INT8 (W4A8)"                (pwwt.cn)
 *   P2 "Kimi 2.7 MoE W4A8: 4-bit storage to INT8, deployment notes"     (xdnf.cn)
 *   P3 "Quantization: formats, error and the real execution path"       (wineandchord.com)
 *   P4 "Choosing a weight-quantization scheme and locating kernel hits" (xbrilliance.ai)
 *   P5 "Inference quantization, chapter 1: the Linear layer"            (sgdbs.github.io)
 *
 * Conventions for every entry point
 *   - Matrices are row-major.  X is [M, K], W is [K, N], Y is [M, N] (P5 section 1:
 *     M = batch * seq_len, K = hidden, N = out features).
 *   - The caller owns every buffer, host and device.  GPU entry points only
 *     enqueue work on `stream` (a hipStream_t, NULL = the null stream) and never
 *     allocate device memory, free or synchronize (w4a8_moe_forward_sets creates
 *     helper streams and events once per device; see there).  Device pointers must
 *     stay valid until the enqueued work completes.
 *   - Return value: W4A8_OK (0) or a negative w4a8_status.  All argument checks
 *     run on the host before anything is enqueued, so an error return means
 *     nothing was launched.  W4A8_EHIP reports a launch failure seen right after
 *     enqueueing.  There is no fallback path: a shape or format the kernels do
 *     not implement returns W4A8_EUNSUPPORTED (P3 "Correctness contract" item 6
 *     and P4: a fallback must be explicit and observable).
 *   - Device buffers read with 128-bit loads (Xq, Hq, blobs) must be 16-byte
 *     aligned; the library checks this and returns W4A8_EINVAL otherwise.
 *   - Calls are thread-safe.  The only state the library keeps is created once per
 *     device and kept until the process ends: the helper streams of
 *     w4a8_moe_forward_sets and the scratch array of w4a8_moe_forward_noalloc.
 *   - Environment: W4A8_LOG set to anything but "0" makes every GEMM and MoE entry
 *     point print one line to stderr before it launches: the call, its shape and the
 *     kernel variant it resolved to (P4: a kernel hit must be observable).
 */
#ifndef W4A8_H
#define W4A8_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    W4A8_OK = 0,
    W4A8_EINVAL = -1,        /* bad argument: null pointer, bad shape, group not tiling K, ... */
    W4A8_ESIZE = -2,         /* a caller-provided buffer is smaller than required             */
    W4A8_EUNSUPPORTED = -3,  /* valid request the kernels do not implement (no fallback)       */
    W4A8_EHIP = -4           /* the HIP runtime reported an error when launching               */
} w4a8_status;

typedef enum { W4A8_OUT_BF16 = 0, W4A8_OUT_F32 = 1 } w4a8_out_dtype;

/* Element types of the router and of the unquantized (W16A16) products; the first two values are
 * those of w4a8_out_dtype. */
typedef enum { W4A8_BF16 = 0, W4A8_F32 = 1, W4A8_F16 = 2 } w4a8_dtype;

/* Weight format description (P3 "Four independent dimensions": object, format,
 * granularity, execution types must each be stated).
 *   K, N        weight matrix W[K, N]
 *   group_size  g: consecutive k sharing one scale per column (P5 section 8.4);
 *               must divide K.  pack accepts g in {32, 64, 128, 256} and g = K (one
 *               scale, and zero point, per output column: the per-channel granularity
 *               of P5 section 8.3).  Kernels implement all of them; 32, 256 and K run on
 *               the dense GEMMs only (the MoE entry points return EUNSUPPORTED), and
 *               g = K needs g * 127 * m < 2^31, the reach of the int32 group sum, where
 *               m is the largest weight operand the kernels feed: 15 (asymmetric), 112
 *               (symmetric 4-bit codes enter as 16 q) or 127 (8-bit codes); so K <= 150912
 *               for symmetric 4-bit per-channel weights; otherwise EUNSUPPORTED.  The GPU entry points also return
 *               EUNSUPPORTED for a blob whose codes reach 2 GiB (32-bit offsets).
 *   asymmetric  0: signed codes q in [-7, 7], zero point 0 (P3 "Basic mapping",
 *                  symmetric form);
 *               1: unsigned codes q in [0, 15] with a uint8 zero point z per
 *                  group, w ~ s (q - z) (P3 "Basic mapping"; P5 section 6).
 *   weight_bits 4 (or 0): the INT4 codes above, two per byte;
 *               8: the W8A8 sibling the pages compare against (P1 section 5): signed
 *                  codes q in [-127, 127], one per byte, symmetric only (qmax of the
 *                  P3 symmetric group-wise reference with bits = 8).  Dense GEMMs
 *                  only: the MoE entry points return EUNSUPPORTED for it.
 *   scale_bits  32 (or 0): float32 group scales;
 *               16: binary16 group scales, the storage P1 section 4.1 names for expert
 *                  weights.  The packer rounds each float32 scale to the nearest binary16
 *                  (ties to even) and computes the codes with the rounded scale, so
 *                  dequantization uses exactly the stored value; a scale past the binary16
 *                  range (65504) makes w4a8_pack return EINVAL.  Kernels take binary16
 *                  scales with 4-bit codes and g in {64, 128} (dense and MoE); other
 *                  combinations return EUNSUPPORTED. */
typedef struct {
    int32_t K;
    int32_t N;
    int32_t group_size;
    int32_t asymmetric;
    int32_t weight_bits;
    int32_t scale_bits;
} w4a8_wdesc;

/* ------------------------------------------------------------------------------------
 * Packed weight blob ("the checkpoint"): header + codes + scales [+ zeros].
 * P3 "Calibration and conversion" asks the converted artifact to record format,
 * signedness, packing, scale axis and group size; the header does.
 *
 *   offset 0    header, W4A8_HEADER_BYTES bytes, little endian:
 *               char magic[8] = "W4A8BLB1"; uint32 version = 1; uint32 layout = 1;
 *               int32 K, N, group_size, asymmetric; uint32 scale_dtype (0 float32,
 *               1 binary16);
 *               uint32 zero_dtype = 0 (uint8); uint64 codes_off, codes_bytes,
 *               scales_off, scales_bytes, zeros_off, zeros_bytes, total_bytes;
 *               uint32 weight_bits (4 or 8; 0 in older headers reads as 4);
 *               the rest is zero.
 *   codes       Np = N rounded up to 16 (padding columns hold code 0, scale 0).
 *               Superblock = 16 columns x 128 rows = 1024 bytes, stored as 64
 *               lanes x 16 bytes; superblocks run over k first, then over the
 *               column tile:  superblock index = (n / 16) * (K / 128) + k / 128.
 *               Inside a superblock, for kk = k % 128 and c = n % 16:
 *                 half = kk / 64, r = kk % 64, lane = (r / 16) * 16 + c, j = r % 16,
 *                 byte = lane * 16 + half * 8 + (j / 8) * 4 + (j % 4),
 *                 nibble = (j % 8) / 4   (0 = low 4 bits, 1 = high 4 bits).
 *               So one 128-bit load per lane fetches 16 k of one column for two
 *               64-deep MFMA steps, and the low/high nibbles of a 32-bit word are
 *               the k and k+4 operands of the same byte position (P1 section 5.1:
 *               tile format matched to the MFMA operand; P1 section 7, third pitfall).
 *               Symmetric codes are stored as 4-bit two's complement; asymmetric
 *               codes as unsigned 0..15.  Two codes per byte (P1 section 5.2).
 *               8-bit codes (weight_bits = 8): superblock = 2048 bytes, 64 lanes x 32
 *               bytes, one int8 code per byte at lane * 32 + half * 16 + j (lane, half
 *               and j as above): the values the 4-bit form unpacks, in the same order.
 *   scales      float32 [Np/16][K/g][16]: scale of (group i, column n) at
 *               ((n/16) * (K/g) + i) * 16 + n % 16.
 *   zeros       (asymmetric only) uint8, same index as scales.
 *   Every section starts on a 256-byte boundary.
 * ------------------------------------------------------------------------------------ */
#define W4A8_HEADER_BYTES 256

/* Bytes of the blob for `d` (header + codes + scales + zeros + alignment padding), the
 * M = N b/8 + N_groups M_meta + M_pad term of P3 "Basic mapping" with the padding
 * explicit.  Returns 0 if `d` is invalid. */
size_t w4a8_packed_size(const w4a8_wdesc* d);

/* Offline RTN quantization + packing on the host (P3 "Basic mapping"; P3 symmetric
 * group-wise reference; P2 section 2.1).  W_host: float32 [K, N] row-major, finite.
 * Per (group, column): symmetric s = fl32(max|w| / 7), q = clamp(rint(fl32(w / s)), -7, 7)
 * (8-bit codes: 127 in place of 7);
 * asymmetric lo = min(0, min w), hi = max(0, max w), s = fl32(fl32(hi - lo) / 15),
 * z = clamp(rint(fl32(-lo / s)), 0, 15), q = clamp(rint(fl32(w / s)) + z, 0, 15); an
 * all-zero group gets s = 0, z = 0, q = 0.  Round half to even, IEEE float32 division.
 * Writes w4a8_packed_size(d) bytes to blob_host.  EINVAL: bad desc, group not tiling K,
 * non-finite weight; ESIZE: blob_bytes too small. */
int w4a8_pack(const w4a8_wdesc* d, const float* W_host, void* blob_host, size_t blob_bytes);

/* Pack externally produced codes (e.g. from GPTQ/AWQ, P2 section 3.2) without
 * re-quantizing.  codes: int8 [K, N] in [-7, 7] (symmetric), [0, 15] (asymmetric) or
 * [-127, 127] (8-bit);
 * scales: float32 [K/g, N]; zeros: uint8 [K/g, N] in [0, 15] (asymmetric) or NULL.
 * EINVAL on out-of-range codes or zero points. */
int w4a8_pack_codes(const w4a8_wdesc* d, const int8_t* codes, const float* scales,
                    const uint8_t* zeros, void* blob_host, size_t blob_bytes);

/* Inverse of the packing, on the host: checks the header and writes codes [K, N],
 * scales [K/g, N] and (asymmetric) zeros [K/g, N]; d_out receives the header's desc.
 * Any output pointer may be NULL to skip it.  EINVAL on a bad header. */
int w4a8_unpack_codes(const void* blob_host, size_t blob_bytes, w4a8_wdesc* d_out,
                      int8_t* codes, float* scales, uint8_t* zeros);

/* Host check that blob_host's header describes `d` and fits in blob_bytes; to be run
 * once when a blob is loaded (GPU entry points trust the desc they are given). */
int w4a8_blob_check(const void* blob_host, size_t blob_bytes, const w4a8_wdesc* d);

/* ------------------------------------------------------------------------------------
 * GPU entry points
 * ------------------------------------------------------------------------------------ */

/* Per-token dynamic INT8 activation quantization (P1 section 3.3; P5 section 8.3;
 * P2 section 3.3: a quantize node before each Linear).
 *   X_bf16  device, bfloat16 [M, K] with row stride ldx >= K elements
 *   Xq      device, int8 [M, K] dense (row stride K), 16-byte aligned, K % 16 == 0
 *   sx      device, float32 [M]
 * Per row: amax = max|x|; s = fl32(amax / 127); q = clamp(rint(fl32(x / s)), -127, 127)
 * (divisor 1 when s == 0).  A row containing NaN or Inf gets s = NaN and q = 0.
 * M == 0 is a no-op. */
int w4a8_quant_act(const void* X_bf16, int M, int K, int ldx, int8_t* Xq, float* sx,
                   void* stream);

/* The same quantization of X diag(alpha)^-1, the activation side of the equivalent
 * per-channel rescaling Y = (X diag(alpha)^-1) (diag(alpha) W) of P3 "Weight-Activation"
 * (SmoothQuant: quantization difficulty moved from activations to weights offline).  The
 * page asks for the scaling to be fused into an adjacent operator; here it is: each
 * x[m, k] is multiplied by inv_alpha[k] (one float32 product, round to nearest even) and
 * the per-token rule above applies to the products.  The weight side, diag(alpha) W, is
 * applied before packing by the caller.
 *   inv_alpha  device float32 [K], 16-byte aligned (1 / alpha per input channel)
 * Other arguments, layouts and errors as w4a8_quant_act; EINVAL if inv_alpha is NULL. */
int w4a8_quant_act_smooth(const void* X_bf16, int M, int K, int ldx, const float* inv_alpha, int8_t* Xq,
                          float* sx, void* stream);

/* Static (calibrated) activation quantization (P1 section 3.2: a scale measured on a
 * calibration set ahead of time replaces the per-batch reduction; the page recommends it for
 * decode).  Every row uses the one given scale:
 *   s       device float32 [1] (a device value, so a captured graph can be recalibrated)
 *   Xq, sx  as w4a8_quant_act; sx[m] = s for every row
 * q = clamp(rint(fl32(x / s)), -127, 127): values beyond the calibrated range saturate at
 * +-127, NaN gives 0, +-Inf gives +-127.  A scale that is not finite and positive gives
 * all-zero codes.  No limit on K besides K % 16 == 0 (one pass, nothing held per row).
 * M == 0 is a no-op; EINVAL for NULL pointers, K % 16, ldx % 8 or misaligned X / Xq. */
int w4a8_quant_act_static(const void* X_bf16, int M, int K, int ldx, const float* s, int8_t* Xq,
                          float* sx, void* stream);

/* Static per-expert quantization of the routed rows (P1 section 3.1: one activation scale
 * per expert; section 3.2: static scales).  Row r of the expert-sorted order (from
 * w4a8_moe_align) quantizes token sorted_rows[r] / k of X with the scale s[e] of the
 * expert e that owns row r (expert_offsets[e] <= r < expert_offsets[e + 1]), by the rule of
 * w4a8_quant_act_static.
 *   X_bf16          device bfloat16 [T, H], row stride ldx
 *   sorted_rows     device int32 [T*k]; expert_offsets device int32 [E+1]; s device float32 [E]
 *   Xq, sx          device int8 [T*k, H] (16-byte aligned), float32 [T*k], sorted order
 * Rows at or past expert_offsets[E] (routing ids outside [0, E)) get zero codes and scale 0.
 * E <= 1024 (EINVAL), T*k <= 2^24 (EUNSUPPORTED). */
int w4a8_moe_quant_static(const void* X_bf16, int T, int H, int ldx, const int32_t* sorted_rows,
                          int k, const int32_t* expert_offsets, int E, const float* s, int8_t* Xq,
                          float* sx, void* stream);

/* W4A8 GEMM Y = (s_x * Xq) (s_w * (q - z)) (P5 section 4 ideal path; P5 section 8.3
 * epilogue Y[i, j] = s_x[i] s_w[j] acc[i, j], applied per K-group of P5 section 8.4).
 *   Xq, sx    device, from w4a8_quant_act ([M, K] int8 dense, [M] float32)
 *   blob_dev  device copy of a blob packed for `d` (K % 128 == 0 required)
 *   Y         device, [M, N] with row stride ldy >= N, bfloat16 or float32 (out_dtype)
 * The INT4 nibbles are unpacked in registers into INT8 MFMA operands; each group's INT32
 * partial sum is scaled by its float32 weight scale into a float32 accumulator, the
 * row scale is applied last, then the bfloat16 cast rounds to nearest even.  No
 * dequantized weight is ever written to memory (P1 section 4.4 step 4; P5 section 3.2).
 * M == 0 is a no-op.  EINVAL for M > 32 with 256 * K >= 2^31 (the 256-row activation tile
 * is addressed with 32-bit offsets). */
int w4a8_gemm(const int8_t* Xq, const float* sx, int M, const void* blob_dev,
              const w4a8_wdesc* d, void* Y, int ldy, int out_dtype, void* stream);

/* Per-token quantization and W4A8 GEMM in one call: Y = GEMM(quant_act(X)).
 *   X_bf16   device bfloat16 [M, K], row stride ldx >= K (ldx % 8 == 0, 16-byte aligned)
 *   Xq, sx   device int8 [M, K] (16-byte aligned) and float32 [M]: always written with the
 *            activation codes and scales (the caller can reuse them)
 *   Y, ldy, out_dtype, blob_dev, d as in w4a8_gemm.
 * For M <= 16 and M * K <= 8192 (M <= 2 at K = 4096) this is one kernel: each
 * workgroup of the decode GEMM quantizes the activation rows itself into its staged
 * activation tile (P2 section 3.3 places the per-token quantization node right before
 * the GEMM; P1 section 8 suggests fusing quantization into the GEMM kernel); otherwise
 * it is w4a8_quant_act followed by w4a8_gemm.  Results are bit-identical either way. */
int w4a8_linear(const void* X_bf16, int M, int K, int ldx, const void* blob_dev, const w4a8_wdesc* d, void* Y,
                int ldy, int out_dtype, int8_t* Xq, float* sx, void* stream);

/* W4A16 sibling (P1 section 5.3 compares W4A16 with W8A8 and W4A8; P5 section 3.2: the
 * weight-only path dequantizes inside the GEMM): Y = X W with the activations kept in bfloat16
 * (no activation quantization) and the 4-bit codes of a W4A8 blob dequantized in registers,
 *   Y[m, n] = sum_i s[i, n] * sum_{k in group i} X[m, k] * (q[k, n] - z[i, n]),
 * accumulated in float32 on bfloat16 MFMA.
 *   X_bf16   device bfloat16 [M, ldx], 16-byte aligned, ldx % 8 == 0, ldx >= K
 *   blob_dev the same blob as w4a8_gemm: 4-bit codes, g in {64, 128}, float32 scales
 *            (other formats: EUNSUPPORTED)
 *   Y        device [M, ldy] bfloat16 or float32
 * M <= 32 runs the streaming (decode) kernel, larger M the 128 x 128-tile kernel; M == 0 is a
 * no-op.  EINVAL for M > 32 when 128 * ldx * 2 reaches 2^31 (32-bit activation offsets). */
int w4a16_gemm(const void* X_bf16, int M, int ldx, const void* blob_dev, const w4a8_wdesc* d, void* Y,
               int ldy, int out_dtype, void* stream);

/* Name of the kernel variant w4a16_gemm resolves to for (d, M), or "unsupported". */
const char* w4a16_kernel_name(const w4a8_wdesc* d, int M);

/* Test export of the same main loop: INT32 per-group partial sums
 * P[m, n, i] = sum_{k in group i} Xq[m, k] (q[k, n] - z[i, n]) written to device
 * int32 [M, N, K/g].  (P3 "Correctness contract" item 3: the accumulator covers the
 * reduction: |P| <= g * 127 * 15, or g * 127 * 127 with 8-bit codes, < 2^31; symmetric
 * 4-bit sums are formed as 16 P, |16 P| <= g * 127 * 112 < 2^31.)  Same
 * EINVAL size limit as w4a8_gemm.  With g = K and M <= 32 (the decode kernels, which split
 * K across waves) it returns EUNSUPPORTED. */
int w4a8_gemm_partials(const int8_t* Xq, int M, const void* blob_dev, const w4a8_wdesc* d,
                       int32_t* P, void* stream);

/* MoE dispatch by expert (P1 section 4.4, steps 2-3).
 *   topk_ids       device int32 [T, k], each in [0, E)
 *   sorted_rows    device int32 [T*k]: routed rows r = t*k + j grouped by expert,
 *                  ascending r inside an expert (stable counting sort)
 *   expert_offsets device int32 [E+1]: exclusive prefix sum of rows per expert
 *   inv            device int32 [T, k]: position of row t*k + j in sorted_rows
 * Ids outside [0, E) are counted nowhere and their inv entry is -1; the host cannot see
 * device ids, so callers validate routing upstream.  E <= 1024, T*k <= 2^24. */
int w4a8_moe_align(const int32_t* topk_ids, int T, int k, int E, int32_t* sorted_rows,
                   int32_t* expert_offsets, int32_t* inv, void* stream);

/* Expert-grouped W4A8 GEMM (P1 section 4.4 step 4, "the performance key").
 *   Xq, sx         device activations [src_rows, K] and [src_rows]; if `gather` is non-NULL,
 *                  output row r (in sorted order) reads Xq/sx row gather[r] / k (token of
 *                  the routed row); if NULL, row r reads row r (rows already permuted)
 *   gather         device int32 [rows] or NULL (pass sorted_rows from w4a8_moe_align)
 *   k              top-k (divisor for gather; ignored when gather is NULL)
 *   expert_offsets device int32 [E+1]; rows [off[e], off[e+1]) use expert e
 *   rows           T*k, total rows (= off[E]); rows of Y
 *   src_rows       rows of Xq and sx: T with a gather, >= rows without one (EINVAL otherwise)
 *   blobs_dev      device, E blobs of desc `d`, expert e at blobs_dev + e * expert_stride
 *   Y              device [rows, N] bfloat16 or float32, dense
 * The kernels bound what the device arrays may name: a gather entry that is negative or
 * names a token at or past src_rows reads no activations and gives an output row of zeros,
 * and expert row ranges are clamped to [0, rows).  Experts with no rows read no weights.
 * All experts of a call share one allocation at a fixed stride: the kernels find an expert's
 * weights by one multiply of ids they already hold, with no further dependent load in front of
 * the weight stream. */
int w4a8_moe_gemm(const int8_t* Xq, const float* sx, const int32_t* gather, int k,
                  const int32_t* expert_offsets, int E, int rows, int src_rows, const void* blobs_dev,
                  size_t expert_stride, const w4a8_wdesc* d, void* Y, int out_dtype,
                  void* stream);

/* Expert-grouped gate/up GEMM with the static SiLU-requant folded into its epilogue (P1
 * section 8: fold the activation quantization into the GEMM; P1 section 3.2: static, calibrated
 * activation scales, so the requantization needs no reduction over a row).  The blob holds the
 * gate columns [0, I) and the up columns [I, 2I) of each expert (d->N = 2I, I % 16 == 0,
 * EINVAL otherwise).  A workgroup computes gate column c and up column I + c side by side; each
 * output is rounded to bfloat16 as w4a8_moe_gemm stores it, h = silu(g) * u is formed in float32
 * and quantized with the scale s[e] of the row's expert (the rule of w4a8_quant_act_static),
 * so Hq and sh equal those of w4a8_moe_gemm followed by w4a8_silu_mul_quant_static, bit for
 * bit, without the [rows, 2I] bfloat16 intermediate.
 *   Xq, sx, gather, k, expert_offsets, E, rows, src_rows, blobs_dev, expert_stride, d
 *                  as for w4a8_moe_gemm
 *   s              device float32 [E], static scales of h
 *   Hq, sh         device int8 [rows, I], float32 [rows]
 * Rows at or past expert_offsets[E] (no expert owns them) are not written.  Same checks and
 * limits as w4a8_moe_gemm. */
int w4a8_moe_gemm_silu_static(const int8_t* Xq, const float* sx, const int32_t* gather, int k,
                              const int32_t* expert_offsets, int E, int rows, int src_rows,
                              const void* blobs_dev, size_t expert_stride, const w4a8_wdesc* d,
                              const float* s, int8_t* Hq, float* sh, void* stream);

/* SiLU-gated expert activation + per-row INT8 requantization for the down projection
 * (P1 section 1 names SiLU; P1 section 3.1: per-expert activation scales).
 *   GU_bf16  device bfloat16 [R, 2I]: gate = columns [0, I), up = [I, 2I)
 *   Hq, sh   device int8 [R, I] (16-byte aligned, I % 16 == 0), float32 [R]
 * h = fl32(g / (1 + exp(-g)) * u) in float32, then the per-token rule of w4a8_quant_act.
 * I <= 16384 (EUNSUPPORTED beyond). */
int w4a8_silu_mul_quant(const void* GU_bf16, int R, int I, int8_t* Hq, float* sh,
                        void* stream);

/* The same with static per-expert scales: row r (expert-sorted order) is quantized by the
 * rule of w4a8_quant_act_static with the scale s[e] of the expert that owns it.
 *   expert_offsets  device int32 [E+1] from w4a8_moe_align; s device float32 [E]
 * Rows at or past expert_offsets[E] get zero codes and scale 0.  E <= 1024 (EINVAL). */
int w4a8_silu_mul_quant_static(const void* GU_bf16, int R, int I, const int32_t* expert_offsets,
                               int E, const float* s, int8_t* Hq, float* sh, void* stream);

/* Un-permute and top-k weighted combine (P1 section 4.3: dequantize to 16-bit, multiply
 * by the gate weight, accumulate; kept out of the integer domain).
 *   Yd_bf16  device bfloat16 [T*k, H] in sorted order
 *   inv      device int32 [T, k] from w4a8_moe_align
 *   topk_w   device float32 [T, k]
 *   out      device bfloat16 [T, H]
 * out[t] = bf16(sum_{j=0..k-1} topk_w[t, j] * Yd[inv[t, j]]) in float32, j ascending. */
int w4a8_moe_combine(const void* Yd_bf16, const int32_t* inv, const float* topk_w, int T,
                     int k, int H, void* out_bf16, void* stream);

/* Workspace bytes needed by w4a8_moe_forward for the given sizes (0 if invalid). */
size_t w4a8_moe_workspace_size(int T, int k, int H, int I, int E);

/* One MoE expert layer, the steps of P1 section 4.4 chained on `stream`:
 * quant_act(X) -> moe_align -> moe_gemm(gate/up, gathered) -> silu_mul_quant ->
 * moe_gemm(down) -> moe_combine.
 *   X_bf16      device [T, H]; topk_ids / topk_w device [T, k]
 *   gu_blobs    E blobs of desc gu_desc (K = H, N = 2I), stride gu_stride
 *   d_blobs     E blobs of desc d_desc (K = I, N = H), stride d_stride
 *   workspace   device, >= w4a8_moe_workspace_size(T, k, H, I, E) bytes, 256-aligned
 *   out_bf16    device [T, H], 16-byte aligned
 * Limits: E <= 1024 (EINVAL), T*k <= 2^24, H <= 65536, I <= 16384 (EUNSUPPORTED); H and I
 * multiples of 16, X 16-byte aligned (EINVAL).  Every argument check of the chained steps
 * runs before the first launch: an error return means that nothing was enqueued. */
int w4a8_moe_forward(const void* X_bf16, const int32_t* topk_ids, const float* topk_w, int T,
                     int k, int E, const void* gu_blobs, size_t gu_stride,
                     const w4a8_wdesc* gu_desc, const void* d_blobs, size_t d_stride,
                     const w4a8_wdesc* d_desc, void* workspace, size_t workspace_bytes,
                     void* out_bf16, void* stream);

/* w4a8_moe_forward for callers that cannot allocate device memory: code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc.  The workspace is a 64 MiB
 * device array that the library holds on each GPU it runs on until the process ends; the call
 * itself allocates nothing.  Layers whose w4a8_moe_workspace_size exceeds 64 MiB return
 * W4A8_ESIZE (the T = 512, E = 64, top-6 layer with H = 4096, I = 1408 needs about 49 MB).
 * Every call on one GPU shares that array: calls that overlap on one GPU (other streams, other
 * threads) race and must be serialized by the caller.  Arguments, results and other errors as
 * w4a8_moe_forward (W4A8_EHIP also if the array's address cannot be obtained). */
int w4a8_moe_forward_noalloc(const void* X_bf16, const int32_t* topk_ids, const float* topk_w, int T,
                             int k, int E, const void* gu_blobs, size_t gu_stride,
                             const w4a8_wdesc* gu_desc, const void* d_blobs, size_t d_stride,
                             const w4a8_wdesc* d_desc, void* out_bf16, void* stream);

/* One format class of experts for w4a8_moe_forward_sets: n_experts consecutive experts
 * whose gate/up blobs (desc gu_desc, stride gu_stride) and down blobs (d_desc, d_stride)
 * share one format.  Experts are numbered set by set: set 0 holds experts [0, n_0), set 1
 * [n_0, n_0 + n_1), and so on. */
typedef struct {
    int32_t n_experts;
    const void* gu_blobs;
    size_t gu_stride;
    const w4a8_wdesc* gu_desc;
    const void* d_blobs;
    size_t d_stride;
    const w4a8_wdesc* d_desc;
} w4a8_expert_set;

/* One MoE expert layer whose experts use different weight formats (P1 section 8: quantize at
 * expert granularity, with a group size and format per expert, so that sensitive experts can
 * be kept at a finer format).  The steps of w4a8_moe_forward.  The group size, zero points and
 * scale width may differ between sets; the shapes (gate/up [H, 2I], down [I, H]) may not (EINVAL).
 * A grouped GEMM whose K (H for gate/up, I for down) is at most 4096 runs every set in one
 * launch pair on `stream` when there are at most four sets: each workgroup takes the format of
 * its expert's set, so the result is that of one launch per set.  Otherwise the GEMM runs once
 * per set, over that set's experts; these launches are independent (disjoint experts, disjoint
 * rows): set 0 runs on `stream`, the others on up to four helper streams of the current device,
 * forked from `stream` and joined back into it with events, so the call completes in `stream`
 * order and can be captured into a graph.  The helpers (default priority) are created by the
 * first call that needs them and is not made under graph capture, and kept until the process
 * ends; a call made before they exist, or where they cannot be created, runs the sets one after
 * another on `stream`.  Calls from several host threads enqueue one at a time.
 *   sets, nsets  host array of the format classes; E = sum of n_experts <= 1024
 *   workspace    device, >= w4a8_moe_workspace_size(T, k, H, I, E) bytes, 256-aligned
 * Other arguments and errors as w4a8_moe_forward. */
int w4a8_moe_forward_sets(const void* X_bf16, const int32_t* topk_ids, const float* topk_w, int T,
                          int k, const w4a8_expert_set* sets, int nsets, void* workspace,
                          size_t workspace_bytes, void* out_bf16, void* stream);

/* Workspace bytes needed by w4a8_moe_forward_static (0 if invalid): the routed rows are
 * quantized one by one, so the activation codes take T*k rows instead of T. */
size_t w4a8_moe_static_workspace_size(int T, int k, int H, int I, int E);

/* One MoE expert layer with static per-expert activation scales (P1 section 3.1 and 3.2:
 * calibrated scales, one per expert, for decode).  The steps of w4a8_moe_forward, with the
 * two quantizations replaced: moe_align -> moe_quant_static(X, s_gu) -> moe_gemm_silu_static
 * (gate/up GEMM, rows already sorted, with the SiLU-requant by s_dn in its epilogue) ->
 * moe_gemm(down) -> moe_combine.
 *   s_gu, s_dn  device float32 [E]: scale of each expert's gate/up and down inputs
 *   workspace   device, >= w4a8_moe_static_workspace_size(T, k, H, I, E) bytes, 256-aligned
 * Other arguments and errors as w4a8_moe_forward. */
int w4a8_moe_forward_static(const void* X_bf16, const int32_t* topk_ids, const float* topk_w, int T,
                            int k, int E, const void* gu_blobs, size_t gu_stride,
                            const w4a8_wdesc* gu_desc, const void* d_blobs, size_t d_stride,
                            const w4a8_wdesc* d_desc, const float* s_gu, const float* s_dn,
                            void* workspace, size_t workspace_bytes, void* out_bf16, void* stream);

/* ------------------------------------------------------------------------------------
 * Router, and the expert-grouped products of the two formats beside W4A8
 * ------------------------------------------------------------------------------------ */

typedef enum { W4A8_ROUTE_SOFTMAX = 0, W4A8_ROUTE_SIGMOID = 1 } w4a8_route_score;

/* How a router chooses experts.
 *   E, k         experts (1..1024) and experts per token (1..min(E, 64))
 *   score        p_i = softmax(x)_i over all E logits, or p_i = 1 / (1 + exp(-x_i))
 *   renormalize  0 or 1: divide the k chosen scores by their sum (weights 0 if the sum is 0)
 *   n_group, topk_group
 *                experts in n_group groups of E / n_group neighbours, of which only the topk_group
 *                best may be chosen from; n_group = 1 (or 0) turns groups off
 *   scale        factor on every weight, applied last */
typedef struct {
    int32_t E;
    int32_t k;
    int32_t score;
    int32_t renormalize;
    int32_t n_group;
    int32_t topk_group;
    float scale;
} w4a8_route_desc;

/* Top-k routing of T tokens (P1 section 4.1 keeps the router in 16 bits, outside the quantized
 * path): the topk_ids and topk_w that w4a8_moe_align, w4a8_moe_combine and the MoE layers take.
 *   logits    device float32, bfloat16 or float16 (dtype) [T, E], row stride ldl >= E elements,
 *             aligned to its element
 *   bias      device float32 [E] or NULL: an offset used for the choice only, not for the weights
 *   topk_ids  device int32 [T, k], best first; topk_w device float32 [T, k]
 * Experts are ranked by their logit, or by p_i + bias_i in float64 if a bias is given, of which 42
 * bits of the mantissa count; a group by its best expert, or with a bias by the sum of its two best
 * ranks, of which again 42 bits count.  Equal ranks go to the lower index.  An expert whose logit (or bias) is -Inf is masked: never chosen;
 * a -Inf logit also has p_i = 0.  Where fewer than k can be chosen, the remaining entries are id -1
 * with weight 0, which w4a8_moe_align leaves out and w4a8_moe_combine skips (a padded token: all
 * logits -Inf).  A row with a NaN logit or rank, or
 * with a +Inf logit under softmax, has no order: it gets the ids 0..k-1 with NaN weights.
 * Scores are computed in float64, without a bias the denominator of the softmax in float32; with a
 * bias and sigmoid scores, logits below -708 may rank as -708.
 * T == 0 is a no-op.  EINVAL: E, k or score out of range, n_group not dividing E, topk_group
 * outside 1..n_group or leaving fewer than k experts, ldl < E, scale not finite, NULL or misaligned pointers;
 * EUNSUPPORTED: E > 1024, k > 64, T > 2^24. */
int w4a8_moe_route(const void* logits, int dtype, int T, int ldl, const float* bias,
                   const w4a8_route_desc* d, int32_t* topk_ids, float* topk_w, void* stream);

/* Expert-grouped W8A8 GEMM (P1 section 5.3: W8A8 beside W4A8; P5 section 8.3: one scale per token
 * and one per output channel): w4a8_moe_gemm for blobs of 8-bit codes with group_size = K,
 *   Y[r, n] = sx[src] sw[e, n] sum_k Xq[src, k] q_e[k, n],
 * the sum exact in int32, then float32, then rounded to nearest even for bfloat16.
 *   d   weight_bits = 8, group_size = K, float32 scales, K < 133144; other formats EUNSUPPORTED
 * Rows at or past expert_offsets[E] are not written.  Other arguments, bounds and errors as
 * w4a8_moe_gemm; additionally E <= 1024 (EINVAL) and EUNSUPPORTED for N > 2^20 or rows > 2^24.  k
 * also tells, with or without a gather, that no expert should have more than rows / k rows: the
 * launches are chosen by it (1 if unknown).  A row's result is the same bit for bit whatever k and
 * the other rows are.  A row whose scale is -0 gives zeros, like
 * a gather entry that names no row. */
int w4a8_moe_gemm_w8a8(const int8_t* Xq, const float* sx, const int32_t* gather, int k,
                       const int32_t* expert_offsets, int E, int rows, int src_rows,
                       const void* blobs_dev, size_t expert_stride, const w4a8_wdesc* d, void* Y,
                       int out_dtype, void* stream);

/* Expert-grouped unquantized GEMM (P1 section 8: sensitive experts kept in a finer format):
 *   Y[r, n] = sum_k X[src, k] W[e, n, k],
 * the products exact and summed in float32, then rounded to nearest even if Y has 16 bits.  A call
 * repeats bit for bit, but the order of a row's sum, and with it its last bits, depend on the kernel
 * that E, rows and k select and on the row's place among the rows of its expert and of the call:
 * the same token may round to a neighbouring value in another batch.
 *   X         device bfloat16 or float16 (dtype) [src_rows, K], row stride ldx elements
 *   W         device, same type, [E, N, K]: output channels by inputs, K contiguous, row stride ldw
 *             and expert stride expert_stride, both in elements
 *   Y         device [rows, N], row stride ldy; out_dtype is dtype or W4A8_F32
 *   gather, k, expert_offsets, E, rows, src_rows   as w4a8_moe_gemm_w8a8
 * K, ldx, ldw and expert_stride are multiples of 8, X and W 16-byte aligned (EINVAL); any N.  Rows
 * at or past expert_offsets[E] are not written, nor is Y past column N.  A gather entry that
 * names no row of X gives a row of zeros.  E <= 1024 (EINVAL).  EUNSUPPORTED: N > 2^20, ldw > 2^23,
 * rows > 2^24. */
int w4a8_moe_gemm_w16a16(const void* X, int dtype, int ldx, const int32_t* gather, int k,
                         const int32_t* expert_offsets, int E, int rows, int src_rows, const void* W,
                         size_t expert_stride, int ldw, int K, int N, void* Y, int ldy, int out_dtype,
                         void* stream);

/* Expert-grouped unquantized gate/up GEMM with the gated activation in its epilogue (P1 section 1):
 *   H[r, c] = silu(g) u,  g = sum_k X[src, k] W[e, c, k],  u = sum_k X[src, k] W[e, I + c, k],
 * formed from the float32 sums and rounded once, so no [rows, 2I] intermediate is stored.  For g < 0
 * silu(g) is g exp(g) / (1 + exp(g)), where exp(g) may count as 0 below 2^-126.
 *   W   device [E, 2I, K]: the I gate rows, then the I up rows; any I
 *   H   device [rows, I], row stride ldh, of type dtype
 * Other arguments and errors as w4a8_moe_gemm_w16a16. */
int w4a8_moe_gemm_silu_w16a16(const void* X, int dtype, int ldx, const int32_t* gather, int k,
                              const int32_t* expert_offsets, int E, int rows, int src_rows,
                              const void* W, size_t expert_stride, int ldw, int K, int I, void* H,
                              int ldh, void* stream);

/* One MoE expert layer on 8-bit per-channel experts: the steps of w4a8_moe_forward with
 * w4a8_moe_gemm_w8a8 for both products.
 *   gu_desc, d_desc  as w4a8_moe_gemm_w8a8 (K = H, N = 2I; K = I, N = H)
 *   workspace        device, >= w4a8_moe_workspace_size(T, k, H, I, E) bytes, 256-aligned
 * Ids outside [0, E) (w4a8_moe_route gives -1 for padded tokens) add nothing to their token.  H <= 65536
 * and I <= 16384 (EUNSUPPORTED).  Other arguments, limits and errors as w4a8_moe_forward. */
int w4a8_moe_forward_w8a8(const void* X_bf16, const int32_t* topk_ids, const float* topk_w, int T,
                          int k, int E, const void* gu_blobs, size_t gu_stride,
                          const w4a8_wdesc* gu_desc, const void* d_blobs, size_t d_stride,
                          const w4a8_wdesc* d_desc, void* workspace, size_t workspace_bytes,
                          void* out_bf16, void* stream);

/* Workspace bytes needed by w4a8_moe_forward_w16a16 (0 if invalid). */
size_t w4a8_moe_w16a16_workspace_size(int T, int k, int H, int I, int E);

/* One MoE expert layer on unquantized bfloat16 experts: w4a8_moe_align ->
 * w4a8_moe_gemm_silu_w16a16 (gate/up, gathered) -> w4a8_moe_gemm_w16a16 (down) -> w4a8_moe_combine.
 *   X_bf16     device bfloat16 [T, H]
 *   Wgu        device bfloat16 [E, 2I, H], gate rows first; Wd [E, H, I]; rows dense, expert strides
 *              gu_stride and d_stride in elements
 *   workspace  device, >= w4a8_moe_w16a16_workspace_size(T, k, H, I, E) bytes, 256-aligned
 *   out        device bfloat16 [T, H]
 * H and I multiples of 8, all pointers 16-byte aligned (EINVAL); T*k <= 2^24 (EUNSUPPORTED).  Every
 * check of the chained steps runs before the first launch. */
int w4a8_moe_forward_w16a16(const void* X_bf16, const int32_t* topk_ids, const float* topk_w, int T,
                            int k, int E, const void* Wgu, size_t gu_stride, const void* Wd,
                            size_t d_stride, int H, int I, void* workspace, size_t workspace_bytes,
                            void* out_bf16, void* stream);

/* ------------------------------------------------------------------------------------
 * Microscaled formats (MXFP4, MXFP8): quantization, products and the expert layer
 * (P3 names them beside the integer formats; the layer's steps are those of P1 section 4.4)
 *
 * Blocks of 32 neighbours along K share one scale 2^(b - 127), kept as the byte b (E8M0; 255 is NaN).
 * Elements are E2M1 (MXFP4: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives; sign, two bits of exponent,
 * one of mantissa; two to a byte, the lower k in the low half) or E4M3 (MXFP8: up to 448, one byte).
 *
 * Quantization of a block: b = max(0, floor(log2 amax) + 127 - e), e = 2 (E2M1) or 8 (E4M3), amax the
 * largest magnitude; element = x / 2^(b - 127) rounded to nearest even, saturating at 6 or 448.  A
 * block of zeros has b = 0.  A block with a NaN or an infinity has b = 255 and elements 0, and makes
 * every product with it NaN.
 *
 * Activations [M, K]: rows are padded to Kp = 128 ceil(K / 128); codes uint8 [M, Kp / 2] (MXFP4) or
 * [M, Kp] (MXFP8), scales uint8 [M, Kp / 32], both dense.  Elements and scales behind K are 0:
 * the quantizing calls write them, and the products rely on it.
 *
 * Packed weights (MXFP4, [N, K] output channels by inputs; no header, the caller keeps N and K):
 *   codes   tile n / 16, then step k / 128, then lane 16 (k % 128 / 32) + n % 16: the 16 bytes of one
 *           block, the operand of an MFMA
 *   scales  (at the next multiple of 256) tile n / 64, then step k / 128, then lane (as above), then
 *           n % 64 / 16: one byte each
 *   N and K are padded to whole tiles and steps with zeros.
 *
 * Limits: K and N at most 2^20, packed codes below 2 GiB (EUNSUPPORTED).
 * ------------------------------------------------------------------------------------ */

/* Formats of activations.  W4A8_QUANT_INT8, the codes and scales of w4a8_quant_act, is taken by
 * w4a8_norm_residual_quant only. */
typedef enum { W4A8_MX_FP4 = 0, W4A8_MX_FP8 = 1, W4A8_QUANT_INT8 = 2 } w4a8_act_format;

/* Block quantization of activations.
 *   X       device bfloat16, float16 or float32 (dtype) [M, K], row stride ldx >= K elements, aligned to
 *           its element; any K
 *   Xq, sx  device, as above; Xq 16-byte, sx 4-byte aligned
 * M == 0 is a no-op.  EINVAL: fmt, dtype, K <= 0, ldx < K, NULL or misaligned pointers. */
int w4a8_mx_quant(const void* X, int dtype, int M, int K, int ldx, int fmt, void* Xq, uint8_t* sx, void* stream);

/* The values that codes and scales stand for: Y [M, K] in bfloat16, float16 or float32 (dtype), row stride
 * ldy (exact in float32 and, where their range has them, in bfloat16; else rounded to nearest even).
 * Nothing behind column K is written. */
int w4a8_mx_dequant(const void* Xq, const uint8_t* sx, int fmt, int M, int K, void* Y, int dtype, int ldy, void* stream);

/* Bytes of packed MXFP4 weights [N, K] (0 if invalid). */
size_t w4a8_mx_packed_size(int K, int N);

/* Quantization and packing of weights on the device.
 *   W      device bfloat16, float16 or float32 (dtype) [E, N, K], row stride ldw and expert stride
 *          expert_stride in elements (ignored for E = 1)
 *   blobs  device, 16-byte aligned, E packed matrices, blob_stride bytes apart (a multiple of 16, >=
 *          w4a8_mx_packed_size)
 * E <= 1024 (EINVAL); E == 0 is a no-op; E N / 64 K / 128 < 2^24 (EUNSUPPORTED). */
int w4a8_mx_pack(const void* W, int dtype, int E, int N, int K, int ldw, size_t expert_stride, void* blobs,
                 size_t blob_stride, void* stream);

/* Packing of existing MXFP4 codes (a checkpoint, or w4a8_mx_quant's of weights): codes uint8 [N, K / 2] with
 * row stride ldc bytes (a multiple of 16), scales uint8 [N, K / 32] with row stride lds; K % 32 == 0
 * (EINVAL).  w4a8_mx_unpack_codes is the inverse, into the layout of activations (rows of Kp). */
int w4a8_mx_pack_codes(const uint8_t* codes, const uint8_t* scales, int N, int K, int ldc, int lds, void* blob, void* stream);
int w4a8_mx_unpack_codes(const void* blob, int N, int K, uint8_t* codes, uint8_t* scales, void* stream);

/* Product of MX activations with MXFP4 weights,
 *   Y[m, n] = sum over blocks i of 2^(sx[m, i] + sw[n, i] - 254) sum_{k in block i} x[m, k] w[n, k],
 * on the scaled MFMA (v_mfma_scale_f32_16x16x128_f8f6f4): exact products summed in float32, rounded to nearest
 * even if Y has 16 bits.  Terms below 2^-126 may count as 0.  A call repeats bit for bit; the order of a sum
 * depends on the kernel, which M, K and N select.
 *   Xq, sx, fmt  device activations [M, K], W4A8_MX_FP4 or W4A8_MX_FP8
 *   blob         device, packed [N, K]
 *   Y            device [M, N] bfloat16, float16 or float32 (out_dtype), row stride ldy; any N
 * M == 0 is a no-op.  EUNSUPPORTED: M > 2^24, (M / 32 + 1) ceil(N / 64) >= 2^32. */
int w4a8_mx_gemm(const void* Xq, const uint8_t* sx, int fmt, int M, const void* blob, int K, int N, void* Y,
                 int ldy, int out_dtype, void* stream);

/* The same by expert: rows [expert_offsets[e], expert_offsets[e + 1]) of Y are products with blob e.
 *   gather, k, expert_offsets, E, rows, src_rows   as w4a8_moe_gemm_w8a8
 *   blobs, expert_stride   E packed [N, K], expert_stride bytes apart (a multiple of 16)
 * Rows at or past expert_offsets[E] are not written, nor is Y past column N.  A gather entry that names no
 * row gives a row of zeros.  E <= 1024 (EINVAL); EUNSUPPORTED: rows or src_rows > 2^24,
 * (rows / 32 + E) ceil(columns of a blob / 64) >= 2^32. */
int w4a8_moe_gemm_mx(const void* Xq, const uint8_t* sx, int fmt, const int32_t* gather, int k,
                     const int32_t* expert_offsets, int E, int rows, int src_rows, const void* blobs,
                     size_t expert_stride, int K, int N, void* Y, int ldy, int out_dtype, void* stream);

/* Grouped gate/up product with the gated activation in its epilogue, H[r, c] = silu(g) u from the float32
 * sums (silu(g) is good to 2^-22 + |g| 2^-24 of itself, and 0 where exp(g) is below 2^-126, g < -87.3).
 *   blobs   packed [2I, K]: the I gate channels, then the I up channels; I % 16 == 0 (EINVAL)
 *   H       device [rows, I] bfloat16 or float16 (out_dtype), row stride ldh
 * Other arguments and errors as w4a8_moe_gemm_mx. */
int w4a8_moe_gemm_silu_mx(const void* Xq, const uint8_t* sx, int fmt, const int32_t* gather, int k,
                          const int32_t* expert_offsets, int E, int rows, int src_rows, const void* blobs,
                          size_t expert_stride, int K, int I, void* H, int ldh, int out_dtype, void* stream);

/* The same with H quantized in the epilogue (a block of 32 columns needs no reduction over the row): codes
 * and scales of the float32 H in h_fmt, the activations [rows, I] of the down product. */
int w4a8_moe_gemm_silu_mx_quant(const void* Xq, const uint8_t* sx, int fmt, const int32_t* gather, int k,
                                const int32_t* expert_offsets, int E, int rows, int src_rows, const void* blobs,
                                size_t expert_stride, int K, int I, int h_fmt, void* Hq, uint8_t* sh, void* stream);

/* Workspace bytes with which w4a8_moe_forward_mx makes all columns at once (0 if invalid). */
size_t w4a8_moe_mx_workspace_size(int T, int k, int H, int I, int E, int fmt);

/* One MoE expert layer on MXFP4 experts with activations in fmt: w4a8_mx_quant(X) -> w4a8_moe_align ->
 * w4a8_moe_gemm_silu_mx_quant (gathered) -> w4a8_moe_gemm_mx (down, float32) -> the weighted sum per token,
 * in float32 and rounded once.
 *   X_bf16     device bfloat16 [T, H]; topk_ids / topk_w device [T, k] (ids outside [0, E) add nothing)
 *   gu_blobs   E packed [2I, H], gate channels first; d_blobs E packed [H, I]; strides in bytes
 *   workspace  device, 256-aligned, w4a8_moe_mx_workspace_size(T, k, H, I, E, fmt) bytes, or less: its last
 *              4 T k H bytes are the experts' outputs, and where only a part of their columns fits (64 at
 *              least, ESIZE), the down product and the sum are made by slices of columns, at two launches a
 *              slice, with the same bits
 *   out_bf16   device bfloat16 [T, H]
 * I % 16 == 0 (EINVAL); T*k <= 2^24 and T ceil(H / 1024) < 2^24 (EUNSUPPORTED).  Every check of the chained
 * steps runs before the first launch. */
int w4a8_moe_forward_mx(const void* X_bf16, const int32_t* topk_ids, const float* topk_w, int T, int k, int E,
                        int fmt, const void* gu_blobs, size_t gu_stride, const void* d_blobs, size_t d_stride,
                        int H, int I, void* workspace, size_t workspace_bytes, void* out_bf16, void* stream);

/* ------------------------------------------------------------------------------------
 * The norm around a block
 * ------------------------------------------------------------------------------------ */

typedef struct {
    float eps;        /* of the norm of the residual stream */
    float eps_post;   /* of the norm of the block's output */
    float alpha;      /* factor on the block's output */
} w4a8_norm_desc;

/* The end of one block and the start of the next, row by row:
 *   u  = X rsqrt(mean(X^2) + eps_post) post_w, or X where post_w is NULL
 *   r' = residual + alpha gate u, rounded to res_dtype       -> residual_out
 *   h  = r' rsqrt(mean(r'^2) + eps) w, rounded to dtype      -> Y
 * in float32 (squares past its range make the mean infinite and h 0 or NaN).  A call repeats bit for bit; the
 * order of a row's sums depends on H and on whether M exceeds 512.
 *   X             device [M, H] of dtype (bfloat16, float16 or float32), row stride ldx
 *   residual      device [M, H] of res_dtype, row stride ldr, or NULL (zeros: with alpha = 1 and no gate the
 *                 call is the norm of X alone)
 *   gate          device of dtype, [M, H] with row stride ldg, or one row for all (ldg = 0), or NULL (ones)
 *   post_w, w     device float32 [H]
 *   residual_out  row stride ldo, or NULL (not stored); may be residual itself
 *   Y             row stride ldy, or NULL (r' only; w is not read)
 * Any H up to 65536 (EUNSUPPORTED beyond, for M > 2^22, and for M = 2^22 with H > 8192), rows aligned to
 * their element.  M == 0 is a no-op.  EINVAL: types, strides below H, eps negative or not finite, alpha not finite, NULL X, no output. */
int w4a8_norm_residual(const void* X, int dtype, int ldx, const void* residual, int res_dtype, int ldr,
                       const void* gate, int ldg, const float* post_w, const float* w, const w4a8_norm_desc* d,
                       int M, int H, void* residual_out, int ldo, void* Y, int ldy, void* stream);

/* The same with h quantized in place of stored: the codes and scales that w4a8_mx_quant (fmt W4A8_MX_FP4 or
 * W4A8_MX_FP8) gives for h, or by the rule of w4a8_quant_act (W4A8_QUANT_INT8: int8 [M, H] and float32 [M],
 * H % 16 == 0; h of any type), bit for bit.  Xq 16-byte, sx 4-byte aligned. */
int w4a8_norm_residual_quant(const void* X, int dtype, int ldx, const void* residual, int res_dtype, int ldr,
                             const void* gate, int ldg, const float* post_w, const float* w,
                             const w4a8_norm_desc* d, int M, int H, void* residual_out, int ldo, int fmt, void* Xq,
                             void* sx, void* stream);

/* Name of the kernel variant w4a8_gemm resolves to for (d, M), or "unsupported"
 * (P4: record target and resolved backend so a silent fallback is visible):
 * {w4a8,w8a8}_{decode_m16,decode_m32,prefill}_{sym,asym}_g{64,128,256,K,32}[_h16], and
 * w4a8_decode_split_m{16,32}_... for the decode GEMMs served by the kernel with one K-slice per
 * wave (4-bit codes, g in {64, 128}, 2048 < K <= 4096, rows w4a8_linear does not quantize
 * inside the GEMM). */
const char* w4a8_kernel_name(const w4a8_wdesc* d, int M);

/* Human-readable text of a w4a8_status. */
const char* w4a8_status_string(int status);

/* Library ABI version (1). */
int w4a8_version(void);

#ifdef __cplusplus
}
#endif

#endif /* W4A8_H */
