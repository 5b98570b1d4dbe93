/*
 * wq.h - W8A8 dynamic-quant linear and FP8 per-token-group quant for MI355X (gfx950).
 *
 * The operation (from "DeepSeek-V4 W8A8 性能分析：小 M、NZ 布局与测量方法", section 一):
 * a dense linear Y = X W with X [M, K], W [K, N], Y [M, N], run as BF16 X -> per-token
 * dynamic quant -> INT8 X + per-token f32 scale -> INT8 x INT8 -> INT32 GEMM against
 * per-output-channel-scaled INT8 weights -> BF16 Y.  The FP8 variant (SGLang PR #34277
 * summary, 功能与动机 / 实现拆解) quantises each 128-wide hidden group of each token to
 * E4M3FN with a power-of-two UE8M0 scale, and writes the scales packed 4 per int32 in the
 * [G, ceil((D/128)/4), align4(T)] layout the grouped FP8 contraction reads directly.
 *
 * Conventions for every call:
 *  - Tensor pointers are DEVICE pointers owned by the caller.  The library never
 *    allocates, frees or synchronises in these calls: it validates the arguments on the
 *    host, enqueues kernels on `stream` (a hipStream_t passed as void*; NULL = the null
 *    stream) and returns.  Device faults surface at the caller's next synchronisation.
 *  - Weights are stored [N, K] with K contiguous (output-channel rows), the logical
 *    W[K, N] transposed once at load time.
 *  - Every base pointer and every leading dimension times the element size must be a
 *    multiple of 16 bytes (the 16-byte scale-base rule of PR #34277, 实现拆解 item 1);
 *    INT8 GEMMs need K % 16 == 0 and N % 16 == 0; FP8 needs D, K and N multiples of 128.
 *  - On any failed check nothing is written and nothing is launched.
 *  - An empty problem (M == 0 or T == 0) returns WQ_OK with no launch (the wrapper in
 *    PR #34277 launches only when x has elements).
 *  - Outputs are deterministic: the same inputs give the same bytes on every call.
 *  - A context and its workspace serve one stream at a time: calls that overlap on two
 *    streams must use two contexts.
 */
#ifndef WQ_H
#define WQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------------------ */
enum {
  WQ_OK = 0,
  WQ_ERR_NULL = 1,        /* a required pointer is NULL                                  */
  WQ_ERR_SHAPE = 2,       /* negative or inconsistent sizes, unsupported divisibility   */
  WQ_ERR_ALIGN = 3,       /* a base pointer or leading dimension not 16-byte aligned    */
  WQ_ERR_WORKSPACE = 4,   /* workspace missing or smaller than wq_workspace_bytes()     */
  WQ_ERR_DEVICE = 5,      /* not a gfx950 device, or the launch failed                  */
  WQ_ERR_UNSUPPORTED = 6  /* a valid but unimplemented combination of options           */
};

/* input element types */
enum { WQ_IN_BF16 = 1, WQ_IN_F32 = 2 };
/* GEMM payload types */
enum {
  WQ_PAYLOAD_INT8 = 1,
  WQ_PAYLOAD_FP8_E4M3 = 2,
  WQ_PAYLOAD_MXFP8 = 3,
  WQ_PAYLOAD_MXFP4 = 4,    /* E2M1 activations on E2M1 weights, 32-element blocks       */
  WQ_PAYLOAD_MXFP8_W4 = 5  /* E4M3 activations on E2M1 weights, 32-element blocks       */
};
/* code types of a paged cache */
enum { WQ_KV_E4M3 = 1, WQ_KV_INT8 = 2 };
/* GEMM epilogues */
enum { WQ_EPI_BF16 = 1, WQ_EPI_SWIGLU_F32 = 2 };
/* weight layout of wq_matmul_desc.b: plain [batch][N][K], or the fragment order of
 * wq_pack_weight_i8 applied to each batch (INT8: segments, or dense M < 256) */
enum { WQ_LAYOUT_PLAIN = 0, WQ_LAYOUT_FRAGMENT = 1 };

/* Human-readable text for a status code (static storage). */
const char* wq_status_str(int status);

/* ABI revision of this header (3: wq_matmul_desc.expected_rows). */
int wq_abi_version(void);

/* ---- context ----------------------------------------------------------------------- */
typedef struct wq_ctx wq_ctx;

/* Bytes of device workspace a context needs (a fixed bound, independent of shapes). */
size_t wq_workspace_bytes(void);

/* Create a context for `device`.  `workspace` is caller-owned device memory of at least
 * wq_workspace_bytes() bytes, 256-byte aligned; its contents need no initialisation.  The
 * library uses it only to stage the INT8 payload and scales between the two launches of
 * wq_fused_quant_matmul when M is above the one-launch limit and the caller passed no
 * x_q_out / x_scale_out.  Fails with WQ_ERR_DEVICE if the device is not gfx950.
 * Reads the environment once:
 *   WQ_LOG=1          one line per call describing the chosen launch;
 *   WQ_FORCE_SPLIT=n  the K-split factor of the quant kernel (tests use it to show every
 *                     split gives the same bytes);
 *   WQ_DECODE_NT=n    columns per workgroup of the decode GEMM of wq_quant_matmul (4, 8
 *                     or 16; 0 = auto);
 *   WQ_DECODE_MT=t    16-row tiles per workgroup of the decode GEMM (1, 2 or 4; 0 = auto);
 *   WQ_FUSED_MAX_M=m  the largest M wq_fused_quant_matmul runs as one launch (0..255,
 *                     default 255; 0 = always two launches);
 *   WQ_FUSED_GEMV_MAX_M=m  up to this M (0..4, default 0) that one launch is the dot4
 *                     GEMV kernel rather than the 8-wave MFMA kernel;
 *   WQ_FUSED_R=r, WQ_FUSED_NT=n  rows (1, 2, 4, 8, 16) and columns (4, 8, 16, 32) per
 *                     workgroup of that MFMA kernel (0 = auto; see wq_ctx_set_fused_shape);
 *   WQ_SEG_SMALL=0    expert segments: run every expert on the tiled kernel instead of
 *                     sending the experts with at most 16 rows to the streaming kernel;
 *   WQ_FP8_RT=r       grouped FP8 contraction at T <= 16: 16-token tiles per workgroup
 *                     (1..4; 0 = auto, all of them);
 *   WQ_FP8_COLS=16    grouped FP8 contraction at 16 < T <= 64: keep the 16-column kernel
 *                     instead of the 32-column one (default 32);
 *   WQ_GQ_PPW=p       FP8 group quant: packs of four hidden groups per wave (1, 2, 4 or
 *                     8; 0 = auto by grid size);
 *   WQ_EXPECTED_TOKENS=n  expert segments: the expected rows per expert when a call's
 *                     descriptor gives none (wq_matmul_desc.expected_rows; 0 = no hint).
 * Values out of range fall back to the default.  Every setting gives bit-identical
 * results except WQ_FP8_COLS, which changes the order of the FP8 contraction's f32 sums
 * (4 or 8 partial sums per output; both within the contraction's stated tolerance).  The
 * knobs exist for tests and measurement. */
int wq_ctx_create(int device, void* workspace, size_t workspace_bytes, wq_ctx** out);
void wq_ctx_destroy(wq_ctx* ctx);

/* Force the K-split factor of later quant calls on this context (the same knob as
 * WQ_FORCE_SPLIT); n = 0 restores the automatic choice.  Results are bit-identical for
 * every split; tests use this to show it.  Returns WQ_ERR_SHAPE for n < 0; a split larger
 * than K / 8 (bf16 input) or K / 4 (f32 input), one 16-byte piece of the row per slice,
 * makes later quant calls return WQ_ERR_SHAPE. */
int wq_ctx_set_split(wq_ctx* ctx, int n);

/* Force the shape of the one-launch fused kernel of wq_fused_quant_matmul on this context
 * (the same knobs as WQ_FUSED_R / WQ_FUSED_NT): rows_per_wg rows (1, 2, 4, 8 or 16) and
 * cols_per_wg output columns (4, 8, 16 or 32) per workgroup; 0 restores the automatic
 * choice of that dimension.  Results are bit-identical for every shape; tests use this to
 * show it.  Returns WQ_ERR_SHAPE for other values and changes nothing then. */
int wq_ctx_set_fused_shape(wq_ctx* ctx, int rows_per_wg, int cols_per_wg);

/* ---- per-token dynamic INT8 quantisation --------------------------------------------
 * Follows section 一 of the W8A8 article (npu_dynamic_quant: BF16 X -> INT8 X plus a
 * per-token scale) and section 二 (row-parallel work whose parallelism is capped by the
 * row count; long rows may additionally be split along K over several workgroups).
 * Optionally fuses an RMSNorm in front and a row gather, following "DeepSeek V4 950 低精度
 * 优化全复盘" section 2.3 (RMSNorm fused with quantisation in registers) and section 3.2
 * (rows gathered in expert-sorted order).
 *
 * For output row r (0 <= r < M), with src = row_index ? row_index[r] : r:
 *   v[k]  = x[src, k]                                  (no RMSNorm)
 *   v[k]  = (x[src, k] * inv) * gamma[k],  inv = 1 / sqrt(f32(sum_k x^2 / K) + rms_eps)
 *                                                      (rms_gamma != NULL; sum in f64)
 *   a     = max_k |v[k]|,   x_scale[r] = RN_f32(a / 127)
 *   x_q[r, k] = clamp(rint(RN_f32(v[k] / x_scale[r])), -127, 127)   (0 when a == 0)
 * x: x_dtype WQ_IN_BF16 or WQ_IN_F32, row stride ldx elements (ldx >= K).
 * rms_gamma: NULL or bf16 [K].  row_index: NULL or int32 [M] (values are not checked).
 * x_q: int8 [M, K] contiguous.  x_scale: f32 [M].  K % 16 == 0, K <= 131072. */
int wq_dynamic_quant(wq_ctx* ctx, const void* x, int x_dtype, int64_t M, int64_t K, int64_t ldx,
                     const void* rms_gamma, float rms_eps, const int32_t* row_index,
                     int8_t* x_q, float* x_scale, void* stream);

/* ---- per-token-group FP8 quantisation with packed UE8M0 scales -----------------------
 * Follows the SGLang PR #34277 summary (实现拆解 items 1-2 and the kernel write-logic and
 * wrapper snippets).  x: bf16 [T, G, D] contiguous, D % 128 == 0.  HG = D / 128,
 * PH = ceil(HG / 4), TA = 4 * ceil(T / 4).  For each (t, g, h):
 *   a = max |x[t, g, 128h .. 128h+127]|,  e = max(-127, smallest e with 2^e >= a / 448)
 *   x_q[t, g, 128h + i] = E4M3FN(x * 2^-e), nearest-even       (uint8 [T, G, D])
 *   byte e + 127 goes to byte (h % 4) of int32 word (g * PH + h / 4) * TA + t of x_s
 * x_s: int32 storage [G, PH, TA] (16-byte aligned).  Every byte of x_s not written this
 * way - the tail of the last pack and the token-padding words t in [T, TA) - is written
 * as zero.  The logical [T, G, PH] view has element strides (1, PH * TA, TA).
 * TA * G * PH < 2^31 (WQ_ERR_SHAPE otherwise). */
int wq_group_quant_fp8_ue8m0(wq_ctx* ctx, const void* x, int64_t T, int64_t G, int64_t D,
                             uint8_t* x_q, int32_t* x_s, void* stream);

/* The MX-like variant of "DeepSeek V4 950 低精度优化全复盘", section 2.1: every 32
 * elements share one 8-bit scale, E4M3 values.  Same contract as wq_group_quant_fp8_ue8m0
 * with 32-element groups: D % 32 == 0, HG = D / 32 (so PH = ceil(D / 128)),
 *   a = max |x[t, g, 32h .. 32h+31]|, e = max(-127, smallest e with 2^e >= a / 448),
 *   x_q = E4M3FN(x * 2^-e), byte e + 127 at byte (h % 4) of word (g * PH + h / 4) * TA + t,
 * every other byte of x_s [G, PH, TA] zero.  One pack word holds the four 32-element
 * scales of one 128-deep K block. */
int wq_group_quant_mxfp8(wq_ctx* ctx, const void* x, int64_t T, int64_t G, int64_t D,
                         uint8_t* x_q, int32_t* x_s, void* stream);

/* ---- microscaled 4-bit blocks ---------------------------------------------------------
 * The same blocks of 32 elements in 4 bits: E2M1 (sign, two exponent bits of bias 1, one
 * fraction bit; magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6), two codes to a byte, the element with
 * the even index in the low four bits.  x: bf16 [T, G, D] contiguous, D % 32 == 0.
 *   a = max |x[t, g, 32h .. 32h+31]|,  e = max(-127, smallest e with 2^e >= a / 6)
 *   code = E2M1(x * 2^-e), nearest-even                       (x_q: uint8 [T, G, D/2])
 *   byte e + 127 at the place wq_group_quant_mxfp8 gives it (x_s: int32 [G, PH, TA],
 *   PH = ceil(D / 128)); every other byte of x_s zero.
 * A block that holds a NaN or an infinity gets byte 255, UE8M0's NaN, and zero codes: what
 * reads it (the inverse below, the products) gives NaN.
 * Weights [N, K] are cast by the same call as [T = N, G = 1, D = K]; the casts of G groups
 * one behind the other are the operand b and its scales of the 4-bit payloads.
 * TA * G * PH < 2^31 (WQ_ERR_SHAPE otherwise). */
int wq_group_quant_mxfp4(wq_ctx* ctx, const void* x, int64_t T, int64_t G, int64_t D, uint8_t* x_q, int32_t* x_s,
                         void* stream);

/* The inverse: y[t, g, d] = code * 2^(byte - 127), bf16 [T, G, D] contiguous (exact: every
 * value of a finite block below 2^128 is a bf16 number; a magnitude from 1.75 * 2^127 on was rounded
 * up to 2^128, which reads as infinity; byte 255 gives NaN). */
int wq_group_dequant_mxfp4(wq_ctx* ctx, const uint8_t* x_q, const int32_t* x_s, int64_t T, int64_t G, int64_t D,
                           void* y, void* stream);

/* ---- residual, RMSNorm and 8-bit rows ---------------------------------------------------
 * What stands in front of a layer's projections, in one pass: the residual's addition, the norm
 * of "DeepSeek V4 950 低精度优化全复盘" section 2.3 and the quantisation that the payload reads.
 * x, residual: bf16 [M, K], row strides ldx, ldr (elements); residual may be NULL.
 *   h[k] = bf16_RN(x[k] + residual[k])                    (x[k] without a residual)
 *   v[k] = (h[k] * inv) * rms_gamma[k],  inv = 1 / sqrt(f32(sum_k h^2 / K) + rms_eps)
 * with the sum in f64 and every other step one f32 rounding; v is not rounded before its codes.
 * sum: bf16 [M, K], row stride lds, gets h; y: bf16 [M, K], row stride ldy, gets bf16_RN(v); either
 * may be NULL, and sum may be x or residual itself, at its own stride (the residual stream in
 * place); outputs overlap nothing else.
 *   WQ_PAYLOAD_INT8: x_q int8 [M, K], x_s f32 [M], as wq_dynamic_quant:
 *     x_s = RN(max |v| / 127), x_q = rint(RN(v / x_s))    (0 where the row is 0); K % 16 == 0
 *   WQ_PAYLOAD_FP8_E4M3, WQ_PAYLOAD_MXFP8: x_q E4M3 codes [M, K], x_s the packed words
 *     [1, PH, TA] of wq_group_quant_fp8_ue8m0 and wq_group_quant_mxfp8 with G = 1 (TA = 4 ceil(M / 4)):
 *     e = max(-127, smallest e with 448 * 2^e >= max |v| of the block), x_q = E4M3FN(v * 2^-e);
 *     K % 128 == 0, K % 32 == 0; every word's byte that stands for no block is zero.
 *   Other payloads: WQ_ERR_UNSUPPORTED.
 * A row whose h holds a NaN or an infinity has v = NaN throughout.  A row of INT8 or a block that
 * holds a value that is not finite gets zero codes and the scale NaN, or byte 255, UE8M0's NaN:
 * products with it give NaN.  1 <= K <= 65536. */
int wq_add_rms_quant(wq_ctx* ctx, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                     const void* rms_gamma, float rms_eps, int64_t M, int64_t K, int payload, void* x_q, void* x_s,
                     void* sum, int64_t lds, void* y, int64_t ldy, void* stream);

/* ---- quantised matmul ---------------------------------------------------------------
 * INT8 (section 一 of the W8A8 article; npu_quant_matmul, and the tuple-reuse path where
 * an upstream producer already gave (x_q, x_scale)):
 *   acc[m, n] = sum_k a[m, k] * b[n, k]                    (exact int32)
 *   y[m, n]   = bf16_RN((f32(acc) * a_scale[m]) * b_scale[n])            (WQ_EPI_BF16)
 * WQ_EPI_SWIGLU_F32 (MoE gate/up, "DeepSeek V4 950" section 2.3): with N = 2I,
 *   g = (f32(acc[m, n]) * a_scale[m]) * b_scale[n],  u likewise for column n + I,
 *   y[m, n] = f32( g / (1 + exp(-g)) * u )  for n < I   (f32 [M, I]; exp is the fixed
 *   f32 sequence: n = rint(x*log2e), Cody-Waite r, degree-7 Taylor Horner, ldexp).
 * Segments (MoE, section 五 of the W8A8 article: group_list = tokens per expert):
 *   batch = E experts and seg_offsets = device int64 [E + 1], non-decreasing, with
 *   seg_offsets[E] == M; rows [seg_offsets[e], seg_offsets[e+1]) use b + e*b_batch_stride
 *   and b_scale + e*N.  Segments need K % 128 == 0, E + ceil(M / 128) <= 4096 and no
 *   acc_out (else WQ_ERR_UNSUPPORTED); WQ_EPI_SWIGLU_F32 is available with segments only
 *   and needs N % 256 == 0 (WQ_ERR_SHAPE otherwise).
 * FP8 (SGLang PR #34277: the grouped contraction that reads the packed scales):
 *   payload WQ_PAYLOAD_FP8_E4M3, batch = G groups, a = E4M3 codes with row stride lda
 *   bytes and group stride a_batch_stride bytes; a_scale = the int32 packed storage
 *   [G, PH, TA] written by wq_group_quant_fp8_ue8m0 with TA = a_scale_tokens; b = E4M3
 *   [G][N][K]; b_scale = f32 powers of two [G][N/128][K/128] (the kernels pass each scale's
 *   exponent field to the matrix unit as its E8M0 scale, so a value that is not a normal
 *   power of two acts as 2^(its biased exponent - 127): its mantissa is ignored, and zero
 *   or a subnormal acts as 2^-127); K <= 131072 (else WQ_ERR_SHAPE);
 *   y[m, g, n] = bf16_RN( sum_kb 2^(e_a(m,g,kb)) * b_scale[g, n/128, kb]
 *                         * sum_{k in block kb} a[m, g, k] * b[g, n, k] )   (f32 accumulate)
 * MX-like 32-element blocks ("DeepSeek V4 950 低精度优化全复盘", section 2.1): payload
 *   WQ_PAYLOAD_MXFP8, as the FP8 payload but a_scale = the storage of wq_group_quant_mxfp8
 *   ([G, K/128, TA]) and b_scale pointing at UE8M0 bytes [G][N][K/32] (not floats);
 *   y[m, g, n] = bf16_RN( sum over 32-deep blocks kb of 2^(e_a(m,g,kb))
 *                         * 2^(b_scale[g, n, kb] - 127) * sum_{k in kb} a[m,g,k] * b[g,n,k] );
 *   any M (decode-sized M on the weight-streaming kernel, larger M on the tiled one).
 * 4-bit weights in 32-element blocks: payload WQ_PAYLOAD_MXFP4 (a = E2M1 pairs of
 *   wq_group_quant_mxfp4, K/2 bytes a row) or WQ_PAYLOAD_MXFP8_W4 (a = E4M3 codes of
 *   wq_group_quant_mxfp8, K bytes a row); lda (< 2^23) and a_batch_stride in bytes; a_scale = that
 *   call's storage [G, K/128, TA]; b = E2M1 pairs [G][N][K/2], b_batch_stride in bytes;
 *   b_scale = int32 words [G][K/128][N], the storage of wq_group_quant_mxfp4 on each group's
 *   weights (not floats); any M, N % 16 == 0, K % 128 == 0, K <= 131072, G <= 65535, fewer than
 *   2^24 tiles of 128 x 256 (WQ_ERR_SHAPE otherwise);
 *   y[m, g, n] = bf16_RN( sum over 32-deep blocks of 2^(e_a + e_b) sum_{k in kb} a b ).
 *   seg_offsets, acc_out, WQ_EPI_SWIGLU_F32 and WQ_LAYOUT_FRAGMENT: WQ_ERR_UNSUPPORTED.
 * acc_out (INT8 dense only, may be NULL): the raw int32 accumulators [M, N], row stride N. */
typedef struct {
  int32_t payload;         /* one of WQ_PAYLOAD_...                                       */
  int32_t epilogue;        /* WQ_EPI_BF16 or WQ_EPI_SWIGLU_F32                            */
  int64_t M, N, K;         /* rows (per batch for strided batches), columns, depth        */
  int64_t batch;           /* 1 = dense; G for FP8 groups; E for segments                 */
  const int64_t* seg_offsets; /* device int64 [batch + 1] for segments, else NULL         */
  const void* a;           /* payload rows                                                */
  int64_t lda;             /* row stride of a in elements (bytes: 1-byte payloads)        */
  int64_t a_batch_stride;  /* elements between batches of a (strided batches)             */
  const void* a_scale;     /* INT8: f32 [M]; FP8: int32 packed storage [batch, PH, TA]    */
  int64_t a_scale_tokens;  /* FP8: TA, the token stride of the packed storage             */
  const void* b;           /* weights [batch][N][K]                                       */
  int64_t b_batch_stride;  /* elements between batches of b                               */
  const float* b_scale;    /* INT8: [batch][N]; FP8: [batch][N/128][K/128]                */
  void* y;                 /* output                                                      */
  int64_t ldy;             /* row stride of y in elements                                 */
  int64_t y_batch_stride;  /* elements between batches of y (strided batches)             */
  int32_t* acc_out;        /* optional raw INT8 accumulators [M, N]                       */
  int32_t b_layout;        /* WQ_LAYOUT_PLAIN, or WQ_LAYOUT_FRAGMENT: the [N][K] weights (of
                              every expert) cast by wq_pack_weight_i8, same b_batch_stride.
                              INT8 only, with seg_offsets, or dense with M < 256,
                              K % 512 == 0, K <= 4096 and WQ_EPI_BF16; other combinations
                              give WQ_ERR_UNSUPPORTED.  Outputs are the same bytes as with
                              the plain layout.                                             */
  int64_t expected_rows;   /* segments: the rows per expert the caller expects (the
                              expected-tokens hint of section 五 of the W8A8 article, which
                              picks the grouped GEMM's tiling from it); 0 = no hint, and the
                              context's WQ_EXPECTED_TOKENS applies.  It selects kernels only:
                              above 64 no expert goes to the 16-row streaming kernel; at
                              most 128, no 256-row tiles (one launch fewer).  Every value
                              gives the same bytes; row counts may differ from it freely.   */
} wq_matmul_desc;

int wq_quant_matmul(wq_ctx* ctx, const wq_matmul_desc* desc, void* stream);

/* Which kernel a product on 4-bit weights (WQ_PAYLOAD_MXFP4, WQ_PAYLOAD_MXFP8_W4) of these sizes
 * takes: the weights' stream in 1 = 16 or 2 = 32 columns a workgroup, or tiles of 3 = 64 x 64,
 * 4 = 64 x 128 or 5 = 128 x 256 outputs.  0 for an empty problem; a negative value is -status.
 * Host only: no device work. */
int wq_mx4_path(const wq_ctx* ctx, int64_t M, int64_t N, int64_t K, int64_t batch);

/* ---- fused quant + INT8 GEMM -------------------------------------------------------
 * The whole chain of section 一 of the W8A8 article: per-token quant of the bf16 x [M, K]
 * (row stride ldx), the INT8 GEMM against w [N, K] and the bf16 epilogue.  Outputs are
 * bit-identical to wq_dynamic_quant followed by wq_quant_matmul.  y: bf16 [M, N] row
 * stride ldy.  For M up to the one-launch limit (WQ_FUSED_MAX_M, default 255) one kernel
 * quantises in registers and never writes the INT8 payload to HBM; above it the call runs
 * the quant and the GEMM as two launches, staging the payload in x_q_out / x_scale_out
 * when given, else in the context workspace (WQ_ERR_WORKSPACE if M*K bytes exceed it).
 * The optional outputs export the (x_q, x_scale) tuple and the int32 accumulators so a
 * downstream Linear can reuse them (the tuple-reuse path of section 一). */
int wq_fused_quant_matmul(wq_ctx* ctx, const void* x, int64_t M, int64_t K, int64_t ldx,
                          const int8_t* w, const float* w_scale, int64_t N, void* y, int64_t ldy,
                          int8_t* x_q_out, float* x_scale_out, int32_t* acc_out, void* stream);

/* For callers that cannot allocate device memory: code under HIP graph capture, serving
 * loops that must not allocate, harnesses that forbid it.  wq_fused_quant_matmul with no
 * context and no workspace: `device` is the HIP device index, every other argument and the
 * outputs are those of wq_fused_quant_matmul, bit for bit (the knobs come from the same
 * environment variables, read on every call).  When M is above the one-launch limit and
 * x_q_out / x_scale_out are NULL, the INT8 payload and its scales are staged in a static
 * device buffer of the library instead of a context workspace: at most 16 MiB of payload
 * (M * K bytes) and 16384 scales (M <= 16384); larger calls return WQ_ERR_WORKSPACE and launch
 * nothing.  Each device the library runs on holds that buffer (16 MiB + 64 KiB) until the
 * process ends; the first call on a device looks up its address there, later calls only
 * launch.  The call allocates nothing (no hipMalloc, no hipFree, no host heap).  Calls on one
 * device share the buffer: two such calls that may overlap in time (on different streams, or
 * from different host threads) race and must be serialised by the caller.  WQ_ERR_DEVICE for
 * an invalid or non-gfx950 device. */
int wq_fused_quant_matmul_static(int device, const void* x, int64_t M, int64_t K, int64_t ldx,
                                 const int8_t* w, const float* w_scale, int64_t N, void* y, int64_t ldy,
                                 int8_t* x_q_out, float* x_scale_out, int32_t* acc_out, void* stream);

/* Which launch sequence wq_fused_quant_matmul takes for these sizes on this context:
 * 0 = the quant kernel, then the GEMM (two launches); 1 = one launch of the dot4 GEMV
 * kernel (M <= WQ_FUSED_GEMV_MAX_M, or M <= 4 with a K the MFMA kernel does not take:
 * K % 512 != 0 or 4096 < K <= 8192); 2 = one launch of the 8-wave MFMA kernel
 * (K % 512 == 0, K <= 4096), its rows and columns per workgroup chosen from M and N.
 * A negative value is -status for invalid sizes (M < 1, or K, N as wq_fused_quant_matmul
 * requires).  Host only: no device work. */
int wq_fused_path(const wq_ctx* ctx, int64_t M, int64_t K, int64_t N);

/* ---- weight pre-pack (fragment order) ------------------------------------------------
 * Section 四 of the W8A8 article: the weights are cast once at load time into the layout
 * the matrix unit reads (FRACTAL_NZ there).  The gfx950 form here is fragment order: for
 * the int8 weight w [N, K] (row stride ldw bytes), byte (n, k) goes to
 *   wp[((k/64 * N/4 + n/4) * 4 + (k%64)/16) * 64 + (n%4) * 16 + k%16],
 * so for each 64-deep K step the 4-column blocks follow one another, each 256 bytes as
 * [K quarter 0..3][column 0..3][16 bytes], and the 16 columns x 64 K bytes of one
 * v_mfma_i32_16x16x64_i8 B operand are 1 KiB contiguous in lane order.  wp: int8, N*K
 * bytes, caller-allocated, 16-byte aligned; w 16-byte aligned, ldw % 16 == 0, ldw >= K.
 * N % 16 == 0, K % 64 == 0 (else WQ_ERR_SHAPE).  One device-side permutation on `stream`;
 * w and wp must not overlap. */
int wq_pack_weight_i8(wq_ctx* ctx, const int8_t* w, int64_t N, int64_t K, int64_t ldw, int8_t* wp,
                      void* stream);

/* wq_fused_quant_matmul with the weights in fragment order (wp from wq_pack_weight_i8),
 * same arguments otherwise and bit-identical outputs.  Only the one-launch MFMA path:
 * 1 <= M <= 255 (and M <= WQ_FUSED_MAX_M), K % 512 == 0, K <= 4096, N % 16 == 0; other
 * sizes give WQ_ERR_SHAPE (M = 0 returns WQ_OK with nothing launched). */
int wq_fused_quant_matmul_packed(wq_ctx* ctx, const void* x, int64_t M, int64_t K, int64_t ldx,
                                 const int8_t* wp, const float* w_scale, int64_t N, void* y, int64_t ldy,
                                 int8_t* x_q_out, float* x_scale_out, int32_t* acc_out, void* stream);

/* ---- paged 8-bit cache of keys and values, and attention over it -------------------------
 * A page holds page_tokens consecutive tokens of a sequence, for every head, in 8-bit codes
 * with one UE8M0 byte for each (page, head) of keys and of values:
 *   x = code * 2^(byte - 127); code E4M3 (WQ_KV_E4M3) or int8 (WQ_KV_INT8).
 * Values lie with the tokens innermost (the order the matrix unit contracts them in).
 * table[b][i] is the page of tokens i * page_tokens .. of sequence b.  A page number outside
 * [0, pages) is no page: what would be written there is dropped, its tokens are not attended.
 * Rows belong to sequences by offsets: device int64 [B + 1], non-decreasing from 0; rows
 * [offsets[b], offsets[b+1]) are the newest tokens of sequence b in order, and lens[b] (device
 * int32) is its token count with them, so row i of n has position lens[b] - n + i.  A token at
 * a negative position or behind max_pages * page_tokens is not written and not attended;
 * rows behind offsets[B] are not read, and their outputs stay as they were. */
typedef struct {
  int32_t code;            /* WQ_KV_E4M3 or WQ_KV_INT8                                    */
  int64_t pages, heads;    /* 1 .. 2^31 - 1 pages, 1 .. 65535 heads                       */
  int64_t page_tokens;     /* a multiple of 16, 16 .. 256                                 */
  int64_t head_dim;        /* 64, 128 or 256                                              */
  void* k;                 /* codes [pages][heads][page_tokens][head_dim]                 */
  void* v;                 /* codes [pages][heads][head_dim][page_tokens]                 */
  uint8_t* k_scale;        /* UE8M0 bytes [pages][heads]                                  */
  uint8_t* v_scale;        /* UE8M0 bytes [pages][heads]                                  */
  const int32_t* table;    /* device [B][table_stride]                                    */
  int64_t table_stride;    /* entries between sequences                                   */
  int64_t max_pages;       /* entries of a sequence, <= table_stride                      */
} wq_kv_cache;

/* Quantise new rows into the cache.  k_new, v_new: bf16 [T, heads * head_dim], row strides
 * ldk, ldv (elements).  For each (page, head) that rows fall in, with a = max |x| of them and
 * e = max(-127, smallest e with 2^e >= a / c), c = 448 (E4M3) or 127 (int8):
 *   a page whose first slot is among them is begun anew with byte e + 127; in any other the
 *   byte becomes max(its byte, e + 127), and where it grows, by d, the codes in front of the
 *   new rows become RN(code * 2^-d);
 *   the new codes are RN(x * 2^(127 - byte)) (nearest-even).  Slots behind them keep their codes.
 * A NaN or an infinity among the rows makes the byte 255 (UE8M0's NaN) and their codes zero:
 * the page's tokens of that head read as NaN until the page is begun anew.
 * Magnitudes from 1.9375 * 2^127 (E4M3) or 1.9921875 * 2^127 (int8) on round up to 2^128, which reads
 * as infinity, and from a page of E4M3 codes may reach as NaN rows of its sequence that do not see it.
 * The same call again writes the same bytes.  A page written by the call stands in one place
 * of the tables (a shared one is copied first). */
int wq_kv_append(wq_ctx* ctx, const wq_kv_cache* cache, const void* k_new, int64_t ldk, const void* v_new, int64_t ldv,
                 int64_t T, int64_t B, const int64_t* offsets, const int32_t* lens, void* stream);

/* wq_kv_append with the keys turned by their tokens' positions on the way (rotary positions), and
 * the queries of the same rows turned by the same angles, in one launch.
 * angles: f32 [positions][2][rot_dim / 2], for each position the cosines and then the sines of its
 * frequencies (made once); 16 <= rot_dim <= head_dim, rot_dim % 16 == 0.  Of each head the first
 * rot_dim elements are turned in pairs (a, b): elements (i, i + rot_dim / 2), or (2 i, 2 i + 1) with
 * interleaved != 0, by frequency i:
 *   a' = a c - b s,  b' = b c + a s                       (f32, each product and sum rounded)
 * The position is the token's in its sequence, lens[b] - n + i for row i of n.  Keys go to their
 * codes from a' and b' as they are (in wq_kv_append's rules read them for x), values as in
 * wq_kv_append; q_out gets bf16_RN of the queries.  q, q_out: bf16 [T, q_heads * head_dim], row
 * strides ldq, ldo, q_heads a multiple of the cache's heads; q_out may be q at the same stride; both
 * NULL: no queries.  A position outside [0, positions) has no angle: its elements in pairs become
 * NaN (a key's page is then marked as wq_kv_append marks it; tokens at negative positions are not
 * written).  Rows of no sequence are left as they are in q_out. */
int wq_kv_append_rotated(wq_ctx* ctx, const wq_kv_cache* cache, const void* k_new, int64_t ldk, const void* v_new,
                         int64_t ldv, const void* q, int64_t ldq, int64_t q_heads, void* q_out, int64_t ldo,
                         const float* angles, int64_t positions, int64_t rot_dim, int interleaved, int64_t T,
                         int64_t B, const int64_t* offsets, const int32_t* lens, void* stream);

/* Attention of T query rows over the cache: q bf16 [T, q_heads * head_dim], row stride ldq;
 * q_heads = R * heads, query head i reads cache head i / R.  Row i of n of sequence b sees the
 * tokens 0 .. lens[b] - n + i (causal != 0) or 0 .. lens[b] - 1:
 *   s_j = scale * sum_d q_d k_jd,  lse = log sum_j exp(s_j),  out_d = sum_j exp(s_j - lse) v_jd
 * out: bf16 [T, q_heads * head_dim], row stride ldo (it may not overlap q); lse: f32
 * [T, q_heads] or NULL.  A row that sees no token gets zeros and lse = -inf; one that sees a
 * token of a page and head whose keys' or values' byte is 255, or that sees a token and holds
 * a NaN itself, gets NaN for both.  Codes behind
 * lens[b] may hold anything; E4M3's NaN patterns in front of it, which wq_kv_append never
 * writes, may reach rows that do not see them.  The products take the codes exactly (bf16),
 * sums and softmax statistics are f32, and a weight exp(s - max) is rounded to bf16.
 * Any finite scale is taken, beside any byte; sum_d |q_d code_jd| and the values' sums weighted by
 * exp(s - max) have to stay below 2^128.
 * workspace: device memory, 16-byte aligned, of at least wq_kv_attention_workspace_bytes()
 * for these sizes, that no other call uses until this one is done (the parts of a sequence
 * that is split over workgroups are joined there); its contents need no initialisation.  NULL:
 * the context's workspace, with the context's rule of one stream at a time. */
int wq_kv_attention(wq_ctx* ctx, const wq_kv_cache* cache, const void* q, int64_t ldq, int64_t T, int64_t q_heads,
                    int64_t B, const int64_t* offsets, const int32_t* lens, float scale, int causal, void* out,
                    int64_t ldo, float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* The bytes of workspace that wq_kv_attention takes for these sizes (of the cache: heads,
 * page_tokens, head_dim and max_pages; no pointer is read), at most 64 MiB; 0 where it needs none; a
 * negative value is -status.  Host only: no device work. */
int64_t wq_kv_attention_workspace_bytes(const wq_ctx* ctx, const wq_kv_cache* cache, int64_t T, int64_t q_heads,
                                        int64_t B);

/* Which kernels wq_kv_attention takes for these sizes (read as for the workspace):
 *   1  whole row tiles of 128 rows (64 for heads of 256) of one sequence and head
 *   2, 3  16-row, 64-row tiles, a workgroup for each (sequence, head, tile)
 *   4, 5  16-row, 64-row tiles, their work cut into equal runs, with a join of the parts;
 *   8 more where the items are few and their parts many, so that a join is split over columns.
 * 0 for an empty problem; a negative value is -status.  Host only: no device work. */
int wq_kv_attention_path(const wq_ctx* ctx, const wq_kv_cache* cache, int64_t T, int64_t q_heads, int64_t B);

/* wq_kv_attention of sequences that begin with the same pages (a system prompt, several answers to
 * one question): the same rows, masks and outputs, with what is shared read once for every 256 of the
 * rows that share it (new rows times q_heads / heads; 128 with heads of 256).  group, shared: device
 * int32 [B].  Neighbouring sequences with the same id, not negative, are a group; shared[b] is the
 * number of tokens from its first on that sequence b has in common with the others of its group, in
 * the same pages: the tables' first floor(shared / page_tokens) entries are equal over the group
 * (where they are not, the entries of its first sequence with rows are taken).  A group's least such
 * number counts, in whole pages and whole steps of 64 tokens, and no more than every row of it sees;
 * the remaining tokens are read for each sequence.  Results differ from wq_kv_attention's by the order of f32 sums and by the weights'
 * rounding to bf16: each is off by at most 2^-8 of itself, as there, but here the largest is rounded
 * too and the quotient is over the rounded weights' sum, so that an output is off by at most 2^-8 of
 * the weighted sum of |value - output| (lse is of the weights as they are).  Weights are up to 2^8
 * here, so that the values' weighted sums have to stay below 2^120, and int8 pages with values that
 * read as infinity may reach as NaN rows that do not see them, as those of E4M3 codes may there.
 * The call shares whatever it is told, also where wq_kv_attention would be quicker: for single tokens
 * it pays from about 1000 shared tokens on (2000 to 4000 for 8 sequences with heads of 64; from a
 * few hundred with heads of 256; at any number for 200 sequences of 500 own tokens with heads of
 * 128), and below that it may take twice as long; prompts of 64 new tokens and more take 1 to 1.6 times
 * as long behind 512 tokens (heads of 64: 1.9) and 0.6 to 1.1 times behind 4096.
 * workspace: as there, of at least wq_kv_attention_shared_workspace_bytes(); NULL: the context's
 * (WQ_ERR_WORKSPACE where that is too small). */
int wq_kv_attention_shared(wq_ctx* ctx, const wq_kv_cache* cache, const void* q, int64_t ldq, int64_t T,
                           int64_t q_heads, int64_t B, const int64_t* offsets, const int32_t* lens,
                           const int32_t* group, const int32_t* shared, float scale, int causal, void* out,
                           int64_t ldo, float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* As wq_kv_attention_workspace_bytes, of wq_kv_attention_shared: two f32 rows for every output row (a row
 * and query head), 8 head_dim + 32 bytes, besides the workgroups' own (51 MB on 256 CUs with heads of
 * 128).  It grows with T and is not bounded by the context's workspace: 64 sequences of 500 new tokens
 * with 32 heads of 128 take 1.1 GB, single tokens of 512 sequences 68 MB. */
int64_t wq_kv_attention_shared_workspace_bytes(const wq_ctx* ctx, const wq_kv_cache* cache, int64_t T,
                                               int64_t q_heads, int64_t B);

/* As wq_kv_attention_path, of wq_kv_attention_shared: 16 where the shared tokens are taken once;
 * sequences of 2048 rows and more on average (rows times q_heads / heads) fill row tiles of their own
 * and take wq_kv_attention's kernels, numbered as there. */
int wq_kv_attention_shared_path(const wq_ctx* ctx, const wq_kv_cache* cache, int64_t T, int64_t q_heads, int64_t B);

/* ---- expert sort (MoE) ---------------------------------------------------------------
 * "DeepSeek V4 950" section 3.2: sort the (token, slot) pairs by expert id before the
 * gather so each expert's rows are contiguous.  topk_ids: int32 [T, topk], values in
 * [0, E).  Outputs: perm int32 [T*topk] (flattened pair index t*topk + slot of each sorted
 * row; stable: ties keep pair order), row_token int32 [T*topk] (= perm / topk),
 * offsets int64 [E + 1] (exclusive prefix sum of rows per expert; the group_list of
 * section 五 of the W8A8 article).  An id outside [0, E) drops its pair: the kept pairs are
 * sorted as above, offsets[E] is their count, and the slots from offsets[E] to T*topk get
 * perm = -1 and row_token = 0, so a gather over all T*topk rows stays in bounds. */
int wq_moe_sort(wq_ctx* ctx, const int32_t* topk_ids, int64_t T, int64_t topk, int64_t E,
                int32_t* perm, int32_t* row_token, int64_t* offsets, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* WQ_H */
