/*
 * svdq.h -- C ABI of the fused SVDQuant W4A4 linear layer for AMD Instinct
 * MI355X (gfx950).
 *
 * The layer (SVDQuant, Li, Lin, Zhang, Cai, Li, Guo, Xie, Meng, Zhu, Han 2024,
 * as described by the practice page "sota-314", section "Do this", and the
 * reading note "note-257", section "Key results"):
 *
 *     Y = X_hat L1 L2  +  Q(X_hat) Q(R)  +  b,     R = W_hat - L1 L2,
 *
 * where X_hat / W_hat are the smoothed activations / weight, L1 L2 is the
 * 16-bit rank-r branch taken off W_hat by truncated SVD, and Q() is per-group
 * symmetric quantization along the reduction axis K.  The two fusions the
 * pages name are the two kernels behind this ABI:
 *   Kernel A  (svdq_quantize_down): quantize X_hat and compute the down
 *             projection T = X_hat L1 in the same pass (same input);
 *   Kernel B  (svdq_gemm_w4a4_up):  the low-bit GEMM with the up projection
 *             T L2 and the bias in its epilogue (same output).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Tensor pointers are DEVICE pointers, owned by the caller, row-major,
 *    16-byte aligned.  The library never allocates or frees memory and keeps
 *    no mutable global state beyond a per-device cache of the compute-unit
 *    count (set atomically on first use); calls are thread-safe.
 *  - `stream` is a hipStream_t (NULL = the default stream).  All work is
 *    enqueued on it asynchronously; nothing synchronizes the device and there
 *    are no host<->device copies.
 *  - Arguments are validated on the host before any HIP call; a failed check
 *    returns an error status and enqueues nothing.  A launch failure reported
 *    by the runtime returns SVDQ_ERR_LAUNCH.  No C++ exception crosses the ABI.
 *  - Shapes: M >= 0 and N >= 0 (0 = nothing to do: SVDQ_OK once the format
 *    and the other dimensions check out, and the pointers may then be NULL,
 *    as a zero-size tensor's are); K > 0 with
 *    K % 64 == 0; N % 16 == 0; r % 16 == 0 and 0 <= r <= 64; M, N, K <= 2^24;
 *    the GEMM entry points also need each code operand (M and N times the
 *    format's code bytes per row) below 4 GiB, and the W4A16 control needs
 *    M * 2K and N * K/2 bytes below 4 GiB.
 *  - Non-finite inputs are undefined behaviour.
 *
 * Formats (group quantization along K; groups per token row for activations,
 * per output column for the weight; "sota-314", "Do this": INT4 group 64 with
 * 16-bit scales, NVFP4 group 16 with FP8 scales, rank 16 at 8 bits):
 *  SVDQ_INT4_G64 : codes in [-7, 7], two's-complement nibbles, two per byte
 *                  (byte b = code 2b | code 2b+1 << 4); fp16 scale per 64.
 *                  scale = fp16_rne(fp32(absmax) / 7.0f); code =
 *                  clamp(rint_half_even(fp32(v) / scale), -7, 7); scale 0 ->
 *                  codes 0.  Codes group-major [K/64][rows][32 bytes] (group g
 *                  of row i at byte (g * rows + i) * 32), fp16 scales
 *                  group-major [K/64][rows]: a GEMM tile's rows of one group
 *                  are one contiguous run.
 *  SVDQ_INT8_G64 : same rule with 127; one int8 code per byte.  Codes
 *                  group-major [K/64][rows][64 bytes] (group g of row i at
 *                  byte (g * rows + i) * 64), fp16 scales group-major
 *                  [K/64][rows]: a GEMM tile's rows of one group are one
 *                  contiguous run.
 *  SVDQ_FP4_G16  : E2M1 codes (sign<<3 | magnitude index, magnitudes
 *                  0,0.5,1,1.5,2,3,4,6), packed as INT4; one E4M3FN scale byte
 *                  per 16: scale = e4m3_rne_sat(fp32(absmax) / 6.0f); code =
 *                  nearest E2M1 to fp32(v)/scale, ties to the even mantissa,
 *                  -0 -> +0.  Codes chunk-major [K/64][rows][32 bytes] (chunk c of
 *                  row i at byte (c * rows + i) * 32, two codes per byte as
 *                  above), E4M3 bytes [K/64][rows][4].
 *  SVDQ_INT4_G64_E2M3 : the SVDQ_INT4_G64 codes and scales, bit for bit, in the
 *                  storage the gfx950 FP6 matrix cores read directly: each code
 *                  q becomes the 6-bit E2M3 pattern of q/8 (a subnormal:
 *                  sign<<5 | |q|).  A row takes 48 bytes per group of 64:
 *                  each half of the group (codes 0..31, 32..63) is a 24-byte
 *                  little-endian field string, code j of the half in bits
 *                  [6j, 6j+6); the 48 bytes hold half 0 bytes 0..15, half 1
 *                  bytes 0..15, half 0 bytes 16..23, half 1 bytes 16..23 (so
 *                  each half is one 16-byte and one 8-byte aligned piece).
 *                  Codes and scales are group-major:
 *                  codes [K/64][rows][48 bytes] (the group-g slice of row i at
 *                  byte (g * rows + i) * 48; 3K/4 bytes per row in total),
 *                  fp16 scales [K/64][rows].  The 4-bit values
 *                  sit in a 6-bit container (1.5x the bytes of SVDQ_INT4_G64)
 *                  so that the GEMM runs on the FP6 matrix cores, which return
 *                  fp32 partials and, measured on MI355X, do 1.57x the INT8
 *                  instruction's work per K element.
 *  SVDQ_MXFP4_G32 : MXFP4 (OCP Microscaling Formats v1.0), the block-scaled
 *                  format gfx950's matrix cores apply natively ("sota-314",
 *                  "Conditions": the format ranking follows the hardware's
 *                  native group support; "Quantization", "KV cache
 *                  quantization": OCP MXFP4 among the production formats).
 *                  E2M1 codes packed as SVDQ_FP4_G16, one E8M0 byte per 32
 *                  along K: e = floor(log2 absmax) - 2 clamped to [-127, 127]
 *                  (-127 for an all-zero group), byte = e + 127; code =
 *                  nearest E2M1 to v / 2^e (exact division), ties to the even
 *                  mantissa, saturating at 6, -0 -> +0.  Codes and scales are
 *                  chunk-major, so that a tile's rows of one 64-wide chunk of K
 *                  are contiguous: codes [K/64][rows][32 bytes] (chunk c of
 *                  row i at byte (c * rows + i) * 32; within it the two 16-byte
 *                  halves are the groups, two codes per byte as SVDQ_FP4_G16),
 *                  E8M0 bytes [K/64][rows][2].
 */
#ifndef SVDQ_H
#define SVDQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SVDQ_OK = 0,
  SVDQ_ERR_NULL = -1,      /* a required pointer is NULL                         */
  SVDQ_ERR_SHAPE = -2,     /* M/N/K/r/C outside the documented constraints       */
  SVDQ_ERR_ALIGN = -3,     /* a pointer is not 16-byte aligned                   */
  SVDQ_ERR_FORMAT = -4,    /* unknown or unsupported format for this entry point */
  SVDQ_ERR_WORKSPACE = -5, /* workspace smaller than the *_workspace_bytes value */
  SVDQ_ERR_DEVICE = -6,    /* the current device is not a gfx950 GPU             */
  SVDQ_ERR_LAUNCH = -7     /* the HIP runtime reported a launch error            */
} svdq_status;

typedef enum {
  SVDQ_INT4_G64 = 0,
  SVDQ_INT8_G64 = 1,
  SVDQ_FP4_G16 = 2,
  SVDQ_INT4_G64_E2M3 = 3,
  SVDQ_MXFP4_G32 = 4,
  /* Not formats: these two make the type span every int, so that any value a caller passes is
   * a valid value of the type (in C++ an enum holds only the values its enumerators' range
   * covers) and an unknown one is rejected with SVDQ_ERR_FORMAT. */
  SVDQ_FORMAT_INT_MIN_ = -2147483647 - 1,
  SVDQ_FORMAT_INT_MAX_ = 2147483647
} svdq_format;

/* Bytes of codes per row for K columns (K/2 for 4-bit formats, K for INT8,
 * 3K/4 for the E2M3 container; the device layouts interleave the rows group by
 * group), and bytes of scales per row (K/64 fp16 for the INT formats, K/16 E4M3
 * bytes for FP4, K/32 E8M0 bytes for MXFP4).  Returns 0 for a bad format. */
size_t svdq_code_row_bytes(int K, svdq_format fmt);
size_t svdq_scale_row_bytes(int K, svdq_format fmt);

/*
 * Kernel A: quantize + down projection ("sota-314", "Do this": the down
 * projection is fused with quantization since both consume X_hat;
 * "note-257", "Key results").
 *   x_hat : fp16 [M, K], the smoothed activations (smoothing already applied).
 *   l1t   : fp16 [r, K] = L1^T; NULL iff r == 0.
 *   xq    : out, codes, M * code_row_bytes(K) bytes in the format's layout.
 *   xs    : out, scales, M * scale_row_bytes(K) bytes in the format's layout.
 *   t     : out, fp16 [M, r] = fp16_rne(X_hat L1), fp32 accumulation; NULL iff r == 0.
 *   workspace, workspace_bytes : caller-owned device scratch for the fp32
 *           partial sums of T when the kernel slices K across workgroups
 *           (svdq_quantize_down_workspace_bytes; 16-byte aligned).  Its
 *           contents need no initialisation and are dead after the call; two
 *           calls in flight at once need two workspaces.  NULL is allowed: K
 *           is then not sliced for r > 0 (same results, slower for long K);
 *           a non-NULL workspace that is too small is SVDQ_ERR_WORKSPACE.
 * The branch reads the unquantized 16-bit X_hat.  Results do not depend on
 * the workspace: the slices' partials are added in a fixed order.
 */
svdq_status svdq_quantize_down(const void* x_hat, const void* l1t, int M, int K, int r,
                               svdq_format fmt, void* xq, void* xs, void* t, void* workspace,
                               size_t workspace_bytes, void* stream);

/* Workspace bytes svdq_quantize_down uses to slice K (0: no slicing for this
 * shape, or r == 0, or a bad format or shape). */
size_t svdq_quantize_down_workspace_bytes(int M, int K, int r, svdq_format fmt);

/*
 * Kernel B: low-bit GEMM + up projection + bias ("sota-314", "Do this": the up
 * projection is fused with the 4-bit compute because both write the same
 * output).
 *   Y = fp16_rne( sum_g sx[m,g] sw[n,g] P_g[m,n] + T L2 + b ),
 *   P_g = sum over the group's K of q_x q_w (exact integers; fp32 accumulation
 *   of the rescaled partials).
 *   xq, xs : Kernel A's codes and scales for M rows.
 *   t      : fp16 [M, r]; NULL iff r == 0.
 *   wq     : codes of the N output columns, N * code_row_bytes(K) bytes in the
 *            format's layout (rows = output columns).
 *   ws     : their scales, N * scale_row_bytes(K) bytes in the format's layout.
 *   l2     : fp16 [r, N]; NULL iff r == 0.
 *   bias   : fp16 [N], or NULL for none.
 *   y      : out, fp16 [M, N].
 * r == 0 selects the bare low-bit GEMM (no branch).
 */
svdq_status svdq_gemm_w4a4_up(const void* xq, const void* xs, const void* t, const void* wq,
                              const void* ws, const void* l2, const void* bias, int M, int N, int K,
                              int r, svdq_format fmt, void* y, void* stream);

/* Workspace svdq_linear needs: codes, scales and T for M rows, and Kernel A's
 * partial sums (svdq_quantize_down_workspace_bytes), each part 256-byte
 * aligned.  0 for a bad format or shape. */
size_t svdq_linear_workspace_bytes(int M, int K, int r, svdq_format fmt);

/*
 * The fused layer: Kernel A then Kernel B on one stream, with codes, scales
 * and T in the caller's workspace (>= svdq_linear_workspace_bytes).
 * Arguments as for the two kernels above.
 */
svdq_status svdq_linear(const void* x_hat, const void* l1t, const void* wq, const void* ws,
                        const void* l2, const void* bias, int M, int N, int K, int r,
                        svdq_format fmt, void* workspace, size_t workspace_bytes, void* y,
                        void* stream);

/*
 * The fused layer without a workspace argument, for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): svdq_linear with its codes, scales, T and Kernel A's partial sums in a static
 * device array of SVDQ_STATIC_SCRATCH_BYTES inside the library.  Each GPU the library runs on
 * holds its own copy of the array until the process ends; the first call on a device looks up
 * that copy's address (hipGetSymbolAddress, with the device current) and keeps it.  The call
 * allocates nothing (no hipMalloc / hipFree, no allocating library routine).
 *   Limit: shapes whose svdq_linear_workspace_bytes(M, K, r, fmt) exceeds
 *   SVDQ_STATIC_SCRATCH_BYTES return SVDQ_ERR_WORKSPACE before anything is enqueued (the FLUX
 *   shapes, M = 4608 with K = 3072 or 12288, fit in every format).
 *   Concurrency: every call on one GPU shares that GPU's array and its contents persist from
 *   call to call (nothing in it needs to start at zero).  Calls that overlap on one GPU -- on
 *   two streams, or from two host threads without ordering -- race on it and give wrong
 *   results: order them on one stream.
 * Other arguments, results (bit for bit those of svdq_linear) and errors as for svdq_linear.
 */
#define SVDQ_STATIC_SCRATCH_BYTES (64u << 20)
svdq_status svdq_linear_noalloc(const void* x_hat, const void* l1t, const void* wq, const void* ws,
                                const void* l2, const void* bias, int M, int N, int K, int r,
                                svdq_format fmt, void* y, void* stream);

/*
 * Offline weight quantizer: the residual R = W_hat - L1 L2, given as
 * R^T fp32 [N, K] (K contiguous per output column), to codes wq and scales ws
 * in the layouts Kernel B reads ("sota-314", "Do this": quantize only the
 * residual; round-to-nearest-even here, where the pages' own pipeline uses
 * GPTQ).
 */
svdq_status svdq_quantize_weight(const float* r_t, int N, int K, svdq_format fmt, void* wq,
                                 void* ws, void* stream);

/*
 * Codes and scales of the residual computed elsewhere -- e.g. GPTQ on the host
 * ("sota-314", "Do this": the authors' pipeline rounds the residual with GPTQ,
 * not to nearest) -- put into the layouts Kernel B reads, for the INT
 * formats (SVDQ_INT4_G64, SVDQ_INT4_G64_E2M3, SVDQ_INT8_G64; others are
 * SVDQ_ERR_FORMAT):
 *   codes  : int8 [N, K], one code per byte (in [-7, 7] or [-127, 127]; not
 *            checked), K contiguous per output column.
 *   scales : fp16 [N, K/64].
 *   wq, ws : out, as svdq_quantize_weight writes them.
 * With round-to-nearest codes and scales this reproduces svdq_quantize_weight
 * bit for bit.  Pointers 16-byte aligned; N % 16 == 0, K % 64 == 0.
 */
svdq_status svdq_pack_weight(const int8_t* codes, const void* scales, int N, int K, svdq_format fmt,
                             void* wq, void* ws, void* stream);

/*
 * Codes and scales between the exchange layout and the layout of the format's kernels
 * (the exchange layout is the one the bit-exact comparisons with a plain implementation of
 * the quantizers are stated in; "sota-314", "Do this": INT4 group 64 with 16-bit scales,
 * NVFP4 group 16 with FP8 scales, rank 16 at 8 bits -- the formats fix codes and scales, not
 * a memory order).
 *   Exchange layout: row-major, K contiguous per row (token, or output column of a weight):
 *     codes  [rows, K/2] for the 4-bit formats (two codes a byte, code 2b in the low nibble;
 *            two's-complement INT4 for SVDQ_INT4_G64 and SVDQ_INT4_G64_E2M3, E2M1 nibbles for
 *            SVDQ_FP4_G16 and SVDQ_MXFP4_G32) or [rows, K] for SVDQ_INT8_G64;
 *     scales [rows, K/G]: fp16 (INT formats), E4M3 bytes (SVDQ_FP4_G16), E8M0 bytes
 *            (SVDQ_MXFP4_G32).
 *   Device layout: the format's layout above (chunk- or group-major).  SVDQ_INT4_G64_E2M3's INT4 codes are
 *   turned into or out of their 6-bit E2M3 fields exactly; exchange codes must lie in [-7, 7].
 *   to_canonical : 1 = device -> exchange, 0 = exchange -> device.
 *   codes_in, scales_in : the source layout; codes_out, scales_out : the destination layout
 *   (caller-allocated, svdq_code_row_bytes(K, SVDQ_INT4_G64 or fmt) and
 *   svdq_scale_row_bytes(K, fmt) bytes a row; may not alias the sources).
 *   rows >= 0 (any count), K % 64 == 0.  Offline / exchange work, not on the layer's path.
 */
svdq_status svdq_relayout(const void* codes_in, const void* scales_in, int rows, int K, svdq_format fmt,
                          int to_canonical, void* codes_out, void* scales_out, void* stream);

/* Workspace of the unfused comparison: svdq_linear's workspace plus an fp16
 * [M, N] intermediate, 256-byte aligned. */
size_t svdq_linear_unfused_workspace_bytes(int M, int N, int K, int r, svdq_format fmt);

/*
 * Unfused comparison (measurement only; "sota-314", "Do this", latency table:
 * a rank-32 branch run as separate kernels): four launches -- quantize;
 * down projection T = X_hat L1 (a second read of X_hat); the low-bit GEMM
 * writing fp16 Y0 = fp16(Q(X_hat) Q(R) + b); up projection
 * Y = fp16(Y0 + T L2) (a second read and write of the output).  Note the extra
 * fp16 rounding of Y0: results agree with svdq_linear to fp16 tolerance, not
 * bitwise.
 */
svdq_status svdq_linear_unfused(const void* x_hat, const void* l1t, const void* wq, const void* ws,
                                const void* l2, const void* bias, int M, int N, int K, int r,
                                svdq_format fmt, void* workspace, size_t workspace_bytes,
                                void* y, void* stream);

/*
 * W4A16 control ("sota-314", "Do this" and "What it buys": the W4A16
 * baseline and the layers kept at W4A16): Y = fp16_rne( X deq(W) + b ) with
 * X fp16 [M, K] unquantized, W as SVDQ_INT4_G64 codes wq and fp16 scales ws
 * (the format's layout, rows = output columns), fp32 accumulation; bias may be
 * NULL.  No branch.
 */
svdq_status svdq_gemm_w4a16(const void* x, const void* wq, const void* ws, const void* bias,
                            int M, int N, int K, void* y, void* stream);

/*
 * GELU(tanh) + smoothing glue between an MLP's two linears:
 *   out[m, c] = fp16_rne( gelu_tanh(float(y[m, c])) / lambda[c] ),
 *   gelu_tanh(v) = 0.5 v (1 + tanh( sqrt(2/pi) (v + 0.044715 v^3) )),
 *   evaluated in fp32 as gelu_div(v, lam) = v / ((1 + exp(-2u)) lam) with
 *   u = sqrt(2/pi) (v + 0.044715 v^3) (the same value; no cancellation for
 *   negative v), exp and the reciprocal from the hardware's approximations:
 *   within one fp16 ulp of the exactly rounded result.
 *   y: fp16 [M, C]; lambda: fp32 [C] (the second layer's smoothing factors);
 *   out: fp16 [M, C] (may not alias y).  C % 8 == 0.
 */
svdq_status svdq_gelu_tanh_smooth(const void* y, const float* lambda, int M, int C, void* out,
                                  void* stream);

/*
 * Folding the neighbouring steps into the two kernels.  The pages fuse the
 * branch with the low-bit kernels because the fused steps share an operand
 * ("sota-314", "Do this"); the same argument carries the steps on either side
 * of a layer into the kernels: the smoothing of the layer's input into Kernel A
 * (both read X) and an MLP's GELU + next-layer smoothing into Kernel B's
 * epilogue (both write the output).  The pages do not describe this fold.
 *
 * Kernel A on the unsmoothed activations ("sota-314", "Do this": smoothing
 * divides each input channel by its factor, X_hat = X diag(lambda)^-1):
 *   x      : fp16 [M, K], unsmoothed.
 *   lambda : fp32 [K], the layer's smoothing factors (> 0), 16-byte aligned.
 *   Every value is first replaced by X_hat = fp16_rne(fp32(x) / lambda[k])
 *   (IEEE fp32 division, then one rounding); codes, scales and T are then
 *   exactly those svdq_quantize_down gives for that X_hat.  Other arguments,
 *   the workspace rules and errors as for svdq_quantize_down; lambda NULL is
 *   SVDQ_ERR_NULL.
 */
svdq_status svdq_quantize_down_smooth(const void* x, const float* lambda, const void* l1t, int M, int K,
                                      int r, svdq_format fmt, void* xq, void* xs, void* t,
                                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * Kernel B with an MLP's glue in its epilogue: writes
 *   y[m, n] = fp16_rne( gelu_div( Y[m, n], lambda_next[n] ) ),
 * where Y is the fp16 output svdq_gemm_w4a4_up would write and gelu_div is the
 * arithmetic of svdq_gelu_tanh_smooth, so the result equals
 * svdq_gelu_tanh_smooth(svdq_gemm_w4a4_up(...), lambda_next) bit for bit
 * without the fp16 round trip of Y through memory.
 *   lambda_next : fp32 [N], the next layer's smoothing factors (> 0), 16-byte
 *                 aligned; NULL is SVDQ_ERR_NULL.
 * Other arguments and errors as for svdq_gemm_w4a4_up.
 */
svdq_status svdq_gemm_w4a4_up_gelu_smooth(const void* xq, const void* xs, const void* t, const void* wq,
                                          const void* ws, const void* l2, const void* bias,
                                          const float* lambda_next, int M, int N, int K, int r,
                                          svdq_format fmt, void* y, void* stream);

/*
 * The fused layer with either fold: svdq_linear's Kernel A then Kernel B, with
 * lambda_in != NULL taking x unsmoothed (as svdq_quantize_down_smooth) and
 * lambda_next != NULL writing fp16(gelu(Y) / lambda_next) (as
 * svdq_gemm_w4a4_up_gelu_smooth).  With both NULL it is svdq_linear.  An
 * MLP's first layer runs with both; its output is then the second layer's
 * X_hat, for svdq_linear.  Workspace as for svdq_linear
 * (svdq_linear_workspace_bytes covers the smoothing variant's plan too).
 */
svdq_status svdq_linear_folded(const void* x, const float* lambda_in, const void* l1t, const void* wq,
                               const void* ws, const void* l2, const void* bias, const float* lambda_next,
                               int M, int N, int K, int r, svdq_format fmt, void* workspace,
                               size_t workspace_bytes, void* y, void* stream);

/* ------------------------------------------------------------------------------------------
 * The operators of a transformer block between its quantized linears: the norm in front of a
 * linear, a matrix product with its neighbours in the epilogue, and the rotary positions of
 * queries and keys.  Beyond the conventions above:
 *  - sizes and strides have their own rules, stated at each operator; strides count elements of
 *    their tensor and the innermost dimension is contiguous;
 *  - a pointer needs its element's alignment only, unless the operator says 16 bytes;
 *  - an output may overlap an input only where the operator says so;
 *  - all arithmetic is fp32 (int32 for INT8 sums) and every output is rounded once, to nearest
 *    even; the library adds in a fixed order, so equal calls give equal bits.
 */
typedef enum {
  SVDQ_TYPE_F16 = 0,
  SVDQ_TYPE_BF16 = 1,
  SVDQ_TYPE_F32 = 2,
  SVDQ_TYPE_INT8 = 3,  /* codes in [-127, 127] */
  SVDQ_TYPE_E4M3 = 4,  /* OCP FP8 E4M3 (finite, largest value 448) */
  SVDQ_TYPE_INT_MIN_ = -2147483647 - 1,   /* not types: see svdq_format */
  SVDQ_TYPE_INT_MAX_ = 2147483647
} svdq_type;

typedef enum {
  SVDQ_ACT_NONE = 0,
  SVDQ_ACT_GELU_TANH = 1,  /* gelu_tanh of svdq_gelu_tanh_smooth, the same fp32 form */
  SVDQ_ACT_SILU = 2,       /* v / (1 + exp(-v)) */
  SVDQ_ACT_INT_MIN_ = -2147483647 - 1,
  SVDQ_ACT_INT_MAX_ = 2147483647
} svdq_activation;

/*
 * Root-mean-square norm of x plus a residual, with an 8-bit output and its scales.  Per row:
 *   h = rnd(x + residual) in the residual's type (h = x without one), written to residual_out;
 *   rstd = 1 / sqrt(mean_k h^2 + eps);  v = h weight;
 *   8-bit out_type: a = max(max_k |v|, 2^-100), code = rnd(v * (qmax / a)) with qmax 127 (INT8,
 *     ties to even) or 448 (E4M3), scale = a * rstd / qmax, so code * scale is the normed value.
 *     rstd is a factor of the whole row and cancels in the codes: they are exact functions of h.
 *   v is an fp32 value (|h weight| below 2^128); the mean of h^2 holds for every finite h.
 *   out_type == x_type: out = rnd(v * rstd), scales unused.  With weight / lambda in place of
 *     weight this is the smoothed input of svdq_linear.
 *   x        : [M, K], x_type SVDQ_TYPE_F16 or _BF16, rows x_stride apart.
 *   residual : [M, K] of residual_type (x_type or SVDQ_TYPE_F32), or NULL for none (residual_out
 *              is then unused and the strides and type are ignored).
 *   weight   : [K] of weight_type (x_type or SVDQ_TYPE_F32).
 *   eps      : finite, > 0.
 *   out      : out, [M, K] contiguous, out_type (SVDQ_TYPE_INT8, _E4M3 or x_type).
 *   scales   : out, fp32 [M]; required for an 8-bit out_type.
 *   residual_out : out, rows residual_out_stride apart; may be residual, or x where the types agree.
 * 1 <= K <= 2^24, 0 <= M <= 2^24 (0 = nothing to do), strides >= K.  SVDQ_ERR_SHAPE also where the
 * rows need 2^32 threads or more (never below 2^34 elements).
 */
svdq_status svdq_add_rmsnorm(const void* x, int64_t x_stride, svdq_type x_type, const void* residual,
                             int64_t residual_stride, svdq_type residual_type, const void* weight,
                             svdq_type weight_type, float eps, int M, int K, svdq_type out_type, void* out,
                             float* scales, void* residual_out, int64_t residual_out_stride, void* stream);

/*
 * Matrix product with bias, activation and residual in its epilogue:
 *   y[m, n] = rnd( act( (sum_k x[m, k] w[n, k]) * xs[m] * ws[n] + bias[n] ) + residual[m, n] )
 *   x  : [M, K] of `type` (SVDQ_TYPE_INT8, _E4M3, _F16 or _BF16), rows x_stride apart.
 *   xs : fp32 [M], or NULL for ones (svdq_add_rmsnorm writes x and xs).
 *   w  : [N, K] contiguous, of `type` (rows = output columns).
 *   ws : fp32 [N], or NULL for ones.
 *   bias     : [N] of out_type, or NULL.
 *   residual : [M, N] of out_type, rows residual_stride apart, or NULL.
 *   y        : out, [M, N] of out_type (SVDQ_TYPE_F16 or _BF16), rows y_stride apart; may be residual.
 * INT8 sums are exact in int32 (K <= 2^17 for INT8: 2^17 * 127^2 < 2^31).  x and w are 16-byte
 * aligned, K and x_stride multiples of 16 bytes, and a row of either (x_stride for x) takes at
 * most 4 MiB.  Any M >= 0 and N >= 0 up to 2^24, at most 2^31 - 1 output tiles of 64 x 64; strides
 * >= the row's length.  E4M3 products are exact and their sums fp32, as for 16-bit types (and at their
 * rate: the FP8 matrix instructions drop small products beside a large one).
 *   workspace, workspace_bytes : caller-owned device scratch, 16-byte aligned, for the sums of K's
 *           splits when few output tiles leave CUs idle (svdq_gemm_act_residual_workspace_bytes).
 *           Its contents need no initialisation and are dead after the call; two calls in flight at
 *           once need two workspaces.  NULL, or fewer bytes, is allowed: K is then split less
 *           or not at all (slower for long K; sums in another order, so fp32 sums may differ in their
 *           last bits).
 */
svdq_status svdq_gemm_act_residual(const void* x, int64_t x_stride, const float* xs, const void* w,
                                   const float* ws, const void* bias, const void* residual,
                                   int64_t residual_stride, int M, int N, int K, svdq_type type,
                                   svdq_activation act, svdq_type out_type, void* y, int64_t y_stride,
                                   void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes svdq_gemm_act_residual uses for these sizes (0: none, or a bad type or size). */
size_t svdq_gemm_act_residual_workspace_bytes(int M, int N, int K, svdq_type type);

/* The kernel that svdq_gemm_act_residual takes for these sizes with this much workspace, by its tiles:
 * "few rows", "64x64", "64x128", "128x192", "128x256" or "256x256"; NULL for a bad type or size or
 * an empty product.  For tests and measurements.  *splits: the parts K is split into.  *tail: with
 * 256x256, the parts each tile of the last partial round is cut into (1, 2 or 4; 0: no such round).
 * Either pointer may be NULL. */
const char* svdq_gemm_act_residual_kernel(int M, int N, int K, svdq_type type, size_t workspace_bytes, int* splits,
                                          int* tail);

/*
 * Rotary positions with several axes on queries and keys, with the heads' root-mean-square norm
 * in front where a weight is given.  For each (batch, token, head) and its `dim` values x:
 *   u = x * weight / sqrt(mean_d x^2 + eps), or u = x without a weight;
 *   pair p of the first 2 P values turns by angle = positions[b, t, axis(p)] * inv_freq[p]:
 *     (u_i, u_j) -> (u_i cos - u_j sin, u_i sin + u_j cos),
 *   (i, j) = (2p, 2p + 1) or, with halves != 0, (p, p + P); axis_pairs[a] consecutive pairs turn
 *   by axis a, P = sum of axis_pairs; the values from 2 P on are u unturned.
 *   inverse != 0 turns by -angle: the inverse map, and the gradient of the output with respect
 *   to x; it takes no weights.
 * The product of position and frequency is taken in fp64 (exact for fp32 positions) up to a size of
 * 2^48; a larger or infinite angle counts as 2^48 with its sign.
 */
typedef struct {
  const void* in;        /* [batch, tokens, heads, dim], strides below, innermost contiguous */
  void* out;             /* same shape; may be `in` with the same strides */
  const float* weight;   /* fp32 [dim], or NULL: no norm */
  int heads;             /* >= 1 */
  int64_t in_batch, in_token, in_head, out_batch, out_token, out_head;   /* strides >= 0, in elements */
} svdq_rope_operand;

#define SVDQ_ROPE_MAX_AXES 4
/*   operands : 1 or 2 operands (queries, keys), `count` of them; host memory, read in the call.
 *   type     : SVDQ_TYPE_F16 or _BF16, of all inputs and outputs.
 *   positions : [batch, tokens, axes] int32, or fp32 with positions_fp32 != 0; token stride
 *              `axes`, batch stride position_batch (0: shared by the batch).
 *   inv_freq : fp32 [P].  axis_pairs : host memory, `axes` (1 ... SVDQ_ROPE_MAX_AXES) counts >= 0.
 * batch, tokens >= 0 (0 = nothing to do); 1 <= dim <= 1024; 1 <= P, 2 P <= dim; eps finite, > 0
 * where a weight is given.  Sizes past one launch's 2^32 threads give SVDQ_ERR_SHAPE (never below
 * 2^25 heads of tokens). */
svdq_status svdq_rope_axes(const svdq_rope_operand* operands, int count, int batch, int tokens, int dim,
                           svdq_type type, const void* positions, int positions_fp32, int64_t position_batch,
                           const float* inv_freq, int axes, const int* axis_pairs, int halves, float eps,
                           int inverse, void* stream);

/* ------------------------------------------------------------------------------------------
 * The operators around a paged cache of keys and values, for decoding.  Conventions as for the block's
 * operators above.  The cache's pages are handed out by the caller; a step adds `tokens` tokens of
 * several sequences, packed one sequence behind the other:
 *   svdq_rope_append      turns the step's queries and keys and writes keys and values to the cache;
 *   svdq_tree_attention   lets the step's queries attend to the cache, the step's own tokens in it;
 *   svdq_cache_keep       of a drafted tree, moves the accepted path's keys and values together.
 */
typedef struct {
  void* k;               /* keys [pages, page_size, heads, dim] of `type`, by the strides below, the values of a */
  void* v;               /* head contiguous; values the same.  16-byte aligned */
  float* k_scales;       /* 8-bit types: [pages, page_size, heads], a head's value is code * scale; else ignored */
  float* v_scales;
  svdq_type type;        /* SVDQ_TYPE_F16 or _BF16 (the type of the step's tokens), _INT8 or _E4M3 */
  int64_t pages;         /* 0 ... 2^31 - 1 */
  int page_size;         /* tokens a page: a power of two up to 2^16 */
  int heads;             /* 1 ... 2^16 */
  int dim;               /* 8 ... 256, a multiple of 8 (16 for an 8-bit type) */
  int64_t page_stride, token_stride, head_stride;   /* of k and v, in elements, multiples of 16 bytes */
  int64_t scale_page_stride, scale_token_stride, scale_head_stride;   /* of the scales, in elements */
} svdq_paged_cache;

typedef struct {
  const int* page_table; /* int32 [sequences, table_width], rows table_stride apart: slot s of a sequence is token
                            s % page_size of page page_table[s / page_size].  An entry outside the cache's pages, or
                            a column past the table, is no page: nothing is written there, and attention does not see it */
  int64_t table_stride;
  int table_width;       /* table_width * page_size <= 2^30 */
  const int* starts;     /* int32 [sequences + 1], not falling: sequence b has the tokens starts[b] ... starts[b + 1] - 1 of
                            the step.  Tokens outside starts[0] ... starts[sequences] - 1 belong to none */
  const int* context;    /* int32 [sequences], 0 ... 2^30: tokens in the cache before the step; token i of the step has
                            slot context[b] + i */
  int sequences;         /* 0 ... 2^24 (0: the pointers may be NULL) */
} svdq_paged_batch;

/*
 * Rotary positions on a step's queries and keys, and its keys and values into the cache, in one launch:
 *   queries: turned as svdq_rope_axes turns them, to q->out;
 *   keys: turned the same way, then rounded once to a 16-bit cache's type, or quantized: a =
 *     max(max_d |u_d|, 2^-100), code = rnd(u * (qmax / a)) with qmax 127 (INT8, ties to even) or 448 (E4M3),
 *     scale = a / qmax;
 *   values: to the cache the same way, unturned.
 *   q : queries ([tokens, heads, dim] by in_token, in_head; `out` by out_token, out_head; may be `in` with the
 *       same strides), or NULL for none.  k : keys, k->heads the cache's; its `out` is unused.  The batch
 *       strides of both are unused.  v : [tokens, cache heads, dim] by v_token, v_head.
 *   positions : [tokens, axes] int32, or fp32 with positions_fp32 != 0; the position of a token need not be
 *       its slot (tokens of a tree share positions).  Other arguments as for svdq_rope_axes.
 * Queries of tokens that belong to no sequence are turned too; their keys and values go nowhere.  Two tokens
 * of a step must not have the same slot of the same page (which one's values stay is then open).  8-bit
 * codes are those of finite values. */
svdq_status svdq_rope_append(const svdq_paged_cache* cache, const svdq_paged_batch* batch, const svdq_rope_operand* q,
                             const svdq_rope_operand* k, const void* v, int64_t v_token, int64_t v_head, int tokens,
                             svdq_type type, const void* positions, int positions_fp32, const float* inv_freq, int axes,
                             const int* axis_pairs, int halves, float eps, void* stream);

/*
 * Attention of a step's tokens over the cache (which svdq_rope_append has brought the step's own keys and
 * values into):
 *   out[t, h] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q[t, h] . k_j - max),
 * over the keys j of cache head h / (heads / cache heads) that token t, the i-th of its sequence in the step, sees:
 * the slots below the sequence's context, and of the step's own tokens the j-th where
 *   tree[t, j] != 0 (a byte; j >= tree_width: not seen)    with a tree,
 *   j <= i                                                 without (a chain: one token, or a chunk of a prompt).
 * A row that sees nothing is zeros (and so is one whose logits are all minus infinity).  What a token does not see
 * has no effect on it, infinities and NaN included.
 *   q, out : [tokens, heads, dim] of `type` by their strides; heads a multiple of the cache's.  out may be q with
 *            the same strides.  Rows of tokens that belong to no sequence are left as they were.
 *   tokens * heads < 2^31, and (tokens * (heads / cache heads) / 16 + sequences) * cache heads <= 2^24.
 *   scale  : 2^-126 ... 2^126.
 *   tree   : bytes [tokens, tree_width], rows tree_stride apart, or NULL.
 * The work is cut by the mean number of rows of a sequence: long chunks and single tokens are best in calls of their own.
 * Logits, the softmax's statistics and sums are fp32; probabilities are rounded to 16 bits for the matrix
 * cores (to fp16 with an 8-bit cache, whose scales of values join them there).  In fp16 one below 2^-21 of the row's
 * largest (of probability times scale) is off by up to 2^-32 of that: values of n keys so far below the rest are good to
 * n 2^-32 of the largest.  Powers are taken relative to a maximum that may lag by 2^8 (2^15 with an fp16 cache): sums of values of a
 * bf16 cache from 2^119 on can leave fp32's range.
 *   workspace, workspace_bytes : caller-owned device scratch, 16-byte aligned, for the sums of the keys' parts
 *            where rows alone do not fill the chip (svdq_tree_attention_workspace_bytes); rules as for
 *            svdq_gemm_act_residual's.
 */
svdq_status svdq_tree_attention(const svdq_paged_cache* cache, const svdq_paged_batch* batch, const void* q,
                                int64_t q_token, int64_t q_head, int heads, int tokens, svdq_type type, float scale,
                                const void* tree, int64_t tree_stride, int tree_width, void* out, int64_t out_token,
                                int64_t out_head, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes svdq_tree_attention uses for these sizes (0: none, or a bad size). */
size_t svdq_tree_attention_workspace_bytes(int sequences, int tokens, int heads, int kv_heads, int dim, int table_width,
                                           int page_size);

/*
 * A draft's accepted path: slot context[b] + i takes the keys, values and scales of slot context[b] + path[b, i]
 * for each i below path_width with path[b, i] >= 0 and i and path[b, i] below the sequence's number of tokens
 * in the step (starts as in the step that drafted them); other entries leave their slot as it is.  The path of
 * a sequence rises (path[b, i] < path[b, i + 1], negative ends apart), so that path[b, i] >= i; two
 * sequences of one call must not share pages that the path writes.
 *   path : int32 [sequences, path_width], rows path_stride apart; path_width <= 2^16. */
svdq_status svdq_cache_keep(const svdq_paged_cache* cache, const svdq_paged_batch* batch, const int* path,
                            int64_t path_stride, int path_width, void* stream);

/* Static description of a status code. */
const char* svdq_status_string(svdq_status s);

/* Library version string. */
const char* svdq_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SVDQ_H */
