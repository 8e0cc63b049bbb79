/*
 * tl.h -- C ABI of the ternary linear-layer library for AMD Instinct MI355X (gfx950).
 *
 * The layer is the quantized linear layer of the ternary 27B model described in
 * qiita.com/nakanokensetsu/items/ecc183fae033565af7cb (cited below as [P1] with
 * its section headings):
 *   - weights are 2-bit codes in {-1, 0, +1} with one fp16 scale per row and per
 *     128-element group along K ([P1] "前提");
 *   - the input is rotated by a block-wise Sylvester Hadamard transform with
 *     1024-wide blocks and an optional sign table ([P1] "前提", "1. TP=2 への移植");
 *   - decode computes y = W (H_blk x) for 1..64 tokens;
 *   - prefill decomposes each scale as q = round(127 s / smax) so that
 *     code * q is exact in int8, quantises the rotated activations to int8 per
 *     token, and runs one int8 x int8 -> int32 GEMM followed by a per-row and
 *     per-token rescale ([P1] "4. 効いた高速化").
 *
 * Conventions for every call
 *   - Every tensor argument is a DEVICE pointer owned by the caller, dense and
 *     row-major (C order).  The library allocates no device memory; scratch, when
 *     a call needs it, is a caller-provided workspace whose size a *_workspace_size
 *     query returns (tl_linear_apply_noalloc instead uses a static device array
 *     of tl_noalloc_scratch_bytes() per GPU, see there).
 *   - `stream` is a hipStream_t passed as void* (NULL = the default stream).  All
 *     work is enqueued on it; no call synchronises.  A device fault surfaces at the
 *     caller's next synchronisation.
 *   - Arguments are checked on the host before anything is launched.  A failed
 *     check returns a non-zero TL_ERR_* code, launches nothing and leaves every
 *     output untouched.  Launch failures return TL_ERR_LAUNCH.
 *   - Counts of zero (T, b, M, N) are valid and do nothing; K must be positive.
 *   - Inputs and outputs must not overlap (TL_ERR_ALIAS).
 *   - Pointers must be 16-byte aligned (TL_ERR_ALIGN).
 *   - Value preconditions (codes in {-1,0,+1}, signs +-1, finite inputs) are not
 *     checked on the device, except that tl_pack_weights can count bad codes.
 *   - Calls are thread-safe; concurrent calls on different streams are
 *     independent (each uses only its own arguments and workspace).
 *
 * Packed weight layout (ABI version 2; the page gives no layout, this one is ours)
 *   Codes are stored two bits each in uint32 words.  Within a word, code j
 *   (j = 0..15, for 16 consecutive k) occupies bits 8*(j mod 4) + 2*(j div 4) and
 *   the bit above it, so ((w >> 2r) & 0x03030303) holds codes 4r..4r+3 in bytes
 *   0..3, in k order.  A field is the code's two's-complement low two bits:
 *   0 -> 00, +1 -> 01, -1 -> 11 (10 is never written).
 *   Words are grouped in 1024-byte tiles that match the lanes of a 64-wide
 *   wavefront: rows are taken in blocks of 16 and K in pairs of 128-groups,
 *   NB = ceil(N/16) row blocks, GP = ceil(K/256) group pairs (a last partial
 *   block or pair is padded with zero codes).  Tile (rb, p) starts at word
 *   256*(rb*GP + p).  Its word 4*l + 2*gi + m (l = 0..63, gi, m in {0, 1}) holds
 *   the codes k = 128*(2p + gi) + 16*(2*(l/16) + m) + j, j = 0..15, of row
 *   n = 16*rb + (l mod 16).  Lane l of a wavefront reading 16 bytes at
 *   4*l words thus gets, for both groups of the pair, the two words an
 *   int8 16x16x64 matrix instruction needs from it.  tl_packed_bytes(N, K)
 *   gives the size.
 */
#ifndef TL_H
#define TL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define TL_ABI_VERSION 2

/* status codes returned by every call */
#define TL_OK 0
#define TL_ERR_NULLPTR 1     /* a required pointer is NULL */
#define TL_ERR_SHAPE 2       /* a size is negative, out of range or not a required multiple */
#define TL_ERR_ALIGN 3       /* a pointer is not 16-byte aligned */
#define TL_ERR_DTYPE 4       /* y_dtype is not TL_BF16 or TL_F32 */
#define TL_ERR_LAUNCH 5      /* the HIP runtime reported an error */
#define TL_ERR_UNSUPPORTED 6 /* no kernel variant for this request */
#define TL_ERR_WORKSPACE 7   /* workspace missing or smaller than the query says */
#define TL_ERR_ALIAS 8       /* an output overlaps an input or another output */
#define TL_ERR_SCRATCH 9     /* beyond the static scratch of tl_linear_apply_noalloc */

/* output element types */
#define TL_BF16 0 /* bfloat16, round to nearest even from fp32 */
#define TL_F32 1  /* IEEE binary32 */
/* element type of an 8-bit K/V cache (not an output type) */
#define TL_E4M3 2 /* 8-bit float: 4 exponent, 3 mantissa bits, largest 448, no infinities */

/* Version of the packed layout and of the signatures below (TL_ABI_VERSION). */
int tl_abi_version(void);

/* Static text for a status code; never NULL. */
const char *tl_status_string(int status);

/* Name of the last kernel this host thread launched through the library
 * ("" before the first launch).  Used to check which variant ran. */
const char *tl_last_kernel_name(void);

/* Text of the HIP runtime error behind the last TL_ERR_LAUNCH returned on this
 * host thread ("" if none).  For diagnostics only. */
const char *tl_last_error_detail(void);

/*
 * tl_pack_weights -- load-time conversion of one ternary layer.
 *   [P1] "前提" (2-bit codes, one fp16 scale per row and 128-group) and
 *   [P1] "4. 効いた高速化" (q[n,g] = round(127 s[n,g] / smax[n])).
 * in  codes      int8   [N, K]     values in {-1, 0, +1}
 * in  scales     fp16   [N, K/128] (raw IEEE half bits), finite
 * out packed     uint32, tl_packed_bytes(N, K) bytes, layout above (padding
 *                included and written)
 * out q          int8   [N, K/128] q = RNE( fl32(fl32(127*s) / smax) ),
 *                                  smax[n] = max_g |s[n,g]|; |q| <= 127
 * out row_scale  f32    [N]        fl32(smax / 127)
 * out invalid_count int32 [1] or NULL: if not NULL, the number of codes outside
 *                  {-1,0,+1} is ADDED to it (the caller zeroes it first).
 * A row whose scales are all zero gets q = 0 and row_scale = 0.
 * Requires K > 0, K % 128 == 0.
 */
size_t tl_packed_bytes(int64_t N, int64_t K);
int tl_pack_weights(const int8_t *codes, const uint16_t *scales, int64_t N, int64_t K,
                    uint32_t *packed, int8_t *q, float *row_scale, int32_t *invalid_count,
                    void *stream);

/*
 * tl_hadamard_blk -- block rotation of the layer input.
 *   [P1] "前提" (Hadamard rotation on the input side) and "1. TP=2 への移植"
 *   (Sylvester type, 1024-wide blocks, sign table keyed by the layer width).
 * in  x      bf16 [T, K] (raw bits)
 * in  signs  int8 [K] of +-1, or NULL for all +1; applied to x before H
 * out xr     f32  [T, K]: for each token and block j,
 *            xr[t, 1024 j + i] = (1/32) sum_m (-1)^popcount(i & m) d[1024 j + m] x[t, 1024 j + m]
 *            computed exactly (binary64 butterflies) and rounded once to f32.
 *            The result is exact before that rounding whenever the x values are
 *            multiples of 2^-31 below 2^8 in magnitude (bf16 with |x| >= 2^-24).
 * Requires K > 0, K % 1024 == 0.
 */
int tl_hadamard_blk(const uint16_t *x, int64_t T, int64_t K, const int8_t *signs, float *xr,
                    void *stream);

/*
 * tl_hadamard_half, tl_hadamard_join -- the rotation of a 1024-block that a
 * K-shard boundary splits in the middle, in two stages with an exchange of the
 * stage results between the two ranks in between.
 *   [P1] "1. TP=2 への移植" (17408 / 2 = 8704 falls in the middle of a block;
 *   H1024 [a; b] = [H512 a + H512 b; H512 a - H512 b]: each rank transforms its
 *   own 512 columns, the results are exchanged, the rank with the first half
 *   keeps the sum, the other the difference).
 * tl_hadamard_half:
 * in  x      bf16 [T, 512] with rows ldx elements apart (ldx >= 512, ldx % 8 == 0,
 *            so a column slice of the rank's [T, K_shard] input can be passed)
 * in  signs  int8 [512] of +-1 for these columns, or NULL for all +1
 * out u      f64  [T, 512] dense: u[t, i] = sum_m (-1)^popcount(i & m) d[m] x[t, m]
 *            (no 1/32), exact in binary64 for inputs that are multiples of 2^-31
 *            below 2^8 in magnitude (bf16 with |x| >= 2^-24).
 * tl_hadamard_join:
 * in  u_lo, u_hi  f64 [T, 512]: the stage results of the block's first and second
 *            512 columns (one computed here, one received from the other rank)
 * in  half   0 for the rank that holds the first half, 1 for the other
 * out xr     f32 [T, 512] with rows ldxr elements apart (ldxr >= 512, ldxr % 4 == 0):
 *            half 0: fl32((u_lo + u_hi) / 32), half 1: fl32((u_lo - u_hi) / 32) --
 *            bit for bit the columns tl_hadamard_blk produces for that half.
 * The exchange itself (512 binary64 values per token each way) is the caller's.
 */
int tl_hadamard_half(const uint16_t *x, int64_t T, int64_t ldx, const int8_t *signs, double *u,
                     void *stream);
int tl_hadamard_join(const double *u_lo, const double *u_hi, int64_t T, int half, float *xr,
                     int64_t ldxr, void *stream);

/*
 * tl_gemv_ternary -- decode GEMV, y = W xr for 1..64 tokens.
 *   [P1] "前提" (y = W (H_blk x), W = code * group scale).
 * in  xr      f32    [b, K]      rotated activations (tl_hadamard_blk output)
 * in  packed  uint32 tiles      from tl_pack_weights (tl_packed_bytes(N, K) bytes)
 * in  scales  fp16   [N, K/128]
 * out y       [b, N] of y_dtype: y[t,n] = sum_g s[n,g] sum_{k in g} code[n,k] xr[t,k]
 * workspace   device scratch of at least tl_gemv_workspace_size(b, K, N) bytes,
 *             16-byte aligned; its contents on entry do not matter.
 * Numerics: each weight is read once for all b tokens; group sums run on int8
 * matrix cores with each token's activations held as a 15-bit fixed-point value
 * split into two int8 limbs, scaled per token and 1024-wide block of K (scale
 * |x|max / 32639 of that block), and group results are accumulated in f32.
 * Relative Frobenius error against exact arithmetic is about 3e-5 on the
 * generator's data (bound used by the tests: 1e-3).  In general each activation
 * is off by at most 2^-16 of the largest magnitude in its own block (15 bits per
 * block, whatever the other blocks hold), so the error of y[t, n] is at most
 * about 2^-16 sum_g |s[n,g]| sum_{k in g} |code[n,k]| max_blk(k) |xr[t,.]|: the
 * relative error stays near 3e-5 unless y itself is small against that sum
 * (heavy cancellation) or a block's values spread over more than 15 bits.
 * One matrix-core operand holds 16 tokens: b > 16 runs ceil(b/16) chunks of 16
 * tokens side by side in the same launch, each streaming the weights itself
 * (chunks of one row range share an L2), so the time grows with the chunk count
 * (tl_linear_path tells when the prefill path is the faster choice).
 * Requires 0 <= b <= 64, K > 0, K % 128 == 0.
 */
size_t tl_gemv_workspace_size(int64_t b, int64_t K, int64_t N);
int tl_gemv_ternary(const float *xr, int64_t b, int64_t K, int64_t N, const uint32_t *packed,
                    const uint16_t *scales, void *y, int y_dtype, void *workspace,
                    size_t workspace_bytes, void *stream);

/*
 * The two stages of tl_gemv_ternary, for callers that apply several weight
 * matrices to the same rotated input (e.g. q/k/v or gate/up as separate
 * layers) or that time the stages apart:
 *   tl_gemv_prepare  writes the activation limbs and their per-block scales of
 *                    xr [b, K] into the workspace (one kernel, one wavefront per
 *                    token and 1024-block);
 *   tl_gemv_prepared runs the weight-streaming kernel on a workspace that
 *                    tl_gemv_prepare filled for the same b and K (one kernel).
 * tl_gemv_ternary(...) is exactly tl_gemv_prepare followed by tl_gemv_prepared.
 * The workspace must stay unmodified between the two calls.
 */
int tl_gemv_prepare(const float *xr, int64_t b, int64_t K, void *workspace,
                    size_t workspace_bytes, void *stream);
int tl_gemv_prepared(const void *workspace, size_t workspace_bytes, int64_t b, int64_t K,
                     int64_t N, const uint32_t *packed, const uint16_t *scales, void *y,
                     int y_dtype, void *stream);

/*
 * tl_gemv_ternary_q8 -- decode GEMV against int8 activations (the int8 decode
 * variant [P1] "5." weighed and set aside for its extra error: the page's dp4a
 * kernel; here int8 matrix cores).
 *   [P1] "前提" (y = W (H_blk x)), "4. 効いた高速化" (per-token int8 activations).
 * in  xq, tok_scale  int8 [b, K], f32 [b]: the rotated activations quantised per
 *                    token by tl_quant_act_int8 (or tl_quant_act_int8_x)
 * in  packed, scales as for tl_gemv_ternary
 * out y       [b, N] of y_dtype:
 *             y[t,n] = tok_scale[t] * sum_g s[n,g] sum_{k in g} code[n,k] xq[t,k]
 *             (group sums exact in int32, f32 accumulation over the groups)
 * One matrix-core chain per group and b*K activation bytes, against two limb
 * chains and 2*b*K for tl_gemv_ternary; the result carries the activation
 * rounding (about 8e-3 relative against the exact layer on the generator's data,
 * against about 3e-5 for tl_gemv_ternary).  No workspace.
 * Requires 0 <= b <= 16, K > 0, K % 128 == 0, and a wave's share of the group
 * pairs must fit its registers: every b is supported for K <= 18432, larger K
 * only while b (K + 16) <= 96 KiB (TL_ERR_UNSUPPORTED otherwise).
 */
int tl_gemv_ternary_q8(const int8_t *xq, const float *tok_scale, int64_t b, int64_t K, int64_t N,
                       const uint32_t *packed, const uint16_t *scales, void *y, int y_dtype,
                       void *stream);

/*
 * tl_quant_act_int8 -- per-token int8 quantisation of rotated activations.
 *   [P1] "4. 効いた高速化" (activations quantised to int8 per token after the
 *   rotation, which evens out outliers).
 * in  xr         f32  [T, K]
 * out xq         int8 [T, K]  clamp( RNE( fl32(xr / sx_t) ), -127, 127 )
 * out tok_scale  f32  [T]     sx_t = fl32(amax_t / 127), amax_t = max_k |xr[t,k]|
 * A token with amax = 0 gets sx = 0 and xq = 0.  Divisions are correctly rounded.
 * Requires K > 0, K % 128 == 0.
 */
int tl_quant_act_int8(const float *xr, int64_t T, int64_t K, int8_t *xq, float *tok_scale,
                      void *stream);

/*
 * Fused layer inputs: the block rotation and the step that consumes it in one
 * launch, so the rotated activations are never written to memory.
 *   [P1] "前提" (rotation of the input), "4. 効いた高速化" (int8 per token after
 *   the rotation).  Outputs are bit-identical to the unfused sequences:
 *     tl_gemv_prepare_x   == tl_hadamard_blk then tl_gemv_prepare
 *     tl_gemv_ternary_x   == tl_hadamard_blk then tl_gemv_ternary
 *     tl_quant_act_int8_x == tl_hadamard_blk then tl_quant_act_int8
 *   except tl_gemv_ternary_x (and the GEMV path of tl_linear_apply) for one
 *   token with N <= 12288 and K <= 6144 (N <= 8192 at K = 6144) or two tokens
 *   with N <= 6144 and K <= 4096, K a multiple of 1024: there a
 *   single kernel rotates, splits into limbs and runs the GEMV, each workgroup
 *   rotating the blocks it needs; its limbs are the same, but it adds the
 *   group results in another order, so its output is not bit-identical to the
 *   sequence (the same error against the exact layer, about 3e-5), and the
 *   workspace (still required) is not used.
 * in  x       bf16 [b or T, K] raw layer input; signs as in tl_hadamard_blk.
 * Requires K % 1024 == 0 and K <= 65536 (TL_ERR_UNSUPPORTED above: use the
 * unfused calls); other arguments as in the unfused entry points.
 */
int tl_gemv_prepare_x(const uint16_t *x, int64_t b, int64_t K, const int8_t *signs,
                      void *workspace, size_t workspace_bytes, void *stream);
int tl_gemv_ternary_x(const uint16_t *x, int64_t b, int64_t K, int64_t N, const int8_t *signs,
                      const uint32_t *packed, const uint16_t *scales, void *y, int y_dtype,
                      void *workspace, size_t workspace_bytes, void *stream);
int tl_quant_act_int8_x(const uint16_t *x, int64_t T, int64_t K, const int8_t *signs, int8_t *xq,
                        float *tok_scale, void *stream);

/*
 * tl_gemm_int8_rescale -- prefill int8 GEMM and rescale.
 *   [P1] "4. 効いた高速化" (W_int8 = code * q exactly in int8; one int8 GEMM,
 *   then a per-row and per-token rescale).
 * in  xq         int8   [M, K]     from tl_quant_act_int8
 * in  tok_scale  f32    [M]
 * in  packed     uint32 tiles     from tl_pack_weights
 * in  q          int8   [N, K/128] from tl_pack_weights
 * in  row_scale  f32    [N]        from tl_pack_weights
 * out y          [M, N] of y_dtype: y = fl32( fl32(acc) * row_scale[n] ) * tok_scale[m]
 * out acc_out    int32  [M, N] or NULL: acc[m,n] = sum_k xq[m,k] code[n,k] q[n,k/128]
 *                (exact; |acc| <= K * 127^2, so K <= 133143 keeps it in int32)
 * workspace      device scratch of at least tl_gemm_workspace_size(M, K, N)
 *                bytes (may be NULL when that size is 0).  Layout: 256 int32
 *                counters (one per K-split tile; at most 256 are ever used),
 *                then the int32 partial tiles of the K-split work.  It must be
 *                zero-filled before its first use; every call leaves the
 *                counters at zero again, so one workspace can be reused, also
 *                across shapes, without clearing.  Calls that overlap in time
 *                must not share one.
 * The size depends only on (M, K, N): the schedule is fixed for the 256
 * compute units of gfx950 (whole rounds of 512 tiles, two per compute unit,
 * of 128 x 256 or, with fewer than 512 such tiles, of 128 x 128; the left-over
 * tiles split along K into up to 6 pieces or cut into sub-tiles).
 * Requires K > 0, K % 128 == 0, K <= 133120.
 */
size_t tl_gemm_workspace_size(int64_t M, int64_t K, int64_t N);
int tl_gemm_int8_rescale(const int8_t *xq, const float *tok_scale, int64_t M, int64_t K,
                         int64_t N, const uint32_t *packed, const int8_t *q,
                         const float *row_scale, void *y, int y_dtype, int32_t *acc_out,
                         void *workspace, size_t workspace_bytes, void *stream);

/*
 * tl_linear_apply -- the whole layer from the raw input, y = W (H_blk x) for T
 * tokens, on the path that tl_linear_path(T, K, N) names:
 *   TL_PATH_GEMV  rotation fused into the limb prep, then the two-limb GEMV
 *                 (tl_gemv_ternary_x); relative error about 3e-5;
 *   TL_PATH_INT8  rotation fused into the per-token int8 quantisation, then the
 *                 int8 GEMM + rescale (tl_quant_act_int8_x, tl_gemm_int8_rescale);
 *                 relative error about 1e-2 against the exact layer (the
 *                 activation and scale rounding of [P1] "4. 効いた高速化").
 *   [P1] "前提" (the layer), "4. 効いた高速化" (the prefill path); the choice by
 *   token count mirrors the page's decode / prefill split.
 * tl_linear_path: up to 16 tokens the GEMV; 17..64 tokens the GEMV while
 * ceil(T/16) * N * K <= 2^27 (every 16-token chunk streams all weights
 * again), else the int8 path; above 64 tokens the int8 path.
 * The rule follows a measured token sweep of both paths at the qkv
 * (5120 -> 10240), gate_up (5120 -> 34816) and down (17408 -> 5120) shapes.
 * in  x          bf16 [T, K] raw layer input; signs as in tl_hadamard_blk
 * in  packed, scales, q, row_scale  from tl_pack_weights (all four are required
 *                whichever path runs)
 * out y          [T, N] of y_dtype
 * workspace      device scratch of at least tl_linear_workspace_size(T, K, N)
 *                bytes, zero-filled before its first use (its first KiB holds the
 *                int8 GEMM's split-K counters, which every call leaves at zero, as
 *                for tl_gemm_int8_rescale); calls that overlap in time must not
 *                share one.
 * Requires K % 1024 == 0 and K <= 65536 (TL_ERR_UNSUPPORTED above).
 */
#define TL_PATH_GEMV 0
#define TL_PATH_INT8 1
int tl_linear_path(int64_t T, int64_t K, int64_t N);
size_t tl_linear_workspace_size(int64_t T, int64_t K, int64_t N);
int tl_linear_apply(const uint16_t *x, int64_t T, int64_t K, int64_t N, const int8_t *signs,
                    const uint32_t *packed, const uint16_t *scales, const int8_t *q,
                    const float *row_scale, void *y, int y_dtype, void *workspace,
                    size_t workspace_bytes, void *stream);

/*
 * tl_read_probe -- measurement helper, not a step of the layer: one launch that
 * only reads `bytes` (a multiple of 16) from src, the way the decode GEMV streams
 * its weights (1 KB per wavefront load, all of a wavefront's loads at once), and
 * writes nothing but possibly one word of *sink.  Its duration is the floor a
 * single launch reading that many bytes reaches on this chip (launch, first
 * memory round trip and tail included), beside which the GEMV's launch time can
 * be put.  src and sink are device pointers, 16-byte aligned.
 */
int tl_read_probe(const void *src, size_t bytes, uint32_t *sink, void *stream);

/*
 * tl_mfma_probe -- measurement helper, not a step of the layer: one launch of 512
 * workgroups of 256 threads (two per compute unit, as the prefill GEMM runs) in
 * which every wavefront issues iters x 8 v_mfma_i32_32x32x32_i8 on eight
 * independent accumulators (65536 int8 operations each) and nothing else, with
 * constant operands (random_operands = 0: every byte 1) or random-looking ones
 * (two sets hashed from the lane and workgroup, alternating from one
 * instruction to the next).  Its duration gives the int8 matrix-core
 * rate the chip sustains with each kind of data, beside which the GEMM's can be
 * put: 512 * 4 * iters * 8 * 65536 operations.  sink is a device pointer,
 * 16-byte aligned, of which at most one word is written.
 * Errors: TL_ERR_SHAPE for iters <= 0, TL_ERR_NULLPTR, TL_ERR_ALIGN.
 */
int tl_mfma_probe(int random_operands, int iters, uint32_t *sink, void *stream);

/*
 * tl_linear_apply_noalloc -- tl_linear_apply without a workspace argument and
 * without any allocation, for callers that cannot allocate device memory: code
 * under HIP graph capture, tight serving loops, harnesses that forbid it.
 * It runs the same kernels as tl_linear_apply (same path rule, same outputs, bit
 * for bit) with the workspace taken from a static device array of
 * tl_noalloc_scratch_bytes() bytes, one per GPU, held until the process ends.
 * The first call on a device looks the array up and zeroes its counter region
 * (one small kernel on `stream`); later calls leave the counters at zero as
 * tl_linear_apply does.  Every call on one GPU shares that GPU's array: calls
 * that overlap in time on one GPU (two streams, two host threads) race and must
 * be serialised by the caller.  A request whose workspace
 * (tl_linear_workspace_size(T, K, N)) exceeds the array returns TL_ERR_SCRATCH
 * before anything is launched; so do all other argument errors of
 * tl_linear_apply, with the same codes.
 */
size_t tl_noalloc_scratch_bytes(void);
int tl_linear_apply_noalloc(const uint16_t *x, int64_t T, int64_t K, int64_t N, const int8_t *signs,
                            const uint32_t *packed, const uint16_t *scales, const int8_t *q,
                            const float *row_scale, void *y, int y_dtype, void *stream);

/* ---------------------------------------------------------------------------
 * One step of speculative decoding over a paged K/V cache.  A step brings R
 * requests new tokens: the nodes of a drafted tree, one token, or a chunk of a
 * prompt.  Its calls, in order:
 *   tl_step_plan       block tables, slots, positions and tree masks from the lengths
 *   (per layer)        the qkv layer, tl_kv_write, tl_tree_attention, the o layer, ...
 *   tl_tree_verify     accepted path and next token of every request from the logits
 *   tl_kv_commit       the accepted rows moved together, for all layers at once
 * Lengths live on the device: no call waits for them on the host, and a step can be
 * captured in a graph with T and R as capacities.
 *
 * The cache.  `pages` pages of `block` tokens (a power of two, 16..4096) for each of
 * H heads of D = 64, 128 or 256 elements, bf16 or e4m3 with one f32 scale per token
 * and head ([pages, H, block]).  The block * D elements of a (page, head) are block/16
 * tiles of 16 tokens, in matrix-operand order:
 *   bf16  K [D/32][4 g][16 p][8 e]       d = 32 c + 8 g + e
 *         V [D/16][2 o][16 m][8 i]       token 8 o + i, d = 16 c + m
 *   e4m3  K [D/64][4 g][16 p][16 e]      d = 64 c + 16 g + e
 *         V [D/32][2 o][16 m][2 u][8 i]  token 8 o + i, d = 32 c + 16 u + m
 * Place p of a K tile holds the token whose bits are (p2, p3, p1, p0).
 * tl_kv_offset gives an element's place.  A slot is page * block + place in the page;
 * request r's token at position pos lies in page table[r, pos / block].  A table entry
 * outside [0, pages) is a page whose tokens are not there; a slot outside
 * [0, pages * block) is not written.
 *
 * Metadata arrays (lengths, tables, slots, masks, paths) need natural alignment only; q, k,
 * v, out, caches and cos_sin 16 bytes, as the scales do where tl_tree_attention reads them.
 * Beside what each call requires: 1 <= H <= 65536, 1 <= pages < 2^31,
 * pages * H * block * D <= 2^50, T < 2^31, and distances of tokens at least a token's
 * elements and below 2^31.  What breaks a limit is refused with TL_ERR_SHAPE.
 */
#define TL_MAX_REQUESTS 4096
#define TL_TREE_NODES 64 /* nodes of a drafted tree */

/* Element offset of (page, head, token in the page, d) in a cache; which = 0 for K,
 * 1 for V; -1 for arguments out of range. */
int64_t tl_kv_offset(int which, int cache_dtype, int64_t H, int64_t D, int64_t block, int64_t page, int64_t head,
                     int64_t token, int64_t d);

/*
 * tl_step_plan
 * in  ctx_lens   int32 [R]  tokens in the cache (negative values count as 0 here and below)
 * in  new_lens   int32 [R]  tokens of this step
 * in  owned      int32 [R]  pages of the table that are the request's
 * io  table      int32 [R, table_width]: entries owned[r] .. are filled with new pages
 * in  free_list  int32 [free_count], free_head int32 [1]: pages free_list[free_head..] are
 *                free, and are taken in this order, request by request
 * in  parents    int32 [T] or NULL: a tree node's parent, as its number inside the request;
 *                a value that is not an earlier node makes a root
 * out q_start    int32 [R + 1]  first token of each request (exclusive sums of new_lens, at most T)
 * out kv_lens    int32 [R]      ctx + new, or 0 for a request that is not served
 * out slots      int64 [T]      where each token's rows go; -1: nowhere
 * out positions  int32 [T]      ctx + depth in the tree, or ctx + number of the token
 * out tree_mask  uint64 [T]     (with parents) the node and its ancestors, a bit each
 * out owned_out  int32 [R], free_head_out int32 [1]: both after this step
 * A request is served if its tokens fit table_width pages, the pages it needs beyond
 * `owned` are free after those of the requests before it, and its tokens are among the T
 * (with those of the requests before it); one that is not served gets slots of -1 and
 * takes no page.  With parents, requests of more than 64 new tokens are
 * chains (mask 0).  Tokens from q_start[R] on get slot -1, position 0 and mask 0.
 * No output may be an input; table is the only in-out argument.
 * Requires 0 <= R <= 4096, T and free_count < 2^31, table_width * block < 2^31.
 */
int tl_step_plan(const int32_t *ctx_lens, const int32_t *new_lens, const int32_t *owned, int64_t R, int32_t *table,
                 int64_t table_width, int64_t block, const int32_t *free_list, int64_t free_count,
                 const int32_t *free_head, const int32_t *parents, int64_t T, int32_t *q_start, int32_t *kv_lens,
                 int64_t *slots, int32_t *positions, uint64_t *tree_mask, int32_t *owned_out,
                 int32_t *free_head_out, void *stream);

/*
 * tl_kv_write
 * in  k, v       bf16 [T, H, D], tokens ldk / ldv elements apart (column ranges of the qkv
 *                layer's output, for instance); multiples of 8
 * in  slots      int64 [T]; two tokens of a call must not share a slot
 * in  q          bf16 [T, Hq, D], tokens ldq apart, or NULL (then q_out is not written)
 * in  positions  int32 [T], cos_sin f32 [max_pos, rot]: rot/2 cosines, then rot/2 sines, of
 *                each position; or cos_sin NULL: no rotation.  The first rot elements of
 *                every q and k row are rotated in pairs (d, d + rot/2), in f32, and rounded
 *                to bf16.  Positions are clamped to the table.
 * out q_out      bf16 [T, Hq, D]
 * io  k_cache, v_cache and, for e4m3, k_scale, v_scale: the tokens' rows.  e4m3: scale =
 *                fl32(amax / 448) of the (rotated, rounded) row, code = RNE(fl32(x / scale)),
 *                both 0 for a row of zeros.
 * Requires rot a multiple of 16, at most D; max_pos < 2^31; Hq <= 65536; finite inputs.
 */
int tl_kv_write(const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv, const int64_t *slots, int64_t T,
                int64_t H, int64_t D, const uint16_t *q, int64_t ldq, int64_t Hq, const int32_t *positions,
                const float *cos_sin, int64_t max_pos, int64_t rot, uint16_t *q_out, void *k_cache, void *v_cache,
                float *k_scale, float *v_scale, int cache_dtype, int64_t pages, int64_t block, void *stream);

/*
 * tl_tree_attention
 * in  q          bf16 [T, H * G, D], tokens ldq elements apart (a multiple of 8); query heads
 *                h G .. h G + G - 1 read cache head h
 * in  caches and scales as tl_kv_write leaves them; the step's own rows are in them
 * in  table      int32 [R, table_width]
 * in  q_start    int32 [R + 1], kv_lens int32 [R]: request r's tokens are q_start[r] ..
 *                q_start[r + 1] - 1 (n of them), its keys the positions 0 .. kv_lens[r] - 1,
 *                of which the last n are its own tokens; positions past the table (and in
 *                table entries that are no page) are not there.  q_start must not fall: where
 *                it does, nothing is written at all
 * in  tree_mask  uint64 [T] or NULL.  A token sees every key before its request's own
 *                tokens and, with a mask in a request of up to 64 tokens, the own token j
 *                where bit j is set; else the own tokens up to itself.
 * out out        bf16 [T, H * G, D]: softmax(scale q K^T) V over the keys it sees, 0 if none
 * out lse        f32 [T, H * G] or NULL: log of the sum of exponentials, -inf if none; NaN
 *                (as out) where a score is NaN
 * max_nodes      the most tokens a request has, as far as the caller knows: it chooses the
 *                kernel and sizes the workspace; lengths above it are still right
 * workspace      tl_tree_attention_workspace_size(max_nodes, G, D, cache_dtype) bytes, 16-byte
 *                aligned, contents free; calls that overlap in time must not share it
 * What lies in keys a token does not see (infinities and NaN among it) does not reach it.
 * Rows of out and lse of tokens that belong to no request are left as they are.
 * Requires scale > 0 and finite, 1 <= G <= 64, 1 <= max_nodes < 2^31, 0 <= R <= 4096,
 * T * G < 2^31, table_width * block <= 2^31 - 4096, and
 *   H * (T * G / 16 + R) * (table_width * block / 128 + 1) < 2^31:
 * the kernels count their work (16 rows by 128 keys a unit, or more) in 32 bits, and the
 * host knows the most there can be.  A longer step is several calls, over fewer of its
 * requests or heads each.
 */
size_t tl_tree_attention_workspace_size(int64_t max_nodes, int64_t G, int64_t D, int cache_dtype);
int tl_tree_attention(const uint16_t *q, int64_t ldq, int64_t T, int64_t H, int64_t G, int64_t D, const void *k_cache,
                      const void *v_cache, const float *k_scale, const float *v_scale, int cache_dtype,
                      int64_t pages, int64_t block, const int32_t *table, int64_t table_width, int64_t R,
                      const int32_t *q_start, const int32_t *kv_lens, const uint64_t *tree_mask, float scale,
                      int64_t max_nodes, uint16_t *out, float *lse, void *workspace, size_t workspace_bytes,
                      void *stream);

/*
 * tl_tree_verify -- greedy check of drafted trees.
 * in  logits     [T, V] of logits_dtype (TL_BF16 or TL_F32), rows ld elements apart
 * in  draft      int32 [T]  the nodes' tokens; parents int32 [T] as for tl_step_plan
 * in  q_start    int32 [R + 1]
 * out target     int32 [T]  index of the row's largest logit, the lowest of equals (-0 equals
 *                +0; a NaN counts as larger than every number)
 * out accepted   int32 [R]  nodes on the accepted path: node 0, then from node c the lowest
 *                node whose parent is c and whose token is target(c), as long as there is one
 * out path       int32 [R, path_width] their numbers, then -1
 * out next       int32 [R]  target of the last accepted node (-1 for a request of no tokens)
 * A request of more than 64 tokens is a prompt: all its tokens count as accepted, path is
 * -1, next its last token's target.
 * Which requests were served is not known here: where tl_step_plan left kv_lens at 0 (and
 * tl_kv_commit leaves the context as it was) the logits, and so these outputs, mean nothing.
 * workspace      tl_tree_verify_workspace_size(T, V) bytes, 16-byte aligned, contents free
 * Requires 1 <= path_width <= 64, 1 <= V <= ld < 2^31, 0 <= R <= 4096, and T times the parts
 * of a row (at most 64) below 2^31.
 */
size_t tl_tree_verify_workspace_size(int64_t T, int64_t V);
int tl_tree_verify(const void *logits, int logits_dtype, int64_t ld, int64_t T, int64_t V, const int32_t *draft,
                   const int32_t *parents, const int32_t *q_start, int64_t R, int32_t *accepted, int32_t *path,
                   int64_t path_width, int32_t *next, int32_t *target, void *workspace, size_t workspace_bytes,
                   void *stream);

/*
 * tl_kv_commit -- the accepted nodes' rows to the positions after the context.
 * in  accepted   int32 [R], path int32 [R, path_width] from tl_tree_verify
 * in  ctx_lens   int32 [R] (before the step), kv_lens int32 [R] from tl_step_plan
 * in  table      int32 [R, table_width]
 * io  k_cache, v_cache [L, pages, H, block, D] and, for e4m3, the scales: for each layer and
 *                head the row of position ctx + path[i] goes to ctx + i, for i < accepted;
 *                every source is read before it is overwritten
 * out ctx_out    int32 [R]: ctx + accepted; ctx for a request that was not served.  Of a request
 *                of up to 64 tokens no more than path_width nodes are committed and counted:
 *                where the later ones' rows lie is not known
 * Entries of path that do not move a row forward inside the request are skipped.
 * Requires 1 <= path_width <= 64, 1 <= L <= 4096, 0 <= R <= 4096, L * R * H < 2^31,
 * L * pages * H * block * D <= 2^50, table_width * block < 2^31.
 */
int tl_kv_commit(const int32_t *accepted, const int32_t *path, int64_t path_width, const int32_t *ctx_lens,
                 const int32_t *kv_lens, const int32_t *table, int64_t table_width, int64_t R, void *k_cache,
                 void *v_cache, float *k_scale, float *v_scale, int cache_dtype, int64_t L, int64_t pages, int64_t H,
                 int64_t block, int64_t D, int32_t *ctx_out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TL_H */
