/*
 * cr_ffn.h -- C ABI of libcr, second part: the operators of a transformer's
 * feed-forward sublayer, whose weight gradients the collectives and the FSDP
 * step of cr.h reduce and apply.
 *
 *   cr_rms_norm            sum = x + residual, RMS norm, 8-bit output
 *   cr_glu                 a = act(x Wg^T) * (x Wu^T) in one kernel
 *   cr_q8_store, cr_q8_load  8-bit activation checkpoints
 *   cr_glu_act_backward    the gate's backward pass from 8-bit checkpoints
 *   cr_glu_backward        dx, dWg, dWu of cr_glu from 8-bit checkpoints
 *   cr_rms_norm_backward   dx, dweight of cr_rms_norm
 *
 * A training step calls them in that order: the norm writes its output y for
 * the block and y's 8-bit checkpoint; the block writes `a` for the down
 * projection and keeps gate and up in 8 bits from its epilogue; backward
 * reads the three checkpoints, and dx of the block is dy of the norm.
 * Weight gradients come out as bf16, the type cr_fsdp_step takes, or fp32.
 *
 * Conventions: those of cr.h (caller-owned buffers, no allocation, one
 * stream argument, status codes, cr_last_error), and
 *  - A matrix is row-major: a device pointer and its row stride `ld` in
 *    elements, ld >= columns (a matrix of at most one row may give any ld).
 *    Columns are contiguous.  Any element-aligned pointer and any ld work;
 *    16-byte aligned pointers and row strides take the fast path.
 *  - Optional matrices are NULL where they are not wanted (then their ld is
 *    ignored).
 *  - Outputs may not overlap inputs or each other, except as each call
 *    allows (CR_ERR_INVALID_ARG).  Two matrices with one row stride that use
 *    different columns of the same rows (halves of a fused buffer) do not
 *    overlap.
 *  - Zero rows or columns are legal: the call writes what remains defined
 *    (sums over nothing are zero) and returns CR_OK.
 *  - Row and column counts of one matrix are below 2^31 (CR_ERR_UNSUPPORTED);
 *    element offsets are 64-bit.
 *  - dtype is CR_F32 or CR_BF16 where a call takes one; the block's calls
 *    take CR_BF16 only (CR_ERR_UNSUPPORTED otherwise: the tensor cores have
 *    no full fp32 product).  Arithmetic is fp32 throughout, rounded once to
 *    the output's type, with the exceptions named at each call.
 *  - Every result is deterministic: no sum depends on the order in which
 *    blocks run.
 */
#ifndef CR_FFN_H
#define CR_FFN_H

#include "cr.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- 8-bit matrices -------------------------------------------------------
 * rows x cols values held as e4m3 codes (1 sign, 4 exponent, 3 fraction bits,
 * bias 7, largest 448, 0x7f = NaN) and one fp32 scale for each row and each
 * group of CR_Q8_GROUP columns (the last group of a row may be shorter).
 * With m the largest finite magnitude of a group:
 *     scale = max(m * (1/448), 2^-126),   code = e4m3(value * (1/scale)),
 * each operation in fp32, nearest even, the code saturated at 448.  A value
 * that is not finite becomes the NaN code, so an overflow stays visible.
 * The matrix stands for code * scale.
 *   codes   rows x cols bytes, row stride ld
 *   scales  rows x ceil(cols / CR_Q8_GROUP) floats, row stride lds */
#define CR_Q8_GROUP 128
typedef struct cr_q8 {
  void* codes;
  size_t ld;
  float* scales;
  size_t lds;
} cr_q8;

/* q = the 8-bit form of x (rows x cols of dtype). */
cr_status cr_q8_store(const void* x, size_t ldx, size_t rows, size_t cols,
                      cr_dtype dtype, const cr_q8* q, cr_stream_t stream);
/* x = the values q stands for, rounded to dtype. */
cr_status cr_q8_load(const cr_q8* q, size_t rows, size_t cols, void* x,
                     size_t ldx, cr_dtype dtype, cr_stream_t stream);

/* ---- RMS norm with the residual's addition --------------------------------
 *     h = x + residual          (fp32; h = x without a residual)
 *     rstd = 1 / sqrt(mean over the row of h^2 + eps)
 *     v = h * rstd * weight
 *   x, residual  rows x cols of dtype (residual optional)
 *   weight       cols of dtype
 *   sum          h rounded to dtype (optional)
 *   y            v rounded to dtype (optional)
 *   y8           8-bit form of v, quantised from fp32 (optional)
 *   rstd         rows floats (optional; cr_rms_norm_backward reads it)
 * sum or y may be x or residual itself (same pointer and ld).  eps is rounded
 * to fp32: >= 0 and finite there (CR_ERR_INVALID_ARG).  A row of zeros with eps
 * 0 gives NaN, as the formula does.  h^2 and its sum are fp32: a row whose sum
 * of squares passes fp32's range (values from about 1e19) has rstd 0. */
cr_status cr_rms_norm(const void* x, size_t ldx, const void* residual,
                      size_t ldr, const void* weight, size_t rows, size_t cols,
                      cr_dtype dtype, double eps, void* sum, size_t ldsum,
                      void* y, size_t ldy, const cr_q8* y8, float* rstd,
                      cr_stream_t stream);

/* With n = h * rstd and c = mean over the row of (dy * weight * n):
 *     dx = rstd * (dy * weight - n * c) + dres
 *     dweight = sum over the rows of dy * n
 * dx is the gradient of both x and residual; dres is the gradient that
 * reaches `sum` along the residual stream (optional).
 *   h or h8      the norm's input (`sum`, or x without a residual), as a
 *                matrix of dtype or as its 8-bit checkpoint: exactly one
 *   rstd         as cr_rms_norm wrote it
 *   dx           rows x cols of dtype (optional); may be dy, dres or h
 *   dweight      cols of dw_dtype, CR_F32 or CR_BF16 (optional)
 *   workspace    cr_rms_norm_backward_workspace_bytes() bytes, 16-byte
 *                aligned (may be NULL without dweight); its contents mean
 *                nothing before and after the call */
size_t cr_rms_norm_backward_workspace_bytes(size_t rows, size_t cols);
cr_status cr_rms_norm_backward(const void* dy, size_t lddy, const void* h,
                               size_t ldh, const cr_q8* h8, const void* weight,
                               const float* rstd, const void* dres,
                               size_t lddres, size_t rows, size_t cols,
                               cr_dtype dtype, void* dx, size_t lddx,
                               void* dweight, cr_dtype dw_dtype,
                               void* workspace, size_t workspace_bytes,
                               cr_stream_t stream);

/* ---- gated feed-forward block ----------------------------------------------
 * act(z): CR_ACT_SILU  z / (1 + exp(-z))
 *         CR_ACT_GELU  z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) */
typedef enum { CR_ACT_SILU = 0, CR_ACT_GELU = 1 } cr_act;

/*     g = x wg^T,  u = x wu^T,  a = act(g) * u
 *   x       tokens x dim, bf16      wg, wu  ffn x dim, bf16
 *   a       tokens x ffn, bf16
 *   g8, u8  8-bit checkpoints of g and u, quantised from the fp32 sums
 *           (each optional)
 * The down projection is a plain matrix product of `a` and is left to the
 * caller.
 *   workspace  cr_glu_workspace_bytes(tokens, dim, ffn) bytes, 16-byte
 *              aligned; contents mean nothing before and after the call. */
size_t cr_glu_workspace_bytes(size_t tokens, size_t dim, size_t ffn);
cr_status cr_glu(const void* x, size_t ldx, const void* wg, size_t ldwg,
                 const void* wu, size_t ldwu, size_t tokens, size_t dim,
                 size_t ffn, cr_dtype dtype, cr_act act, void* a, size_t lda,
                 const cr_q8* g8, const cr_q8* u8, void* workspace,
                 size_t workspace_bytes, cr_stream_t stream);

/* The elementwise part of the block's backward pass, from its checkpoints:
 *     dg = da * u * act'(g),  du = da * act(g),  a = act(g) * u
 * g and u are the values g8 and u8 stand for.  `a`, recomputed here, is what
 * the down projection's weight gradient needs.
 *   da, dg, du, a  tokens x ffn, bf16; dg, du and a are each optional, and
 *                  any one of them may be da itself (same pointer and ld) */
cr_status cr_glu_act_backward(const void* da, size_t ldda, const cr_q8* g8,
                              const cr_q8* u8, size_t tokens, size_t ffn,
                              cr_dtype dtype, cr_act act, void* dg, size_t lddg,
                              void* du, size_t lddu, void* a, size_t lda,
                              cr_stream_t stream);

/* The whole backward pass of cr_glu:
 *     dx = dg wg + du wu,  dwg = dg^T x,  dwu = du^T x,  a = act(g) * u
 * with dg and du as above.  They enter the products of dx, and those of dwg and
 * dwu over more than 64 tokens, rounded to bf16: a relative error of 2^-8 at
 * most in every term, about 0.0017 of the result's norm however long the sum
 * is, also where dw_dtype is CR_F32.  For dwg and dwu over at most 64 tokens
 * they enter as sums of two bf16 numbers (2^-16), so that a CR_F32 result there
 * is within 2^-14 of its norm.
 *   x or x8    the block's input, tokens x dim, as bf16 or as its 8-bit
 *              checkpoint (whose values enter the products as a sum of two
 *              bf16 numbers, exact to 2^-16): exactly one
 *   dx         tokens x dim, bf16 (optional)
 *   dwg, dwu   ffn x dim, row stride dim, of dw_dtype CR_BF16 or CR_F32 (each
 *              optional)
 *   a          tokens x ffn, bf16 (optional)
 *   workspace  cr_glu_backward_workspace_bytes(tokens, dim, ffn) bytes,
 *              16-byte aligned; contents mean nothing before and after. */
size_t cr_glu_backward_workspace_bytes(size_t tokens, size_t dim, size_t ffn);
cr_status cr_glu_backward(const void* da, size_t ldda, const cr_q8* g8,
                          const cr_q8* u8, const void* x, size_t ldx,
                          const cr_q8* x8, const void* wg, size_t ldwg,
                          const void* wu, size_t ldwu, size_t tokens,
                          size_t dim, size_t ffn, cr_dtype dtype, cr_act act,
                          void* dx, size_t lddx, void* dwg, void* dwu,
                          cr_dtype dw_dtype, void* a, size_t lda,
                          void* workspace, size_t workspace_bytes,
                          cr_stream_t stream);

/* The calls above from one array of 64-bit words, for bindings whose cost grows
 * with the number of arguments: words[] holds the call's arguments in order
 * (pointers, sizes, enum values and the stream as unsigned integers, a double
 * as its bits). */
typedef enum {
  CR_CALL_Q8_STORE = 0,
  CR_CALL_Q8_LOAD = 1,
  CR_CALL_RMS_NORM = 2,
  CR_CALL_RMS_NORM_BACKWARD = 3,
  CR_CALL_GLU = 4,
  CR_CALL_GLU_ACT_BACKWARD = 5,
  CR_CALL_GLU_BACKWARD = 6
} cr_ffn_op;
cr_status cr_ffn_call(cr_ffn_op op, const void* words);

/* The block's products wait on barriers inside the kernel, each wait for about
 * half a second at most; the wait for a sum, 8 ms more for every 65536 of its K.
 * A wait that runs out (it never should) ends the kernel, leaves its results
 * undefined and sets this word, which stays set until it is cleared.  The call
 * has returned CR_OK by then, so a training loop reads the word where it waits
 * for the device anyway.  Returns the word (0: no wait ever ran out), or -2 if
 * reading it failed; waits for the device. */
long long cr_glu_wait_word(int clear);

#ifdef __cplusplus
}
#endif
#endif /* CR_FFN_H */
