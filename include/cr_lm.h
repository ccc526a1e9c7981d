/*
 * cr_lm.h -- C ABI of libcr, third part: the two ends of a language model's
 * training step, and the dropout between its sublayers.
 *
 *   cr_embedding            rows of a table, scaled
 *   cr_embedding_backward   the table's dense gradient, by sorted tokens
 *   cr_dropout              residual + dropout(x); the mask is never stored
 *   cr_log_probs            log probabilities of given tokens, entropy, log-sum-exp
 *                           and the most likely tokens, in one read of the logits
 *   cr_log_probs_backward   the logits' gradient
 *
 * With the sublayer of cr_ffn.h in between, a training step goes from token
 * ids to gradients through this library.  The embedding's gradient comes out
 * dense, as the collectives and the FSDP step of cr.h take it.
 *
 * Conventions: those of cr_ffn.h (row-major matrices with a row stride in
 * elements, any alignment to the element, caller-owned buffers, one stream,
 * overlaps refused except where a call allows them, zero sizes legal,
 * deterministic results, fp32 arithmetic rounded once to the output's type),
 * and
 *  - Token ids are integers of id_bits 32 or 64 (CR_ERR_INVALID_ARG
 *    otherwise), signed, in device memory.  An id outside [0, vocab) is no
 *    token (padding): each call says what it does there.  None is an error.
 *  - dtype is CR_F32 or CR_BF16.
 */
#ifndef CR_LM_H
#define CR_LM_H

#include "cr_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- embedding -------------------------------------------------------------
 *     out[t] = scale * table[ids[t]]        (zeros where ids[t] is no token)
 *   table  vocab x dim of dtype
 *   ids    tokens integers
 *   out    tokens x dim of out_dtype
 * scale is rounded to fp32, in which it has to be finite (CR_ERR_INVALID_ARG). */
cr_status cr_embedding(const void* table, size_t ldt, size_t vocab,
                       const void* ids, int id_bits, size_t tokens, size_t dim,
                       cr_dtype dtype, double scale, void* out, size_t ldo,
                       cr_dtype out_dtype, cr_stream_t stream);

/*     dtable[v] = base[v] + scale * sum over the t with ids[t] = v of dout[t]
 *   dout    tokens x dim of dtype
 *   base    vocab x dim of dt_dtype: the gradient so far (optional; zeros
 *           without it).  It may be dtable itself (same pointer and ld): rows
 *           that no token names are then neither read nor written, which
 *           makes a small batch's call cheap.
 *   dtable  vocab x dim of dt_dtype, every row written (but see base)
 * A row's sum is fp32 and its order depends on the ids alone: the row's tokens in
 * order, or sums of consecutive parts of them.
 * vocab is at most 2^21 (CR_ERR_UNSUPPORTED).
 *   workspace  cr_embedding_backward_workspace_bytes(tokens, vocab, dim)
 *              bytes, 16-byte aligned; contents mean nothing before and after
 *              the call.  Calls that may run at the same time (two streams, two
 *              graphs) need one each. */
size_t cr_embedding_backward_workspace_bytes(size_t tokens, size_t vocab,
                                             size_t dim);
cr_status cr_embedding_backward(const void* dout, size_t lddo, cr_dtype dtype,
                                const void* ids, int id_bits, size_t tokens,
                                size_t vocab, size_t dim, double scale,
                                const void* base, size_t ldb, void* dtable,
                                size_t ldt, cr_dtype dt_dtype, void* workspace,
                                size_t workspace_bytes, cr_stream_t stream);

/* ---- dropout ----------------------------------------------------------------
 *     out = residual + (kept ? x * c : 0)      (without a residual: 0 + ...)
 * With limit = p * 65536 rounded to the nearest integer (halves up), an element is kept
 * where its random number is at least limit, and c = 65536 / (65536 - limit)
 * rounded to fp32 (p = 1: nothing is kept): the mean of out - residual over the random numbers is
 * exactly x's but for that rounding.  An element that is dropped leaves
 * residual even where x is not finite.  p = 0 keeps everything.
 *
 * Random numbers: 16 bits for each element, a function of seed, offset, row and
 * column alone.  Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel
 * random numbers: as easy as 1, 2, 3", 2011) under the key {seed's low word,
 * high word} takes the counter {column / 8, row, offset's low word, high word}
 * to four words; column c has, of word (c mod 8) / 2, the low half where c is
 * even and the high half where it is odd.
 *   rng        two 64-bit integers in device memory: seed, and an offset to
 *              which `call` is added (modulo 2^64).  They are read when the
 *              call runs, so a captured step gets new masks where the step (or
 *              the loop between replays) moves the offset.
 *   call       tells the calls of a step apart: its number in the step, from 0.  Since it is
 *              added to the offset, a step of n calls has to move the offset by n or more: moved by one,
 *              call 1 of a step would have the mask of call 0 of the next.
 *   first_row  the row counter of the matrix's first row: a slab of rows has
 *              the mask of its part of the whole.  first_row + rows is at
 *              most 2^32 (CR_ERR_INVALID_ARG).
 * p is in [0, 1] (CR_ERR_INVALID_ARG).  out may be x or residual itself (same
 * pointer and ld).
 *
 * The backward pass is the same call on the gradient: with the same p, rng
 * contents, call and first_row, cr_dropout(dout, no residual) is x's gradient,
 * and the residual's is dout itself. */
cr_status cr_dropout(const void* x, size_t ldx, const void* residual,
                     size_t ldr, size_t rows, size_t cols, cr_dtype dtype,
                     double p, const uint64_t* rng, uint64_t call,
                     uint64_t first_row, void* out, size_t ldo,
                     cr_stream_t stream);

/* ---- log probabilities -------------------------------------------------------
 * With z = scale * logits[r] and p = softmax(z), for each row r:
 *     lse = log(sum over v of exp(z_v))
 *     logp = z_target - lse                 (0 where the target is no token)
 *     entropy = -sum over v of p_v log(p_v)
 * A logit of -infinity rules its token out (p_v = 0, and 0 log 0 = 0); a
 * row of them only has lse = -infinity, logp -infinity and entropy 0.  A row masked with
 * the type's lowest value throughout is one of equal logits.  A NaN or a logit of +infinity
 * makes the row's lse, logp, entropy and top_logp NaN.
 *   logits   rows x vocab of dtype, vocab >= 1 where there are rows
 *            (CR_ERR_INVALID_ARG)
 *   targets  rows ids (may be NULL without logp)
 *   logp, entropy, lse   rows floats, each optional
 *   top      how many of the most likely tokens are wanted, 0 to
 *            CR_MAX_TOP and at most vocab (CR_ERR_INVALID_ARG)
 *   top_ids, top_logp    rows x top packed, int32 and float: tokens in the order of
 *            falling logits, equal ones by rising id, NaN behind all others;
 *            and their log probabilities (each optional)
 * scale is rounded to fp32: > 0 and at most 2^126 there, one over the temperature
 * (CR_ERR_INVALID_ARG).  A product with it past fp32's end is infinite: in lse, and in logp where a token is that
 * far below the largest.  vocab is below 2^31 - 65536 (CR_ERR_UNSUPPORTED). */
#define CR_MAX_TOP 32
cr_status cr_log_probs(const void* logits, size_t ldl, const void* targets,
                       int id_bits, size_t rows, size_t vocab, cr_dtype dtype,
                       double scale, float* logp, float* entropy, float* lse,
                       int top, int32_t* top_ids, float* top_logp,
                       cr_stream_t stream);

/* The gradient of  sum over the rows of dlogp logp + dentropy entropy + dlse lse:
 *     dlogits_v = scale * (dlogp [v = target]
 *                          + p_v (dlse - dlogp - dentropy (log(p_v) + entropy)))
 * with p_v = exp(z_v - lse).  dlogp counts as 0 where the target is no token.
 *  - p_v = 0 (also: below 2^-126) gives 0 where the row's dlogp, dlse and 100 dentropy are finite in fp32,
 *    scaled or not.
 *  - A row whose lse is -2^100 or less (every token ruled out, by -infinity or by the type's
 *    lowest value) gets zeros, be dlogp, dentropy and dlse finite there or not.
 *  - A row whose lse is otherwise 256 or more in magnitude (filled with a finite mask value, say) goes by its own
 *    maximum and sum: rounded to fp32, such an lse leaves too little of z_v - lse.
 *   lse, entropy   as cr_log_probs wrote them of these logits (entropy may be NULL without
 *                  dentropy)
 *   targets        rows ids (may be NULL without dlogp)
 *   dlogp, dentropy, dlse  rows floats, each optional
 *   dlogits        rows x vocab of dtype; may be logits itself (same pointer
 *                  and ld) */
cr_status cr_log_probs_backward(const void* logits, size_t ldl,
                                const void* targets, int id_bits, size_t rows,
                                size_t vocab, cr_dtype dtype, double scale,
                                const float* lse, const float* entropy,
                                const float* dlogp, const float* dentropy,
                                const float* dlse, void* dlogits, size_t lddl,
                                cr_stream_t stream);

/* The calls above from one array of 64-bit words, as cr_ffn_call takes those of
 * cr_ffn.h. */
typedef enum {
  CR_CALL_EMBEDDING = 0,
  CR_CALL_EMBEDDING_BACKWARD = 1,
  CR_CALL_DROPOUT = 2,
  CR_CALL_LOG_PROBS = 3,
  CR_CALL_LOG_PROBS_BACKWARD = 4
} cr_lm_op;
cr_status cr_lm_call(cr_lm_op op, const void* words);

#ifdef __cplusplus
}
#endif
#endif /* CR_LM_H */
