// api_lm.cu -- entry points of include/cr_lm.h: argument checks, the choice
// between vector and scalar kernels, and the workspace.
#include <math.h>

#include "api_matrix.h"
#include "lm_internal.cuh"

using namespace cr;
using namespace cr::host;

namespace {

cr_status check_id_bits(int bits) {
  if (bits == 32 || bits == 64) return CR_OK;
  return fail(CR_ERR_INVALID_ARG, "id_bits=%d is neither 32 nor 64", bits);
}

// A scale that is finite in fp32.
cr_status check_scale(double scale) {
  if (isfinite((float)scale)) return CR_OK;
  return fail(CR_ERR_INVALID_ARG, "scale=%g must be finite in fp32", scale);
}

// One over a temperature.  Past 2^126 its product with log2(e) may not be finite.
cr_status check_softmax_scale(double scale) {
  if ((float)scale > 0.0f && (float)scale <= 8.507059173023462e37f) return CR_OK;
  return fail(CR_ERR_INVALID_ARG, "scale=%g must be above 0 and at most 2^126 in fp32", scale);
}

cr_status check_vocab(uint64_t vocab, uint64_t rows) {
  if (rows && vocab == 0) return fail(CR_ERR_INVALID_ARG, "vocab is 0");
  if (vocab >= (1ull << 31) - 65536)
    return fail(CR_ERR_UNSUPPORTED, "vocab=%llu is 2^31 - 65536 or more", (unsigned long long)vocab);
  return CR_OK;
}

size_t id_size(int bits) { return bits / 8; }

}  // namespace

extern "C" {

cr_status cr_embedding(const void* table, size_t ldt, size_t vocab, const void* ids, int id_bits,
                       size_t tokens, size_t dim, cr_dtype dtype, double scale, void* out,
                       size_t ldo, cr_dtype out_dtype, cr_stream_t stream) {
  cr_status st = check_float(dtype, "dtype");
  if (st != CR_OK || (st = check_float(out_dtype, "out_dtype")) != CR_OK) return st;
  if ((st = check_id_bits(id_bits)) != CR_OK || (st = check_scale(scale)) != CR_OK) return st;
  if ((st = check_size(vocab, "vocab")) != CR_OK || (st = check_size(tokens, "tokens")) != CR_OK ||
      (st = check_size(dim, "dim")) != CR_OK)
    return st;
  Args a;
  a.matrix("table", table, tokens ? vocab : 0, dim, ldt, esize_of(dtype), false);
  a.raw("ids", ids, 1, dim ? tokens : 0, tokens, id_size(id_bits), false);
  a.matrix("out", out, tokens, dim, ldo, esize_of(out_dtype), true);
  if ((st = a.disjoint(never)) != CR_OK) return st;
  if (tokens == 0 || dim == 0) return ok();
  const EmbedArgs k = {mat(table, ldt), mat(out, ldo), Ids{ids, id_bits}, tokens,
                       (uint32_t)vocab, (uint32_t)dim, (float)scale};
  return launched(launch_embed(dtype, out_dtype, k, a.vec(), stream_of(stream)), "cr_embedding");
}

size_t cr_embedding_backward_workspace_bytes(size_t tokens, size_t vocab, size_t dim) {
  if (tokens >= (1ull << 31) || vocab > kEmbedVocab || dim >= (1ull << 31)) return 0;
  if (vocab == 0 || dim == 0) return 0;
  return (size_t)embed_back_workspace(tokens, vocab, dim);
}

cr_status cr_embedding_backward(const void* dout, size_t lddo, cr_dtype dtype, const void* ids,
                                int id_bits, size_t tokens, size_t vocab, size_t dim, double scale,
                                const void* base, size_t ldb, void* dtable, size_t ldt,
                                cr_dtype dt_dtype, void* workspace, size_t workspace_bytes,
                                cr_stream_t stream) {
  cr_status st = check_float(dtype, "dtype");
  if (st != CR_OK || (st = check_float(dt_dtype, "dt_dtype")) != CR_OK) return st;
  if ((st = check_id_bits(id_bits)) != CR_OK || (st = check_scale(scale)) != CR_OK) return st;
  if ((st = check_size(tokens, "tokens")) != CR_OK || (st = check_size(dim, "dim")) != CR_OK) return st;
  if (vocab > kEmbedVocab)
    return fail(CR_ERR_UNSUPPORTED, "vocab=%zu is above %llu", vocab, (unsigned long long)kEmbedVocab);
  const size_t need = cr_embedding_backward_workspace_bytes(tokens, vocab, dim);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != CR_OK) return st;
  Args a;
  a.matrix("dout", dout, vocab ? tokens : 0, dim, lddo, esize_of(dtype), false);
  a.raw("ids", ids, 1, vocab && dim ? tokens : 0, tokens, id_size(id_bits), false);
  if (base) a.matrix("base", base, vocab, dim, ldb, esize_of(dt_dtype), false);
  a.matrix("dtable", dtable, vocab, dim, ldt, esize_of(dt_dtype), true);
  if (need) a.raw("workspace", workspace, 1, need, need, 1, true);
  st = a.disjoint([](const char* out, const char* in) { return is(out, "dtable") && is(in, "base"); });
  if (st != CR_OK) return st;
  if (vocab == 0 || dim == 0) return ok();
  const EmbedBackArgs k = {mat(dout, lddo), mat(base, ldb),  mat(dtable, ldt), Ids{ids, id_bits},
                           tokens,          (uint32_t)vocab, (uint32_t)dim,    (float)scale,
                           base == dtable};
  return launched(launch_embed_back(dtype, dt_dtype, k, workspace, a.vec(), stream_of(stream)),
                  "cr_embedding_backward");
}

cr_status cr_dropout(const void* x, size_t ldx, const void* residual, size_t ldr, size_t rows,
                     size_t cols, cr_dtype dtype, double p, const uint64_t* rng, uint64_t call,
                     uint64_t first_row, void* out, size_t ldo, cr_stream_t stream) {
  cr_status st = check_float(dtype, "dtype");
  if (st != CR_OK) return st;
  if (!(p >= 0.0 && p <= 1.0)) return fail(CR_ERR_INVALID_ARG, "p=%g outside [0, 1]", p);
  if ((st = check_size(rows, "rows")) != CR_OK || (st = check_size(cols, "cols")) != CR_OK) return st;
  if (first_row > (1ull << 32) || first_row + rows > (1ull << 32))
    return fail(CR_ERR_INVALID_ARG, "first_row=%llu + %zu rows pass 2^32",
                (unsigned long long)first_row, rows);
  const size_t es = esize_of(dtype);
  Args a;
  a.matrix("x", x, rows, cols, ldx, es, false);
  if (residual) a.matrix("residual", residual, rows, cols, ldr, es, false);
  a.raw("rng", rng, 1, rows && cols ? 2 : 0, 2, 8, false);
  a.matrix("out", out, rows, cols, ldo, es, true);
  st = a.disjoint([](const char*, const char* in) { return is(in, "x") || is(in, "residual"); });
  if (st != CR_OK) return st;
  if (rows == 0 || cols == 0) return ok();
  DropoutArgs k = {};
  k.x = mat(x, ldx), k.residual = mat(residual, ldr), k.out = mat(out, ldo);
  k.rng = rng;
  k.call = call;
  k.rows = rows;
  k.cols = (uint32_t)cols;
  k.first_row = (uint32_t)first_row;
  k.limit = (uint32_t)floor(p * 65536.0 + 0.5);
  k.by = k.limit == 65536 ? 0.0f : (float)(65536.0 / (65536.0 - k.limit));
  return launched(launch_dropout(dtype, k, a.vec(), stream_of(stream)), "cr_dropout");
}

cr_status cr_log_probs(const void* logits, size_t ldl, const void* targets, int id_bits,
                       size_t rows, size_t vocab, cr_dtype dtype, double scale, float* logp,
                       float* entropy, float* lse, int top, int32_t* top_ids, float* top_logp,
                       cr_stream_t stream) {
  cr_status st = check_float(dtype, "dtype");
  if (st != CR_OK || (st = check_id_bits(id_bits)) != CR_OK ||
      (st = check_softmax_scale(scale)) != CR_OK || (st = check_size(rows, "rows")) != CR_OK ||
      (st = check_vocab(vocab, rows)) != CR_OK)
    return st;
  if (top < 0 || top > CR_MAX_TOP || (rows && (size_t)top > vocab))
    return fail(CR_ERR_INVALID_ARG, "top=%d outside [0, %d] or above vocab=%zu", top, CR_MAX_TOP, vocab);
  Args a;
  a.matrix("logits", logits, rows, vocab, ldl, esize_of(dtype), false);
  if (logp) a.raw("targets", targets, 1, rows, rows, id_size(id_bits), false);
  if (logp) a.raw("logp", logp, 1, rows, rows, 4, true);
  if (entropy) a.raw("entropy", entropy, 1, rows, rows, 4, true);
  if (lse) a.raw("lse", lse, 1, rows, rows, 4, true);
  if (top_ids) a.raw("top_ids", top_ids, rows, top, top, 4, true);
  if (top_logp) a.raw("top_logp", top_logp, rows, top, top, 4, true);
  if ((st = a.disjoint(never)) != CR_OK) return st;
  if (!top_ids && !top_logp) top = 0;
  if (rows == 0 || !(logp || entropy || lse || top)) return ok();
  LogProbArgs k = {};
  k.logits = mat(logits, ldl);
  k.targets = Ids{targets, id_bits};
  k.rows = rows;
  k.vocab = (uint32_t)vocab;
  k.scale = (float)scale;
  k.logp = logp, k.entropy = entropy, k.lse = lse;
  k.top = top;
  k.top_ids = top_ids;
  k.top_logp = top_logp;
  return launched(launch_log_probs(dtype, k, stream_of(stream)), "cr_log_probs");
}

cr_status cr_log_probs_backward(const void* logits, size_t ldl, const void* targets, int id_bits,
                                size_t rows, size_t vocab, cr_dtype dtype, double scale,
                                const float* lse, const float* entropy, const float* dlogp,
                                const float* dentropy, const float* dlse, void* dlogits,
                                size_t lddl, cr_stream_t stream) {
  cr_status st = check_float(dtype, "dtype");
  if (st != CR_OK || (st = check_id_bits(id_bits)) != CR_OK ||
      (st = check_softmax_scale(scale)) != CR_OK || (st = check_size(rows, "rows")) != CR_OK ||
      (st = check_vocab(vocab, rows)) != CR_OK)
    return st;
  const size_t es = esize_of(dtype);
  Args a;
  a.matrix("logits", logits, rows, vocab, ldl, es, false);
  if (dlogp) a.raw("targets", targets, 1, rows, rows, id_size(id_bits), false);
  a.raw("lse", lse, 1, rows, rows, 4, false);
  if (dentropy) a.raw("entropy", entropy, 1, rows, rows, 4, false);
  if (dlogp) a.raw("dlogp", dlogp, 1, rows, rows, 4, false);
  if (dentropy) a.raw("dentropy", dentropy, 1, rows, rows, 4, false);
  if (dlse) a.raw("dlse", dlse, 1, rows, rows, 4, false);
  a.matrix("dlogits", dlogits, rows, vocab, lddl, es, true);
  st = a.disjoint([](const char*, const char* in) { return is(in, "logits"); });
  if (st != CR_OK) return st;
  if (rows == 0) return ok();
  LogProbBackArgs k = {};
  k.logits = mat(logits, ldl), k.dlogits = mat(dlogits, lddl);
  k.targets = Ids{targets, id_bits};
  k.rows = rows;
  k.vocab = (uint32_t)vocab;
  k.scale = (float)scale;
  k.lse = lse, k.entropy = entropy;
  k.dlogp = dlogp, k.dentropy = dentropy, k.dlse = dlse;
  return launched(launch_log_probs_back(dtype, k, a.vec(), stream_of(stream)),
                  "cr_log_probs_backward");
}

cr_status cr_lm_call(cr_lm_op op, const void* words) {
  if (!words) return fail(CR_ERR_INVALID_ARG, "words is NULL");
  const uint64_t* w = static_cast<const uint64_t*>(words);
  const auto in = [&](int i) { return reinterpret_cast<const void*>(w[i]); };
  const auto out = [&](int i) { return reinterpret_cast<void*>(w[i]); };
  const auto floats = [&](int i) { return reinterpret_cast<float*>(w[i]); };
  const auto bits = [&](int i) { return (int)(int64_t)w[i]; };
  const auto type = [&](int i) { return (cr_dtype)w[i]; };
  const auto real = [&](int i) {
    double v;
    memcpy(&v, &w[i], sizeof(v));
    return v;
  };
  const auto stream = [&](int i) { return reinterpret_cast<cr_stream_t>(w[i]); };
  switch (op) {
    case CR_CALL_EMBEDDING:
      return cr_embedding(in(0), w[1], w[2], in(3), bits(4), w[5], w[6], type(7), real(8), out(9),
                          w[10], type(11), stream(12));
    case CR_CALL_EMBEDDING_BACKWARD:
      return cr_embedding_backward(in(0), w[1], type(2), in(3), bits(4), w[5], w[6], w[7], real(8),
                                   in(9), w[10], out(11), w[12], type(13), out(14), w[15],
                                   stream(16));
    case CR_CALL_DROPOUT:
      return cr_dropout(in(0), w[1], in(2), w[3], w[4], w[5], type(6), real(7),
                        reinterpret_cast<const uint64_t*>(w[8]), w[9], w[10], out(11), w[12],
                        stream(13));
    case CR_CALL_LOG_PROBS:
      return cr_log_probs(in(0), w[1], in(2), bits(3), w[4], w[5], type(6), real(7), floats(8),
                          floats(9), floats(10), bits(11), reinterpret_cast<int32_t*>(w[12]),
                          floats(13), stream(14));
    case CR_CALL_LOG_PROBS_BACKWARD:
      return cr_log_probs_backward(in(0), w[1], in(2), bits(3), w[4], w[5], type(6), real(7),
                                   floats(8), floats(9), floats(10), floats(11), floats(12),
                                   out(13), w[14], stream(15));
  }
  return fail(CR_ERR_INVALID_ARG, "unknown call %d", (int)op);
}

}  // extern "C"
