// api_ffn.cu -- entry points of include/cr_ffn.h: argument checks, the choice
// between vector and scalar kernels, and the workspaces.
#include <math.h>

#include <algorithm>

#include "api_host.h"
#include "ffn_internal.cuh"

using namespace cr;
using namespace cr::host;

namespace {

// One matrix argument: its bytes and how the call uses it.
struct Arg {
  const char* name;
  uintptr_t p;
  uint64_t pitch;  // bytes from row to row
  uint64_t width;  // bytes of a row
  uint64_t rows;
  bool out;
};

// The arguments of one call, checked as they are added.
struct Args {
  Arg list[20];
  int n = 0;
  bool vec16 = true;  // every bf16/fp32 pointer and pitch, and every code pointer and
                      // pitch, is a multiple of 16 bytes
  bool vec32 = true;  // every bf16/fp32 pointer and pitch is a multiple of 32 bytes
  cr_status status = CR_OK;

  void fails(cr_status st) {
    if (status == CR_OK) status = st;
  }

  void raw(const char* name, const void* p, uint64_t rows, uint64_t cols, uint64_t ld, size_t es,
           bool out) {
    if (status != CR_OK || rows == 0 || cols == 0) return;
    if (!p) return fails(fail(CR_ERR_INVALID_ARG, "%s is NULL", name));
    if (!aligned(p, es))
      return fails(fail(CR_ERR_ALIGNMENT, "%s=%p not aligned to %zu bytes", name, p, es));
    if (rows > 1 && ld < cols)
      return fails(fail(CR_ERR_INVALID_ARG, "%s: row stride %llu below %llu columns", name,
                        (unsigned long long)ld, (unsigned long long)cols));
    if (rows == 1) ld = cols;
    if (ld > (1ull << 60) / es / rows)
      return fails(fail(CR_ERR_INVALID_ARG, "%s: row stride %llu too large", name,
                        (unsigned long long)ld));
    const Arg a = {name, reinterpret_cast<uintptr_t>(p), ld * es, cols * es, rows, out};
    list[n++] = a;
  }

  void matrix(const char* name, const void* p, uint64_t rows, uint64_t cols, uint64_t ld, size_t es,
              bool out) {
    raw(name, p, rows, cols, ld, es, out);
    if (status != CR_OK || rows == 0 || cols == 0) return;
    const uint64_t bits = reinterpret_cast<uintptr_t>(p) | (rows == 1 ? 0 : ld * es);
    vec16 = vec16 && bits % 16 == 0;
    vec32 = vec32 && bits % 32 == 0;
  }

  void q8(const char* name, const cr_q8* q, uint64_t rows, uint64_t cols, bool out) {
    if (status != CR_OK || rows == 0 || cols == 0) return;
    raw(name, q->codes, rows, cols, q->ld, 1, out);
    raw(name, q->scales, rows, (cols + CR_Q8_GROUP - 1) / CR_Q8_GROUP, q->lds, 4, out);
    vec16 = vec16 && aligned(q->codes, 16) && (rows == 1 || q->ld % 16 == 0);
  }

  // The accesses the elementwise kernels may use (ffn_internal.cuh).
  int vec() const { return !vec16 ? 0 : vec32 ? 2 : 1; }

  // Whether some row of x and some row of y share a byte.
  static bool meet(const Arg& x, const Arg& y) {
    const uintptr_t xe = x.p + (x.rows - 1) * x.pitch + x.width;
    const uintptr_t ye = y.p + (y.rows - 1) * y.pitch + y.width;
    if (x.p >= ye || y.p >= xe) return false;
    if (x.rows == 1 || y.rows == 1 || x.pitch != y.pitch) {
      // one row against the other's rows: look at the rows it may fall in
      const Arg& one = x.rows == 1 ? x : y;
      const Arg& many = x.rows == 1 ? y : x;
      if (one.rows != 1) return true;
      if (many.rows == 1 || one.p < many.p) return true;
      const uint64_t at = (one.p - many.p) % many.pitch;
      return at < many.width || at + one.width > many.pitch;
    }
    const uint64_t d = x.p <= y.p ? (y.p - x.p) % x.pitch
                                  : (x.pitch - (x.p - y.p) % x.pitch) % x.pitch;
    return d < x.width || d + y.width > x.pitch;
  }

  // No output may meet another argument; `in_place(out, other)` exempts a pair
  // that is the same matrix.
  template <typename InPlace>
  cr_status disjoint(InPlace in_place) {
    for (int i = 0; i < n && status == CR_OK; ++i) {
      if (!list[i].out) continue;
      for (int j = 0; j < n; ++j) {
        if (i == j || (list[j].out && j < i) || !meet(list[i], list[j])) continue;
        const bool same = list[i].p == list[j].p && list[i].width == list[j].width &&
                          list[i].rows == list[j].rows && list[i].pitch == list[j].pitch;
        if (same && !list[j].out && in_place(list[i].name, list[j].name)) continue;
        fails(fail(CR_ERR_INVALID_ARG, "output %s overlaps %s", list[i].name, list[j].name));
        break;
      }
    }
    return status;
  }
};

bool never(const char*, const char*) { return false; }
bool is(const char* a, const char* b) { return strcmp(a, b) == 0; }

Mat mat(const void* p, uint64_t ld) { return Mat{const_cast<void*>(p), p ? ld : 0}; }

Q8 q8_of(const cr_q8* q) {
  if (!q) return Q8{nullptr, 0, nullptr, 0};
  return Q8{static_cast<uint8_t*>(q->codes), q->ld, q->scales, q->lds};
}

cudaStream_t stream_of(cr_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

cr_status launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? ok() : cuda_fail(e, what);
}

cr_status check_float(cr_dtype d, const char* what) {
  if (esize_of(d) == 0) return fail(CR_ERR_INVALID_ARG, "%s: unknown dtype %d", what, (int)d);
  if (!is_float(d)) return fail(CR_ERR_UNSUPPORTED, "%s must be CR_F32 or CR_BF16", what);
  return CR_OK;
}

cr_status check_size(uint64_t n, const char* what) {
  if (n >= (1ull << 31))
    return fail(CR_ERR_UNSUPPORTED, "%s=%llu is 2^31 or more", what, (unsigned long long)n);
  return CR_OK;
}

cr_status check_block(cr_dtype dtype, cr_act act, uint64_t tokens, uint64_t dim, uint64_t ffn) {
  cr_status st = check_float(dtype, "dtype");
  if (st != CR_OK) return st;
  if (dtype != CR_BF16) return fail(CR_ERR_UNSUPPORTED, "the gated block takes CR_BF16 only");
  if (act != CR_ACT_SILU && act != CR_ACT_GELU)
    return fail(CR_ERR_INVALID_ARG, "unknown activation %d", (int)act);
  if ((st = check_size(tokens, "tokens")) != CR_OK) return st;
  if ((st = check_size(dim, "dim")) != CR_OK) return st;
  return check_size(ffn, "ffn");
}

cr_status check_workspace(const void* p, size_t have, size_t need) {
  if (need == 0) return CR_OK;
  if (!p) return fail(CR_ERR_INVALID_ARG, "workspace is NULL, %zu bytes needed", need);
  if (have < need)
    return fail(CR_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", have, need);
  if (!aligned(p, 16)) return fail(CR_ERR_ALIGNMENT, "workspace=%p not aligned to 16 bytes", p);
  return CR_OK;
}

uint64_t round_up(uint64_t v, uint64_t m) { return (v + m - 1) / m * m; }

// Row stride, and elements, of a bf16 workspace matrix: rows a multiple of 128
// bytes apart, which a K block's rows then fill (4001 tokens, 1001 x 4001, backward
// 149 us against 158 at multiples of 32).
uint64_t padded_ld(uint64_t cols) { return round_up(cols, 64); }
uint64_t padded(uint64_t rows, uint64_t cols) { return rows * padded_ld(cols); }

// `vec`, for a call that reads or writes a workspace matrix at p too (the
// workspace itself is 16-byte aligned).
int vec_with(int vec, const void* p) { return vec == 2 && !aligned(p, 32) ? 1 : vec; }

// Tokens up to which dW's products take dg and du in two bf16 parts: one K block,
// to which the second product adds another.  What rounding dg and du to one part
// adds to dW's error, relative to dW, is the same for any number of tokens
// (0.0017 of its norm, 0.0024 with the result's own rounding): the rule goes by
// the cost.  A backward pass of 2048 x 8192 with two parts and with one: 1 token
// 65.7 us and 60.8, 64 tokens 61.5 and 59.0, 65 tokens 64.3 and 60.5, 128 tokens
// 68.2 and 63.3, 257 tokens 86.1 and 72.0, 2048 tokens 300 and 216; 512 x 2048,
// 64 tokens 17.9 and 17.5, 128 tokens 18.4 and 18.0.
constexpr uint64_t kExactTokens = 64;

// TMA reads operands whose rows start on 16-byte boundaries; any other is
// copied to `ws` first.
void operand(CopyBf16* copies, Mat* m, uint64_t rows, uint64_t cols, uint16_t* ws) {
  if (!m->p || rows == 0 || cols == 0) return;
  if (aligned(m->p, 16) && (rows == 1 || m->ld % 8 == 0)) return;
  const Mat copy = {ws, padded_ld(cols)};
  add_copy(copies, *m, copy, rows, (uint32_t)cols);
  *m = copy;
}

}  // namespace

extern "C" {

cr_status cr_q8_store(const void* x, size_t ldx, size_t rows, size_t cols, cr_dtype dtype,
                      const cr_q8* q, cr_stream_t stream) {
  cr_status st = check_float(dtype, "dtype");
  if (st != CR_OK) return st;
  if (!q) return fail(CR_ERR_INVALID_ARG, "q is NULL");
  if ((st = check_size(rows, "rows")) != CR_OK || (st = check_size(cols, "cols")) != CR_OK) return st;
  Args a;
  a.matrix("x", x, rows, cols, ldx, esize_of(dtype), false);
  a.q8("q", q, rows, cols, true);
  if ((st = a.disjoint(never)) != CR_OK) return st;
  if (rows == 0 || cols == 0) return ok();
  return launched(launch_q8_store(dtype, mat(x, ldx), q8_of(q), rows, (uint32_t)cols, a.vec(),
                                  stream_of(stream)), "cr_q8_store");
}

cr_status cr_q8_load(const cr_q8* q, size_t rows, size_t cols, void* x, size_t ldx, cr_dtype dtype,
                     cr_stream_t stream) {
  cr_status st = check_float(dtype, "dtype");
  if (st != CR_OK) return st;
  if (!q) return fail(CR_ERR_INVALID_ARG, "q is NULL");
  if ((st = check_size(rows, "rows")) != CR_OK || (st = check_size(cols, "cols")) != CR_OK) return st;
  Args a;
  a.q8("q", q, rows, cols, false);
  a.matrix("x", x, rows, cols, ldx, esize_of(dtype), true);
  if ((st = a.disjoint(never)) != CR_OK) return st;
  if (rows == 0 || cols == 0) return ok();
  return launched(launch_q8_load(dtype, q8_of(q), mat(x, ldx), rows, (uint32_t)cols, a.vec(),
                                 stream_of(stream)), "cr_q8_load");
}

cr_status cr_rms_norm(const void* x, size_t ldx, const void* residual, size_t ldr,
                      const void* weight, size_t rows, size_t cols, cr_dtype dtype, double eps,
                      void* sum, size_t ldsum, void* y, size_t ldy, const cr_q8* y8, float* rstd,
                      cr_stream_t stream) {
  cr_status st = check_float(dtype, "dtype");
  if (st != CR_OK) return st;
  if (!(eps >= 0.0) || !isfinite((float)eps))
    return fail(CR_ERR_INVALID_ARG, "eps=%g must be >= 0 and finite in fp32", eps);
  if ((st = check_size(rows, "rows")) != CR_OK || (st = check_size(cols, "cols")) != CR_OK) return st;
  const size_t es = esize_of(dtype);
  Args a;
  a.matrix("x", x, rows, cols, ldx, es, false);
  if (residual) a.matrix("residual", residual, rows, cols, ldr, es, false);
  a.matrix("weight", weight, 1, rows ? cols : 0, cols, es, false);
  if (sum) a.matrix("sum", sum, rows, cols, ldsum, es, true);
  if (y) a.matrix("y", y, rows, cols, ldy, es, true);
  if (y8) a.q8("y8", y8, rows, cols, true);
  if (rstd) a.raw("rstd", rstd, 1, rows, rows, 4, true);
  st = a.disjoint([](const char* out, const char* in) {
    return (is(out, "sum") || is(out, "y")) && (is(in, "x") || is(in, "residual"));
  });
  if (st != CR_OK) return st;
  if (rows == 0 || cols == 0) return ok();
  NormArgs k = {};
  k.x = mat(x, ldx), k.residual = mat(residual, ldr), k.sum = mat(sum, ldsum), k.y = mat(y, ldy);
  k.y8 = q8_of(y8);
  k.weight = weight;
  k.rstd = rstd;
  k.rows = rows;
  k.cols = (uint32_t)cols;
  k.eps = (float)eps;
  k.inv_cols = 1.0f / (float)cols;
  return launched(launch_rms_norm(dtype, k, a.vec(), stream_of(stream)), "cr_rms_norm");
}

size_t cr_rms_norm_backward_workspace_bytes(size_t rows, size_t cols) {
  if (rows >= (1ull << 31) || cols >= (1ull << 31)) return 0;
  return (size_t)norm_back_parts(rows, (uint32_t)cols) * cols * sizeof(float);
}

cr_status cr_rms_norm_backward(const void* dy, size_t lddy, const void* h, size_t ldh,
                               const cr_q8* h8, const void* weight, const float* rstd,
                               const void* dres, size_t lddres, size_t rows, size_t cols,
                               cr_dtype dtype, void* dx, size_t lddx, void* dweight,
                               cr_dtype dw_dtype, void* workspace, size_t workspace_bytes,
                               cr_stream_t stream) {
  cr_status st = check_float(dtype, "dtype");
  if (st != CR_OK || (dweight && (st = check_float(dw_dtype, "dw_dtype")) != CR_OK)) return st;
  if ((h != nullptr) == (h8 != nullptr) && rows && cols)
    return fail(CR_ERR_INVALID_ARG, "exactly one of h and h8 must be given");
  if ((st = check_size(rows, "rows")) != CR_OK || (st = check_size(cols, "cols")) != CR_OK) return st;
  const size_t es = esize_of(dtype);
  const size_t need = dweight && cols ? cr_rms_norm_backward_workspace_bytes(rows, cols) : 0;
  if ((st = check_workspace(workspace, workspace_bytes, need)) != CR_OK) return st;
  Args a;
  a.matrix("dy", dy, rows, cols, lddy, es, false);
  if (h) a.matrix("h", h, rows, cols, ldh, es, false);
  if (h8) a.q8("h8", h8, rows, cols, false);
  a.matrix("weight", weight, 1, rows ? cols : 0, cols, es, false);
  a.raw("rstd", rstd, 1, cols ? rows : 0, rows, 4, false);
  if (dres) a.matrix("dres", dres, rows, cols, lddres, es, false);
  if (dx) a.matrix("dx", dx, rows, cols, lddx, es, true);
  if (dweight) a.raw("dweight", dweight, 1, cols, cols, esize_of(dw_dtype), true);
  if (need) a.raw("workspace", workspace, 1, need, need, 1, true);
  st = a.disjoint([](const char* out, const char* in) {
    return is(out, "dx") && (is(in, "dy") || is(in, "dres") || is(in, "h"));
  });
  if (st != CR_OK) return st;
  if (cols == 0 || (rows == 0 && !dweight) || (!dx && !dweight)) return ok();
  NormBackArgs k = {};
  k.dy = mat(dy, lddy), k.h = mat(h, ldh), k.dres = mat(dres, lddres);
  k.dx = mat(rows ? dx : nullptr, lddx);
  k.h8 = q8_of(h8);
  k.weight = weight;
  k.rstd = rstd;
  k.dweight = dweight;
  k.partial = dweight ? static_cast<float*>(workspace) : nullptr;
  k.rows = rows;
  k.cols = (uint32_t)cols;
  k.inv_cols = 1.0f / (float)cols;
  return launched(launch_rms_norm_back(dtype, dw_dtype, k, a.vec(), stream_of(stream)),
                  "cr_rms_norm_backward");
}

cr_status cr_glu_act_backward(const void* da, size_t ldda, const cr_q8* g8, const cr_q8* u8,
                              size_t tokens, size_t ffn, cr_dtype dtype, cr_act act, void* dg,
                              size_t lddg, void* du, size_t lddu, void* a_out, size_t lda,
                              cr_stream_t stream) {
  cr_status st = check_block(dtype, act, tokens, 0, ffn);
  if (st != CR_OK) return st;
  if (!g8 || !u8) return fail(CR_ERR_INVALID_ARG, "%s is NULL", g8 ? "u8" : "g8");
  Args a;
  a.matrix("da", da, tokens, ffn, ldda, 2, false);
  a.q8("g8", g8, tokens, ffn, false);
  a.q8("u8", u8, tokens, ffn, false);
  if (dg) a.matrix("dg", dg, tokens, ffn, lddg, 2, true);
  if (du) a.matrix("du", du, tokens, ffn, lddu, 2, true);
  if (a_out) a.matrix("a", a_out, tokens, ffn, lda, 2, true);
  st = a.disjoint([](const char*, const char* in) { return is(in, "da"); });
  if (st != CR_OK) return st;
  if (tokens == 0 || ffn == 0 || (!dg && !du && !a_out)) return ok();
  ActBackArgs k = {mat(da, ldda), mat(dg, lddg), mat(du, lddu), mat(a_out, lda),
                   q8_of(g8),     q8_of(u8),     tokens,        (uint32_t)ffn, {}, {}};
  return launched(launch_act_back(act, k, nullptr, a.vec(), stream_of(stream)),
                  "cr_glu_act_backward");
}

size_t cr_glu_workspace_bytes(size_t tokens, size_t dim, size_t ffn) {
  if (tokens >= (1ull << 31) || dim >= (1ull << 31) || ffn >= (1ull << 31)) return 0;
  if (tokens == 0 || ffn == 0) return 0;
  // room for copies of operands that are not aligned
  return 2 * (padded(tokens, dim) + 2 * padded(ffn, dim));
}

cr_status cr_glu(const void* x, size_t ldx, const void* wg, size_t ldwg, const void* wu,
                 size_t ldwu, size_t tokens, size_t dim, size_t ffn, cr_dtype dtype, cr_act act,
                 void* a_out, size_t lda, const cr_q8* g8, const cr_q8* u8, void* workspace,
                 size_t workspace_bytes, cr_stream_t stream) {
  cr_status st = check_block(dtype, act, tokens, dim, ffn);
  if (st != CR_OK) return st;
  const size_t need = cr_glu_workspace_bytes(tokens, dim, ffn);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != CR_OK) return st;
  Args a;
  a.matrix("x", x, tokens, dim, ldx, 2, false);
  a.matrix("wg", wg, tokens ? ffn : 0, dim, ldwg, 2, false);
  a.matrix("wu", wu, tokens ? ffn : 0, dim, ldwu, 2, false);
  a.matrix("a", a_out, tokens, ffn, lda, 2, true);
  if (g8) a.q8("g8", g8, tokens, ffn, true);
  if (u8) a.q8("u8", u8, tokens, ffn, true);
  if (need) a.raw("workspace", workspace, 1, need, need, 1, true);
  if ((st = a.disjoint(never)) != CR_OK) return st;
  if (tokens == 0 || ffn == 0) return ok();
  GluArgs k = {mat(x, ldx), mat(wg, ldwg), mat(wu, ldwu),   mat(a_out, lda), q8_of(g8),
               q8_of(u8),   (uint32_t)tokens, (uint32_t)dim, (uint32_t)ffn};
  const cudaStream_t s = stream_of(stream);
  if (glu_few(tokens, dim, g8 || u8)) {
    Args w;
    w.matrix("wg", wg, ffn, dim, ldwg, 2, false);
    w.matrix("wu", wu, ffn, dim, ldwu, 2, false);
    return launched(launch_glu_few(act, k, w.vec(), s), "cr_glu");
  }
  uint16_t* ws = static_cast<uint16_t*>(workspace);
  CopyBf16 copies = {};
  operand(&copies, &k.x, tokens, dim, ws);
  ws += padded(tokens, dim);
  operand(&copies, &k.wg, ffn, dim, ws);
  ws += padded(ffn, dim);
  operand(&copies, &k.wu, ffn, dim, ws);
  cudaError_t e = launch_copy_bf16(copies, s);
  if (e == cudaSuccess) e = launch_glu(act, k, s);
  return launched(e, "cr_glu");
}

size_t cr_glu_backward_workspace_bytes(size_t tokens, size_t dim, size_t ffn) {
  if (tokens >= (1ull << 31) || dim >= (1ull << 31) || ffn >= (1ull << 31)) return 0;
  // dg and du; x restored from its checkpoint, in two parts; copies of
  // weights that are not aligned; what dg and du were rounded by
  const size_t rest = tokens <= kExactTokens ? 2 * padded(tokens, ffn) : 0;
  return 2 * (2 * padded(tokens, ffn) + 2 * padded(tokens, dim) + 2 * padded(ffn, dim) + rest);
}

cr_status cr_glu_backward(const void* da, size_t ldda, const cr_q8* g8, const cr_q8* u8,
                          const void* x, size_t ldx, const cr_q8* x8, const void* wg, size_t ldwg,
                          const void* wu, size_t ldwu, size_t tokens, size_t dim, size_t ffn,
                          cr_dtype dtype, cr_act act, void* dx, size_t lddx, void* dwg, void* dwu,
                          cr_dtype dw_dtype, void* a_out, size_t lda, void* workspace,
                          size_t workspace_bytes, cr_stream_t stream) {
  cr_status st = check_block(dtype, act, tokens, dim, ffn);
  if (st != CR_OK) return st;
  const bool dw = dwg || dwu;
  if (dw && (st = check_float(dw_dtype, "dw_dtype")) != CR_OK) return st;
  if (!g8 || !u8) return fail(CR_ERR_INVALID_ARG, "%s is NULL", g8 ? "u8" : "g8");
  if ((x != nullptr) == (x8 != nullptr) && dw && tokens && dim)
    return fail(CR_ERR_INVALID_ARG, "exactly one of x and x8 must be given");
  const size_t need = cr_glu_backward_workspace_bytes(tokens, dim, ffn);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != CR_OK) return st;
  const size_t des = dw ? esize_of(dw_dtype) : 0;
  Args a;
  a.matrix("da", da, tokens, ffn, ldda, 2, false);
  a.q8("g8", g8, tokens, ffn, false);
  a.q8("u8", u8, tokens, ffn, false);
  if (a_out) a.matrix("a", a_out, tokens, ffn, lda, 2, true);
  const int act_vec = a.vec();
  Args xa;
  if (dw && x8) {
    a.q8("x8", x8, tokens, dim, false);
    xa.q8("x8", x8, tokens, dim, false);
  } else if (dw) {
    a.matrix("x", x, tokens, dim, ldx, 2, false);
  }
  if (dx) {
    a.matrix("wg", wg, tokens ? ffn : 0, dim, ldwg, 2, false);
    a.matrix("wu", wu, tokens ? ffn : 0, dim, ldwu, 2, false);
    a.matrix("dx", dx, tokens, dim, lddx, 2, true);
  }
  if (dwg) a.raw("dwg", dwg, ffn, dim, dim, des, true);
  if (dwu) a.raw("dwu", dwu, ffn, dim, dim, des, true);
  if (need) a.raw("workspace", workspace, 1, need, need, 1, true);
  if ((st = a.disjoint(never)) != CR_OK) return st;

  const cudaStream_t s = stream_of(stream);
  uint16_t* ws = static_cast<uint16_t*>(workspace);
  const Mat dg = {ws, padded_ld(ffn)};
  const Mat du = {ws + padded(tokens, ffn), padded_ld(ffn)};
  uint16_t* const xs = ws + 2 * padded(tokens, ffn);
  Mat dg_lo = {}, du_lo = {};
  if (dw && tokens <= kExactTokens) {
    dg_lo = Mat{xs + 2 * padded(tokens, dim) + 2 * padded(ffn, dim), padded_ld(ffn)};
    du_lo = Mat{static_cast<uint16_t*>(dg_lo.p) + padded(tokens, ffn), padded_ld(ffn)};
  }
  cudaError_t e = cudaSuccess;
  const SplitArgs split = {q8_of(x8), Mat{xs, padded_ld(dim)},
                           Mat{xs + padded(tokens, dim), padded_ld(dim)}, tokens, (uint32_t)dim,
                           xa.vec()};
  const bool splits = dw && x8 && tokens && dim;
  if (tokens && ffn) {
    ActBackArgs k = {mat(da, ldda), dg,     du, mat(a_out, lda), q8_of(g8), q8_of(u8),
                     tokens,        (uint32_t)ffn, dg_lo, du_lo};
    if (!dx && !dw) k.dg = k.du = Mat{nullptr, 0};
    if (k.dg.p || k.a.p)
      e = launch_act_back(act, k, splits ? &split : nullptr, vec_with(act_vec, ws), s);
    if (e != cudaSuccess) return cuda_fail(e, "cr_glu_backward: activation");
  }
  if (dim == 0 || (!dw && !(dx && tokens))) return ok();
  GluBackArgs k = {};
  k.dg = dg, k.du = du;
  k.dg_lo = dg_lo, k.du_lo = du_lo;
  k.x = mat(x, ldx);
  k.wg = mat(wg, ldwg), k.wu = mat(wu, ldwu);
  ws = xs;
  CopyBf16 copies = {};
  if (splits) {
    k.x = split.hi, k.x_lo = split.lo;
  } else if (dw) {
    operand(&copies, &k.x, tokens, dim, ws);
  }
  ws += 2 * padded(tokens, dim);
  if (dx) operand(&copies, &k.wg, ffn, dim, ws);
  ws += padded(ffn, dim);
  if (dx) operand(&copies, &k.wu, ffn, dim, ws);
  if (e == cudaSuccess) e = launch_copy_bf16(copies, s);
  if (e != cudaSuccess) return cuda_fail(e, "cr_glu_backward: operands");
  k.dx = mat(tokens ? dx : nullptr, lddx);
  k.dwg = ffn ? dwg : nullptr;
  k.dwu = ffn ? dwu : nullptr;
  k.tokens = (uint32_t)tokens, k.dim = (uint32_t)dim, k.ffn = (uint32_t)ffn;
  return launched(launch_glu_back(dw_dtype, k, s), "cr_glu_backward");
}

cr_status cr_ffn_call(cr_ffn_op op, const void* words) {
  if (!words) return fail(CR_ERR_INVALID_ARG, "words is NULL");
  const uint64_t* w = static_cast<const uint64_t*>(words);
  const auto in = [&](int i) { return reinterpret_cast<const void*>(w[i]); };
  const auto out = [&](int i) { return reinterpret_cast<void*>(w[i]); };
  const auto q = [&](int i) { return reinterpret_cast<const cr_q8*>(w[i]); };
  const auto type = [&](int i) { return (cr_dtype)w[i]; };
  const auto act = [&](int i) { return (cr_act)w[i]; };
  const auto stream = [&](int i) { return reinterpret_cast<cr_stream_t>(w[i]); };
  switch (op) {
    case CR_CALL_Q8_STORE: return cr_q8_store(in(0), w[1], w[2], w[3], type(4), q(5), stream(6));
    case CR_CALL_Q8_LOAD: return cr_q8_load(q(0), w[1], w[2], out(3), w[4], type(5), stream(6));
    case CR_CALL_RMS_NORM: {
      double eps;
      memcpy(&eps, &w[8], sizeof(eps));
      return cr_rms_norm(in(0), w[1], in(2), w[3], in(4), w[5], w[6], type(7), eps, out(9), w[10],
                         out(11), w[12], q(13), static_cast<float*>(out(14)), stream(15));
    }
    case CR_CALL_RMS_NORM_BACKWARD:
      return cr_rms_norm_backward(in(0), w[1], in(2), w[3], q(4), in(5),
                                  static_cast<const float*>(in(6)), in(7), w[8], w[9], w[10],
                                  type(11), out(12), w[13], out(14), type(15), out(16), w[17],
                                  stream(18));
    case CR_CALL_GLU:
      return cr_glu(in(0), w[1], in(2), w[3], in(4), w[5], w[6], w[7], w[8], type(9), act(10),
                    out(11), w[12], q(13), q(14), out(15), w[16], stream(17));
    case CR_CALL_GLU_ACT_BACKWARD:
      return cr_glu_act_backward(in(0), w[1], q(2), q(3), w[4], w[5], type(6), act(7), out(8), w[9],
                                 out(10), w[11], out(12), w[13], stream(14));
    case CR_CALL_GLU_BACKWARD:
      return cr_glu_backward(in(0), w[1], q(2), q(3), in(4), w[5], q(6), in(7), w[8], in(9), w[10],
                             w[11], w[12], w[13], type(14), act(15), out(16), w[17], out(18),
                             out(19), type(20), out(21), w[22], out(23), w[24], stream(25));
  }
  return fail(CR_ERR_INVALID_ARG, "unknown call %d", (int)op);
}

long long cr_glu_wait_word(int clear) {
  unsigned int word = 0;
  const cudaError_t e = glu_wait_word(clear != 0, &word);
  if (e != cudaSuccess) {
    cuda_fail(e, "cr_glu_wait_word");
    return -2;
  }
  return (long long)word;
}

}  // extern "C"
