// api_matrix.h -- host-side checks of matrix arguments, shared by the entry
// points of include/cr_ffn.h and include/cr_lm.h (api_ffn.cu, api_lm.cu).
#pragma once

#include "api_host.h"
#include "ffn_internal.cuh"

namespace cr {
namespace host {

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

inline bool never(const char*, const char*) { return false; }
inline bool is(const char* a, const char* b) { return strcmp(a, b) == 0; }

inline Mat mat(const void* p, uint64_t ld) { return Mat{const_cast<void*>(p), p ? ld : 0}; }

inline Q8 q8_of(const cr_q8* q) {
  if (!q) return Q8{nullptr, 0, nullptr, 0};
  return Q8{static_cast<uint8_t*>(q->codes), q->ld, q->scales, q->lds};
}

inline cudaStream_t stream_of(cr_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

inline cr_status launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? ok() : cuda_fail(e, what);
}

inline cr_status check_float(cr_dtype d, const char* what) {
  if (esize_of(d) == 0) return fail(CR_ERR_INVALID_ARG, "%s: unknown dtype %d", what, (int)d);
  if (!is_float(d)) return fail(CR_ERR_UNSUPPORTED, "%s must be CR_F32 or CR_BF16", what);
  return CR_OK;
}

inline cr_status check_size(uint64_t n, const char* what) {
  if (n >= (1ull << 31))
    return fail(CR_ERR_UNSUPPORTED, "%s=%llu is 2^31 or more", what, (unsigned long long)n);
  return CR_OK;
}

inline cr_status check_workspace(const void* p, size_t have, size_t need) {
  if (need == 0) return CR_OK;
  if (!p) return fail(CR_ERR_INVALID_ARG, "workspace is NULL, %zu bytes needed", need);
  if (have < need)
    return fail(CR_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", have, need);
  if (!aligned(p, 16)) return fail(CR_ERR_ALIGNMENT, "workspace=%p not aligned to 16 bytes", p);
  return CR_OK;
}

}  // namespace host
}  // namespace cr
