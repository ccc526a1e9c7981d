// lm_internal.cuh -- types and device helpers shared by the language model
// operators (include/cr_lm.h).
#pragma once

#include "cr_lm.h"
#include "ffn_internal.cuh"
#include "span.cuh"

namespace cr {

// Token ids of 32 or 64 bits.
struct Ids {
  const void* p;
  int bits;
};

struct EmbedArgs {
  Mat table, out;
  Ids ids;
  uint64_t tokens;
  uint32_t vocab, dim;
  float scale;
};

struct EmbedBackArgs {
  Mat dout, base, dtable;
  Ids ids;
  uint64_t tokens;
  uint32_t vocab, dim;
  float scale;
  bool in_place;  // base is dtable: rows without tokens stay as they are
};

struct DropoutArgs {
  Mat x, residual, out;
  const uint64_t* rng;
  uint64_t call;
  uint64_t rows;
  uint32_t cols;
  uint32_t first_row;
  uint32_t limit;  // of 65536
  float by;        // what kept values are multiplied by
};

struct LogProbArgs {
  Mat logits;
  Ids targets;
  uint64_t rows;
  uint32_t vocab;
  float scale;
  float *logp, *entropy, *lse;
  int top;
  int32_t* top_ids;
  float* top_logp;
};

struct LogProbBackArgs {
  Mat logits, dlogits;
  Ids targets;
  uint64_t rows;
  uint32_t vocab;
  float scale;
  const float *lse, *entropy, *dlogp, *dentropy, *dlse;
};

// vec: the accesses every pointer and row stride of the call allows, 0 to 2.
cudaError_t launch_embed(cr_dtype d, cr_dtype out, const EmbedArgs& a, int vec, cudaStream_t s);
constexpr uint64_t kEmbedVocab = 1ull << 21;  // largest vocabulary of the backward pass
uint64_t embed_back_workspace(uint64_t tokens, uint64_t vocab, uint64_t dim);
cudaError_t launch_embed_back(cr_dtype d, cr_dtype out, const EmbedBackArgs& a, void* workspace,
                              int vec, cudaStream_t s);
cudaError_t launch_dropout(cr_dtype d, const DropoutArgs& a, int vec, cudaStream_t s);
cudaError_t launch_log_probs(cr_dtype d, const LogProbArgs& a, cudaStream_t s);
cudaError_t launch_log_probs_back(cr_dtype d, const LogProbBackArgs& a, int vec, cudaStream_t s);

#if defined(__CUDACC__)

// Id k, or -1 where it is outside [0, vocab).
__device__ __forceinline__ int32_t token_id(const Ids& ids, uint64_t k, uint32_t vocab) {
  const int64_t v = ids.bits == 64 ? static_cast<const int64_t*>(ids.p)[k]
                                   : (int64_t)static_cast<const int32_t*>(ids.p)[k];
  return (uint64_t)v < vocab ? (int32_t)v : -1;
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// How a warp's lanes share a chunk of a row.
//   0 to 2  ffn_internal.cuh's chunks: single values, 16- and 32-byte vectors
//   3       spans (span.cuh): bf16 rows off the vector grid, led by the output
constexpr int kSpan = 3;
__host__ __device__ constexpr int place_vals(int mode) { return mode == kSpan ? 8 : lane_vals(mode); }
__host__ __device__ constexpr uint32_t place_cols(int mode) { return 32 * place_vals(mode); }
inline uint32_t place_chunks(uint32_t cols, int mode) {
  const uint32_t lead = mode == kSpan ? 7 : 0;
  return (uint32_t)(((uint64_t)cols + lead + place_cols(mode) - 1) / place_cols(mode));
}

// A lane's columns of chunk `base` of a row, whose output row is `out`.
template <int MODE>
struct Place {
  uint32_t base, cols;
  int lane;
  Span8 span;

  __device__ __forceinline__ Place(uint32_t b, uint32_t c, int l, const void* out)
      : base(b), cols(c), lane(l) {
    if constexpr (MODE == kSpan) span = span8((int64_t)b + 8 * l - lead_of<2>(out), c);
  }
};

// Those columns of a row, as loaded.
template <int DT, int MODE>
struct Loaded {
  Raw<DT, MODE> raw;
  __device__ __forceinline__ void load(const void* row, const Place<MODE>& p) {
    raw.load(row, p.base, p.cols, p.lane);
  }
  __device__ __forceinline__ void ready() {}
  __device__ __forceinline__ float value(int i) const { return raw.value(i); }
};

template <int DT>
struct Loaded<DT, kSpan> {
  static_assert(DT == CR_BF16, "spans are bf16's");
  Granules<16> g;
  __device__ __forceinline__ void load(const void* row, const Place<kSpan>& p) { g.load(row, p.span); }
  __device__ __forceinline__ void ready() { g.align(); }
  __device__ __forceinline__ float value(int i) const {
    return __uint_as_float(i & 1 ? g.w[i / 2] & 0xffff0000u : g.w[i / 2] << 16);
  }
};

template <int DT, int MODE>
__device__ __forceinline__ void st_place(void* row, const Place<MODE>& p, const float* v) {
  if constexpr (MODE == kSpan) {
    if (p.span.hi > p.span.lo) st_span<DT>(row, p.span, v);
  } else {
    st_chunk<DT, MODE>(row, p.base, p.cols, p.lane, v);
  }
}

#endif  // __CUDACC__

}  // namespace cr
