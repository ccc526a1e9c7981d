// k_logp_back.cu -- the gradient of log probabilities, entropies and log-sum-exps with
// respect to the logits.
//
// One pass: a logit is read, its probability made from the row's log-sum-exp with
// one exponential, and its gradient written (in place of it, where that is wanted).  A warp
// takes a chunk of a row (ffn_internal.cuh; bf16 rows off the vector grid in spans,
// span.cuh).
//
// Measured: 8192 x 32000 bf16 (1.05 GB) 149.5 us a call in a loop, 7.0 TB/s; with the entropy's gradient
// 161; 8192 x 31999, in spans, 194.  Two chunks a warp, which share the row's numbers, at five blocks an SM:
// one chunk 183, four blocks 158.
#include <type_traits>

#include "lm_internal.cuh"
#include "pdl.cuh"

namespace cr {

namespace {

constexpr int kAhead = 2;  // chunks of a warp in flight

// An lse at or below this has no token left: nothing of the row's logits is known better than that.
constexpr float kNoToken = -1.2676506e30f;  // -2^100

// A row's numbers: gradient of column v = p (by - ent log(p)), and `hit` more at the target.
struct RowTerms {
  float lse, by, ent, hit;
  int32_t target;
};

template <bool ENT>
__device__ __forceinline__ RowTerms row_terms(const LogProbBackArgs& a, uint64_t row) {
  RowTerms r;
  r.lse = a.lse[row];
  r.target = a.dlogp ? token_id(a.targets, row, a.vocab) : -1;
  const float dlogp = r.target >= 0 ? a.dlogp[row] : 0.0f, dlse = a.dlse ? a.dlse[row] : 0.0f;
  r.by = dlse - dlogp;
  r.ent = 0.0f;
  if constexpr (ENT) {
    r.ent = a.dentropy[row];
    r.by -= r.ent * a.entropy[row];
  }
  r.by *= a.scale, r.ent *= a.scale, r.hit = a.scale * dlogp;
  if (r.lse <= kNoToken) {
    r.lse = __builtin_huge_valf();  // p = 0
    r.target = -1;
  }
  return r;
}

template <bool ENT>
__device__ __forceinline__ float gradient(float x, float scale, const RowTerms& r) {
  const float log_p = fmaf(x, scale, -r.lse), p = fast_exp2(log_p * kLog2E);
  if constexpr (!ENT) return p * r.by;
  return p * fmaf(-r.ent, fmaxf(log_p, -1e30f), r.by);  // 0 times -infinity is 0 here
}

// A warp takes kAhead chunks of a row, next to each other, so that the row's numbers are read once.
template <int DT, int MODE, bool ENT>
__global__ void __launch_bounds__(kBlock, 5) k_logp_back(const __grid_constant__ LogProbBackArgs a,
                                                      const __grid_constant__ ChunkRange r) {
  constexpr int vals = place_vals(MODE);
  constexpr uint32_t cols = place_cols(MODE);
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const uint64_t stride = (uint64_t)gridDim.x * (kBlock / 32);
  for (uint64_t k = (uint64_t)blockIdx.x * (kBlock / 32) + (threadIdx.x >> 5); k < r.chunks;
       k += stride) {
    const uint64_t row = fastdiv_div(r.per_row, k);
    const uint32_t base = (uint32_t)(k - row * r.per_row.d) * kAhead * cols;
    const char* from = row_at<DT>(a.logits, row);
    char* out = row_at<DT>(a.dlogits, row);
    Loaded<DT, MODE> in[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      in[j].load(from, Place<MODE>(base + j * cols, a.vocab, lane, out));
    const RowTerms terms = row_terms<ENT>(a, row);
    const uint32_t near = (uint32_t)terms.target - base + 7;  // spans lead by up to 7 columns
    const bool hit = terms.target >= 0 && near < kAhead * cols + 7;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const Place<MODE> at(base + j * cols, a.vocab, lane, out);
      float v[vals];
      in[j].ready();
#pragma unroll
      for (int i = 0; i < vals; ++i) v[i] = gradient<ENT>(in[j].value(i), a.scale, terms);
      if (hit) {
        int64_t first = base + j * cols + (MODE == 0 ? lane : lane * vals);
        if constexpr (MODE == kSpan) first = at.span.first;
        const int64_t d = terms.target - first;
#pragma unroll
        for (int i = 0; i < vals; ++i)
          if (d == (MODE == 0 ? 32 * i : i)) v[i] += terms.hit;
      }
      st_place<DT, MODE>(out, at, v);
    }
  }
}

template <int DT, int MODE>
cudaError_t run(const LogProbBackArgs& a, cudaStream_t s) {
  const uint64_t per_row = (place_chunks(a.vocab, MODE) + kAhead - 1) / kAhead;
  const ChunkRange r = {a.rows * per_row, fastdiv_make(per_row, a.rows * per_row)};
  return launch_pdl(a.dentropy ? k_logp_back<DT, MODE, true> : k_logp_back<DT, MODE, false>,
                    chunk_grid(r, 1), kBlock, s, a, r);
}

}  // namespace

cudaError_t launch_log_probs_back(cr_dtype d, const LogProbBackArgs& a, int vec, cudaStream_t s) {
  if (d == CR_BF16)
    return vec == 2 ? run<CR_BF16, 2>(a, s) : vec == 1 ? run<CR_BF16, 1>(a, s) : run<CR_BF16, kSpan>(a, s);
  return vec == 2 ? run<CR_F32, 2>(a, s) : vec == 1 ? run<CR_F32, 1>(a, s) : run<CR_F32, 0>(a, s);
}

}  // namespace cr
