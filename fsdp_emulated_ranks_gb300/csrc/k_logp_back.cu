// k_logp_back.cu -- the gradient of log probabilities, entropies and log-sum-exps with
// respect to the logits.
//
// One pass: a logit is read, its probability made from the row's log-sum-exp with
// one exponential, and its gradient written (in place of it, where that is wanted).  A warp
// takes a chunk of a row (ffn_internal.cuh; bf16 rows off the vector grid in spans,
// span.cuh).
//
// exp(z - lse) is off by the rounding of the stored lse: by a factor as large as the number of tokens in a row
// filled with -1e9, whose lse is -1e9.  Rows of a large lse are therefore left to blocks of their own, which read a row
// twice: for its maximum and sum, and to write
//     p = exp(scale (x - max)) / sum.
// A block takes the whole row, so that dlogits may be logits there too.
//
// Measured: 8192 x 32000 bf16 (1.05 GB) 150 us a call in a loop, 7.0 TB/s; with the entropy's gradient
// 159; 8192 x 31999, in spans, 198.  Two chunks a warp, which share the row's numbers, at five blocks an SM:
// one chunk 183, four blocks 158.  One row in 32 of a large lse: 154; every row: 500.
#include <algorithm>

#include "lm_internal.cuh"
#include "pdl.cuh"

namespace cr {

namespace {

constexpr int kAhead = 2;  // chunks of a warp in flight

// An lse at or below this has no token left: nothing of the row's logits is known better than that.
constexpr float kNoToken = -1.2676506e30f;  // -2^100

// Rows of such an lse go by their own maximum and sum.  Below it half a step of lse is at most 2^-17, the share
// by which p is off: a few roundings of log(p) next to bf16's 2^-9.  Infinity (a product with the
// scale past the type's end) is one, NaN is none.
constexpr float kFarLse = 256.0f;
__device__ __forceinline__ bool is_far(float lse) { return fabsf(lse) >= kFarLse && lse > kNoToken; }

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
    r.lse = __builtin_huge_valf();  // p = 0, of factors that may not be finite (a z-loss's dlse is -infinity there)
    r.by = r.ent = r.hit = 0.0f;
    r.target = -1;
  }
  return r;
}

// exp of this and of all below is 0 (2^-126 is exp(-87.3)), and so has to be its product with log(p), which
// stays finite from here up.
constexpr float kLeastLog = -100.0f;

template <bool ENT>
__device__ __forceinline__ float gradient(float x, float scale, const RowTerms& r) {
  const float log_p = fmaf(x, scale, -r.lse), p = fast_exp2(log_p * kLog2E);
  if constexpr (!ENT) return p * r.by;
  return p * fmaf(-r.ent, fmaxf(log_p, kLeastLog), r.by);
}

// The column of a lane's value 0; value i's is i further, or 32 i where lanes have single values.
template <int MODE>
__device__ __forceinline__ int64_t first_col(const Place<MODE>& at) {
  if constexpr (MODE == kSpan) return at.span.first;
  return (int64_t)at.base + (MODE == 0 ? at.lane : at.lane * place_vals(MODE));
}
template <int MODE>
constexpr int kColStep = MODE == 0 ? 32 : 1;

// v[i] += hit for the target's column, if it is among them.
template <int MODE>
__device__ __forceinline__ void add_hit(const Place<MODE>& at, const RowTerms& r, float* v) {
  const int64_t d = r.target - first_col(at);
#pragma unroll
  for (int i = 0; i < place_vals(MODE); ++i)
    if (d == i * kColStep<MODE>) v[i] += r.hit;
}

// A row of a large lse, by a block.  `part`: a maximum and a sum a warp, in shared memory.
template <int DT, int MODE, bool ENT>
__device__ __forceinline__ void far_row(const LogProbBackArgs& a, uint64_t row, float2* part) {
  constexpr int vals = place_vals(MODE), warps = kBlock / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const char* from = row_at<DT>(a.logits, row);
  char* out = row_at<DT>(a.dlogits, row);
  const float c = a.scale * kLog2E;
  const uint32_t end = a.vocab + (MODE == kSpan ? 7 : 0);  // spans lead by up to 7 columns
  float most = -__builtin_huge_valf(), sum = 0.0f;  // of 2^((x - most) c)
  // What is subtracted of a logit, and the sum with another reference: -infinity less itself is not to be formed.
  const auto reference = [](float m) { return m == -__builtin_huge_valf() ? 0.0f : m; };
  const auto moved = [&](float s, float m, float to) { return s * fast_exp2((m - reference(to)) * c); };
#pragma unroll 1
  for (uint32_t base = warp * place_cols(MODE); base < end; base += warps * place_cols(MODE)) {
    const Place<MODE> at(base, a.vocab, lane, out);
    Loaded<DT, MODE> in;
    in.load(from, at);
    in.ready();
    const int64_t first = first_col(at);
    const auto held = [&](int i) { return (uint64_t)(first + i * kColStep<MODE>) < a.vocab; };
    float m = most;
#pragma unroll
    for (int i = 0; i < vals; ++i)
      if (held(i)) m = fmaxf(m, in.value(i));
    sum = moved(sum, most, m);
    most = m;
#pragma unroll
    for (int i = 0; i < vals; ++i)
      if (held(i)) sum += fast_exp2((in.value(i) - reference(most)) * c);
  }
  float m = most;
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  sum = moved(sum, most, m);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  if (lane == 0) part[warp] = make_float2(m, sum);
  __syncthreads();
  most = part[0].x;
#pragma unroll
  for (int w = 1; w < warps; ++w) most = fmaxf(most, part[w].x);
  sum = 0.0f;
#pragma unroll
  for (int w = 0; w < warps; ++w) sum += moved(part[w].y, part[w].x, most);
  RowTerms terms = row_terms<ENT>(a, row);
  terms.lse = kLn2 * log2f(sum);  // of the logits less their maximum
#pragma unroll 1
  for (uint32_t base = warp * place_cols(MODE); base < end; base += warps * place_cols(MODE)) {
    const Place<MODE> at(base, a.vocab, lane, out);
    Loaded<DT, MODE> in;
    in.load(from, at);
    in.ready();
    float v[vals];
#pragma unroll
    for (int i = 0; i < vals; ++i) v[i] = gradient<ENT>(in.value(i) - reference(most), a.scale, terms);
    if (terms.target >= 0) add_hit(at, terms, v);
    st_place<DT, MODE>(out, at, v);
  }
  __syncthreads();  // `part` has been read
}

// The rows of a large lse, by the first `blocks` blocks of the grid: a thread looks at a row.
template <int DT, int MODE, bool ENT>
__device__ __forceinline__ void far_rows(const LogProbBackArgs& a, uint32_t blocks) {
  __shared__ uint32_t found[kBlock / 32];
  __shared__ float2 part[kBlock / 32];
#pragma unroll 1
  for (uint64_t first = blockIdx.x; first < a.rows; first += (uint64_t)blocks * kBlock) {
    const uint64_t mine = first + (uint64_t)threadIdx.x * blocks;
    const uint32_t any = __ballot_sync(~0u, mine < a.rows && is_far(a.lse[mine]));
    if (threadIdx.x % 32 == 0) found[threadIdx.x / 32] = any;
    __syncthreads();
#pragma unroll 1
    for (uint32_t w = 0; w < kBlock / 32; ++w)
#pragma unroll 1
      for (uint32_t left = found[w]; left; left &= left - 1)
        far_row<DT, MODE, ENT>(a, first + (uint64_t)(32 * w + __ffs(left) - 1) * blocks, part);
    __syncthreads();
  }
}

// A warp takes kAhead chunks of a row, next to each other, so that the row's numbers are read once.
template <int DT, int MODE, bool ENT>
__global__ void __launch_bounds__(kBlock, 5) k_logp_back(const __grid_constant__ LogProbBackArgs a,
                                                      const __grid_constant__ ChunkRange r, uint32_t far) {
  constexpr int vals = place_vals(MODE);
  constexpr uint32_t cols = place_cols(MODE);
  pdl_enter();
  if (blockIdx.x < far) return far_rows<DT, MODE, ENT>(a, far);
  const int lane = threadIdx.x & 31;
  const uint64_t stride = (uint64_t)(gridDim.x - far) * (kBlock / 32);
  for (uint64_t k = (uint64_t)(blockIdx.x - far) * (kBlock / 32) + (threadIdx.x >> 5); k < r.chunks;
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
    const bool far_off = is_far(a.lse[row]);  // another block's
    const uint32_t near = (uint32_t)terms.target - base + 7;  // spans lead by up to 7 columns
    const bool hit = terms.target >= 0 && near < kAhead * cols + 7;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const Place<MODE> at(base + j * cols, a.vocab, lane, out);
      float v[vals];
      in[j].ready();
#pragma unroll
      for (int i = 0; i < vals; ++i) v[i] = gradient<ENT>(in[j].value(i), a.scale, terms);
      if (hit) add_hit(at, terms, v);
      if (!far_off) st_place<DT, MODE>(out, at, v);
    }
  }
}

template <int DT, int MODE>
cudaError_t run(const LogProbBackArgs& a, cudaStream_t s) {
  const uint64_t per_row = (place_chunks(a.vocab, MODE) + kAhead - 1) / kAhead;
  const ChunkRange r = {a.rows * per_row, fastdiv_make(per_row, a.rows * per_row)};
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  // Blocks for rows of a large lse: two an SM at most (they end at once where there are none), an odd number so that
  // such rows at even distances spread over them.
  const uint32_t far = (uint32_t)std::min<uint64_t>(a.rows, 2 * (uint64_t)sms + 1);
  dim3 grid = chunk_grid(r, 1);
  grid.x += far;
  return launch_pdl(a.dentropy ? k_logp_back<DT, MODE, true> : k_logp_back<DT, MODE, false>, grid, kBlock, s,
                    a, r, far);
}

}  // namespace

cudaError_t launch_log_probs_back(cr_dtype d, const LogProbBackArgs& a, int vec, cudaStream_t s) {
  if (d == CR_BF16)
    return vec == 2 ? run<CR_BF16, 2>(a, s) : vec == 1 ? run<CR_BF16, 1>(a, s) : run<CR_BF16, kSpan>(a, s);
  return vec == 2 ? run<CR_F32, 2>(a, s) : vec == 1 ? run<CR_F32, 1>(a, s) : run<CR_F32, 0>(a, s);
}

}  // namespace cr
