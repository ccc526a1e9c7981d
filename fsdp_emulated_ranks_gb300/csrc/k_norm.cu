// k_norm.cu -- RMS norm with the residual's addition and an 8-bit output,
// and its backward pass.
//
// Forward, per row of h = x + residual:  v = h * rstd * weight with
// rstd = 1/sqrt(mean h^2 + eps).  A row is held in registers between its one
// read and its writes, a chunk a warp, the sum of squares reduced by shuffles
// and, across the row's warps, through shared memory.  Rows too wide for that
// are read twice; the second read comes from L2.
//
// Backward, per row with n = h * rstd and c = mean(dy * weight * n):
// dx = rstd * (dy * weight - n * c) + dres.  dweight sums dy * n down the
// columns: a block keeps the sums of its columns in registers over all the
// rows it takes (persistent grid) and writes one partial row; a second
// kernel adds the partials in order.  Wide rows take a second pass over dy
// and h for dweight.
//
// Measured, bf16, a call in a loop: the forward pass of 8192 x 2048 with residual,
// sum, y and 8-bit y (151 MB) 26.4 us, 5.7 TB/s (a copy that moves as many
// bytes takes 29.6 in such a loop); the backward pass (134 MB) 28.3, of which 24
// in the rows (5.6 TB/s, bound by latency: 117 registers, 16 warps an SM; at 80
// registers it spills and takes 41) and 4 in the partials.  fp32, 4096 x 2048:
// 23.4 us forward, 6.1 TB/s, and 28.4 backward.  Rows above kWideFrom columns are
// read twice: 2048 x 16384 bf16 63.4 us forward, 4.8 TB/s of what has to be
// moved, and 106 backward, 2.5 TB/s, where dweight takes a pass of its own.
//
// Rows off the vector grid (an odd width or address) come to shared memory as
// the aligned 16-byte granules that hold them, a row ahead of the one at work,
// and are read there value by value.
#include <algorithm>
#include <map>
#include <mutex>
#include <tuple>

#include "ffn_internal.cuh"
#include "pdl.cuh"

namespace cr {

namespace {

constexpr int kWideThreads = 1024;      // threads of a block on a wide row
constexpr uint32_t kWideFrom = 8192;    // columns above which a row is wide
constexpr uint32_t kBackParts = 912;    // partial rows of dweight, at most
constexpr uint32_t kWideParts = 64;
constexpr int kMaxWarps = kWideThreads / 32;
constexpr uint32_t kSpanFrom = 256;     // columns above which a row off the vector grid is staged

// Sum over the row's warps (blockDim.x / 32 of them, row threadIdx.y of the
// block).  `buf` alternates between two halves of `part`, so one barrier a
// call is enough.  APART: the barrier is the row's own, so that the rows of a
// block do not wait for each other.  That helps the backward pass (8000 x 1025:
// 30.0 -> 27.0 us) and not the forward pass (35.2 -> 37.2), which takes the
// block's.
template <bool APART>
__device__ __forceinline__ float row_sum(float s, float (*part)[kMaxWarps], int buf) {
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return s;
  float* p = part[buf];
  const int w0 = threadIdx.y * nw;
  if ((threadIdx.x & 31) == 0) p[w0 + (threadIdx.x >> 5)] = s;
  if constexpr (APART)
    asm volatile("bar.sync %0, %1;" ::"r"(threadIdx.y + 1), "r"(blockDim.x) : "memory");
  else
    __syncthreads();
  if (nw <= 4) {
    s = 0.0f;
    for (int w = 0; w < nw; ++w) s += p[w0 + w];
    return s;
  }
  const int lane = threadIdx.x & 31;
  s = lane < nw ? p[w0 + lane] : 0.0f;
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
  return s;
}

template <int DT>
__device__ __forceinline__ const void* row_of(const Mat& m, uint64_t row) {
  return static_cast<const char*>(m.p) + row * m.ld * (DT == CR_BF16 ? 2 : 4);
}

template <int DT>
__device__ __forceinline__ void* row_of_out(const Mat& m, uint64_t row) {
  return static_cast<char*>(m.p) + row * m.ld * (DT == CR_BF16 ? 2 : 4);
}

// x and residual of a row's chunk.
template <int DT, int VEC>
struct NormIn {
  Raw<DT, VEC> x, r;

  __device__ __forceinline__ void load(const NormArgs& a, uint64_t row, uint32_t base, int lane) {
    x.load(row_of<DT>(a.x, row), base, a.cols, lane);
    if (a.residual.p)
      r.load(row_of<DT>(a.residual, row), base, a.cols, lane);
    else
      r.clear();
  }
  __device__ __forceinline__ void clear() { x.clear(), r.clear(); }
  __device__ __forceinline__ void values(float* h) const {
#pragma unroll
    for (int i = 0; i < lane_vals(VEC); ++i) h[i] = x.value(i) + r.value(i);
  }
};

template <int DT, int VEC>
__device__ __forceinline__ void norm_st(const NormArgs& a, uint64_t row, uint32_t base, int lane,
                                        float* h, const Raw<DT, VEC>& w, float rstd) {
  if (a.sum.p) st_chunk<DT, VEC>(row_of_out<DT>(a.sum, row), base, a.cols, lane, h);
#pragma unroll
  for (int i = 0; i < lane_vals(VEC); ++i) h[i] = h[i] * rstd * w.value(i);
  if (a.y.p) st_chunk<DT, VEC>(row_of_out<DT>(a.y, row), base, a.cols, lane, h);
  if (a.y8.codes) st_chunk_q8<VEC>(a.y8, row, base, a.cols, lane, h);
}

// Threads of a block that holds rows in registers, at most: a chunk a warp up
// to kWideFrom columns; off the vector grid, 8 rows of a chunk.
constexpr int row_threads(int vec) {
  return vec ? (int)(kWideFrom / chunk_cols(vec)) * 32 : 256;
}

// Block (32 * warps per row, rows per block), persistent.  The next row is
// loaded while this one is reduced and written.
template <int DT, int VEC>
__global__ void __launch_bounds__(row_threads(VEC)) __maxnreg__(VEC ? 128 : 64) k_rms_norm(const __grid_constant__ NormArgs a) {
  pdl_enter();
  __shared__ float part[2][kMaxWarps];
  const int lane = threadIdx.x & 31;
  const uint32_t base = (threadIdx.x >> 5) * chunk_cols(VEC);
  const uint64_t step = (uint64_t)gridDim.x * blockDim.y;
  NormIn<DT, VEC> in;
  Raw<DT, VEC> w;
  const auto load = [&](uint64_t row) {
    if (row < a.rows)
      in.load(a, row, base, lane);
    else
      in.clear();
  };
  load((uint64_t)blockIdx.x * blockDim.y + threadIdx.y);
  w.load(a.weight, base, a.cols, lane);
  int buf = 0;
  // every row of a block's turn takes part in the barriers
  for (uint64_t first = (uint64_t)blockIdx.x * blockDim.y; first < a.rows; first += step, buf ^= 1) {
    const uint64_t row = first + threadIdx.y;
    float h[lane_vals(VEC)], s = 0.0f;
    in.values(h);
#pragma unroll
    for (int i = 0; i < lane_vals(VEC); ++i) s = fmaf(h[i], h[i], s);
    load(row + step);
    const float rstd = rsqrtf(fmaf(row_sum<false>(s, part, buf), a.inv_cols, a.eps));
    if (row >= a.rows) continue;
    norm_st<DT, VEC>(a, row, base, lane, h, w, rstd);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
  }
}

// ---- rows off the vector grid --------------------------------------------------------
//
// Staged, the loads need neither registers nor a check a value, and a lane has
// 16 values, over which the sums' shuffles and the codes' scales spread (40
// instructions a value forward; 57 with 8 values from global memory, whose loads
// ahead filled the registers).  Bound by instructions: 53 % of the issue slots,
// at 24 to 36 warps an SM.  Measured against loads of single values:
// bf16 2700 x 6001 with residual, sum, y and 8-bit y, which is read back after
// it, 49 us (80; 37 of the 49 in the norm), backward 36 (55); 4000 x 4097 50
// (66), backward 33 (46); fp32 1777 x 4099 21.9 (24.5).  At
// up to kSpanFrom columns, where a warp holds a row, single values are as fast:
// 20000 x 129 17.0 us against 18.1, 77 columns 14.8 against 16.5.

// The aligned 16-byte granules that hold `bytes` bytes at `src`, copied to
// `dst` by threads t of n.  Each granule holds at least one of the bytes, so no
// load leaves the memory they lie in.
__device__ __forceinline__ void span_copy(char* dst, const void* src, uint32_t bytes, int t, int n) {
  const uint32_t lead = (uint32_t)(uintptr_t)src & 15;
  const char* from = static_cast<const char*>(src) - lead;
  const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
  for (uint32_t o = t * 16; o < lead + bytes; o += n * 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + o), "l"(from + o) : "memory");
}

// The span's first byte.
__device__ __forceinline__ const char* span_at(const char* dst, const void* src) {
  return dst + ((uint32_t)(uintptr_t)src & 15);
}

constexpr uint32_t span_bytes(uint32_t bytes) { return (bytes + 15 + 15) & ~15u; }

__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The barrier of row threadIdx.y of the block.
__device__ __forceinline__ void row_sync() {
  if (blockDim.x == 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(threadIdx.y + 1), "r"(blockDim.x) : "memory");
}

constexpr int kSpanVals = 16;                   // values of a lane: columns l, l + 32, ...
constexpr uint32_t kSpanCols = 32 * kSpanVals;  // columns of a warp
constexpr int kSpanThreads = (int)(kWideFrom / kSpanCols) * 32;
// Shared memory of a block, at most: two stages of dy, h and dres and the
// weights of one wide fp32 row.
constexpr int kSpanSmem = 7 * (int)span_bytes(kWideFrom * 4);
static_assert(kSpanSmem + 2 * kMaxWarps * 4 <= 227 << 10);

// Value c of a row at any address.
template <int DT>
__device__ __forceinline__ float value_at(const char* p, uint32_t c) {
  if constexpr (DT == CR_BF16)
    return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[c] << 16);
  else
    return reinterpret_cast<const float*>(p)[c];
}

template <int DT>
__device__ __forceinline__ void value_to(char* p, uint32_t c, float v) {
  if constexpr (DT == CR_BF16)
    reinterpret_cast<uint16_t*>(p)[c] = (uint16_t)ffn_bf16x2(v, 0.0f);
  else
    reinterpret_cast<float*>(p)[c] = v;
}

template <int DT, bool FULL>
__device__ __forceinline__ void span_values(const char* p, uint32_t c0, uint32_t cols, float* v) {
#pragma unroll
  for (int i = 0; i < kSpanVals; ++i)
    v[i] = FULL || c0 + 32 * i < cols ? value_at<DT>(p, c0 + 32 * i) : 0.0f;
}

template <int DT, bool FULL>
__device__ __forceinline__ void span_st(const Mat& m, uint64_t row, uint32_t c0, uint32_t cols, const float* v) {
  char* const p = static_cast<char*>(row_of_out<DT>(m, row));
#pragma unroll
  for (int i = 0; i < kSpanVals; ++i)
    if (FULL || c0 + 32 * i < cols) value_to<DT>(p, c0 + 32 * i, v[i]);
}

// h of a row in shared memory, and its sum of squares.
template <int DT, bool FULL>
__device__ __forceinline__ float span_in(const NormArgs& a, const char* x, const char* res,
                                         uint32_t c0, float* h) {
  span_values<DT, FULL>(x, c0, a.cols, h);
  if (a.residual.p) {
    float r[kSpanVals];
    span_values<DT, FULL>(res, c0, a.cols, r);
#pragma unroll
    for (int i = 0; i < kSpanVals; ++i) h[i] += r[i];
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kSpanVals; ++i) s = fmaf(h[i], h[i], s);
  return s;
}

template <int DT, bool FULL>
__device__ __forceinline__ void span_out(const NormArgs& a, uint64_t row, uint32_t base, int lane,
                                         const char* weight, float rstd, float* h) {
  const uint32_t c0 = base + lane;
  if (a.sum.p) span_st<DT, FULL>(a.sum, row, c0, a.cols, h);
  float w[kSpanVals];
  span_values<DT, FULL>(weight, c0, a.cols, w);
#pragma unroll
  for (int i = 0; i < kSpanVals; ++i) h[i] = h[i] * rstd * w[i];
  if (a.y.p) span_st<DT, FULL>(a.y, row, c0, a.cols, h);
  if (a.y8.codes) st_groups_q8<kSpanVals / 4, FULL>(a.y8, row, base, a.cols, lane, h);
}

// Block (32 * warps per row, rows per block), persistent; each row of the block
// has two stages in shared memory, behind the weights.
template <int DT>
__global__ void __launch_bounds__(kSpanThreads, 2) k_rms_norm_span(const __grid_constant__ NormArgs a) {
  pdl_enter();
  extern __shared__ __align__(16) char smem[];
  __shared__ float part[2][kMaxWarps];
  const int lane = threadIdx.x & 31;
  const uint32_t bytes = a.cols * (DT == CR_BF16 ? 2 : 4), span = span_bytes(bytes);
  const uint32_t stage = span * (a.residual.p ? 2 : 1);
  char* const ring = smem + span + threadIdx.y * 2 * stage;
  const auto copy = [&](uint64_t row, int k) {
    span_copy(ring + k * stage, row_of<DT>(a.x, row), bytes, threadIdx.x, blockDim.x);
    if (a.residual.p)
      span_copy(ring + k * stage + span, row_of<DT>(a.residual, row), bytes, threadIdx.x, blockDim.x);
  };
  const uint64_t step = (uint64_t)gridDim.x * blockDim.y;
  uint64_t row = (uint64_t)blockIdx.x * blockDim.y + threadIdx.y;
  span_copy(smem, a.weight, bytes, threadIdx.y * blockDim.x + threadIdx.x, blockDim.x * blockDim.y);
  if (row < a.rows) copy(row, 0);
  copies_wait();
  __syncthreads();
  const char* const weight = span_at(smem, a.weight);
  const uint32_t base = (threadIdx.x >> 5) * kSpanCols;
  const bool full = base + kSpanCols <= a.cols;
  for (int k = 0; row < a.rows; row += step, k ^= 1) {
    copies_wait();
    row_sync();
    if (row + step < a.rows) copy(row + step, k ^ 1);
    const char* const x = span_at(ring + k * stage, row_of<DT>(a.x, row));
    const char* const res = span_at(ring + k * stage + span, row_of<DT>(a.residual, row));
    float h[kSpanVals];
    const float s = full ? span_in<DT, true>(a, x, res, base + lane, h)
                         : span_in<DT, false>(a, x, res, base + lane, h);
    const float rstd = rsqrtf(fmaf(row_sum<true>(s, part, k), a.inv_cols, a.eps));
    if (full)
      span_out<DT, true>(a, row, base, lane, weight, rstd, h);
    else
      span_out<DT, false>(a, row, base, lane, weight, rstd, h);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
  }
}

// Wide rows, one block each, read twice: the second time from L2.
template <int DT, int VEC>
__global__ void __launch_bounds__(kWideThreads)
    k_rms_norm_wide(const __grid_constant__ NormArgs a) {
  pdl_enter();
  __shared__ float part[2][kMaxWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int buf = 0;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x, buf ^= 1) {
    NormIn<DT, VEC> in;
    float h[lane_vals(VEC)], s = 0.0f;
    for (uint64_t base = (uint64_t)warp * chunk_cols(VEC); base < a.cols; base += (uint64_t)nw * chunk_cols(VEC)) {
      in.load(a, row, (uint32_t)base, lane);
      in.values(h);
#pragma unroll
      for (int i = 0; i < lane_vals(VEC); ++i) s = fmaf(h[i], h[i], s);
    }
    const float rstd = rsqrtf(fmaf(row_sum<false>(s, part, buf), a.inv_cols, a.eps));
    for (uint64_t base = (uint64_t)warp * chunk_cols(VEC); base < a.cols; base += (uint64_t)nw * chunk_cols(VEC)) {
      Raw<DT, VEC> w;
      w.load(a.weight, (uint32_t)base, a.cols, lane);
      in.load(a, row, (uint32_t)base, lane);
      in.values(h);
      norm_st<DT, VEC>(a, row, (uint32_t)base, lane, h, w, rstd);
    }
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
  }
}

// ---- backward -----------------------------------------------------------------------

// h of a chunk, from the matrix or from its 8-bit form.
template <int DT, int VEC, bool HELD8>
struct HeldIn {
  Raw<DT, VEC> r;
  __device__ __forceinline__ void load(const NormBackArgs& a, uint64_t row, uint32_t base, int lane) {
    r.load(row_of<DT>(a.h, row), base, a.cols, lane);
  }
  __device__ __forceinline__ void clear() { r.clear(); }
  __device__ __forceinline__ void values(float* h) const {
#pragma unroll
    for (int i = 0; i < lane_vals(VEC); ++i) h[i] = r.value(i);
  }
};

template <int DT, int VEC>
struct HeldIn<DT, VEC, true> {
  RawQ8<VEC> r;
  __device__ __forceinline__ void load(const NormBackArgs& a, uint64_t row, uint32_t base, int lane) {
    r.load(a.h8, row, base, a.cols, lane);
  }
  __device__ __forceinline__ void clear() { r.clear(); }
  __device__ __forceinline__ void values(float* h) const { r.values(h); }
};

// t = dy * weight, n = h * rstd; res: dres, or zeros.
template <int DT, int VEC>
__device__ __forceinline__ void back_st(const NormBackArgs& a, uint64_t row, uint32_t base,
                                        int lane, const float* t, const float* n,
                                        const Raw<DT, VEC>& res, float rstd, float c) {
  float dx[lane_vals(VEC)];
#pragma unroll
  for (int i = 0; i < lane_vals(VEC); ++i) dx[i] = rstd * (t[i] - n[i] * c) + res.value(i);
  st_chunk<DT, VEC>(row_of_out<DT>(a.dx, row), base, a.cols, lane, dx);
}

// The sums of the block's other rows join the first's, in order; `sums` holds
// VALS x threads of a row.
template <int VALS>
__device__ __forceinline__ void join_rows(float* dw, float* sums) {
  for (unsigned y = 1; y < blockDim.y; ++y) {
    __syncthreads();
    if (threadIdx.y == y) {
#pragma unroll
      for (int i = 0; i < VALS; ++i) sums[i * blockDim.x + threadIdx.x] = dw[i];
    }
    __syncthreads();
    if (threadIdx.y == 0) {
#pragma unroll
      for (int i = 0; i < VALS; ++i) dw[i] += sums[i * blockDim.x + threadIdx.x];
    }
  }
}

// Rows of at most kWideFrom columns: block (32 * warps per row, rows per
// block), persistent; partial row blockIdx.x of dweight, whose sums stay in
// registers.  Everything the next row needs is loaded while this one is
// reduced and written.
template <int DT, int VEC, bool HELD8>
__global__ void __launch_bounds__(row_threads(VEC))
    k_rms_norm_back(const __grid_constant__ NormBackArgs a) {
  pdl_enter();
  __shared__ float part[2][kMaxWarps];
  constexpr int vals = lane_vals(VEC);
  const int lane = threadIdx.x & 31;
  const uint32_t base = (threadIdx.x >> 5) * chunk_cols(VEC);
  const uint64_t step = (uint64_t)gridDim.x * blockDim.y;
  Raw<DT, VEC> dy, res, w;
  HeldIn<DT, VEC, HELD8> held;
  float next_rstd = 0.0f;
  const auto load = [&](uint64_t row) {
    if (row < a.rows) {
      next_rstd = a.rstd[row];
      dy.load(row_of<DT>(a.dy, row), base, a.cols, lane);
      held.load(a, row, base, lane);
      if (a.dres.p) res.load(row_of<DT>(a.dres, row), base, a.cols, lane);
    } else {
      dy.clear();
      held.clear();
    }
  };
  float dw[vals];
#pragma unroll
  for (int i = 0; i < vals; ++i) dw[i] = 0.0f;
  res.clear();
  load((uint64_t)blockIdx.x * blockDim.y + threadIdx.y);
  if (a.rows) w.load(a.weight, base, a.cols, lane);
  int buf = 0;
  for (uint64_t row = (uint64_t)blockIdx.x * blockDim.y + threadIdx.y; row < a.rows;
       row += step, buf ^= 1) {
    const float rstd = next_rstd;
    float t[vals], n[vals], s = 0.0f;
    held.values(n);
    const Raw<DT, VEC> r = res;
#pragma unroll
    for (int i = 0; i < vals; ++i) {
      n[i] *= rstd;
      const float d = dy.value(i);
      dw[i] = fmaf(d, n[i], dw[i]);
      t[i] = d * w.value(i);
      s = fmaf(t[i], n[i], s);
    }
    load(row + step);
    if (!a.dx.p) continue;
    const float c = row_sum<true>(s, part, buf) * a.inv_cols;
    back_st<DT, VEC>(a, row, base, lane, t, n, r, rstd, c);
  }
  if (!a.partial) return;
  extern __shared__ float sums[];
  join_rows<vals>(dw, sums);
  if (threadIdx.y) return;
  float* p = a.partial + (uint64_t)blockIdx.x * a.cols;
#pragma unroll
  for (int i = 0; i < vals; ++i) {
    const uint32_t c = chunk_col<VEC>(base, lane, i);
    if (c < a.cols) p[c] = dw[i];
  }
}

// One row's part of a block's shared memory in the backward pass: dy, then h (or
// its codes and scales), then dres.
struct BackStage {
  uint32_t dy, held, scales, res, end;
};

__host__ __device__ inline BackStage back_stage(const NormBackArgs& a, uint32_t es) {
  const uint32_t span = span_bytes(a.cols * es);
  BackStage b;
  b.dy = 0;
  b.held = span;
  b.scales = b.held + (a.h8.codes ? span_bytes(a.cols) : span);
  b.res = b.scales + (a.h8.codes ? span_bytes((a.cols + CR_Q8_GROUP - 1) / CR_Q8_GROUP * 4) : 0);
  b.end = b.res + (a.dres.p ? span : 0);
  return b;
}

template <bool FULL>
__device__ __forceinline__ void span_q8_values(const char* codes, const char* scales, uint32_t base,
                                               int lane, uint32_t cols, float* v) {
#pragma unroll
  for (int i = 0; i < kSpanVals; ++i) {
    const uint32_t c = base + lane + 32 * i;
    v[i] = FULL || c < cols
               ? from_e4m3x2(reinterpret_cast<const uint8_t*>(codes)[c]).x *
                     reinterpret_cast<const float*>(scales)[base / CR_Q8_GROUP + i / 4]
               : 0.0f;
  }
}

// t = dy * weight, n = h * rstd; dw += dy * n; the sum of t * n.
template <int DT, bool HELD8, bool FULL>
__device__ __forceinline__ float span_back_in(const NormBackArgs& a, const char* dy, const char* held,
                                              const char* scales, const char* weight, uint32_t base,
                                              int lane, float rstd, float* t, float* n, float* dw) {
  const uint32_t c0 = base + lane;
  float s = 0.0f;
  if constexpr (HELD8)
    span_q8_values<FULL>(held, scales, base, lane, a.cols, n);
  else
    span_values<DT, FULL>(held, c0, a.cols, n);
  span_values<DT, FULL>(dy, c0, a.cols, t);
#pragma unroll
  for (int i = 0; i < kSpanVals; ++i) {
    n[i] *= rstd;
    dw[i] = fmaf(t[i], n[i], dw[i]);
    t[i] *= FULL || c0 + 32 * i < a.cols ? value_at<DT>(weight, c0 + 32 * i) : 0.0f;
    s = fmaf(t[i], n[i], s);
  }
  return s;
}

template <int DT, bool FULL>
__device__ __forceinline__ void span_back_out(const NormBackArgs& a, uint64_t row, const char* res,
                                              uint32_t c0, float rstd, float c, float* t,
                                              const float* n) {
#pragma unroll
  for (int i = 0; i < kSpanVals; ++i) t[i] = rstd * (t[i] - n[i] * c);
  if (a.dres.p) {
#pragma unroll
    for (int i = 0; i < kSpanVals; ++i)
      if (FULL || c0 + 32 * i < a.cols) t[i] += value_at<DT>(res, c0 + 32 * i);
  }
  span_st<DT, FULL>(a.dx, row, c0, a.cols, t);
}

// The backward pass of such rows: partial row blockIdx.x of dweight.  80
// registers: two blocks of 12 warps an SM.
template <int DT, bool HELD8>
__global__ void __maxnreg__(80)
    k_rms_norm_back_span(const __grid_constant__ NormBackArgs a) {
  pdl_enter();
  extern __shared__ __align__(16) char smem[];
  __shared__ float part[2][kMaxWarps];
  constexpr uint32_t es = DT == CR_BF16 ? 2 : 4;
  const int lane = threadIdx.x & 31;
  const uint32_t bytes = a.cols * es;
  const BackStage at = back_stage(a, es);
  char* const ring = smem + span_bytes(bytes) + threadIdx.y * 2 * at.end;
  float next_rstd = 0.0f;
  const auto scales_of = [&](uint64_t row) { return a.h8.scales + row * a.h8.lds; };
  const auto codes_of = [&](uint64_t row) { return a.h8.codes + row * a.h8.ld; };
  const auto copy = [&](uint64_t row, int k) {
    char* const to = ring + k * at.end;
    const int n = blockDim.x;
    next_rstd = a.rstd[row];
    span_copy(to, row_of<DT>(a.dy, row), bytes, threadIdx.x, n);
    if constexpr (HELD8) {
      span_copy(to + at.held, codes_of(row), a.cols, threadIdx.x, n);
      span_copy(to + at.scales, scales_of(row), (a.cols + CR_Q8_GROUP - 1) / CR_Q8_GROUP * 4, threadIdx.x, n);
    } else {
      span_copy(to + at.held, row_of<DT>(a.h, row), bytes, threadIdx.x, n);
    }
    if (a.dres.p) span_copy(to + at.res, row_of<DT>(a.dres, row), bytes, threadIdx.x, n);
  };
  const uint64_t step = (uint64_t)gridDim.x * blockDim.y;
  uint64_t row = (uint64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (a.rows) span_copy(smem, a.weight, bytes, threadIdx.y * blockDim.x + threadIdx.x, blockDim.x * blockDim.y);
  if (row < a.rows) copy(row, 0);
  copies_wait();
  __syncthreads();
  const char* const weight = span_at(smem, a.weight);
  const uint32_t base = (threadIdx.x >> 5) * kSpanCols;
  const bool full = base + kSpanCols <= a.cols;
  float dw[kSpanVals];
#pragma unroll
  for (int i = 0; i < kSpanVals; ++i) dw[i] = 0.0f;
  for (int k = 0; row < a.rows; row += step, k ^= 1) {
    const float rstd = next_rstd;
    copies_wait();
    row_sync();
    if (row + step < a.rows) copy(row + step, k ^ 1);
    const char* const from = ring + k * at.end;
    const char* const dy = span_at(from, row_of<DT>(a.dy, row));
    const char* const held = span_at(from + at.held, HELD8 ? codes_of(row) : row_of<DT>(a.h, row));
    const char* const scales = span_at(from + at.scales, scales_of(row));
    float t[kSpanVals], n[kSpanVals];
    const float s =
        full ? span_back_in<DT, HELD8, true>(a, dy, held, scales, weight, base, lane, rstd, t, n, dw)
             : span_back_in<DT, HELD8, false>(a, dy, held, scales, weight, base, lane, rstd, t, n, dw);
    if (!a.dx.p) continue;
    const float c = row_sum<true>(s, part, k) * a.inv_cols;
    const char* const res = span_at(from + at.res, row_of<DT>(a.dres, row));
    if (full)
      span_back_out<DT, true>(a, row, res, base + lane, rstd, c, t, n);
    else
      span_back_out<DT, false>(a, row, res, base + lane, rstd, c, t, n);
  }
  if (!a.partial) return;
  join_rows<kSpanVals>(dw, reinterpret_cast<float*>(smem));
  if (threadIdx.y) return;
  float* p = a.partial + (uint64_t)blockIdx.x * a.cols;
#pragma unroll
  for (int i = 0; i < kSpanVals; ++i) {
    const uint32_t c = base + lane + 32 * i;
    if (c < a.cols) p[c] = dw[i];
  }
}

template <int DT, int VEC>
__device__ __forceinline__ void ld_chunk(const void* row, uint32_t base, uint32_t cols, int lane,
                                         float* v) {
  Raw<DT, VEC> r;
  r.load(row, base, cols, lane);
#pragma unroll
  for (int i = 0; i < lane_vals(VEC); ++i) v[i] = r.value(i);
}

template <int DT, int VEC>
__device__ __forceinline__ void back_ld(const NormBackArgs& a, uint64_t row, uint32_t base,
                                        int lane, float* dy, float* h) {
  ld_chunk<DT, VEC>(row_of<DT>(a.dy, row), base, a.cols, lane, dy);
  if (a.h8.codes) {
    RawQ8<VEC> r;
    r.load(a.h8, row, base, a.cols, lane);
    r.values(h);
  } else {
    ld_chunk<DT, VEC>(row_of<DT>(a.h, row), base, a.cols, lane, h);
  }
}

// Wide rows, dx: one block a row, read twice.
template <int DT, int VEC>
__global__ void __launch_bounds__(kWideThreads)
    k_rms_norm_back_wide(const __grid_constant__ NormBackArgs a) {
  pdl_enter();
  __shared__ float part[2][kMaxWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int buf = 0;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x, buf ^= 1) {
    const float rstd = a.rstd[row];
    float t[lane_vals(VEC)], n[lane_vals(VEC)], w[lane_vals(VEC)], s = 0.0f;
    for (uint64_t base = (uint64_t)warp * chunk_cols(VEC); base < a.cols; base += (uint64_t)nw * chunk_cols(VEC)) {
      back_ld<DT, VEC>(a, row, (uint32_t)base, lane, t, n);
      ld_chunk<DT, VEC>(a.weight, (uint32_t)base, a.cols, lane, w);
#pragma unroll
      for (int i = 0; i < lane_vals(VEC); ++i) s = fmaf(t[i] * w[i], n[i] * rstd, s);
    }
    const float c = row_sum<false>(s, part, buf) * a.inv_cols;
    for (uint64_t base = (uint64_t)warp * chunk_cols(VEC); base < a.cols; base += (uint64_t)nw * chunk_cols(VEC)) {
      back_ld<DT, VEC>(a, row, (uint32_t)base, lane, t, n);
      ld_chunk<DT, VEC>(a.weight, (uint32_t)base, a.cols, lane, w);
#pragma unroll
      for (int i = 0; i < lane_vals(VEC); ++i) t[i] *= w[i], n[i] *= rstd;
      Raw<DT, VEC> res;
      if (a.dres.p)
        res.load(row_of<DT>(a.dres, row), (uint32_t)base, a.cols, lane);
      else
        res.clear();
      back_st<DT, VEC>(a, row, (uint32_t)base, lane, t, n, res, rstd, c);
    }
  }
}

// Wide rows, dweight partials: warp (blockIdx.x, warp) takes one chunk of
// columns, blockIdx.y every gridDim.y-th row.
template <int DT, int VEC>
__global__ void __launch_bounds__(kBlock)
    k_rms_norm_back_wide_dw(const __grid_constant__ NormBackArgs a) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const uint64_t base = ((uint64_t)blockIdx.x * (kBlock / 32) + (threadIdx.x >> 5)) * chunk_cols(VEC);
  if (base >= a.cols) return;
  float dw[lane_vals(VEC)] = {0.0f};
  for (uint64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    float dy[lane_vals(VEC)], h[lane_vals(VEC)];
    back_ld<DT, VEC>(a, row, (uint32_t)base, lane, dy, h);
    const float rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < lane_vals(VEC); ++i) dw[i] = fmaf(dy[i], h[i] * rstd, dw[i]);
  }
  float* p = a.partial + (uint64_t)blockIdx.y * a.cols;
#pragma unroll
  for (int i = 0; i < lane_vals(VEC); ++i) {
    const uint32_t c = chunk_col<VEC>((uint32_t)base, lane, i);
    if (c < a.cols) p[c] = dw[i];
  }
}

// dweight = sum of the partial rows: block (16 columns, 64 row classes), each
// class in order, then the classes in order.
constexpr int kDwCols = 16, kDwClasses = 64;

template <int DW>
__global__ void __launch_bounds__(kDwCols* kDwClasses)
    k_norm_dw(const float* partial, uint32_t parts, uint32_t cols, void* dweight) {
  pdl_enter();
  __shared__ float sum[kDwClasses][kDwCols + 1];
  const uint64_t c = (uint64_t)blockIdx.x * kDwCols + threadIdx.x;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (uint32_t k = threadIdx.y; k < parts; k += kDwClasses) s += partial[(uint64_t)k * cols + c];
  }
  sum[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < cols) {
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < kDwClasses; ++k) s += sum[k][threadIdx.x];
    if constexpr (DW == CR_BF16)
      static_cast<uint16_t*>(dweight)[c] = (uint16_t)ffn_bf16x2(s, 0.0f);
    else
      static_cast<float*>(dweight)[c] = s;
  }
}

struct RowShape {
  unsigned warps;  // per row, a chunk each
  unsigned rows;   // per block, at most the matrix's
};

// Short rows share a block of 8 to 12 warps.
RowShape row_shape(uint64_t rows, uint32_t cols, int vec) {
  const unsigned warps = (unsigned)(((uint64_t)cols + chunk_cols(vec) - 1) / chunk_cols(vec));
  const unsigned fit = warps <= 8 ? std::max(warps > 4 && warps <= 6 ? 12 / warps : 8 / warps, 1u) : 1u;
  return {warps, (unsigned)std::min<uint64_t>(fit, std::max<uint64_t>(rows, 1))};
}

uint32_t wide_parts(uint64_t rows) {
  return (uint32_t)std::min<uint64_t>(std::max<uint64_t>(rows, 1), kWideParts);
}

template <typename... KArgs, typename... Args>
cudaError_t launch2_smem(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                         cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename... KArgs, typename... Args>
cudaError_t launch2(void (*kernel)(KArgs...), dim3 grid, dim3 block, cudaStream_t s,
                    Args... args) {
  return launch2_smem(kernel, grid, block, 0, s, args...);
}

// Blocks of `threads` that all SMs hold at once (cached: the query costs
// microseconds).
cudaError_t resident_blocks(const void* kernel, int threads, size_t smem, unsigned* blocks) {
  static std::mutex mu;
  static std::map<std::tuple<const void*, int, size_t, int>, unsigned> cache;
  int dev = 0, sms = 0, per_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const auto key = std::make_tuple(kernel, threads, smem, dev);
  {
    std::lock_guard<std::mutex> lock(mu);
    const auto it = cache.find(key);
    if (it != cache.end()) {
      *blocks = it->second;
      return cudaSuccess;
    }
  }
  if ((e = sm_count(&sms)) != cudaSuccess) return e;
  if (smem) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSpanSmem);
    if (e != cudaSuccess) return e;
  }
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
  if (e != cudaSuccess) return e;
  *blocks = (unsigned)(sms * std::max(per_sm, 1));
  std::lock_guard<std::mutex> lock(mu);
  cache[key] = *blocks;
  return cudaSuccess;
}

// Blocks of r for `rows` rows: at most what the SMs hold at once.
template <typename K>
cudaError_t row_grid(K kernel, const RowShape& r, uint64_t rows, unsigned* grid, size_t smem = 0) {
  unsigned most = 0;
  const cudaError_t e = resident_blocks(reinterpret_cast<const void*>(kernel), r.warps * 32 * r.rows, smem, &most);
  *grid = (unsigned)std::min<uint64_t>((rows + r.rows - 1) / r.rows, most);
  return e;
}

template <int DT, int VEC>
cudaError_t norm_run(const NormArgs& a, const RowShape& r, cudaStream_t s) {
  unsigned grid = 0;
  const cudaError_t e = row_grid(k_rms_norm<DT, VEC>, r, a.rows, &grid);
  if (e != cudaSuccess) return e;
  return launch2(k_rms_norm<DT, VEC>, dim3(grid), dim3(r.warps * 32, r.rows), s, a);
}

// Staged rows: a warp takes kSpanCols columns; short rows share a block of 8 warps.
RowShape span_shape(uint64_t rows, uint32_t cols) {
  const unsigned warps = (cols + kSpanCols - 1) / kSpanCols;
  return {warps, (unsigned)std::min<uint64_t>(std::max(8 / warps, 1u), std::max<uint64_t>(rows, 1))};
}

template <int DT>
cudaError_t span_run(const NormArgs& a, cudaStream_t s) {
  const uint32_t span = span_bytes(a.cols * (DT == CR_BF16 ? 2 : 4));
  const RowShape r = span_shape(a.rows, a.cols);
  const size_t smem = span + (size_t)r.rows * 2 * span * (a.residual.p ? 2 : 1);
  unsigned grid = 0;
  const cudaError_t e = row_grid(k_rms_norm_span<DT>, r, a.rows, &grid, smem);
  if (e != cudaSuccess) return e;
  return launch2_smem(k_rms_norm_span<DT>, dim3(grid), dim3(r.warps * 32, r.rows), smem, s, a);
}

template <int DT, int VEC>
cudaError_t norm_dispatch(const NormArgs& a, cudaStream_t s) {
  if constexpr (VEC == 0) {
    if (a.cols > kSpanFrom && a.cols <= kWideFrom) return span_run<DT>(a, s);
  }
  if (a.cols <= kWideFrom) return norm_run<DT, VEC>(a, row_shape(a.rows, a.cols, VEC), s);
  const unsigned g = (unsigned)std::min<uint64_t>(a.rows, 1u << 30);
  return launch2(k_rms_norm_wide<DT, VEC>, dim3(g), dim3(kWideThreads), s, a);
}

template <int DT, int VEC>
cudaError_t back_run(NormBackArgs& a, const RowShape& r, cudaStream_t s) {
  void (*kernel)(const NormBackArgs) =
      a.h8.codes ? k_rms_norm_back<DT, VEC, true> : k_rms_norm_back<DT, VEC, false>;
  unsigned grid = 0;
  const cudaError_t e = row_grid(kernel, r, a.rows, &grid);
  if (e != cudaSuccess) return e;
  grid = std::min(std::max(grid, 1u), kBackParts);  // no rows: one block writes zeros
  a.parts = grid;
  const size_t smem = r.rows > 1 ? (size_t)lane_vals(VEC) * r.warps * 32 * sizeof(float) : 0;
  return launch2_smem(kernel, dim3(grid), dim3(r.warps * 32, r.rows), smem, s, a);
}

template <int DT>
cudaError_t back_span_run(NormBackArgs& a, const RowShape& r, size_t smem, cudaStream_t s) {
  void (*kernel)(const NormBackArgs) =
      a.h8.codes ? k_rms_norm_back_span<DT, true> : k_rms_norm_back_span<DT, false>;
  unsigned grid = 0;
  const cudaError_t e = row_grid(kernel, r, a.rows, &grid, smem);
  if (e != cudaSuccess) return e;
  grid = std::min(std::max(grid, 1u), kBackParts);  // no rows: one block writes zeros
  a.parts = grid;
  return launch2_smem(kernel, dim3(grid), dim3(r.warps * 32, r.rows), smem, s, a);
}

template <int DT, int VEC>
cudaError_t back_dispatch(NormBackArgs& a, cudaStream_t s) {
  if constexpr (VEC == 0) {
    const uint32_t es = DT == CR_BF16 ? 2 : 4;
    const RowShape r = span_shape(a.rows, a.cols);
    const size_t smem = std::max(span_bytes(a.cols * es) + (size_t)r.rows * 2 * back_stage(a, es).end,
                                 (size_t)(r.rows > 1 ? r.warps * kSpanCols * sizeof(float) : 0));
    if (a.cols > kSpanFrom && a.cols <= kWideFrom)
      return back_span_run<DT>(a, r, smem, s);
  }
  if (a.cols <= kWideFrom) return back_run<DT, VEC>(a, row_shape(a.rows, a.cols, VEC), s);
  a.parts = wide_parts(a.rows);
  // dweight first: dx may be written over dy or h
  if (a.partial) {
    const unsigned gx = (a.cols / chunk_cols(VEC) + 1 + kBlock / 32 - 1) / (kBlock / 32);
    cudaError_t e = launch2(k_rms_norm_back_wide_dw<DT, VEC>, dim3(gx, a.parts), dim3(kBlock), s, a);
    if (e != cudaSuccess || !a.dx.p) return e;
  }
  const unsigned g = (unsigned)std::min<uint64_t>(a.rows, 1u << 30);
  return launch2(k_rms_norm_back_wide<DT, VEC>, dim3(g), dim3(kWideThreads), s, a);
}

template <int DT>
cudaError_t norm_by_vec(const NormArgs& a, int vec, cudaStream_t s) {
  return vec == 2 ? norm_dispatch<DT, 2>(a, s)
                  : vec == 1 ? norm_dispatch<DT, 1>(a, s) : norm_dispatch<DT, 0>(a, s);
}

template <int DT>
cudaError_t back_by_vec(NormBackArgs& a, int vec, cudaStream_t s) {
  return vec == 2 ? back_dispatch<DT, 2>(a, s)
                  : vec == 1 ? back_dispatch<DT, 1>(a, s) : back_dispatch<DT, 0>(a, s);
}

}  // namespace

cudaError_t launch_rms_norm(cr_dtype d, const NormArgs& a, int vec, cudaStream_t s) {
  return d == CR_BF16 ? norm_by_vec<CR_BF16>(a, vec, s) : norm_by_vec<CR_F32>(a, vec, s);
}

uint32_t norm_back_parts(uint64_t rows, uint32_t cols) {
  const uint32_t narrow = (uint32_t)std::min<uint64_t>(std::max<uint64_t>(rows, 1), kBackParts);
  return cols > kWideFrom ? wide_parts(rows) : narrow;
}

cudaError_t launch_rms_norm_back(cr_dtype d, cr_dtype dw, NormBackArgs a, int vec, cudaStream_t s) {
  const cudaError_t e = d == CR_BF16 ? back_by_vec<CR_BF16>(a, vec, s) : back_by_vec<CR_F32>(a, vec, s);
  if (e != cudaSuccess || !a.partial) return e;
  const dim3 grid((a.cols + kDwCols - 1) / kDwCols), block(kDwCols, kDwClasses);
  return launch2(dw == CR_BF16 ? k_norm_dw<CR_BF16> : k_norm_dw<CR_F32>, grid, block, s,
                 (const float*)a.partial, a.parts, a.cols, a.dweight);
}

}  // namespace cr
