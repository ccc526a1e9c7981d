// k_q8.cu -- 8-bit activation checkpoints: store, load, and the gate's
// backward pass, which reads gate and up from their checkpoints.
//
// All are one pass over memory, bound by HBM: a warp takes a 256-column chunk
// of a row (ffn_internal.cuh), so the 128-column group's largest magnitude is
// a shuffle reduction over 16 lanes.  A warp loads kAhead chunks before it
// works on the first, to keep enough bytes in flight.
#include "ffn_internal.cuh"
#include "pdl.cuh"

namespace cr {

namespace {

// Chunks of a rows x cols matrix, in row order.
struct ChunkRange {
  uint64_t chunks;
  FastDiv per_row;
};

ChunkRange chunk_range(uint64_t rows, uint32_t cols) {
  const uint64_t per_row = ((uint64_t)cols + kChunk - 1) / kChunk;
  return {rows * per_row, fastdiv_make(per_row, rows * per_row)};
}

// Calls load(j, row, base) for up to AHEAD chunks, then work(j, row, base) for
// the same: chunk w, w + W, ..., of the warp w of W in the grid.
template <int AHEAD, typename Load, typename Work>
__device__ __forceinline__ void for_chunks(const ChunkRange& r, Load load, Work work) {
  const uint64_t stride = (uint64_t)gridDim.x * (kBlock / 32);
  for (uint64_t k = (uint64_t)blockIdx.x * (kBlock / 32) + (threadIdx.x >> 5); k < r.chunks;
       k += AHEAD * stride) {
    uint64_t row[AHEAD];
    uint32_t base[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const uint64_t c = k + j * stride;
      if (c >= r.chunks) break;
      row[j] = fastdiv_div(r.per_row, c);
      base[j] = (uint32_t)(c - row[j] * r.per_row.d) * kChunk;
      load(j, row[j], base[j]);
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      if (k + j * stride >= r.chunks) break;
      work(j, row[j], base[j]);
    }
  }
}

template <int DT>
__device__ __forceinline__ char* row_at(const Mat& m, uint64_t row) {
  return static_cast<char*>(m.p) + row * m.ld * (DT == CR_BF16 ? 2 : 4);
}

constexpr int kAhead = 2;

template <int DT, bool VEC>
__global__ void __launch_bounds__(kBlock) k_q8_store(const __grid_constant__ Mat x,
                                                     const __grid_constant__ Q8 q, uint32_t cols,
                                                     const __grid_constant__ ChunkRange r) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  Raw<DT, VEC> in[kAhead];
  for_chunks<kAhead>(
      r,
      [&](int j, uint64_t row, uint32_t base) { in[j].load(row_at<DT>(x, row), base, cols, lane); },
      [&](int j, uint64_t row, uint32_t base) {
        float v[kLaneVals];
#pragma unroll
        for (int i = 0; i < kLaneVals; ++i) v[i] = in[j].value(i);
        st_chunk_q8<VEC>(q, row, base, cols, lane, v);
      });
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kBlock) k_q8_load(const __grid_constant__ Q8 q,
                                                    const __grid_constant__ Mat x, uint32_t cols,
                                                    const __grid_constant__ ChunkRange r) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  RawQ8<VEC> in[2 * kAhead];
  for_chunks<2 * kAhead>(
      r, [&](int j, uint64_t row, uint32_t base) { in[j].load(q, row, base, cols, lane); },
      [&](int j, uint64_t row, uint32_t base) {
        float v[kLaneVals];
        in[j].values(v);
        st_chunk<DT, VEC>(row_at<DT>(x, row), base, cols, lane, v);
      });
}

template <bool VEC>
__global__ void __launch_bounds__(kBlock) k_q8_split(const __grid_constant__ Q8 q,
                                                     const __grid_constant__ Mat hi,
                                                     const __grid_constant__ Mat lo, uint32_t cols,
                                                     const __grid_constant__ ChunkRange r) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  RawQ8<VEC> in[kAhead];
  for_chunks<kAhead>(
      r, [&](int j, uint64_t row, uint32_t base) { in[j].load(q, row, base, cols, lane); },
      [&](int j, uint64_t row, uint32_t base) {
        float v[kLaneVals], rest[kLaneVals];
        in[j].values(v);
#pragma unroll
        for (int i = 0; i < kLaneVals; ++i)
          rest[i] = v[i] - ffn_bf16((uint16_t)ffn_bf16x2(v[i], 0.0f));
        st_chunk<CR_BF16, VEC>(row_at<CR_BF16>(hi, row), base, cols, lane, v);
        st_chunk<CR_BF16, VEC>(row_at<CR_BF16>(lo, row), base, cols, lane, rest);
      });
}

__global__ void __launch_bounds__(kBlock) k_copy_bf16(const __grid_constant__ Mat src,
                                                      const __grid_constant__ Mat dst,
                                                      uint32_t cols,
                                                      const __grid_constant__ ChunkRange r) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  Raw<CR_BF16, false> in[kAhead];
  for_chunks<kAhead>(
      r,
      [&](int j, uint64_t row, uint32_t base) {
        in[j].load(row_at<CR_BF16>(src, row), base, cols, lane);
      },
      [&](int j, uint64_t row, uint32_t base) {
        float v[kLaneVals];
#pragma unroll
        for (int i = 0; i < kLaneVals; ++i) v[i] = in[j].value(i);
        st_chunk<CR_BF16, false>(row_at<CR_BF16>(dst, row), base, cols, lane, v);
      });
}

template <int ACT, bool VEC>
__global__ void __launch_bounds__(kBlock) k_act_back(const __grid_constant__ ActBackArgs a,
                                                     const __grid_constant__ ChunkRange r) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  Raw<CR_BF16, VEC> in[kAhead];
  RawQ8<VEC> gate[kAhead], up[kAhead];
  for_chunks<kAhead>(
      r,
      [&](int j, uint64_t row, uint32_t base) {
        in[j].load(row_at<CR_BF16>(a.da, row), base, a.cols, lane);
        gate[j].load(a.g8, row, base, a.cols, lane);
        up[j].load(a.u8, row, base, a.cols, lane);
      },
      [&](int j, uint64_t row, uint32_t base) {
        float g[kLaneVals], u[kLaneVals], dg[kLaneVals], du[kLaneVals];
        gate[j].values(g);
        up[j].values(u);
#pragma unroll
        for (int i = 0; i < kLaneVals; ++i) {
          const float da = in[j].value(i);
          const float2 v = act_gate_slope<ACT>(g[i]);
          dg[i] = da * u[i] * v.y;
          du[i] = da * v.x;
          u[i] *= v.x;
        }
        if (a.dg.p) st_chunk<CR_BF16, VEC>(row_at<CR_BF16>(a.dg, row), base, a.cols, lane, dg);
        if (a.du.p) st_chunk<CR_BF16, VEC>(row_at<CR_BF16>(a.du, row), base, a.cols, lane, du);
        if (a.a.p) st_chunk<CR_BF16, VEC>(row_at<CR_BF16>(a.a, row), base, a.cols, lane, u);
      });
}

// A warp for every `ahead` chunks.
dim3 chunk_grid(const ChunkRange& r, int ahead) {
  return dim3(flat_grid((r.chunks + ahead - 1) / ahead * 32));
}

}  // namespace

cudaError_t launch_q8_store(cr_dtype d, const Mat& x, const Q8& q, uint64_t rows, uint32_t cols,
                            bool vec, cudaStream_t s) {
  const ChunkRange r = chunk_range(rows, cols);
  const dim3 grid = chunk_grid(r, kAhead);
  if (d == CR_BF16)
    return vec ? launch_pdl(k_q8_store<CR_BF16, true>, grid, kBlock, s, x, q, cols, r)
               : launch_pdl(k_q8_store<CR_BF16, false>, grid, kBlock, s, x, q, cols, r);
  return vec ? launch_pdl(k_q8_store<CR_F32, true>, grid, kBlock, s, x, q, cols, r)
             : launch_pdl(k_q8_store<CR_F32, false>, grid, kBlock, s, x, q, cols, r);
}

cudaError_t launch_q8_load(cr_dtype d, const Q8& q, const Mat& x, uint64_t rows, uint32_t cols,
                           bool vec, cudaStream_t s) {
  const ChunkRange r = chunk_range(rows, cols);
  const dim3 grid = chunk_grid(r, 2 * kAhead);
  if (d == CR_BF16)
    return vec ? launch_pdl(k_q8_load<CR_BF16, true>, grid, kBlock, s, q, x, cols, r)
               : launch_pdl(k_q8_load<CR_BF16, false>, grid, kBlock, s, q, x, cols, r);
  return vec ? launch_pdl(k_q8_load<CR_F32, true>, grid, kBlock, s, q, x, cols, r)
             : launch_pdl(k_q8_load<CR_F32, false>, grid, kBlock, s, q, x, cols, r);
}

cudaError_t launch_q8_split(const Q8& q, const Mat& hi, const Mat& lo, uint64_t rows, uint32_t cols,
                            bool vec, cudaStream_t s) {
  const ChunkRange r = chunk_range(rows, cols);
  const dim3 grid = chunk_grid(r, kAhead);
  return vec ? launch_pdl(k_q8_split<true>, grid, kBlock, s, q, hi, lo, cols, r)
             : launch_pdl(k_q8_split<false>, grid, kBlock, s, q, hi, lo, cols, r);
}

cudaError_t launch_copy_bf16(const Mat& src, const Mat& dst, uint64_t rows, uint32_t cols,
                             cudaStream_t s) {
  const ChunkRange r = chunk_range(rows, cols);
  return launch_pdl(k_copy_bf16, chunk_grid(r, kAhead), kBlock, s, src, dst, cols, r);
}

cudaError_t launch_act_back(cr_act act, const ActBackArgs& a, bool vec, cudaStream_t s) {
  const ChunkRange r = chunk_range(a.rows, a.cols);
  const dim3 grid = chunk_grid(r, kAhead);
  if (act == CR_ACT_SILU)
    return vec ? launch_pdl(k_act_back<CR_ACT_SILU, true>, grid, kBlock, s, a, r)
               : launch_pdl(k_act_back<CR_ACT_SILU, false>, grid, kBlock, s, a, r);
  return vec ? launch_pdl(k_act_back<CR_ACT_GELU, true>, grid, kBlock, s, a, r)
             : launch_pdl(k_act_back<CR_ACT_GELU, false>, grid, kBlock, s, a, r);
}

}  // namespace cr
