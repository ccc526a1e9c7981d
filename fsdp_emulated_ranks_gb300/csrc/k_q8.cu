// k_q8.cu -- 8-bit activation checkpoints: store, load, and the gate's
// backward pass, which reads gate and up from their checkpoints.
//
// All three are one pass over memory, bound by HBM: a warp takes a 256-column
// chunk of a row (ffn_internal.cuh), so the 128-column group's largest
// magnitude is a shuffle reduction over 16 lanes.
#include "ffn_internal.cuh"
#include "pdl.cuh"

namespace cr {

namespace {

// Chunks of a rows x cols matrix, in row order: the warp's first, then every
// `stride`-th.
struct ChunkRange {
  uint64_t chunks;
  FastDiv per_row;
};

ChunkRange chunk_range(uint64_t rows, uint32_t cols) {
  const uint64_t per_row = ((uint64_t)cols + kChunk - 1) / kChunk;
  return {rows * per_row, fastdiv_make(per_row, rows * per_row)};
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kBlock) k_q8_store(const __grid_constant__ Mat x,
                                                     const __grid_constant__ Q8 q, uint32_t cols,
                                                     const __grid_constant__ ChunkRange r) {
  pdl_enter();
  constexpr int es = DT == CR_BF16 ? 2 : 4;
  const int lane = threadIdx.x & 31;
  const uint64_t stride = (uint64_t)gridDim.x * (kBlock / 32);
  for (uint64_t k = (uint64_t)blockIdx.x * (kBlock / 32) + (threadIdx.x >> 5); k < r.chunks;
       k += stride) {
    const uint64_t row = fastdiv_div(r.per_row, k);
    const uint32_t base = (uint32_t)(k - row * r.per_row.d) * kChunk;
    float v[kLaneVals];
    ld_chunk<DT, VEC>(static_cast<const char*>(x.p) + row * x.ld * es, base, cols, lane, v);
    st_chunk_q8<VEC>(q, row, base, cols, lane, v);
  }
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kBlock) k_q8_load(const __grid_constant__ Q8 q,
                                                    const __grid_constant__ Mat x, uint32_t cols,
                                                    const __grid_constant__ ChunkRange r) {
  pdl_enter();
  constexpr int es = DT == CR_BF16 ? 2 : 4;
  const int lane = threadIdx.x & 31;
  const uint64_t stride = (uint64_t)gridDim.x * (kBlock / 32);
  for (uint64_t k = (uint64_t)blockIdx.x * (kBlock / 32) + (threadIdx.x >> 5); k < r.chunks;
       k += stride) {
    const uint64_t row = fastdiv_div(r.per_row, k);
    const uint32_t base = (uint32_t)(k - row * r.per_row.d) * kChunk;
    float v[kLaneVals];
    ld_chunk_q8<VEC>(q, row, base, cols, lane, v);
    st_chunk<DT, VEC>(static_cast<char*>(x.p) + row * x.ld * es, base, cols, lane, v);
  }
}

template <bool VEC>
__global__ void __launch_bounds__(kBlock) k_q8_split(const __grid_constant__ Q8 q,
                                                     const __grid_constant__ Mat hi,
                                                     const __grid_constant__ Mat lo, uint32_t cols,
                                                     const __grid_constant__ ChunkRange r) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const uint64_t stride = (uint64_t)gridDim.x * (kBlock / 32);
  for (uint64_t k = (uint64_t)blockIdx.x * (kBlock / 32) + (threadIdx.x >> 5); k < r.chunks;
       k += stride) {
    const uint64_t row = fastdiv_div(r.per_row, k);
    const uint32_t base = (uint32_t)(k - row * r.per_row.d) * kChunk;
    float v[kLaneVals], rest[kLaneVals];
    ld_chunk_q8<VEC>(q, row, base, cols, lane, v);
#pragma unroll
    for (int i = 0; i < kLaneVals; ++i)
      rest[i] = v[i] - ffn_bf16((uint16_t)ffn_bf16x2(v[i], 0.0f));
    st_chunk<CR_BF16, VEC>(static_cast<uint16_t*>(hi.p) + row * hi.ld, base, cols, lane, v);
    st_chunk<CR_BF16, VEC>(static_cast<uint16_t*>(lo.p) + row * lo.ld, base, cols, lane, rest);
  }
}

__global__ void __launch_bounds__(kBlock) k_copy_bf16(const __grid_constant__ Mat src,
                                                      const __grid_constant__ Mat dst,
                                                      uint32_t cols,
                                                      const __grid_constant__ ChunkRange r) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const uint64_t stride = (uint64_t)gridDim.x * (kBlock / 32);
  for (uint64_t k = (uint64_t)blockIdx.x * (kBlock / 32) + (threadIdx.x >> 5); k < r.chunks;
       k += stride) {
    const uint64_t row = fastdiv_div(r.per_row, k);
    const uint32_t base = (uint32_t)(k - row * r.per_row.d) * kChunk;
    float v[kLaneVals];
    ld_chunk<CR_BF16, false>(static_cast<const uint16_t*>(src.p) + row * src.ld, base, cols, lane, v);
    st_chunk<CR_BF16, false>(static_cast<uint16_t*>(dst.p) + row * dst.ld, base, cols, lane, v);
  }
}

template <int ACT, bool VEC>
__global__ void __launch_bounds__(kBlock) k_act_back(const __grid_constant__ ActBackArgs a,
                                                     const __grid_constant__ ChunkRange r) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const uint64_t stride = (uint64_t)gridDim.x * (kBlock / 32);
  for (uint64_t k = (uint64_t)blockIdx.x * (kBlock / 32) + (threadIdx.x >> 5); k < r.chunks;
       k += stride) {
    const uint64_t row = fastdiv_div(r.per_row, k);
    const uint32_t base = (uint32_t)(k - row * r.per_row.d) * kChunk;
    float g[kLaneVals], u[kLaneVals], da[kLaneVals];
    ld_chunk<CR_BF16, VEC>(static_cast<const uint16_t*>(a.da.p) + row * a.da.ld, base, a.cols,
                           lane, da);
    ld_chunk_q8<VEC>(a.g8, row, base, a.cols, lane, g);
    ld_chunk_q8<VEC>(a.u8, row, base, a.cols, lane, u);
    float dg[kLaneVals], du[kLaneVals];
#pragma unroll
    for (int i = 0; i < kLaneVals; ++i) {
      const float2 v = act_gate_slope<ACT>(g[i]);
      dg[i] = da[i] * u[i] * v.y;
      du[i] = da[i] * v.x;
      u[i] *= v.x;
    }
    if (a.dg.p)
      st_chunk<CR_BF16, VEC>(static_cast<uint16_t*>(a.dg.p) + row * a.dg.ld, base, a.cols, lane, dg);
    if (a.du.p)
      st_chunk<CR_BF16, VEC>(static_cast<uint16_t*>(a.du.p) + row * a.du.ld, base, a.cols, lane, du);
    if (a.a.p)
      st_chunk<CR_BF16, VEC>(static_cast<uint16_t*>(a.a.p) + row * a.a.ld, base, a.cols, lane, u);
  }
}

unsigned chunk_grid(const ChunkRange& r) { return flat_grid(r.chunks * 32); }

}  // namespace

cudaError_t launch_q8_store(cr_dtype d, const Mat& x, const Q8& q, uint64_t rows, uint32_t cols,
                            bool vec, cudaStream_t s) {
  const ChunkRange r = chunk_range(rows, cols);
  const dim3 grid(chunk_grid(r));
  if (d == CR_BF16)
    return vec ? launch_pdl(k_q8_store<CR_BF16, true>, grid, kBlock, s, x, q, cols, r)
               : launch_pdl(k_q8_store<CR_BF16, false>, grid, kBlock, s, x, q, cols, r);
  return vec ? launch_pdl(k_q8_store<CR_F32, true>, grid, kBlock, s, x, q, cols, r)
             : launch_pdl(k_q8_store<CR_F32, false>, grid, kBlock, s, x, q, cols, r);
}

cudaError_t launch_q8_load(cr_dtype d, const Q8& q, const Mat& x, uint64_t rows, uint32_t cols,
                           bool vec, cudaStream_t s) {
  const ChunkRange r = chunk_range(rows, cols);
  const dim3 grid(chunk_grid(r));
  if (d == CR_BF16)
    return vec ? launch_pdl(k_q8_load<CR_BF16, true>, grid, kBlock, s, q, x, cols, r)
               : launch_pdl(k_q8_load<CR_BF16, false>, grid, kBlock, s, q, x, cols, r);
  return vec ? launch_pdl(k_q8_load<CR_F32, true>, grid, kBlock, s, q, x, cols, r)
             : launch_pdl(k_q8_load<CR_F32, false>, grid, kBlock, s, q, x, cols, r);
}

cudaError_t launch_q8_split(const Q8& q, const Mat& hi, const Mat& lo, uint64_t rows, uint32_t cols,
                            bool vec, cudaStream_t s) {
  const ChunkRange r = chunk_range(rows, cols);
  return vec ? launch_pdl(k_q8_split<true>, dim3(chunk_grid(r)), kBlock, s, q, hi, lo, cols, r)
             : launch_pdl(k_q8_split<false>, dim3(chunk_grid(r)), kBlock, s, q, hi, lo, cols, r);
}

cudaError_t launch_copy_bf16(const Mat& src, const Mat& dst, uint64_t rows, uint32_t cols,
                             cudaStream_t s) {
  const ChunkRange r = chunk_range(rows, cols);
  return launch_pdl(k_copy_bf16, dim3(chunk_grid(r)), kBlock, s, src, dst, cols, r);
}

cudaError_t launch_act_back(cr_act act, const ActBackArgs& a, bool vec, cudaStream_t s) {
  const ChunkRange r = chunk_range(a.rows, a.cols);
  const dim3 grid(chunk_grid(r));
  if (act == CR_ACT_SILU)
    return vec ? launch_pdl(k_act_back<CR_ACT_SILU, true>, grid, kBlock, s, a, r)
               : launch_pdl(k_act_back<CR_ACT_SILU, false>, grid, kBlock, s, a, r);
  return vec ? launch_pdl(k_act_back<CR_ACT_GELU, true>, grid, kBlock, s, a, r)
             : launch_pdl(k_act_back<CR_ACT_GELU, false>, grid, kBlock, s, a, r);
}

}  // namespace cr
