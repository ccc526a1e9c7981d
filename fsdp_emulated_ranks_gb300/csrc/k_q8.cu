// k_q8.cu -- 8-bit activation checkpoints: store, load, and the gate's
// backward pass, which reads gate and up from their checkpoints.
//
// All are one pass over memory: a warp takes a chunk of a row
// (ffn_internal.cuh), so the 128-column group's largest magnitude is a shuffle
// reduction.  A warp that loads few bytes a chunk loads several chunks before
// it works on the first.
#include <algorithm>
#include <type_traits>

#include "ffn_internal.cuh"
#include "pdl.cuh"

namespace cr {

namespace {

// Chunks of a rows x cols matrix, in row order.
struct ChunkRange {
  uint64_t chunks;
  FastDiv per_row;
};

ChunkRange chunk_range(uint64_t rows, uint32_t cols, int vec) {
  const uint64_t per_row = ((uint64_t)cols + chunk_cols(vec) - 1) / chunk_cols(vec);
  return {rows * per_row, fastdiv_make(per_row, rows * per_row)};
}

// Calls load(j, row, base) for up to AHEAD chunks, then work(j, row, base) for
// the same: chunk w, w + W, ..., of the warp w of W in the grid.
template <int VEC, int AHEAD, typename Load, typename Work>
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
      base[j] = (uint32_t)(c - row[j] * r.per_row.d) * chunk_cols(VEC);
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

constexpr int kAhead = 2;  // chunks of a warp in flight, where a chunk is few bytes

template <int DT, int VEC>
__global__ void __launch_bounds__(kBlock) k_q8_store(const __grid_constant__ Mat x,
                                                     const __grid_constant__ Q8 q, uint32_t cols,
                                                     const __grid_constant__ ChunkRange r) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  Raw<DT, VEC> in[kAhead];
  for_chunks<VEC, kAhead>(
      r,
      [&](int j, uint64_t row, uint32_t base) { in[j].load(row_at<DT>(x, row), base, cols, lane); },
      [&](int j, uint64_t row, uint32_t base) {
        float v[lane_vals(VEC)];
#pragma unroll
        for (int i = 0; i < lane_vals(VEC); ++i) v[i] = in[j].value(i);
        st_chunk_q8<VEC>(q, row, base, cols, lane, v);
      });
}

template <int DT, int VEC>
__global__ void __launch_bounds__(kBlock) k_q8_load(const __grid_constant__ Q8 q,
                                                    const __grid_constant__ Mat x, uint32_t cols,
                                                    const __grid_constant__ ChunkRange r) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  RawQ8<VEC> in[kAhead];
  for_chunks<VEC, kAhead>(
      r, [&](int j, uint64_t row, uint32_t base) { in[j].load(q, row, base, cols, lane); },
      [&](int j, uint64_t row, uint32_t base) {
        float v[lane_vals(VEC)];
        in[j].values(v);
        st_chunk<DT, VEC>(row_at<DT>(x, row), base, cols, lane, v);
      });
}

// What rounding v to bf16 leaves; nothing where the rounded value is not finite.
__device__ __forceinline__ float bf16_rest(float v) {
  const float hi = ffn_bf16((uint16_t)ffn_bf16x2(v, 0.0f));
  return fabsf(hi) <= kFloatMax ? v - hi : 0.0f;
}

// The values of q's chunks as hi + lo.
template <int VEC>
__device__ __forceinline__ void split_chunks(const SplitArgs& a, const ChunkRange& r) {
  const int lane = threadIdx.x & 31;
  RawQ8<VEC> in[1];
  for_chunks<VEC, 1>(
      r, [&](int j, uint64_t row, uint32_t base) { in[j].load(a.q, row, base, a.cols, lane); },
      [&](int j, uint64_t row, uint32_t base) {
        float v[lane_vals(VEC)], rest[lane_vals(VEC)];
        in[j].values(v);
#pragma unroll
        for (int i = 0; i < lane_vals(VEC); ++i) rest[i] = bf16_rest(v[i]);
        st_chunk<CR_BF16, VEC>(row_at<CR_BF16>(a.hi, row), base, a.cols, lane, v);
        st_chunk<CR_BF16, VEC>(row_at<CR_BF16>(a.lo, row), base, a.cols, lane, rest);
      });
}

// 8 bf16 at p, which is 2-byte aligned, the first `n` of them in bounds: the
// one or two 16-byte granules that hold them, shifted.  A granule is read only
// if it holds an element that is in bounds.
__device__ __forceinline__ void ld_shifted(const uint16_t* p, int n, uint4* lo, uint4* hi) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const uint4* g = reinterpret_cast<const uint4*>(at & ~(uintptr_t)15);
  *lo = n > 0 ? g[0] : make_uint4(0, 0, 0, 0);
  *hi = (int)(at & 15) + 2 * n > 16 ? g[1] : make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ uint4 shifted(const uint4& lo, const uint4& hi, uint32_t bytes) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = bytes & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = bytes & 4 ? w[i + 1] : w[i];
  const uint32_t bits = (bytes & 2) * 8;
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// blockIdx.y: which copy.  Rows of dst start on 16-byte boundaries, so a lane
// writes 8 columns at once and reads them as shifted granules: with 2-byte
// loads and stores the three operands of 1531 x 1001 x 2731 took 11 us.
__global__ void __launch_bounds__(kBlock) k_copy_bf16(const __grid_constant__ CopyBf16 c) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const CopyBf16::One& m = c.one[blockIdx.y];
  uint4 lo[kAhead], hi[kAhead];
  for_chunks<0, kAhead>(
      ChunkRange{m.chunks, m.per_row},
      [&](int j, uint64_t row, uint32_t base) {
        const uint32_t col = base + 8 * lane;
        const int n = col < m.cols ? (int)min(m.cols - col, 8u) : 0;
        ld_shifted(reinterpret_cast<const uint16_t*>(row_at<CR_BF16>(m.src, row)) + col, n, &lo[j], &hi[j]);
      },
      [&](int j, uint64_t row, uint32_t base) {
        const uint32_t col = base + 8 * lane;
        if (col >= m.cols) return;
        const uintptr_t src = reinterpret_cast<uintptr_t>(row_at<CR_BF16>(m.src, row));
        const uint4 v = shifted(lo[j], hi[j], (uint32_t)((src + 2 * col) & 15));
        // columns past the row's end are the row's padding
        *reinterpret_cast<uint4*>(row_at<CR_BF16>(m.dst, row) + 2 * col) = v;
      });
}

// blockIdx.y 1: x's checkpoint, split for the products that follow.  REST: dg_lo
// and du_lo are wanted too.
template <int ACT, int VEC, bool REST>
__global__ void __launch_bounds__(kBlock, 4) k_act_back(const __grid_constant__ ActBackArgs a,
                                                        const __grid_constant__ ChunkRange r,
                                                        const __grid_constant__ SplitArgs x,
                                                        const __grid_constant__ ChunkRange xr) {
  pdl_enter();
  if (blockIdx.y) return x.vec ? split_chunks<1>(x, xr) : split_chunks<0>(x, xr);
  const int lane = threadIdx.x & 31;
  Raw<CR_BF16, VEC> in[1];
  RawQ8<VEC> gate[1], up[1];
  for_chunks<VEC, 1>(
      r,
      [&](int j, uint64_t row, uint32_t base) {
        in[j].load(row_at<CR_BF16>(a.da, row), base, a.cols, lane);
        gate[j].load(a.g8, row, base, a.cols, lane);
        up[j].load(a.u8, row, base, a.cols, lane);
      },
      [&](int j, uint64_t row, uint32_t base) {
        float g[lane_vals(VEC)], u[lane_vals(VEC)], dg[lane_vals(VEC)], du[lane_vals(VEC)];
        gate[j].values(g);
        up[j].values(u);
#pragma unroll
        for (int i = 0; i < lane_vals(VEC); ++i) {
          const float da = in[j].value(i);
          const float2 v = act_gate_slope<ACT>(g[i]);
          dg[i] = da * u[i] * v.y;
          du[i] = da * v.x;
          u[i] *= v.x;
        }
        if (a.dg.p) st_chunk<CR_BF16, VEC>(row_at<CR_BF16>(a.dg, row), base, a.cols, lane, dg);
        if (a.du.p) st_chunk<CR_BF16, VEC>(row_at<CR_BF16>(a.du, row), base, a.cols, lane, du);
        if (a.a.p) st_chunk<CR_BF16, VEC>(row_at<CR_BF16>(a.a, row), base, a.cols, lane, u);
        if constexpr (REST) {
#pragma unroll
          for (int i = 0; i < lane_vals(VEC); ++i) dg[i] = bf16_rest(dg[i]), du[i] = bf16_rest(du[i]);
          st_chunk<CR_BF16, VEC>(row_at<CR_BF16>(a.dg_lo, row), base, a.cols, lane, dg);
          st_chunk<CR_BF16, VEC>(row_at<CR_BF16>(a.du_lo, row), base, a.cols, lane, du);
        }
      });
}

// A warp for every `ahead` chunks.
dim3 chunk_grid(const ChunkRange& r, int ahead) {
  return dim3(flat_grid((r.chunks + ahead - 1) / ahead * 32));
}

}  // namespace

// f(integral constant) for the access width.
template <typename F>
cudaError_t with_vec(int vec, F f) {
  switch (vec) {
    case 2: return f(std::integral_constant<int, 2>());
    case 1: return f(std::integral_constant<int, 1>());
    default: return f(std::integral_constant<int, 0>());
  }
}

cudaError_t launch_q8_store(cr_dtype d, const Mat& x, const Q8& q, uint64_t rows, uint32_t cols,
                            int vec, cudaStream_t s) {
  const ChunkRange r = chunk_range(rows, cols, vec);
  return with_vec(vec, [&](auto v) {
    return launch_pdl(d == CR_BF16 ? k_q8_store<CR_BF16, v()> : k_q8_store<CR_F32, v()>,
                      chunk_grid(r, kAhead), kBlock, s, x, q, cols, r);
  });
}

cudaError_t launch_q8_load(cr_dtype d, const Q8& q, const Mat& x, uint64_t rows, uint32_t cols,
                           int vec, cudaStream_t s) {
  const ChunkRange r = chunk_range(rows, cols, vec);
  return with_vec(vec, [&](auto v) {
    return launch_pdl(d == CR_BF16 ? k_q8_load<CR_BF16, v()> : k_q8_load<CR_F32, v()>,
                      chunk_grid(r, kAhead), kBlock, s, q, x, cols, r);
  });
}

void add_copy(CopyBf16* c, const Mat& src, const Mat& dst, uint64_t rows, uint32_t cols) {
  const ChunkRange r = chunk_range(rows, cols, 0);
  c->one[c->n++] = CopyBf16::One{src, dst, r.chunks, r.per_row, cols};
}

cudaError_t launch_copy_bf16(const CopyBf16& c, cudaStream_t s) {
  if (c.n == 0) return cudaSuccess;
  uint64_t most = 0;
  for (int k = 0; k < c.n; ++k) most = c.one[k].chunks > most ? c.one[k].chunks : most;
  dim3 grid = chunk_grid(ChunkRange{most, FastDiv{}}, 2);
  grid.y = c.n;
  return launch_pdl(k_copy_bf16, grid, kBlock, s, c);
}

cudaError_t launch_act_back(cr_act act, const ActBackArgs& a, const SplitArgs* x, int vec,
                            cudaStream_t s) {
  const ChunkRange r = chunk_range(a.rows, a.cols, vec);
  const ChunkRange xr = x ? chunk_range(x->rows, x->cols, x->vec) : ChunkRange{};
  dim3 grid = chunk_grid(ChunkRange{std::max(r.chunks, xr.chunks), FastDiv{}}, 1);
  grid.y = x ? 2 : 1;
  return with_vec(vec, [&](auto v) {
    const bool silu = act == CR_ACT_SILU;
    const auto kernel = a.dg_lo.p ? silu ? k_act_back<CR_ACT_SILU, v(), true> : k_act_back<CR_ACT_GELU, v(), true>
                                  : silu ? k_act_back<CR_ACT_SILU, v(), false> : k_act_back<CR_ACT_GELU, v(), false>;
    return launch_pdl(kernel, grid, kBlock, s, a, r, x ? *x : SplitArgs{}, xr);
  });
}

}  // namespace cr
