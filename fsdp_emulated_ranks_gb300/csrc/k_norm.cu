// k_norm.cu -- RMS norm with the residual's addition and an 8-bit output,
// and its backward pass.
//
// Forward, per row of h = x + residual:  v = h * rstd * weight with
// rstd = 1/sqrt(mean h^2 + eps).  A row is held in registers between its one
// read and its writes: warps x chunks of 256 columns (V chunks a warp), the
// sum of squares reduced by shuffles and, across the row's warps, through
// shared memory.  Rows too wide for that (V = 0) are read twice; the second
// read comes from L2.
//
// Backward, per row with n = h * rstd and c = mean(dy * weight * n):
// dx = rstd * (dy * weight - n * c) + dres.  dweight sums dy * n down the
// columns: a block keeps the sums of its columns in registers over all the
// rows it takes (persistent grid) and writes one partial row; a second
// kernel adds the partials in order.  Wide rows take a second pass over dy
// and h for dweight.
#include <algorithm>

#include "ffn_internal.cuh"
#include "pdl.cuh"

namespace cr {

namespace {

constexpr int kRowThreads = 256;        // threads of a block that holds rows in registers
constexpr int kWideThreads = 1024;      // threads of a block on a wide row
constexpr uint32_t kWideFrom = 8192;    // columns above which a row is wide: 8 warps x 4 chunks
constexpr int kMaxWarps = kWideThreads / 32;

// Sum over the row's warps (blockDim.x / 32 of them, row threadIdx.y of the
// block).  `buf` alternates between two halves of `part`, so one barrier a
// call is enough.
__device__ __forceinline__ float row_sum(float s, float (*part)[kMaxWarps], int buf) {
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return s;
  float* p = part[buf];
  const int w0 = threadIdx.y * nw;
  if ((threadIdx.x & 31) == 0) p[w0 + (threadIdx.x >> 5)] = s;
  __syncthreads();
  s = 0.0f;
  for (int w = 0; w < nw; ++w) s += p[w0 + w];
  return s;
}

template <int DT, bool VEC>
__device__ __forceinline__ void norm_ld(const NormArgs& a, uint64_t row, uint32_t base, int lane,
                                        float* h) {
  constexpr int es = DT == CR_BF16 ? 2 : 4;
  ld_chunk<DT, VEC>(static_cast<const char*>(a.x.p) + row * a.x.ld * es, base, a.cols, lane, h);
  if (a.residual.p) {
    float r[kLaneVals];
    ld_chunk<DT, VEC>(static_cast<const char*>(a.residual.p) + row * a.residual.ld * es, base,
                      a.cols, lane, r);
#pragma unroll
    for (int i = 0; i < kLaneVals; ++i) h[i] += r[i];
  }
}

template <int DT, bool VEC>
__device__ __forceinline__ void norm_st(const NormArgs& a, uint64_t row, uint32_t base, int lane,
                                        float* h, float rstd) {
  constexpr int es = DT == CR_BF16 ? 2 : 4;
  if (a.sum.p)
    st_chunk<DT, VEC>(static_cast<char*>(a.sum.p) + row * a.sum.ld * es, base, a.cols, lane, h);
  float w[kLaneVals];
  ld_chunk<DT, VEC>(a.weight, base, a.cols, lane, w);
#pragma unroll
  for (int i = 0; i < kLaneVals; ++i) h[i] = h[i] * rstd * w[i];
  if (a.y.p)
    st_chunk<DT, VEC>(static_cast<char*>(a.y.p) + row * a.y.ld * es, base, a.cols, lane, h);
  if (a.y8.codes) st_chunk_q8<VEC>(a.y8, row, base, a.cols, lane, h);
}

// Block (32 * warps per row, rows per block).
template <int DT, int V, bool VEC>
__global__ void __launch_bounds__(V ? kRowThreads : kWideThreads)
    k_rms_norm(const __grid_constant__ NormArgs a) {
  pdl_enter();
  __shared__ float part[2][kMaxWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const uint64_t step = (uint64_t)gridDim.x * blockDim.y;
  int buf = 0;
  // every row of a block's iteration takes part in the barriers
  for (uint64_t first = (uint64_t)blockIdx.x * blockDim.y; first < a.rows; first += step) {
    const uint64_t row = first + threadIdx.y;
    const bool live = row < a.rows;
    float s = 0.0f;
    if constexpr (V > 0) {
      float h[V][kLaneVals];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const uint32_t base = (uint32_t)(warp + k * nw) * kChunk;
#pragma unroll
        for (int i = 0; i < kLaneVals; ++i) h[k][i] = 0.0f;
        if (live && base < a.cols) norm_ld<DT, VEC>(a, row, base, lane, h[k]);
      }
#pragma unroll
      for (int k = 0; k < V; ++k)
#pragma unroll
        for (int i = 0; i < kLaneVals; ++i) s = fmaf(h[k][i], h[k][i], s);
      const float rstd = 1.0f / sqrtf(row_sum(s, part, buf) * a.inv_cols + a.eps);
      if (live) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const uint32_t base = (uint32_t)(warp + k * nw) * kChunk;
          if (base < a.cols) norm_st<DT, VEC>(a, row, base, lane, h[k], rstd);
        }
        if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
      }
    } else {
      float h[kLaneVals];
      if (live)
        for (uint64_t base = (uint64_t)warp * kChunk; base < a.cols; base += (uint64_t)nw * kChunk) {
          norm_ld<DT, VEC>(a, row, (uint32_t)base, lane, h);
#pragma unroll
          for (int i = 0; i < kLaneVals; ++i) s = fmaf(h[i], h[i], s);
        }
      const float rstd = 1.0f / sqrtf(row_sum(s, part, buf) * a.inv_cols + a.eps);
      if (live) {
        for (uint64_t base = (uint64_t)warp * kChunk; base < a.cols; base += (uint64_t)nw * kChunk) {
          norm_ld<DT, VEC>(a, row, (uint32_t)base, lane, h);
          norm_st<DT, VEC>(a, row, (uint32_t)base, lane, h, rstd);
        }
        if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
      }
    }
    buf ^= 1;
  }
}

// ---- backward -----------------------------------------------------------------------

template <int DT, bool VEC>
__device__ __forceinline__ void back_ld(const NormBackArgs& a, uint64_t row, uint32_t base,
                                        int lane, float* dy, float* h) {
  constexpr int es = DT == CR_BF16 ? 2 : 4;
  ld_chunk<DT, VEC>(static_cast<const char*>(a.dy.p) + row * a.dy.ld * es, base, a.cols, lane, dy);
  if (a.h8.codes)
    ld_chunk_q8<VEC>(a.h8, row, base, a.cols, lane, h);
  else
    ld_chunk<DT, VEC>(static_cast<const char*>(a.h.p) + row * a.h.ld * es, base, a.cols, lane, h);
}

// t = dy * weight in, dx out.
template <int DT, bool VEC>
__device__ __forceinline__ void back_st(const NormBackArgs& a, uint64_t row, uint32_t base,
                                        int lane, const float* t, const float* n, float rstd,
                                        float c) {
  constexpr int es = DT == CR_BF16 ? 2 : 4;
  float dx[kLaneVals];
#pragma unroll
  for (int i = 0; i < kLaneVals; ++i) dx[i] = rstd * (t[i] - n[i] * c);
  if (a.dres.p) {
    float r[kLaneVals];
    ld_chunk<DT, VEC>(static_cast<const char*>(a.dres.p) + row * a.dres.ld * es, base, a.cols,
                      lane, r);
#pragma unroll
    for (int i = 0; i < kLaneVals; ++i) dx[i] += r[i];
  }
  st_chunk<DT, VEC>(static_cast<char*>(a.dx.p) + row * a.dx.ld * es, base, a.cols, lane, dx);
}

// Rows of at most kWideFrom columns: block (32 * warps per row, 1), rows
// blockIdx.x, + gridDim.x, ...; partial row blockIdx.x of dweight.
template <int DT, int V, bool VEC>
__global__ void __launch_bounds__(kRowThreads)
    k_rms_norm_back(const __grid_constant__ NormBackArgs a) {
  pdl_enter();
  __shared__ float part[2][kMaxWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  float dw[V][kLaneVals];
#pragma unroll
  for (int k = 0; k < V; ++k)
#pragma unroll
    for (int i = 0; i < kLaneVals; ++i) dw[k][i] = 0.0f;
  int buf = 0;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x, buf ^= 1) {
    const float rstd = a.rstd[row];
    float t[V][kLaneVals], n[V][kLaneVals], s = 0.0f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const uint32_t base = (uint32_t)(warp + k * nw) * kChunk;
      if (base < a.cols) {
        back_ld<DT, VEC>(a, row, base, lane, t[k], n[k]);
      } else {
#pragma unroll
        for (int i = 0; i < kLaneVals; ++i) t[k][i] = n[k][i] = 0.0f;
      }
    }
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const uint32_t base = (uint32_t)(warp + k * nw) * kChunk;
      float w[kLaneVals];
      if (base < a.cols) {
        ld_chunk<DT, VEC>(a.weight, base, a.cols, lane, w);
#pragma unroll
        for (int i = 0; i < kLaneVals; ++i) {
          n[k][i] *= rstd;
          dw[k][i] = fmaf(t[k][i], n[k][i], dw[k][i]);
          t[k][i] *= w[i];
          s = fmaf(t[k][i], n[k][i], s);
        }
      }
    }
    if (a.dx.p) {
      const float c = row_sum(s, part, buf) * a.inv_cols;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const uint32_t base = (uint32_t)(warp + k * nw) * kChunk;
        if (base < a.cols) back_st<DT, VEC>(a, row, base, lane, t[k], n[k], rstd, c);
      }
    }
  }
  if (a.partial) {
    float* p = a.partial + (uint64_t)blockIdx.x * a.cols;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const uint32_t base = (uint32_t)(warp + k * nw) * kChunk;
#pragma unroll
      for (int i = 0; i < kLaneVals; ++i) {
        const uint32_t c = chunk_col<VEC>(base, lane, i);
        if (c < a.cols) p[c] = dw[k][i];
      }
    }
  }
}

// Wide rows, dx: one block a row, read twice.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kWideThreads)
    k_rms_norm_back_wide(const __grid_constant__ NormBackArgs a) {
  pdl_enter();
  __shared__ float part[2][kMaxWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int buf = 0;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x, buf ^= 1) {
    const float rstd = a.rstd[row];
    float t[kLaneVals], n[kLaneVals], w[kLaneVals], s = 0.0f;
    for (uint64_t base = (uint64_t)warp * kChunk; base < a.cols; base += (uint64_t)nw * kChunk) {
      back_ld<DT, VEC>(a, row, (uint32_t)base, lane, t, n);
      ld_chunk<DT, VEC>(a.weight, (uint32_t)base, a.cols, lane, w);
#pragma unroll
      for (int i = 0; i < kLaneVals; ++i) s = fmaf(t[i] * w[i], n[i] * rstd, s);
    }
    const float c = row_sum(s, part, buf) * a.inv_cols;
    for (uint64_t base = (uint64_t)warp * kChunk; base < a.cols; base += (uint64_t)nw * kChunk) {
      back_ld<DT, VEC>(a, row, (uint32_t)base, lane, t, n);
      ld_chunk<DT, VEC>(a.weight, (uint32_t)base, a.cols, lane, w);
#pragma unroll
      for (int i = 0; i < kLaneVals; ++i) t[i] *= w[i], n[i] *= rstd;
      back_st<DT, VEC>(a, row, (uint32_t)base, lane, t, n, rstd, c);
    }
  }
}

// Wide rows, dweight partials: warp (blockIdx.x, warp) takes one chunk of
// columns, blockIdx.y every gridDim.y-th row.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kRowThreads)
    k_rms_norm_back_wide_dw(const __grid_constant__ NormBackArgs a) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const uint64_t base = ((uint64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5)) * kChunk;
  if (base >= a.cols) return;
  float dw[kLaneVals] = {0.0f};
  for (uint64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    float dy[kLaneVals], h[kLaneVals];
    back_ld<DT, VEC>(a, row, (uint32_t)base, lane, dy, h);
    const float rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < kLaneVals; ++i) dw[i] = fmaf(dy[i], h[i] * rstd, dw[i]);
  }
  float* p = a.partial + (uint64_t)blockIdx.y * a.cols;
#pragma unroll
  for (int i = 0; i < kLaneVals; ++i) {
    const uint32_t c = chunk_col<VEC>((uint32_t)base, lane, i);
    if (c < a.cols) p[c] = dw[i];
  }
}

// dweight = sum of the partial rows: block (32 columns, 8 row classes), each
// class in order, then the classes in order.
template <int DW>
__global__ void __launch_bounds__(256) k_norm_dw(const float* partial, uint32_t parts,
                                                 uint32_t cols, void* dweight) {
  pdl_enter();
  __shared__ float sum[8][32];
  const uint64_t c = (uint64_t)blockIdx.x * 32 + threadIdx.x;
  float s = 0.0f;
  if (c < cols)
    for (uint32_t k = threadIdx.y; k < parts; k += 8) s += partial[(uint64_t)k * cols + c];
  sum[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < cols) {
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += sum[k][threadIdx.x];
    if constexpr (DW == CR_BF16)
      static_cast<uint16_t*>(dweight)[c] = (uint16_t)ffn_bf16x2(s, 0.0f);
    else
      static_cast<float*>(dweight)[c] = s;
  }
}

struct RowShape {
  int v;          // chunks per warp; 0: wide
  unsigned warps;  // per row
  unsigned rows;   // per block
};

// One chunk a warp up to 8 warps, then 2 and 4 chunks; wide rows 32 warps.
RowShape row_shape(uint32_t cols) {
  const uint32_t chunks = (uint32_t)(((uint64_t)cols + kChunk - 1) / kChunk);
  if (cols > kWideFrom) return {0, kMaxWarps, 1};
  const int v = chunks <= 8 ? 1 : chunks <= 16 ? 2 : 4;
  const unsigned warps = (chunks + v - 1) / v;
  return {v, warps, (kRowThreads / 32) / warps};
}

template <typename... KArgs, typename... Args>
cudaError_t launch2(void (*kernel)(KArgs...), dim3 grid, dim3 block, cudaStream_t s,
                    Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int DT, bool VEC>
cudaError_t norm_dispatch(const NormArgs& a, cudaStream_t s) {
  const RowShape r = row_shape(a.cols);
  uint64_t g = (a.rows + r.rows - 1) / r.rows;
  if (g > (1u << 30)) g = 1u << 30;
  const dim3 grid((unsigned)g), block(r.warps * 32, r.rows);
  switch (r.v) {
    case 1: return launch2(k_rms_norm<DT, 1, VEC>, grid, block, s, a);
    case 2: return launch2(k_rms_norm<DT, 2, VEC>, grid, block, s, a);
    case 4: return launch2(k_rms_norm<DT, 4, VEC>, grid, block, s, a);
    default: return launch2(k_rms_norm<DT, 0, VEC>, grid, block, s, a);
  }
}

template <int DT, bool VEC>
cudaError_t back_dispatch(const NormBackArgs& a, cudaStream_t s) {
  const RowShape r = row_shape(a.cols);
  const dim3 grid(a.parts), block(r.warps * 32);
  switch (r.v) {
    case 1: return launch2(k_rms_norm_back<DT, 1, VEC>, grid, block, s, a);
    case 2: return launch2(k_rms_norm_back<DT, 2, VEC>, grid, block, s, a);
    case 4: return launch2(k_rms_norm_back<DT, 4, VEC>, grid, block, s, a);
    default: break;
  }
  // dweight first: dx may be written over dy or h
  if (a.partial) {
    const unsigned gx = (a.cols / kChunk + 1 + kRowThreads / 32 - 1) / (kRowThreads / 32);
    cudaError_t e = launch2(k_rms_norm_back_wide_dw<DT, VEC>, dim3(gx, a.parts), dim3(kRowThreads),
                            s, a);
    if (e != cudaSuccess || !a.dx.p) return e;
  }
  const unsigned g = (unsigned)std::min<uint64_t>(a.rows, 1u << 30);
  return launch2(k_rms_norm_back_wide<DT, VEC>, dim3(g), block, s, a);
}

}  // namespace

cudaError_t launch_rms_norm(cr_dtype d, const NormArgs& a, bool vec, cudaStream_t s) {
  if (d == CR_BF16) return vec ? norm_dispatch<CR_BF16, true>(a, s) : norm_dispatch<CR_BF16, false>(a, s);
  return vec ? norm_dispatch<CR_F32, true>(a, s) : norm_dispatch<CR_F32, false>(a, s);
}

uint32_t norm_back_parts(uint64_t rows, uint32_t cols) {
  const uint32_t most = cols > kWideFrom ? 64 : 608;  // 4 blocks on each of 152 SMs
  return (uint32_t)std::min<uint64_t>(rows ? rows : 1, most);
}

cudaError_t launch_rms_norm_back(cr_dtype d, cr_dtype dw, const NormBackArgs& a, bool vec,
                                 cudaStream_t s) {
  cudaError_t e;
  if (d == CR_BF16)
    e = vec ? back_dispatch<CR_BF16, true>(a, s) : back_dispatch<CR_BF16, false>(a, s);
  else
    e = vec ? back_dispatch<CR_F32, true>(a, s) : back_dispatch<CR_F32, false>(a, s);
  if (e != cudaSuccess || !a.partial) return e;
  const dim3 grid((a.cols + 31) / 32), block(32, 8);
  if (dw == CR_BF16)
    return launch2(k_norm_dw<CR_BF16>, grid, block, s, (const float*)a.partial, a.parts, a.cols, a.dweight);
  return launch2(k_norm_dw<CR_F32>, grid, block, s, (const float*)a.partial, a.parts, a.cols, a.dweight);
}

}  // namespace cr
