// k_glu.cu -- the gated feed-forward block: both projections, the activation
// and the product in one kernel, and the products of its backward pass.
#include "ffn_internal.cuh"
#include "pdl.cuh"

namespace cr {

namespace {

constexpr int kTile = 64, kTileK = 16;

// acc[i][j] += sum over k of A(m0 + .., k) * B(n0 + .., k), A(m, k) at
// am * m + ak * k; 16 x 16 threads, 4 x 4 outputs each.
__device__ void tile_product(const uint16_t* A, uint64_t am, uint64_t ak, const uint16_t* B,
                             uint64_t bn, uint64_t bk, uint32_t m0, uint32_t n0, uint32_t M,
                             uint32_t N, uint32_t K, float (*sa)[kTile], float (*sb)[kTile],
                             float (&acc)[4][4]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (uint32_t k0 = 0; k0 < K; k0 += kTileK) {
    for (int i = threadIdx.x; i < kTile * kTileK; i += 256) {
      // consecutive threads along the operand's contiguous dimension
      const int r = ak == 1 ? i / kTileK : i % kTile, k = ak == 1 ? i % kTileK : i / kTile;
      sa[k][r] = m0 + r < M && k0 + k < K ? ffn_bf16(A[(m0 + r) * am + (k0 + k) * ak]) : 0.0f;
      const int c = bk == 1 ? i / kTileK : i % kTile, l = bk == 1 ? i % kTileK : i / kTile;
      sb[l][c] = n0 + c < N && k0 + l < K ? ffn_bf16(B[(n0 + c) * bn + (k0 + l) * bk]) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kTileK; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
}

// Block (64 columns of a 128-column group pair of g and u) -- tile
// (blockIdx.x, blockIdx.y) of a; g and u go to shared memory for the 8-bit
// form, whose groups are two tiles wide.
template <int ACT>
__global__ void __launch_bounds__(256) k_glu(const __grid_constant__ GluArgs a) {
  pdl_enter();
  __shared__ float sa[kTileK][kTile], sb[kTileK][kTile];
  __shared__ float tile[16][CR_Q8_GROUP];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const uint32_t n0 = blockIdx.x * CR_Q8_GROUP;
  for (uint32_t m0 = blockIdx.y * kTile; m0 < a.tokens; m0 += gridDim.y * kTile) {
    float g[2][4][4] = {}, u[2][4][4] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      tile_product(static_cast<const uint16_t*>(a.x.p), a.x.ld, 1,
                   static_cast<const uint16_t*>(a.wg.p), a.wg.ld, 1, m0, n0 + h * kTile, a.tokens,
                   a.ffn, a.dim, sa, sb, g[h]);
      tile_product(static_cast<const uint16_t*>(a.x.p), a.x.ld, 1,
                   static_cast<const uint16_t*>(a.wu.p), a.wu.ld, 1, m0, n0 + h * kTile, a.tokens,
                   a.ffn, a.dim, sa, sb, u[h]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t m = m0 + ty * 4 + i, n = n0 + h * kTile + tx * 4 + j;
          if (m < a.tokens && n < a.ffn)
            static_cast<uint16_t*>(a.a.p)[m * a.a.ld + n] =
                (uint16_t)ffn_bf16x2(act_gate<ACT>(g[h][i][j]) * u[h][i][j], 0.0f);
        }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const Q8& q = which ? a.u8 : a.g8;
      if (!q.codes) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            tile[ty][h * kTile + tx * 4 + j] = which ? u[h][i][j] : g[h][i][j];
        __syncthreads();
        const int lane = threadIdx.x & 31;
        for (int r = threadIdx.x >> 5; r < 16; r += 8) {
          const uint32_t m = m0 + r * 4 + i;
          if (m >= a.tokens) continue;
          float v[kLaneVals] = {0.0f};
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = tile[r][k * 32 + lane];
          // columns past this group are another block's
          const uint32_t end = n0 + CR_Q8_GROUP < a.ffn ? n0 + CR_Q8_GROUP : a.ffn;
          st_chunk_q8<false>(q, m, n0, end, lane, v);
        }
      }
    }
    __syncthreads();
  }
}

// out = A1 B1 (+ A2 B2), the operands' strides as tile_product takes them.
struct Product {
  const uint16_t *A1, *B1, *A2, *B2;
  uint64_t am, ak, bn, bk, bk2;
  uint32_t M, N, K;
  Mat out;
};

template <int DT>
__global__ void __launch_bounds__(256) k_product(const __grid_constant__ Product p) {
  pdl_enter();
  __shared__ float sa[kTileK][kTile], sb[kTileK][kTile];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const uint32_t n0 = blockIdx.x * kTile;
  for (uint32_t m0 = blockIdx.y * kTile; m0 < p.M; m0 += gridDim.y * kTile) {
    float acc[4][4] = {};
    tile_product(p.A1, p.am, p.ak, p.B1, p.bn, p.bk, m0, n0, p.M, p.N, p.K, sa, sb, acc);
    if (p.A2) tile_product(p.A2, p.am, p.ak, p.B2, p.bn, p.bk2, m0, n0, p.M, p.N, p.K, sa, sb, acc);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
        if (m >= p.M || n >= p.N) continue;
        if constexpr (DT == CR_BF16)
          static_cast<uint16_t*>(p.out.p)[m * p.out.ld + n] = (uint16_t)ffn_bf16x2(acc[i][j], 0.0f);
        else
          static_cast<float*>(p.out.p)[m * p.out.ld + n] = acc[i][j];
      }
  }
}

dim3 tiles(uint32_t cols, uint32_t width, uint32_t rows) {
  const uint64_t y = ((uint64_t)rows + kTile - 1) / kTile;
  return dim3((unsigned)(((uint64_t)cols + width - 1) / width), (unsigned)(y < 65535 ? y : 65535));
}

cudaError_t product(cr_dtype out, const Product& p, cudaStream_t s) {
  const dim3 grid = tiles(p.N, kTile, p.M);
  return out == CR_BF16 ? launch_pdl(k_product<CR_BF16>, grid, 256, s, p)
                        : launch_pdl(k_product<CR_F32>, grid, 256, s, p);
}

}  // namespace

cudaError_t launch_glu(cr_act act, const GluArgs& a, cudaStream_t s) {
  const dim3 grid = tiles(a.ffn, CR_Q8_GROUP, a.tokens);
  return act == CR_ACT_SILU ? launch_pdl(k_glu<CR_ACT_SILU>, grid, 256, s, a)
                            : launch_pdl(k_glu<CR_ACT_GELU>, grid, 256, s, a);
}

cudaError_t launch_glu_back(cr_dtype dw, const GluBackArgs& a, cudaStream_t s) {
  const uint16_t *dg = static_cast<const uint16_t*>(a.dg.p), *du = static_cast<const uint16_t*>(a.du.p),
                 *x = static_cast<const uint16_t*>(a.x.p), *wg = static_cast<const uint16_t*>(a.wg.p),
                 *wu = static_cast<const uint16_t*>(a.wu.p);
  if (a.dx.p) {
    Product p = {dg, wg, du, wu, a.dg.ld, 1, 1, a.wg.ld, a.wu.ld, a.tokens, a.dim, a.ffn, a.dx};
    cudaError_t e = product(CR_BF16, p, s);
    if (e != cudaSuccess) return e;
  }
  for (int k = 0; k < 2; ++k) {
    void* out = k ? a.dwu : a.dwg;
    if (!out) continue;
    Product p = {k ? du : dg, x, nullptr, nullptr, 1, a.dg.ld, 1, a.x.ld, a.x.ld, a.ffn, a.dim, a.tokens,
                 Mat{out, a.dim}};
    cudaError_t e = product(dw, p, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace cr
