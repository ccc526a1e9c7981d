// k_glu_few.cu -- the gated block for a few tokens (generation): every weight
// is read once and used once per token, so the call is bound by the weights'
// bytes and by how many of them are in flight.
//
// A warp takes one hidden unit at a time: rows f of Wg and of Wu, streamed in
// 256-column chunks, kDeep of each in flight, against the tokens' x in shared
// memory.  Sums stay in fp32 registers and meet in a shuffle reduction.
#include <algorithm>

#include "ffn_internal.cuh"
#include "pdl.cuh"

namespace cr {

namespace {

constexpr int kDeep = 4;  // chunks of each weight row loaded before the first is used

template <int T, bool VEC>
__device__ __forceinline__ void add_chunk(const Raw<CR_BF16, VEC>& g, const Raw<CR_BF16, VEC>& u,
                                          const uint16_t* x, uint32_t pitch, uint32_t base,
                                          int lane, float* ag, float* au) {
#pragma unroll
  for (int t = 0; t < T; ++t) {
    Raw<CR_BF16, VEC> v;
    if constexpr (VEC) {
      const uint4 q = *reinterpret_cast<const uint4*>(x + t * pitch + base + lane * kLaneVals);
      v.w[0] = q.x, v.w[1] = q.y, v.w[2] = q.z, v.w[3] = q.w;
    } else {
#pragma unroll
      for (int i = 0; i < kLaneVals; ++i)
        v.w[i] = (uint32_t)x[t * pitch + chunk_col<false>(base, lane, i)] << 16;
    }
#pragma unroll
    for (int i = 0; i < kLaneVals; ++i) {
      ag[t] = fmaf(g.value(i), v.value(i), ag[t]);
      au[t] = fmaf(u.value(i), v.value(i), au[t]);
    }
  }
}

// x in shared memory is zero past dim, up to `pitch`, a multiple of kChunk.
template <int ACT, int T, bool VEC>
__global__ void __launch_bounds__(kBlock) k_glu_few(const __grid_constant__ GluArgs a,
                                                    uint32_t pitch) {
  extern __shared__ uint16_t x[];
  pdl_enter();
  // a warp a chunk, all of them loaded before the first is stored
  for (uint32_t k = threadIdx.x >> 5; k < T * (pitch / kChunk); k += kBlock / 32) {
    const uint32_t t = k / (pitch / kChunk), base = (k - t * (pitch / kChunk)) * kChunk;
    Raw<CR_BF16, false> r;
    r.clear();
    if (t < a.tokens)
      r.load(static_cast<const uint16_t*>(a.x.p) + t * a.x.ld, base, a.dim, threadIdx.x & 31);
#pragma unroll
    for (int i = 0; i < kLaneVals; ++i)
      x[t * pitch + chunk_col<false>(base, threadIdx.x & 31, i)] = (uint16_t)(r.w[i] >> 16);
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const uint32_t warps = gridDim.x * (kBlock / 32);
  for (uint32_t f = blockIdx.x * (kBlock / 32) + (threadIdx.x >> 5); f < a.ffn; f += warps) {
    const uint16_t* wg = static_cast<const uint16_t*>(a.wg.p) + f * a.wg.ld;
    const uint16_t* wu = static_cast<const uint16_t*>(a.wu.p) + f * a.wu.ld;
    float g[T], u[T];
#pragma unroll
    for (int t = 0; t < T; ++t) g[t] = u[t] = 0.0f;
    for (uint32_t base = 0; base < a.dim; base += kDeep * kChunk) {
      Raw<CR_BF16, VEC> rg[kDeep], ru[kDeep];
#pragma unroll
      for (int j = 0; j < kDeep; ++j) {
        rg[j].load(wg, base + j * kChunk, a.dim, lane);
        ru[j].load(wu, base + j * kChunk, a.dim, lane);
      }
#pragma unroll
      for (int j = 0; j < kDeep; ++j)
        if (base + j * kChunk < a.dim)
          add_chunk<T, VEC>(rg[j], ru[j], x, pitch, base + j * kChunk, lane, g, u);
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        g[t] += __shfl_xor_sync(~0u, g[t], o);
        u[t] += __shfl_xor_sync(~0u, u[t], o);
      }
      if (lane == t && t < a.tokens)
        static_cast<uint16_t*>(a.a.p)[t * a.a.ld + f] =
            (uint16_t)ffn_bf16x2(act_gate<ACT>(g[t]) * u[t], 0.0f);
    }
  }
}

template <int ACT, int T, bool VEC>
cudaError_t run(const GluArgs& a, uint32_t pitch, cudaStream_t s) {
  int full = 0;
  cudaError_t e = persistent_grid(reinterpret_cast<const void*>(k_glu_few<ACT, T, VEC>), ~0ull >> 8, &full);
  if (e != cudaSuccess) return e;
  const uint32_t blocks = (a.ffn + kBlock / 32 - 1) / (kBlock / 32);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(std::min(blocks, (uint32_t)full));
  cfg.blockDim = dim3(kBlock);
  cfg.dynamicSmemBytes = (size_t)T * pitch * 2;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_glu_few<ACT, T, VEC>, a, pitch);
}

template <int ACT, bool VEC>
cudaError_t by_tokens(const GluArgs& a, uint32_t pitch, cudaStream_t s) {
  if (a.tokens == 1) return run<ACT, 1, VEC>(a, pitch, s);
  if (a.tokens == 2) return run<ACT, 2, VEC>(a, pitch, s);
  return run<ACT, 4, VEC>(a, pitch, s);
}

constexpr uint32_t kFewTokens = 4;
constexpr uint32_t kFewSmem = 48 << 10;  // what a block gets without asking

uint32_t pitch_of(uint32_t dim) { return (uint32_t)(((uint64_t)dim + kChunk - 1) / kChunk * kChunk); }

}  // namespace

bool glu_few(uint64_t tokens, uint64_t dim, bool keeps) {
  if (keeps || tokens > kFewTokens || dim > kFewSmem / 2) return false;
  const uint64_t rows = tokens > 2 ? 4 : tokens;
  return rows * pitch_of((uint32_t)dim) * 2 <= kFewSmem;
}

cudaError_t launch_glu_few(cr_act act, const GluArgs& a, bool vec, cudaStream_t s) {
  const uint32_t pitch = pitch_of(a.dim);
  if (act == CR_ACT_SILU)
    return vec ? by_tokens<CR_ACT_SILU, true>(a, pitch, s) : by_tokens<CR_ACT_SILU, false>(a, pitch, s);
  return vec ? by_tokens<CR_ACT_GELU, true>(a, pitch, s) : by_tokens<CR_ACT_GELU, false>(a, pitch, s);
}

}  // namespace cr
