// k_glu_few.cu -- the gated block for a few tokens (generation): every weight
// is read once and used once per token, so the call is bound by the weights'
// bytes and by how many of them are in flight.
//
// A warp takes one hidden unit at a time: rows f of Wg and of Wu, streamed in
// chunks (ffn_internal.cuh), kDeep of each in flight, against the tokens' x in shared
// memory.  Sums stay in fp32 registers and meet in a shuffle reduction.
//
// Measured, one token of 2048 x 8192 (67 MB of weights): 12.6 us a call, 5.3
// TB/s with the call's start and end in it; the floor is 9.9.  Two blocks an SM
// of as many warps as divide the hidden units evenly: 9 there, three units a
// warp (8 warps left the fourth turn a third full: 13.1 us).
#include <algorithm>

#include "ffn_internal.cuh"
#include "pdl.cuh"

namespace cr {

namespace {

constexpr int kMaxThreads = 320;  // of a block; two blocks an SM
constexpr int kDeep = 4;  // chunks of each weight row loaded before the first is used

template <int T, int VEC>
__device__ __forceinline__ void add_chunk(const Raw<CR_BF16, VEC>& g, const Raw<CR_BF16, VEC>& u,
                                          const uint16_t* x, uint32_t pitch, uint32_t base,
                                          int lane, float* ag, float* au) {
#pragma unroll
  for (int t = 0; t < T; ++t) {
    Raw<CR_BF16, VEC> v;
    if constexpr (VEC) {
      const uint4* p = reinterpret_cast<const uint4*>(x + t * pitch + base + lane * lane_vals(VEC));
      const uint4 q = p[0], r = p[1];
      v.w[0] = q.x, v.w[1] = q.y, v.w[2] = q.z, v.w[3] = q.w;
      v.w[4] = r.x, v.w[5] = r.y, v.w[6] = r.z, v.w[7] = r.w;
    } else {
#pragma unroll
      for (int i = 0; i < lane_vals(VEC); ++i)
        v.w[i] = (uint32_t)x[t * pitch + chunk_col<0>(base, lane, i)] << 16;
    }
#pragma unroll
    for (int i = 0; i < lane_vals(VEC); ++i) {
      ag[t] = fmaf(g.value(i), v.value(i), ag[t]);
      au[t] = fmaf(u.value(i), v.value(i), au[t]);
    }
  }
}

// x in shared memory is zero past dim, up to `pitch`, a multiple of any chunk.
template <int ACT, int T, int VEC>
__global__ void __launch_bounds__(kMaxThreads, 2) k_glu_few(const __grid_constant__ GluArgs a,
                                                    uint32_t pitch) {
  extern __shared__ __align__(16) uint16_t x[];
  pdl_enter();
  // a warp a chunk, all of them loaded before the first is stored
  const uint32_t per = pitch / chunk_cols(0);
  for (uint32_t k = threadIdx.x >> 5; k < T * per; k += blockDim.x / 32) {
    const uint32_t t = k / per, base = (k - t * per) * chunk_cols(0);
    Raw<CR_BF16, 0> r;
    r.clear();
    if (t < a.tokens)
      r.load(static_cast<const uint16_t*>(a.x.p) + t * a.x.ld, base, a.dim, threadIdx.x & 31);
#pragma unroll
    for (int i = 0; i < lane_vals(0); ++i)
      x[t * pitch + chunk_col<0>(base, threadIdx.x & 31, i)] = (uint16_t)(r.w[i] >> 16);
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const uint32_t warps = gridDim.x * (blockDim.x / 32);
  for (uint32_t f = blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5); f < a.ffn; f += warps) {
    const uint16_t* wg = static_cast<const uint16_t*>(a.wg.p) + f * a.wg.ld;
    const uint16_t* wu = static_cast<const uint16_t*>(a.wu.p) + f * a.wu.ld;
    float g[T], u[T];
#pragma unroll
    for (int t = 0; t < T; ++t) g[t] = u[t] = 0.0f;
    for (uint32_t base = 0; base < a.dim; base += kDeep * chunk_cols(VEC)) {
      Raw<CR_BF16, VEC> rg[kDeep], ru[kDeep];
#pragma unroll
      for (int j = 0; j < kDeep; ++j) {
        rg[j].load(wg, base + j * chunk_cols(VEC), a.dim, lane);
        ru[j].load(wu, base + j * chunk_cols(VEC), a.dim, lane);
      }
#pragma unroll
      for (int j = 0; j < kDeep; ++j)
        if (base + j * chunk_cols(VEC) < a.dim)
          add_chunk<T, VEC>(rg[j], ru[j], x, pitch, base + j * chunk_cols(VEC), lane, g, u);
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

template <int ACT, int T, int VEC>
cudaError_t run(const GluArgs& a, uint32_t pitch, cudaStream_t s) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  // Two blocks an SM, of as many warps (5 to 10) as leave the fewest idle in
  // the last turn, the larger block where that is even.
  uint32_t best = 0, least = ~0u;
  for (uint32_t w = 5; w <= kMaxThreads / 32; ++w) {
    const uint32_t all = 2 * (uint32_t)sms * w, slots = (a.ffn + all - 1) / all * all;
    if (slots <= least) least = slots, best = w;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(std::min((a.ffn + best - 1) / best, 2 * (uint32_t)sms));
  cfg.blockDim = dim3(best * 32);
  cfg.dynamicSmemBytes = (size_t)T * pitch * 2;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_glu_few<ACT, T, VEC>, a, pitch);
}

template <int ACT, int VEC>
cudaError_t by_tokens(const GluArgs& a, uint32_t pitch, cudaStream_t s) {
  return a.tokens == 1 ? run<ACT, 1, VEC>(a, pitch, s) : run<ACT, 2, VEC>(a, pitch, s);
}

// 2048 x 8192, a call: 1 token 12.6 us and 2 tokens 15.3 here, 3 tokens 22.7
// (a third row of sums leaves too few registers for loads); in tiles 3 tokens
// 21.3, 4 20.8, 16 20.4, 64 18.7 and 128 19.2.
constexpr uint32_t kFewTokens = 2;
constexpr uint32_t kFewSmem = 48 << 10;  // what a block gets without asking

uint32_t pitch_of(uint32_t dim) { return (dim + 511) / 512 * 512; }

}  // namespace

bool glu_few(uint64_t tokens, uint64_t dim, bool keeps) {
  if (keeps || tokens > kFewTokens || dim > kFewSmem / 2) return false;
  return tokens * pitch_of((uint32_t)dim) * 2 <= kFewSmem;
}

template <int ACT>
cudaError_t by_vec(const GluArgs& a, int vec, cudaStream_t s) {
  const uint32_t pitch = pitch_of(a.dim);
  return vec == 2 ? by_tokens<ACT, 2>(a, pitch, s)
                  : vec == 1 ? by_tokens<ACT, 1>(a, pitch, s) : by_tokens<ACT, 0>(a, pitch, s);
}

cudaError_t launch_glu_few(cr_act act, const GluArgs& a, int vec, cudaStream_t s) {
  return act == CR_ACT_SILU ? by_vec<CR_ACT_SILU>(a, vec, s) : by_vec<CR_ACT_GELU>(a, vec, s);
}

}  // namespace cr
