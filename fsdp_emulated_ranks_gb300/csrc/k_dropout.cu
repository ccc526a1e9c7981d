// k_dropout.cu -- dropout with the residual's addition, from a counter-based generator.
//
// One pass over memory.  Eight consecutive columns share one Philox4x32-10 (twenty
// 32 x 32-bit products), so a lane works on whole groups of eight: 16 columns in vectors; 8
// from shifted granules where bf16 rows are off the vector grid (span.cuh); and for fp32
// there, column by column, with the random numbers handed over in shared memory.  The
// mask exists in registers only.
//
// Measured: 8192 x 2048 bf16 with a residual (101 MB) 16.3 us a call in a loop, 6.2 TB/s; without one
// 15.2, bound by instructions: 160 for a lane's eight elements, of which the generator's ten rounds (two
// products, two exclusive-ors, two key sums) are about 60 and the rest unpacks, compares, packs and starts a
// warp for each 512 columns; 1777 x 4099 fp32 10.8, 5.4 TB/s.
#include "lm_internal.cuh"
#include "pdl.cuh"

namespace cr {

namespace {

struct Key {
  uint32_t k0, k1, off0, off1;
};

__device__ __forceinline__ Key read_key(const DropoutArgs& a) {
  const uint64_t seed = a.rng[0], off = a.rng[1] + a.call;
  return {(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)off, (uint32_t)(off >> 32)};
}

// Philox4x32-10 with the paper's multipliers and key increments.
__device__ __forceinline__ uint4 philox(uint32_t group, uint32_t row, const Key& key) {
  uint32_t c0 = group, c1 = row, c2 = key.off0, c3 = key.off1, k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p = (uint64_t)c0 * 0xD2511F53u, q = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(q >> 32) ^ c1 ^ k0;
    c2 = (uint32_t)(p >> 32) ^ c3 ^ k1;
    c1 = (uint32_t)q;
    c3 = (uint32_t)p;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// Column i's number in the upper half of a word whose lower half means nothing: against
// limit << 16 it compares as the number does against limit.
__device__ __forceinline__ uint32_t half_of(const uint4& w, int i) {
  const uint32_t x = i < 2 ? w.x : i < 4 ? w.y : i < 6 ? w.z : w.w;
  return i & 1 ? x : x << 16;
}

// Blocks an SM, by what was fastest: 8192 x 2048 bf16 with a residual 16.3 us at six (19.3 at four), fp32 30.5 at
// five (36.0 at six), 1777 x 4099 fp32 10.8 at seven (12.2 at four).
constexpr int blocks_of(int dt, int mode) { return dt == CR_BF16 ? 6 : mode ? 5 : 7; }

// A lane's columns in modes 0 to 2 are ffn_internal.cuh's.  Mode kSpan: spans without a
// lead, so that a lane's columns are one group; only the stores are shifted.
template <int DT, int MODE, bool RES>
__global__ void __launch_bounds__(kBlock, blocks_of(DT, MODE)) k_dropout(const __grid_constant__ DropoutArgs a,
                                                    const __grid_constant__ ChunkRange r) {
  constexpr int vals = place_vals(MODE);
  __shared__ __align__(16) uint16_t turned[MODE == 0 ? kBlock / 32 : 1][MODE == 0 ? 256 : 8];
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const Key key = read_key(a);
  const bool some = a.limit < 65536;
  const uint32_t limit = a.limit << 16;
  const uint64_t stride = (uint64_t)gridDim.x * (kBlock / 32);
  for (uint64_t k = (uint64_t)blockIdx.x * (kBlock / 32) + (threadIdx.x >> 5); k < r.chunks;
       k += stride) {
    const uint64_t row = fastdiv_div(r.per_row, k);
    const uint32_t base = (uint32_t)(k - row * r.per_row.d) * place_cols(MODE);
    const Place<MODE> at(base, a.cols, lane, nullptr);
    Loaded<DT, MODE> x, res;
    x.load(row_at<DT>(a.x, row), at);
    if constexpr (RES) res.load(row_at<DT>(a.residual, row), at);
    x.ready();
    if constexpr (RES) res.ready();
    const uint32_t rc = a.first_row + (uint32_t)row;
    float v[vals];
    const auto set = [&](int i, uint32_t number) {
      const float kept = some && number >= limit ? x.value(i) : 0.0f;
      if constexpr (RES)
        v[i] = fmaf(kept, a.by, res.value(i));
      else
        v[i] = kept * a.by;
    };
    if constexpr (MODE == 0) {
      uint16_t* t = turned[threadIdx.x >> 5];
      __syncwarp();
      reinterpret_cast<uint4*>(t)[lane] = philox(base / 8 + lane, rc, key);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < vals; ++i) set(i, (uint32_t)t[32 * i + lane] << 16);
    } else {
#pragma unroll
      for (int g = 0; g < vals / 8; ++g) {
        const uint4 w = philox(base / 8 + lane * (vals / 8) + g, rc, key);
#pragma unroll
        for (int i = 0; i < 8; ++i) set(8 * g + i, half_of(w, i));
      }
    }
    char* out = row_at<DT>(a.out, row);
    if constexpr (MODE == kSpan)
      st_spans(out, at.span, a.cols, lane, v);
    else
      st_chunk<DT, MODE>(out, base, a.cols, lane, v);
  }
}

template <int DT, int MODE>
cudaError_t run(const DropoutArgs& a, cudaStream_t s) {
  const uint64_t per_row = ((uint64_t)a.cols + place_cols(MODE) - 1) / place_cols(MODE);
  const ChunkRange r = {a.rows * per_row, fastdiv_make(per_row, a.rows * per_row)};
  return launch_pdl(a.residual.p ? k_dropout<DT, MODE, true> : k_dropout<DT, MODE, false>,
                    chunk_grid(r, 1), kBlock, s, a, r);
}

}  // namespace

cudaError_t launch_dropout(cr_dtype d, const DropoutArgs& a, int vec, cudaStream_t s) {
  if (d == CR_BF16)
    return vec == 2 ? run<CR_BF16, 2>(a, s) : vec == 1 ? run<CR_BF16, 1>(a, s) : run<CR_BF16, kSpan>(a, s);
  return vec == 2 ? run<CR_F32, 2>(a, s) : vec == 1 ? run<CR_F32, 1>(a, s) : run<CR_F32, 0>(a, s);
}

}  // namespace cr
