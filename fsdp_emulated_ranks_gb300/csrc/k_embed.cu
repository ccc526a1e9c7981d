// k_embed.cu -- embedding lookup: rows of a table, scaled.
//
// A gather: bound by memory (each distinct row of the table read once, every output
// written once).  A warp copies a chunk of a row (ffn_internal.cuh; rows off the vector
// grid in spans, span.cuh): two next to each other, which share the id, since a row's load
// waits for the id's.
//
// Measured: 8192 x 2048 bf16 of 32000 rows (47 MB) 9.3 us a call in a loop, 5.1 TB/s, with the start and
// end of a short launch in it (one chunk a warp 10.3, four 9.2 but idle for narrow rows); 8192 x
// 2047, in spans, 15.1.
#include "lm_internal.cuh"
#include "pdl.cuh"

namespace cr {

namespace {

constexpr int kAhead = 2;  // chunks of a warp in flight

// A warp takes kAhead chunks of a row, next to each other, which share the id.
template <int DT, int OT, int MODE>
__global__ void __launch_bounds__(kBlock) k_embed(const __grid_constant__ EmbedArgs a,
                                                  const __grid_constant__ ChunkRange r) {
  constexpr uint32_t cols = place_cols(MODE);
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const uint64_t stride = (uint64_t)gridDim.x * (kBlock / 32);
  for (uint64_t k = (uint64_t)blockIdx.x * (kBlock / 32) + (threadIdx.x >> 5); k < r.chunks;
       k += stride) {
    const uint64_t row = fastdiv_div(r.per_row, k);
    const uint32_t base = (uint32_t)(k - row * r.per_row.d) * kAhead * cols;
    const int32_t id = token_id(a.ids, row, a.vocab);
    char* out = row_at<OT>(a.out, row);
    Loaded<DT, MODE> in[kAhead];
    if (id >= 0) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        in[j].load(row_at<DT>(a.table, id), Place<MODE>(base + j * cols, a.dim, lane, out));
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const Place<MODE> at(base + j * cols, a.dim, lane, out);
      float v[place_vals(MODE)];
      if (id >= 0) in[j].ready();
#pragma unroll
      for (int i = 0; i < place_vals(MODE); ++i) v[i] = id >= 0 ? in[j].value(i) * a.scale : 0.0f;
      st_place<OT, MODE>(out, at, v);
    }
  }
}

template <int DT, int OT, int MODE>
cudaError_t run(const EmbedArgs& a, cudaStream_t s) {
  const uint64_t per_row = (place_chunks(a.dim, MODE) + kAhead - 1) / kAhead;
  const ChunkRange r = {a.tokens * per_row, fastdiv_make(per_row, a.tokens * per_row)};
  return launch_pdl(k_embed<DT, OT, MODE>, chunk_grid(r, 1), kBlock, s, a, r);
}

template <int DT, int OT>
cudaError_t by_mode(const EmbedArgs& a, int vec, cudaStream_t s) {
  if (vec == 2) return run<DT, OT, 2>(a, s);
  if (vec == 1) return run<DT, OT, 1>(a, s);
  if constexpr (DT == CR_BF16 && OT == CR_BF16) return run<DT, OT, kSpan>(a, s);
  return run<DT, OT, 0>(a, s);
}

}  // namespace

cudaError_t launch_embed(cr_dtype d, cr_dtype out, const EmbedArgs& a, int vec, cudaStream_t s) {
  if (d == CR_BF16)
    return out == CR_BF16 ? by_mode<CR_BF16, CR_BF16>(a, vec, s) : by_mode<CR_BF16, CR_F32>(a, vec, s);
  return out == CR_BF16 ? by_mode<CR_F32, CR_BF16>(a, vec, s) : by_mode<CR_F32, CR_F32>(a, vec, s);
}

}  // namespace cr
