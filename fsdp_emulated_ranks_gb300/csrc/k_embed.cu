// k_embed.cu -- embedding lookup: rows of a table, scaled.
//
// A gather: bound by memory (each distinct row of the table read once, every output
// written once).  A warp copies a chunk of a row (ffn_internal.cuh; rows off the vector
// grid in spans, span.cuh), two chunks in flight, since each begins with two dependent
// loads, the id and the row.
#include <type_traits>

#include "lm_internal.cuh"
#include "pdl.cuh"

namespace cr {

namespace {

constexpr int kAhead = 2;  // chunks of a warp in flight

template <int DT, int OT, int MODE>
__global__ void __launch_bounds__(kBlock) k_embed(const __grid_constant__ EmbedArgs a,
                                                  const __grid_constant__ ChunkRange r) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const uint64_t stride = (uint64_t)gridDim.x * (kBlock / 32);
  for (uint64_t k = (uint64_t)blockIdx.x * (kBlock / 32) + (threadIdx.x >> 5); k < r.chunks;
       k += kAhead * stride) {
    Loaded<DT, MODE> in[kAhead];
    uint64_t row[kAhead];
    uint32_t base[kAhead];
    int32_t id[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const uint64_t c = k + j * stride;
      if (c >= r.chunks) break;
      row[j] = fastdiv_div(r.per_row, c);
      base[j] = (uint32_t)(c - row[j] * r.per_row.d) * place_cols(MODE);
      id[j] = token_id(a.ids, row[j], a.vocab);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (k + j * stride >= r.chunks) break;
      const Place<MODE> at(base[j], a.dim, lane, row_at<OT>(a.out, row[j]));
      if (id[j] >= 0) in[j].load(row_at<DT>(a.table, id[j]), at);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (k + j * stride >= r.chunks) break;
      char* out = row_at<OT>(a.out, row[j]);
      const Place<MODE> at(base[j], a.dim, lane, out);
      float v[place_vals(MODE)];
      in[j].ready();
#pragma unroll
      for (int i = 0; i < place_vals(MODE); ++i) v[i] = id[j] >= 0 ? in[j].value(i) * a.scale : 0.0f;
      st_place<OT, MODE>(out, at, v);
    }
  }
}

template <int DT, int OT, int MODE>
cudaError_t run(const EmbedArgs& a, cudaStream_t s) {
  const uint64_t per_row = place_chunks(a.dim, MODE);
  const ChunkRange r = {a.tokens * per_row, fastdiv_make(per_row, a.tokens * per_row)};
  return launch_pdl(k_embed<DT, OT, MODE>, chunk_grid(r, kAhead), kBlock, s, a, r);
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
