// span.cuh -- walking the chunks of a matrix, and rows off the vector grid
// (ffn_internal.cuh has the chunks of rows on it).
#pragma once

#include "ffn_internal.cuh"

namespace cr {

// Chunks of a rows x cols matrix, in row order.
struct ChunkRange {
  uint64_t chunks;
  FastDiv per_row;
};

inline ChunkRange chunk_range(uint64_t rows, uint32_t cols, int vec) {
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

// ---- rows off the vector grid ---------------------------------------------------------
//
// Where a row's start is not aligned, a lane's 8 columns are moved instead:
// they start `lead` columns earlier, so that what is written is whole 16-byte
// granules in spite of the row, and what is read is taken from the granules
// that hold it, shifted.  Only the granules at a row's two ends are written by
// elements.  (With a column a lane and 2-byte accesses the gate's backward
// pass of 1777 x 4099 ran at 2.9 TB/s.)

// A lane's columns first .. first + 7, of which lo .. hi - 1 (counted from
// first) are in the row.
struct Span8 {
  int64_t first;
  int lo, hi;
};

__device__ __forceinline__ Span8 span8(int64_t first, uint32_t cols) {
  return {first, (int)max((int64_t)0, -first), (int)min((int64_t)8, (int64_t)cols - first)};
}

// Columns by which lanes start early, so that `p` + first * ES is a multiple of 16.
template <int ES>
__device__ __forceinline__ uint32_t lead_of(const void* p) {
  return (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15) / ES;
}

// The two granules that hold a span of bf16 (SIZE 16) or of codes (SIZE 8); one
// is read only if it holds an element of the span.
template <int SIZE>
struct Granules {
  static constexpr int kWords = SIZE / 4, es = SIZE / 8;
  uint32_t w[2 * kWords];
  uint32_t shift;  // bytes

  __device__ __forceinline__ void load(const void* row, const Span8& s) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row) + (uintptr_t)(s.first * es);
    shift = (uint32_t)(at & (SIZE - 1));
    const uintptr_t g = at - shift;
    const int split = (int)(SIZE - shift) / es;  // elements of the first granule
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const bool any = s.hi > s.lo && (k ? s.hi > split : s.lo < split);
      if constexpr (SIZE == 16) {
        const uint4 v = any ? reinterpret_cast<const uint4*>(g)[k] : make_uint4(0, 0, 0, 0);
        w[4 * k] = v.x, w[4 * k + 1] = v.y, w[4 * k + 2] = v.z, w[4 * k + 3] = v.w;
      } else {
        const uint2 v = any ? reinterpret_cast<const uint2*>(g)[k] : make_uint2(0, 0);
        w[2 * k] = v.x, w[2 * k + 1] = v.y;
      }
    }
  }

  // The span's SIZE bytes in w[0 .. kWords - 1].
  __device__ __forceinline__ void align() {
    if (SIZE == 16) {
#pragma unroll
      for (int i = 0; i < kWords + 2; ++i)
        if (i + 2 < 2 * kWords) w[i] = shift & 8 ? w[i + 2] : w[i];
    }
#pragma unroll
    for (int i = 0; i <= kWords; ++i)
      if (i + 1 < 2 * kWords) w[i] = shift & 4 ? w[i + 1] : w[i];
    const uint32_t bits = (shift & 3) * 8;
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], bits);
  }
};

// A span's results: whole granules, or element by element at a row's ends.
template <int DT>
__device__ __forceinline__ void st_span(void* row, const Span8& s, const float* v) {
  if constexpr (DT == CR_BF16) {
    uint16_t* p = static_cast<uint16_t*>(row) + s.first;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = ffn_bf16x2(v[2 * i], v[2 * i + 1]);
    if (s.lo == 0 && s.hi == 8) {
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i >= s.lo && i < s.hi) p[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
    }
  } else {
    float* p = static_cast<float*>(row) + s.first;
    if (s.lo == 0 && s.hi == 8) {
      reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i >= s.lo && i < s.hi) p[i] = v[i];
    }
  }
}

// bf16 results of a whole warp's spans where another matrix set the lead, so
// that a granule begins `d` columns into a span: it is made of this lane's last
// 8 - d results and the next lane's first d.  Lane 0's first and lane 31's last
// go out by elements, as a row's ends do.
__device__ __forceinline__ void st_spans(void* row, const Span8& s, uint32_t cols, int lane,
                                         const float* v) {
  uint16_t* p = static_cast<uint16_t*>(row) + s.first;
  const int d = (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / 2;
  if (d == 0) {  // the same in every lane
    if (s.hi > s.lo) st_span<CR_BF16>(row, s, v);
    return;
  }
  Granules<16> g;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    g.w[i] = ffn_bf16x2(v[2 * i], v[2 * i + 1]);
    g.w[4 + i] = __shfl_down_sync(~0u, g.w[i], 1);
  }
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < d && i >= s.lo && i < s.hi) p[i] = (uint16_t)(g.w[i / 2] >> (16 * (i & 1)));
  }
  g.shift = 2 * d;
  g.align();
  const Span8 own = span8(s.first + d, cols);
  const int end = lane == 31 ? min(own.hi, 8 - d) : own.hi;
  if (own.lo == 0 && end == 8) {
    *reinterpret_cast<uint4*>(p + d) = make_uint4(g.w[0], g.w[1], g.w[2], g.w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i >= own.lo && i < end) p[d + i] = (uint16_t)(g.w[i / 2] >> (16 * (i & 1)));
  }
}

// Chunks of a matrix whose rows are walked in spans: one more column chunk
// where a lead of up to 7 columns can push the last ones out.
inline ChunkRange span_range(uint64_t rows, uint32_t cols) {
  const uint64_t per_row = ((uint64_t)cols + 7 + 255) / 256;
  return {rows * per_row, fastdiv_make(per_row, rows * per_row)};
}

// A warp for every `ahead` chunks.
inline dim3 chunk_grid(const ChunkRange& r, int ahead) {
  return dim3(flat_grid((r.chunks + ahead - 1) / ahead * 32));
}

}  // namespace cr
