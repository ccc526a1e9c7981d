// k_q8.cu -- 8-bit activation checkpoints: store, load, and the gate's
// backward pass, which reads gate and up from their checkpoints.
//
// All are one pass over memory: a warp takes a chunk of a row
// (ffn_internal.cuh), so the 128-column group's largest magnitude is a shuffle
// reduction.  A warp that loads few bytes a chunk loads several chunks before
// it works on the first.
//
// Measured at 8192 x 8192, a call in a loop: store from bf16 (203 MB) 34.0 us, 6.0
// TB/s, load 32.5, 6.2 TB/s; the gate's backward pass (675 MB) 105.9 us with
// SiLU, 6.4 TB/s, and 113 with GELU, bound by memory.  5000 x 5001, off the vector
// grid: store 27.1 (a column a lane, a byte a store), load 20.1, gate 57.9.
// The gate's pass runs at 64 registers and four blocks an SM, with a few spills: 122 us at 96
// registers and two.
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

// A span of an 8-bit matrix: its codes, and the scales of the one or two groups
// it reaches into.
struct SpanQ8 {
  Granules<8> codes;
  float s[2];
  int next;  // first column (counted from the span's) of the second group

  __device__ __forceinline__ void load(const Q8& q, uint64_t row, const Span8& sp) {
    codes.load(q.codes + row * q.ld, sp);
    const float* scales = q.scales + row * q.lds;
    const int64_t group = (sp.first + sp.lo) / CR_Q8_GROUP;
    next = (int)((group + 1) * CR_Q8_GROUP - sp.first);
    s[0] = sp.hi > sp.lo ? scales[group] : 0.0f;
    s[1] = sp.hi > next ? scales[group + 1] : 0.0f;
  }

  __device__ __forceinline__ void values(float* v) {
    codes.align();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = from_e4m3x2(codes.w[i >> 1] >> (16 * (i & 1)));
      v[2 * i] = f.x * (2 * i < next ? s[0] : s[1]);
      v[2 * i + 1] = f.y * (2 * i + 1 < next ? s[0] : s[1]);
    }
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
ChunkRange span_range(uint64_t rows, uint32_t cols) {
  const uint64_t per_row = ((uint64_t)cols + 7 + 255) / 256;
  return {rows * per_row, fastdiv_make(per_row, rows * per_row)};
}

template <int DT>
__global__ void __launch_bounds__(kBlock) k_q8_load_span(const __grid_constant__ Q8 q,
                                                         const __grid_constant__ Mat x,
                                                         uint32_t cols,
                                                         const __grid_constant__ ChunkRange r) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  SpanQ8 in[kAhead];
  Span8 span[kAhead];
  for_chunks<0, kAhead>(
      r,
      [&](int j, uint64_t row, uint32_t base) {
        const uint32_t lead = lead_of<DT == CR_BF16 ? 2 : 4>(row_at<DT>(x, row));
        span[j] = span8((int64_t)base + 8 * lane - lead, cols);
        in[j].load(q, row, span[j]);
      },
      [&](int j, uint64_t row, uint32_t) {
        float v[8];
        in[j].values(v);
        if (span[j].hi > span[j].lo) st_span<DT>(row_at<DT>(x, row), span[j], v);
      });
}

// blockIdx.y: which copy.  Rows of dst start on 16-byte boundaries.  (With
// 2-byte loads and stores the three operands of 1531 x 1001 x 2731 took 11 us
// instead of 6.)
__global__ void __launch_bounds__(kBlock) k_copy_bf16(const __grid_constant__ CopyBf16 c) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const CopyBf16::One& m = c.one[blockIdx.y];
  Granules<16> in[kAhead];
  for_chunks<0, kAhead>(
      ChunkRange{m.chunks, m.per_row},
      [&](int j, uint64_t row, uint32_t base) {
        in[j].load(row_at<CR_BF16>(m.src, row), span8((int64_t)base + 8 * lane, m.cols));
      },
      [&](int j, uint64_t row, uint32_t base) {
        const uint32_t col = base + 8 * lane;
        if (col >= m.cols) return;
        in[j].align();
        // columns past the row's end are the row's padding
        *reinterpret_cast<uint4*>(row_at<CR_BF16>(m.dst, row) + 2 * (uint64_t)col) =
            make_uint4(in[j].w[0], in[j].w[1], in[j].w[2], in[j].w[3]);
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

// The same on spans, led by the first output there is.
template <int ACT, bool REST>
__global__ void __launch_bounds__(kBlock, 4) k_act_back_span(const __grid_constant__ ActBackArgs a,
                                                             const __grid_constant__ ChunkRange r,
                                                             const __grid_constant__ SplitArgs x,
                                                             const __grid_constant__ ChunkRange xr) {
  pdl_enter();
  if (blockIdx.y) return x.vec ? split_chunks<1>(x, xr) : split_chunks<0>(x, xr);
  const int lane = threadIdx.x & 31;
  const Mat& lead_mat = a.dg.p ? a.dg : a.du.p ? a.du : a.a;
  Granules<16> in[1];
  SpanQ8 gate[1], up[1];
  Span8 span[1];
  for_chunks<0, 1>(
      r,
      [&](int j, uint64_t row, uint32_t base) {
        const uint32_t lead = lead_of<2>(row_at<CR_BF16>(lead_mat, row));
        span[j] = span8((int64_t)base + 8 * lane - lead, a.cols);
        in[j].load(row_at<CR_BF16>(a.da, row), span[j]);
        gate[j].load(a.g8, row, span[j]);
        up[j].load(a.u8, row, span[j]);
      },
      [&](int j, uint64_t row, uint32_t) {
        float g[8], u[8], dg[8], du[8];
        in[j].align();
        gate[j].values(g);
        up[j].values(u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t w = in[j].w[i / 2];
          const float da = __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
          const float2 v = act_gate_slope<ACT>(g[i]);
          dg[i] = da * u[i] * v.y;
          du[i] = da * v.x;
          u[i] *= v.x;
        }
        if (a.dg.p) st_spans(row_at<CR_BF16>(a.dg, row), span[j], a.cols, lane, dg);
        if (a.du.p) st_spans(row_at<CR_BF16>(a.du, row), span[j], a.cols, lane, du);
        if (a.a.p) st_spans(row_at<CR_BF16>(a.a, row), span[j], a.cols, lane, u);
        if constexpr (REST) {
#pragma unroll
          for (int i = 0; i < 8; ++i) dg[i] = bf16_rest(dg[i]), du[i] = bf16_rest(du[i]);
          st_spans(row_at<CR_BF16>(a.dg_lo, row), span[j], a.cols, lane, dg);
          st_spans(row_at<CR_BF16>(a.du_lo, row), span[j], a.cols, lane, du);
        }
      });
}

// A warp for every `ahead` chunks.
dim3 chunk_grid(const ChunkRange& r, int ahead) {
  return dim3(flat_grid((r.chunks + ahead - 1) / ahead * 32));
}

}  // namespace

cudaError_t launch_q8_store(cr_dtype d, const Mat& x, const Q8& q, uint64_t rows, uint32_t cols,
                            int vec, cudaStream_t s) {
  const ChunkRange r = chunk_range(rows, cols, vec);
  const auto run = [&](auto v) {
    return launch_pdl(d == CR_BF16 ? k_q8_store<CR_BF16, v()> : k_q8_store<CR_F32, v()>,
                      chunk_grid(r, kAhead), kBlock, s, x, q, cols, r);
  };
  return vec == 2 ? run(std::integral_constant<int, 2>())
                  : vec == 1 ? run(std::integral_constant<int, 1>()) : run(std::integral_constant<int, 0>());
}

cudaError_t launch_q8_load(cr_dtype d, const Q8& q, const Mat& x, uint64_t rows, uint32_t cols,
                           int vec, cudaStream_t s) {
  if (vec == 0) {
    const ChunkRange r = span_range(rows, cols);
    return launch_pdl(d == CR_BF16 ? k_q8_load_span<CR_BF16> : k_q8_load_span<CR_F32>,
                      chunk_grid(r, kAhead), kBlock, s, q, x, cols, r);
  }
  const ChunkRange r = chunk_range(rows, cols, vec);
  const auto run = [&](auto v) {
    return launch_pdl(d == CR_BF16 ? k_q8_load<CR_BF16, v()> : k_q8_load<CR_F32, v()>,
                      chunk_grid(r, kAhead), kBlock, s, q, x, cols, r);
  };
  return vec == 2 ? run(std::integral_constant<int, 2>()) : run(std::integral_constant<int, 1>());
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
  const ChunkRange xr = x ? chunk_range(x->rows, x->cols, x->vec) : ChunkRange{};
  const bool silu = act == CR_ACT_SILU;
  if (vec == 0) {
    const ChunkRange sr = span_range(a.rows, a.cols);
    dim3 grid = chunk_grid(ChunkRange{std::max(sr.chunks, xr.chunks), FastDiv{}}, 1);
    grid.y = x ? 2 : 1;
    const auto kernel = a.dg_lo.p ? silu ? k_act_back_span<CR_ACT_SILU, true> : k_act_back_span<CR_ACT_GELU, true>
                                  : silu ? k_act_back_span<CR_ACT_SILU, false> : k_act_back_span<CR_ACT_GELU, false>;
    return launch_pdl(kernel, grid, kBlock, s, a, sr, x ? *x : SplitArgs{}, xr);
  }
  const ChunkRange r = chunk_range(a.rows, a.cols, vec);
  dim3 grid = chunk_grid(ChunkRange{std::max(r.chunks, xr.chunks), FastDiv{}}, 1);
  grid.y = x ? 2 : 1;
  const auto run = [&](auto v) {
    const auto kernel = a.dg_lo.p ? silu ? k_act_back<CR_ACT_SILU, v(), true> : k_act_back<CR_ACT_GELU, v(), true>
                                  : silu ? k_act_back<CR_ACT_SILU, v(), false> : k_act_back<CR_ACT_GELU, v(), false>;
    return launch_pdl(kernel, grid, kBlock, s, a, r, x ? *x : SplitArgs{}, xr);
  };
  return vec == 2 ? run(std::integral_constant<int, 2>()) : run(std::integral_constant<int, 1>());
}

}  // namespace cr
