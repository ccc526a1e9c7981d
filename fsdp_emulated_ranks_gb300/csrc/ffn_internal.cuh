// ffn_internal.cuh -- types and device helpers shared by the feed-forward
// operators (include/cr_ffn.h): strided matrices, 8-bit matrices, and the
// 256-column chunk every elementwise kernel works in.
//
// A warp handles 256 consecutive columns of a row, 8 values a lane: two of
// the 8-bit form's 128-column groups.  Where pointers and row strides allow
// it (VEC) a lane owns 8 consecutive columns (16 bytes of bf16, 8 codes);
// otherwise lane l owns columns l, l + 32, ..., so that scalar accesses of a
// warp still cover consecutive addresses.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "cr_ffn.h"
#include "cr_internal.cuh"

namespace cr {

constexpr int kChunk = 256;   // columns a warp handles at a time
constexpr int kLaneVals = 8;  // values per lane of a chunk
constexpr float kQ8Max = 448.0f;
constexpr float kQ8InvMax = 1.0f / 448.0f;
constexpr float kQ8Tiny = 1.17549435e-38f;  // 2^-126

// p == nullptr: the matrix is absent.
struct Mat {
  void* p;
  uint64_t ld;  // elements
};

struct Q8 {
  uint8_t* codes;  // nullptr: absent
  uint64_t ld;
  float* scales;
  uint64_t lds;
};

struct NormArgs {
  Mat x, residual, sum, y;
  Q8 y8;
  const void* weight;
  float* rstd;
  uint64_t rows;
  uint32_t cols;
  float eps;
  float inv_cols;
};

struct NormBackArgs {
  Mat dy, h, dres, dx;
  Q8 h8;
  const void* weight;
  const float* rstd;
  void* dweight;
  float* partial;  // [parts][cols] sums of dy * n over a block's rows
  uint64_t rows;
  uint32_t cols;
  uint32_t parts;
  float inv_cols;
};

struct ActBackArgs {
  Mat da, dg, du, a;
  Q8 g8, u8;
  uint64_t rows;
  uint32_t cols;
};

// Operands of the products (x, wg, wu, dg, du): 16-byte aligned rows.
struct GluArgs {
  Mat x, wg, wu, a;
  Q8 g8, u8;
  uint32_t tokens, dim, ffn;
};

struct GluBackArgs {
  Mat dg, du, x, x_lo, wg, wu, dx;  // x_lo: what x lacks to a checkpoint's value, or absent
  void *dwg, *dwu;  // [ffn][dim]
  uint32_t tokens, dim, ffn;
};

// vec: every pointer and row stride of the call allows the VEC accesses.
cudaError_t launch_rms_norm(cr_dtype d, const NormArgs& a, bool vec, cudaStream_t s);
// Row partials the backward pass writes for its dweight, at most.
uint32_t norm_back_parts(uint64_t rows, uint32_t cols);
cudaError_t launch_rms_norm_back(cr_dtype d, cr_dtype dw, NormBackArgs a, bool vec,
                                 cudaStream_t s);
cudaError_t launch_q8_store(cr_dtype d, const Mat& x, const Q8& q, uint64_t rows, uint32_t cols,
                            bool vec, cudaStream_t s);
cudaError_t launch_q8_load(cr_dtype d, const Q8& q, const Mat& x, uint64_t rows, uint32_t cols,
                           bool vec, cudaStream_t s);
// The values q stands for as bf16 hi + lo (lo: what the rounding of hi left).
cudaError_t launch_q8_split(const Q8& q, const Mat& hi, const Mat& lo, uint64_t rows, uint32_t cols,
                            bool vec, cudaStream_t s);
// dst = src, rows x cols bf16 at any alignment.
cudaError_t launch_copy_bf16(const Mat& src, const Mat& dst, uint64_t rows, uint32_t cols,
                             cudaStream_t s);
cudaError_t launch_act_back(cr_act act, const ActBackArgs& a, bool vec, cudaStream_t s);
cudaError_t launch_glu(cr_act act, const GluArgs& a, cudaStream_t s);
// Whether the block's call is one for k_glu_few.cu: few tokens, whose x fits
// in shared memory, and no checkpoints (keeps).  Operands at any alignment;
// vec: 16-byte aligned rows of both weights.
bool glu_few(uint64_t tokens, uint64_t dim, bool keeps);
cudaError_t launch_glu_few(cr_act act, const GluArgs& a, bool vec, cudaStream_t s);
cudaError_t launch_glu_back(cr_dtype dw, const GluBackArgs& a, cudaStream_t s);
// Reads (and clears) the word a block sets that gave up a wait.
cudaError_t glu_wait_word(bool clear, unsigned int* word);

#if defined(__CUDACC__)

// ---- bf16 and e4m3 ---------------------------------------------------------------

__device__ __forceinline__ float ffn_bf16(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// Two fp32 values rounded to bf16 (nearest even), `lo` in the low half.
__device__ __forceinline__ uint32_t ffn_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two fp32 values as e4m3 codes (nearest even, saturated), `lo` in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float2 from_e4m3x2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  float2 f;
  asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b; }"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

__device__ __forceinline__ bool finite(float v) { return fabsf(v) < __int_as_float(0x7f800000); }

__device__ __forceinline__ float q8_magnitude(float v) { return finite(v) ? fabsf(v) : 0.0f; }

__device__ __forceinline__ float q8_scale(float m) { return fmaxf(m * kQ8InvMax, kQ8Tiny); }

// A value that is not finite becomes NaN, which e4m3x2 keeps.
__device__ __forceinline__ float q8_scaled(float v, float inv) {
  return finite(v) ? v * inv : __int_as_float(0x7fc00000);
}

// ---- chunks -----------------------------------------------------------------------

template <bool VEC>
__device__ __forceinline__ uint32_t chunk_col(uint32_t base, int lane, int i) {
  return VEC ? base + lane * kLaneVals + i : base + i * 32 + lane;
}

// A chunk as loaded, before it is widened to fp32: what a kernel that loads
// ahead keeps.  Values of columns past `cols` are zero.
template <int DT, bool VEC>
struct Raw {
  static constexpr int kWords = DT == CR_BF16 ? (VEC ? 4 : 8) : 8;
  uint32_t w[kWords];

  // `row` points at the row's column 0.
  __device__ __forceinline__ void load(const void* row, uint32_t base, uint32_t cols, int lane) {
    const uint32_t c0 = chunk_col<VEC>(base, lane, 0);
    if constexpr (VEC) {
      if (c0 + kLaneVals <= cols) {
        if constexpr (DT == CR_BF16) {
          const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + c0);
          w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
        } else {
          const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(row) + c0);
          const uint4 q = p[0], r = p[1];
          w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
          w[4] = r.x, w[5] = r.y, w[6] = r.z, w[7] = r.w;
        }
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
#pragma unroll
    for (int i = 0; i < kLaneVals; ++i) {
      const uint32_t c = chunk_col<VEC>(base, lane, i);
      if (c >= cols) continue;
      if constexpr (DT == CR_F32)
        w[i] = static_cast<const uint32_t*>(row)[c];
      else if constexpr (VEC)
        w[i / 2] |= (uint32_t) static_cast<const uint16_t*>(row)[c] << (16 * (i & 1));
      else
        w[i] = (uint32_t) static_cast<const uint16_t*>(row)[c] << 16;
    }
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }

  __device__ __forceinline__ float value(int i) const {
    if constexpr (DT == CR_BF16 && VEC)
      return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    else
      return __uint_as_float(w[i]);
  }
};

template <int DT, bool VEC>
__device__ __forceinline__ void ld_chunk(const void* row, uint32_t base, uint32_t cols, int lane,
                                         float* v) {
  Raw<DT, VEC> r;
  r.load(row, base, cols, lane);
#pragma unroll
  for (int i = 0; i < kLaneVals; ++i) v[i] = r.value(i);
}

template <int DT, bool VEC>
__device__ __forceinline__ void st_chunk(void* row, uint32_t base, uint32_t cols, int lane,
                                         const float* v) {
  const uint32_t c0 = chunk_col<VEC>(base, lane, 0);
  if (VEC && c0 + kLaneVals <= cols) {
    if constexpr (DT == CR_BF16) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(row) + c0) =
          make_uint4(ffn_bf16x2(v[0], v[1]), ffn_bf16x2(v[2], v[3]), ffn_bf16x2(v[4], v[5]),
                     ffn_bf16x2(v[6], v[7]));
    } else {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(row) + c0);
      p[0] = make_float4(v[0], v[1], v[2], v[3]);
      p[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kLaneVals; ++i) {
    const uint32_t c = chunk_col<VEC>(base, lane, i);
    if (c >= cols) continue;
    if constexpr (DT == CR_BF16)
      static_cast<uint16_t*>(row)[c] = (uint16_t)ffn_bf16x2(v[i], 0.0f);
    else
      static_cast<float*>(row)[c] = v[i];
  }
}

// 8-bit form of a chunk: every lane of the warp calls it.
template <bool VEC>
__device__ __forceinline__ void st_chunk_q8(const Q8& q, uint64_t row, uint32_t base,
                                            uint32_t cols, int lane, const float* v) {
  uint8_t* codes = q.codes + row * q.ld;
  float* scales = q.scales + row * q.lds;
  const uint32_t group = base / CR_Q8_GROUP;
  if constexpr (VEC) {  // lanes 0-15 hold one group, 16-31 the next
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < kLaneVals; ++i) m = fmaxf(m, q8_magnitude(v[i]));
#pragma unroll
    for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    const float s = q8_scale(m), inv = 1.0f / s;
    const uint32_t c0 = chunk_col<VEC>(base, lane, 0);
    if ((lane & 15) == 0 && c0 < cols) scales[group + (lane >> 4)] = s;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = e4m3x2(q8_scaled(v[2 * i], inv), q8_scaled(v[2 * i + 1], inv));
    const uint32_t lo = w[0] | w[1] << 16, hi = w[2] | w[3] << 16;
    if (c0 + kLaneVals <= cols) {
      *reinterpret_cast<uint2*>(codes + c0) = make_uint2(lo, hi);
    } else {
#pragma unroll
      for (int i = 0; i < kLaneVals; ++i)
        if (c0 + i < cols) codes[c0 + i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
    }
  } else {  // values 0-3 of every lane are one group, 4-7 the next
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) m = fmaxf(m, q8_magnitude(v[4 * h + i]));
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
      const float s = q8_scale(m), inv = 1.0f / s;
      if (lane == 0 && base + h * CR_Q8_GROUP < cols) scales[group + h] = s;
#pragma unroll
      for (int i = 4 * h; i < 4 * h + 4; ++i) {
        const uint32_t c = chunk_col<VEC>(base, lane, i);
        if (c < cols) codes[c] = (uint8_t)e4m3x2(q8_scaled(v[i], inv), 0.0f);
      }
    }
  }
}

// A chunk of an 8-bit matrix as loaded.  VEC: 8 codes and the one scale of the
// lane's half; otherwise a code a word and both scales.
template <bool VEC>
struct RawQ8 {
  uint32_t w[VEC ? 2 : 8];
  float s[VEC ? 1 : 2];

  __device__ __forceinline__ void load(const Q8& q, uint64_t row, uint32_t base, uint32_t cols,
                                       int lane) {
    const uint8_t* codes = q.codes + row * q.ld;
    const float* scales = q.scales + row * q.lds + base / CR_Q8_GROUP;
    const uint32_t c0 = chunk_col<VEC>(base, lane, 0);
    if constexpr (VEC) {
      s[0] = c0 < cols ? scales[lane >> 4] : 0.0f;
      w[0] = w[1] = 0;
      if (c0 + kLaneVals <= cols) {
        const uint2 t = *reinterpret_cast<const uint2*>(codes + c0);
        w[0] = t.x, w[1] = t.y;
      } else {
#pragma unroll
        for (int i = 0; i < kLaneVals; ++i)
          if (c0 + i < cols) w[i >> 2] |= (uint32_t)codes[c0 + i] << (8 * (i & 3));
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) s[h] = base + h * CR_Q8_GROUP < cols ? scales[h] : 0.0f;
#pragma unroll
      for (int i = 0; i < kLaneVals; ++i) {
        const uint32_t c = chunk_col<VEC>(base, lane, i);
        w[i] = c < cols ? codes[c] : 0u;
      }
    }
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (VEC ? 2 : 8); ++i) w[i] = 0;
    s[0] = s[VEC ? 0 : 1] = 0.0f;
  }

  // The values the codes stand for (fp32, not rounded further).
  __device__ __forceinline__ void values(float* v) const {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = from_e4m3x2(w[i >> 1] >> (16 * (i & 1)));
        v[2 * i] = f.x * s[0], v[2 * i + 1] = f.y * s[0];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kLaneVals; ++i) v[i] = from_e4m3x2(w[i]).x * s[i / 4];
    }
  }
};

template <bool VEC>
__device__ __forceinline__ void ld_chunk_q8(const Q8& q, uint64_t row, uint32_t base,
                                            uint32_t cols, int lane, float* v) {
  RawQ8<VEC> r;
  r.load(q, row, base, cols, lane);
  r.values(v);
}

// ---- the gate's activation -----------------------------------------------------------

// act(g) = g p and act'(g), with p = 1 / (1 + exp(-z)): z = g for SiLU; for
// GELU 1/2 (1 + tanh t) = 1 / (1 + exp(-2t)), so z = 2t.  exp and the
// division are the fast ones, within a few fp32 ulps: the results are
// rounded to bf16 (2^-9) right after.
template <int ACT>
__device__ __forceinline__ float act_gate(float g) {
  float z = g;
  if constexpr (ACT == CR_ACT_GELU) z = 1.5957691216f * (g + 0.044715f * g * g * g);
  return __fdividef(g, 1.0f + __expf(-z));
}

template <int ACT>
__device__ __forceinline__ float2 act_gate_slope(float g) {
  float z = g, dz = 1.0f;
  if constexpr (ACT == CR_ACT_GELU) {
    z = 1.5957691216f * (g + 0.044715f * g * g * g);
    dz = 1.5957691216f + 0.2140643f * g * g;
  }
  const float p = __fdividef(1.0f, 1.0f + __expf(-z));
  const float a = g * p;
  return make_float2(a, p + a * (1.0f - p) * dz);
}

#endif  // __CUDACC__

}  // namespace cr
