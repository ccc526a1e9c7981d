// ffn_internal.cuh -- types and device helpers shared by the feed-forward
// operators (include/cr_ffn.h): strided matrices, 8-bit matrices, and the
// chunk of a row every elementwise kernel works in.
//
// A warp handles a chunk of consecutive columns.  Where pointers and row
// strides allow it (VEC: 1 for 16-byte vectors, 2 for 32-byte ones) a lane
// owns 16 consecutive columns, 512 a chunk; otherwise (VEC 0) lane l owns
// columns l, l + 32, ... of 256, so that a warp's scalar accesses still cover
// consecutive addresses.  These kernels are bound by instructions before they
// are by memory (with 8 columns a lane the norm issued 47 a value and
// reached 73 % of its issue slots at 4.7 TB/s): hence the wide lanes, which
// share addresses, reductions and divisions among more values.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "cr_ffn.h"
#include "cr_internal.cuh"

namespace cr {

// Values of a lane, and columns of a chunk.
__host__ __device__ constexpr int lane_vals(int vec) { return vec ? 16 : 8; }
__host__ __device__ constexpr uint32_t chunk_cols(int vec) { return 32 * lane_vals(vec); }
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
  Mat dg_lo, du_lo;  // what dg and du were rounded by (optional)
};

// The values q stands for as bf16 hi + lo (lo: what the rounding of hi left).
struct SplitArgs {
  Q8 q;
  Mat hi, lo;
  uint64_t rows;
  uint32_t cols;
  int vec;  // the accesses q allows
};

// Operands of the products (x, wg, wu, dg, du): 16-byte aligned rows.
struct GluArgs {
  Mat x, wg, wu, a;
  Q8 g8, u8;
  uint32_t tokens, dim, ffn;
};

struct GluBackArgs {
  Mat dg, du, x, wg, wu, dx;
  Mat dg_lo, du_lo, x_lo;  // what dg, du and x were rounded by, or absent
  void *dwg, *dwu;  // [ffn][dim]
  uint32_t tokens, dim, ffn;
};

// vec: the accesses every pointer and row stride of the call allows, 0 to 2.
cudaError_t launch_rms_norm(cr_dtype d, const NormArgs& a, int vec, cudaStream_t s);
// Row partials the backward pass writes for its dweight, at most.
uint32_t norm_back_parts(uint64_t rows, uint32_t cols);
cudaError_t launch_rms_norm_back(cr_dtype d, cr_dtype dw, NormBackArgs a, int vec,
                                 cudaStream_t s);
cudaError_t launch_q8_store(cr_dtype d, const Mat& x, const Q8& q, uint64_t rows, uint32_t cols,
                            int vec, cudaStream_t s);
cudaError_t launch_q8_load(cr_dtype d, const Q8& q, const Mat& x, uint64_t rows, uint32_t cols,
                           int vec, cudaStream_t s);
// dst = src for up to three bf16 matrices at any alignment, in one launch.
struct CopyBf16 {
  struct One {
    Mat src, dst;
    uint64_t chunks;
    FastDiv per_row;
    uint32_t cols;
  } one[3];
  int n;
};
void add_copy(CopyBf16* c, const Mat& src, const Mat& dst, uint64_t rows, uint32_t cols);
cudaError_t launch_copy_bf16(const CopyBf16& c, cudaStream_t s);
// The gate's backward pass and, in the same launch, x's split (or nullptr).
cudaError_t launch_act_back(cr_act act, const ActBackArgs& a, const SplitArgs* x, int vec,
                            cudaStream_t s);
cudaError_t launch_glu(cr_act act, const GluArgs& a, cudaStream_t s);
// Whether the block's call is one for k_glu_few.cu: few tokens, whose x fits
// in shared memory, and no checkpoints (keeps).  Operands at any alignment;
// vec: the accesses both weights allow.
bool glu_few(uint64_t tokens, uint64_t dim, bool keeps);
cudaError_t launch_glu_few(cr_act act, const GluArgs& a, int vec, cudaStream_t s);
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

constexpr float kFloatMax = 3.402823466e38f;

__device__ __forceinline__ float q8_scale(float m) { return fmaxf(m * kQ8InvMax, kQ8Tiny); }

// Largest finite magnitude of a group held by several lanes, and the values
// with infinities made NaN.  `reduce` takes a lane's maximum to the group's;
// the whole warp calls.  fmaxf passes NaN over, so only an infinity needs
// the second look, and NaN times anything stays NaN, which the codes keep.
template <int N, typename Reduce>
__device__ __forceinline__ float q8_magnitude(float* v, Reduce reduce) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(v[i]));
  m = reduce(m);
  if (__any_sync(~0u, m > kFloatMax)) {
    m = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (fabsf(v[i]) > kFloatMax) v[i] = __int_as_float(0x7fc00000);
      m = fmaxf(m, fabsf(v[i]));
    }
    m = reduce(m);
  }
  return m;
}

// ---- chunks -----------------------------------------------------------------------

template <int VEC>
__device__ __forceinline__ uint32_t chunk_col(uint32_t base, int lane, int i) {
  return VEC ? base + lane * lane_vals(VEC) + i : base + i * 32 + lane;
}

__device__ __forceinline__ void ld_words8(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                 "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}

__device__ __forceinline__ void st_words8(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// 8 words at p, 32-byte (VEC 2) or 16-byte aligned.
template <int VEC>
__device__ __forceinline__ void ld_words(const void* p, uint32_t* w) {
  if constexpr (VEC == 2) {
    ld_words8(p, w);
  } else {
    const uint4 q = static_cast<const uint4*>(p)[0], r = static_cast<const uint4*>(p)[1];
    w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    w[4] = r.x, w[5] = r.y, w[6] = r.z, w[7] = r.w;
  }
}

template <int VEC>
__device__ __forceinline__ void st_words(void* p, const uint32_t* w) {
  if constexpr (VEC == 2) {
    st_words8(p, w);
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// A chunk as loaded, before it is widened to fp32: what a kernel that loads
// ahead keeps.  Values of columns past `cols` are zero.
template <int DT, int VEC>
struct Raw {
  static constexpr int kVals = lane_vals(VEC);
  static constexpr int kWords = DT == CR_BF16 && VEC ? kVals / 2 : kVals;
  uint32_t w[kWords];

  // `row` points at the row's column 0.
  __device__ __forceinline__ void load(const void* row, uint32_t base, uint32_t cols, int lane) {
    const uint32_t c0 = chunk_col<VEC>(base, lane, 0);
    const uint16_t* half = static_cast<const uint16_t*>(row) + c0;
    const uint32_t* word = static_cast<const uint32_t*>(row) + c0;
    if constexpr (VEC) {
      if (c0 + kVals <= cols) {
        if constexpr (DT == CR_BF16) {
          ld_words<VEC>(half, w);
        } else {
          ld_words<VEC>(word, w);
          ld_words<VEC>(word + 8, w + 8);
        }
        return;
      }
    }
    clear();
    if (VEC && c0 >= cols) return;
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      const int at = VEC ? i : i * 32;
      if (c0 + at >= cols) continue;
      if constexpr (DT == CR_F32)
        w[i] = word[at];
      else if constexpr (VEC)
        w[i / 2] |= (uint32_t)half[at] << (16 * (i & 1));
      else
        w[i] = (uint32_t)half[at] << 16;
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

template <int DT, int VEC>
__device__ __forceinline__ void st_chunk(void* row, uint32_t base, uint32_t cols, int lane,
                                         const float* v) {
  constexpr int vals = lane_vals(VEC);
  const uint32_t c0 = chunk_col<VEC>(base, lane, 0);
  uint16_t* half = static_cast<uint16_t*>(row) + c0;
  float* word = static_cast<float*>(row) + c0;
  if constexpr (VEC) {
    if (c0 + vals <= cols) {
      uint32_t w[8];
      if constexpr (DT == CR_BF16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = ffn_bf16x2(v[2 * i], v[2 * i + 1]);
        st_words<VEC>(half, w);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[8 * h + i]);
          st_words<VEC>(word + 8 * h, w);
        }
      }
      return;
    }
  }
  if (VEC && c0 >= cols) return;
#pragma unroll
  for (int i = 0; i < vals; ++i) {
    const int at = VEC ? i : i * 32;
    if (c0 + at >= cols) continue;
    if constexpr (DT == CR_BF16)
      half[at] = (uint16_t)ffn_bf16x2(v[i], 0.0f);
    else
      word[at] = v[i];
  }
}

// 8-bit form of GROUPS groups from column `base` on: v[i] is column base + lane
// + 32 i's value, and is changed.  Every lane of the warp calls it.  A group's
// magnitude is one integer maximum over the lanes (bits of floats from 0 up
// order as the floats do), and lane g makes group g's scale for all.
template <int GROUPS, bool FULL>
__device__ __forceinline__ void st_groups_q8(const Q8& q, uint64_t row, uint32_t base,
                                             uint32_t cols, int lane, float* v) {
  uint8_t* codes = q.codes + row * q.ld + base + lane;
  float m[GROUPS];
  bool inf = false;
  for (int look = 0; look < 2; ++look) {
    float most = 0.0f;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      m[g] = 0.0f;
#pragma unroll
      for (int i = 4 * g; i < 4 * g + 4; ++i) {
        if (inf && fabsf(v[i]) > kFloatMax) v[i] = __int_as_float(0x7fc00000);
        m[g] = fmaxf(m[g], fabsf(v[i]));
      }
      m[g] = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(m[g])));
      most = fmaxf(most, m[g]);
    }
    inf = most > kFloatMax;  // the same in every lane
    if (!inf) break;
  }
  float mine = m[0];
#pragma unroll
  for (int g = 1; g < GROUPS; ++g) mine = lane == g ? m[g] : mine;
  const float s = q8_scale(mine), inv = 1.0f / s;
  if (lane < GROUPS && (FULL || base + lane * CR_Q8_GROUP < cols))
    q.scales[row * q.lds + base / CR_Q8_GROUP + lane] = s;
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
    const float by = __shfl_sync(~0u, inv, g);
#pragma unroll
    for (int i = 4 * g; i < 4 * g + 4; ++i)
      if (FULL || base + lane + 32 * i < cols) codes[32 * i] = (uint8_t)e4m3x2(v[i] * by, 0.0f);
  }
}

// 8-bit form of a chunk: every lane of the warp calls it.  v may be changed.
template <int VEC>
__device__ __forceinline__ void st_chunk_q8(const Q8& q, uint64_t row, uint32_t base,
                                            uint32_t cols, int lane, float* v) {
  if constexpr (VEC) {  // 8 lanes hold a group
    const uint32_t c0 = chunk_col<VEC>(base, lane, 0);
    uint8_t* codes = q.codes + row * q.ld + c0;
    float* scales = q.scales + row * q.lds + base / CR_Q8_GROUP;
    const float m = q8_magnitude<16>(v, [](float x) {
#pragma unroll
      for (int o = 4; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, o));
      return x;
    });
    const float s = q8_scale(m), inv = 1.0f / s;
    if (c0 >= cols) return;
    if ((lane & 7) == 0) scales[lane >> 3] = s;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = e4m3x2(v[4 * i] * inv, v[4 * i + 1] * inv) |
             e4m3x2(v[4 * i + 2] * inv, v[4 * i + 3] * inv) << 16;
    if (c0 + 16 <= cols) {
      *reinterpret_cast<uint4*>(codes) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (c0 + i < cols) codes[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
  } else {
    st_groups_q8<2, false>(q, row, base, cols, lane, v);
  }
}

// A chunk of an 8-bit matrix as loaded.  VEC: 16 codes and the one scale of
// the lane's group; otherwise a code a word and both scales.
template <int VEC>
struct RawQ8 {
  static constexpr int kWords = VEC ? 4 : 8, kScales = VEC ? 1 : 2;
  uint32_t w[kWords];
  float s[kScales];

  __device__ __forceinline__ void load(const Q8& q, uint64_t row, uint32_t base, uint32_t cols,
                                       int lane) {
    const uint32_t c0 = chunk_col<VEC>(base, lane, 0);
    const uint8_t* codes = q.codes + row * q.ld + c0;
    const float* scales = q.scales + row * q.lds + base / CR_Q8_GROUP;
    clear();
    if constexpr (VEC) {
      if (c0 >= cols) return;
      s[0] = scales[lane >> 3];
      if (c0 + 16 <= cols) {
        const uint4 t = *reinterpret_cast<const uint4*>(codes);
        w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w;
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (c0 + i < cols) w[i >> 2] |= (uint32_t)codes[i] << (8 * (i & 3));
      }
    } else {
      if (base < cols) s[0] = scales[0];
      if (base + CR_Q8_GROUP < cols) s[1] = scales[1];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c0 + 32 * i < cols) w[i] = codes[32 * i];
    }
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
#pragma unroll
    for (int i = 0; i < kScales; ++i) s[i] = 0.0f;
  }

  // The values the codes stand for (fp32, not rounded further).
  __device__ __forceinline__ void values(float* v) const {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = from_e4m3x2(w[i >> 1] >> (16 * (i & 1)));
        v[2 * i] = f.x * s[0], v[2 * i + 1] = f.y * s[0];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = from_e4m3x2(w[i]).x * s[i / 4];
    }
  }
};

// ---- the gate's activation -----------------------------------------------------------

// act(g) = g p and act'(g), with p = 1 / (1 + exp(-z)): z = g for SiLU; for
// GELU 1/2 (1 + tanh t) = 1 / (1 + exp(-2t)), so z = 2t.  2^x and 1/x are the
// hardware's approximations, each within 2 fp32 ulps (results below 2^-126
// become 0): what follows is rounded to bf16 (2^-9).
__device__ __forceinline__ float logistic(float z) {
  float e, p;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * z));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(1.0f + e));
  return p;
}

template <int ACT>
__device__ __forceinline__ float act_gate(float g) {
  if constexpr (ACT == CR_ACT_GELU)
    return g * logistic(g * fmaf(0.0713548163f, g * g, 1.5957691216f));
  return g * logistic(g);
}

template <int ACT>
__device__ __forceinline__ float2 act_gate_slope(float g) {
  float z = g, dz = 1.0f;
  if constexpr (ACT == CR_ACT_GELU) {
    const float sq = fminf(g * g, 1e4f);  // finite: past |g| = 100 p is 0 or 1, and 0 * dz has to be 0
    z = g * fmaf(0.0713548163f, sq, 1.5957691216f);
    dz = fmaf(0.2140644488f, sq, 1.5957691216f);
  }
  const float p = logistic(z), a = g * p;
  const float rest = ACT == CR_ACT_GELU ? (1.0f - p) * dz : 1.0f - p;
  return make_float2(a, fmaf(a, rest, p));
}

#endif  // __CUDACC__

}  // namespace cr
