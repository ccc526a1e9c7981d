// k_glu.cu -- the gated feed-forward block: both projections, the activation
// and the product in one kernel, and the products of its backward pass.
//
// One persistent kernel, three uses (T tokens, D dim, F ffn; a tile is 128
// rows x 256 accumulator columns, K in blocks of 64):
//   kGlu  a = act(x Wg^T) * (x Wu^T): a tile's 256 columns are the same 128
//         columns of g and of u, so the epilogue has both in one thread's row,
//         and a tile's width is the 8-bit checkpoints' group.
//   kDx   dx = dg Wg + du Wu: one accumulator over both products.
//   kDw   dWg = dg^T x and dWu = du^T x: tiles of both in one launch.
// Operands are read as they lie in memory: rows of K (x, W of kGlu, dg and du
// of kDx) or rows of M or N (W of kDx, everything of kDw), which the tensor
// cores take directly, so nothing is transposed.
//
// Block: warp 0 loads tiles by TMA into a ring of kStages buffers, warp 1
// issues the tcgen05 products into one of two accumulators in tensor memory,
// warps 2-5 read the other accumulator out and write the results.  TMA fills
// rows and columns outside a matrix with zeros, so ragged sizes need no masks
// before the epilogue.  Every wait is bounded (tc.cuh); a block that gives up
// sets g_wait_word and leaves.
#include <algorithm>

#include "ffn_internal.cuh"
#include "pdl.cuh"
#include "tc.cuh"

namespace cr {

__device__ unsigned int g_wait_word = 0;

namespace {

enum TileMode { kGlu = 0, kDx = 1, kDw = 2 };

constexpr int kM = 128;       // rows of a tile
constexpr int kN = 256;       // accumulator columns of a tile
constexpr int kK = 64;        // K of a block: 128 bytes of bf16
constexpr int kStages = 4;
constexpr uint32_t kABytes = kM * kK * 2, kBBytes = kN * kK * 2;
constexpr uint32_t kStageBytes = kABytes + kBBytes;
constexpr uint32_t kTileSmem = kStages * kStageBytes + 1024;  // + room to align to 1024
constexpr int kTileThreads = 192;
constexpr uint32_t kGroupM = 8;  // tile rows walked together, so that their operands stay in L2

struct TileArgs {
  CUtensorMap a[2], b[2];
  Mat out[2];
  Q8 g8, u8;
  uint32_t rows, cols;        // of an output
  uint32_t seg_blocks;        // K blocks of one product
  uint32_t blocks;            // K blocks of a tile: one or two products
  uint32_t tiles_m, tiles_n;  // of an output
  uint32_t tiles;             // of all outputs
  int width;                  // bytes of the output stores all rows allow: 32, 16 or 0
  int width8;                 // the same for the codes
};

__device__ __forceinline__ void st32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// n 32-byte words of a row, all inside it.
template <int WORDS>
__device__ __forceinline__ void st_words(void* p, const uint32_t* w, int width) {
  if (width == 32) {
#pragma unroll
    for (int i = 0; i < WORDS; i += 8) st32(static_cast<uint32_t*>(p) + i, w + i);
  } else {
#pragma unroll
    for (int i = 0; i < WORDS; i += 4)
      *reinterpret_cast<uint4*>(static_cast<uint32_t*>(p) + i) =
          make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  }
}

// 32 values at columns c .. c + 31 of a row.
template <int DT>
__device__ __forceinline__ void st_values(const Mat& m, uint64_t row, uint32_t c, uint32_t cols,
                                          int width, const float* v) {
  if constexpr (DT == CR_BF16) {
    uint16_t* p = static_cast<uint16_t*>(m.p) + row * m.ld + c;
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = ffn_bf16x2(v[2 * i], v[2 * i + 1]);
    if (width && c + 32 <= cols) return st_words<16>(p, w, width);
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (c + i < cols) p[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
  } else {
    float* p = static_cast<float*>(m.p) + row * m.ld + c;
    uint32_t w[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(v[i]);
    if (width && c + 32 <= cols) return st_words<32>(p, w, width);
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (c + i < cols) p[i] = v[i];
  }
}

__device__ __forceinline__ void st_codes(uint8_t* p, uint32_t c, uint32_t cols, int width,
                                         const float* v, float inv) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i] = e4m3x2(q8_scaled(v[4 * i], inv), q8_scaled(v[4 * i + 1], inv)) |
           e4m3x2(q8_scaled(v[4 * i + 2], inv), q8_scaled(v[4 * i + 3], inv)) << 16;
  if (width && c + 32 <= cols) return st_words<8>(p + c, w, width);
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (c + i < cols) p[c + i] = (uint8_t)(w[i / 4] >> (8 * (i & 3)));
}

// Tile `t` of an output, tile rows walked kGroupM at a time.
__device__ __forceinline__ void tile_at(const TileArgs& a, uint32_t t, uint32_t* which,
                                        uint32_t* tm, uint32_t* tn) {
  const uint32_t per_out = a.tiles_m * a.tiles_n;
  *which = t / per_out;
  t -= *which * per_out;
  const uint32_t per_group = kGroupM * a.tiles_n;
  const uint32_t group = t / per_group, first = group * kGroupM;
  const uint32_t height = min(kGroupM, a.tiles_m - first);
  t -= group * per_group;
  *tm = first + t % height;
  *tn = t / height;
}

// Zeros where a tile has no K at all (its accumulator was never written).
__device__ __forceinline__ void ld_acc(uint32_t addr, bool any, float* v) {
  if (any) return tc::tmem_ld32(addr, v);
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = 0.0f;
}

// EPI: the activation (kGlu) or the output's dtype.
template <int MODE, int EPI>
__device__ __forceinline__ void epilogue(const TileArgs& a, uint32_t acc, uint32_t which,
                                         uint32_t tm, uint32_t tn, int quarter, int lane) {
  const uint64_t row = (uint64_t)tm * kM + quarter * 32 + lane;
  const bool live = row < a.rows;
  const bool any = a.blocks != 0;
  acc += (uint32_t)(quarter * 32) << 16;
  if constexpr (MODE == kGlu) {
    const uint32_t c0 = tn * (kN / 2);
    float inv_g = 0.0f, inv_u = 0.0f;
    if (a.g8.codes || a.u8.codes) {
      // columns past the matrix hold zeros, which no magnitude is below
      float mg = 0.0f, mu = 0.0f;
#pragma unroll 1
      for (int c = 0; c < kN / 2; c += 32) {
        float g[32], u[32];
        ld_acc(acc + c, any, g);
        ld_acc(acc + kN / 2 + c, any, u);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          mg = fmaxf(mg, q8_magnitude(g[i])), mu = fmaxf(mu, q8_magnitude(u[i]));
      }
      const float sg = q8_scale(mg), su = q8_scale(mu);
      inv_g = 1.0f / sg, inv_u = 1.0f / su;
      if (live && a.g8.codes) a.g8.scales[row * a.g8.lds + tn] = sg;
      if (live && a.u8.codes) a.u8.scales[row * a.u8.lds + tn] = su;
    }
#pragma unroll 1
    for (int c = 0; c < kN / 2; c += 32) {
      float g[32], u[32];
      __syncwarp();  // rows past the matrix leave the last turn early
      ld_acc(acc + c, any, g);
      ld_acc(acc + kN / 2 + c, any, u);
      if (!live || c0 + c >= a.cols) continue;
      if (a.g8.codes) st_codes(a.g8.codes + row * a.g8.ld, c0 + c, a.cols, a.width8, g, inv_g);
      if (a.u8.codes) st_codes(a.u8.codes + row * a.u8.ld, c0 + c, a.cols, a.width8, u, inv_u);
#pragma unroll
      for (int i = 0; i < 32; ++i) g[i] = act_gate<EPI>(g[i]) * u[i];
      st_values<CR_BF16>(a.out[0], row, c0 + c, a.cols, a.width, g);
    }
  } else {
    const uint32_t c0 = tn * kN;
#pragma unroll 1
    for (int c = 0; c < kN; c += 32) {
      float v[32];
      __syncwarp();
      ld_acc(acc + c, any, v);
      if (live && c0 + c < a.cols) st_values<EPI>(a.out[which], row, c0 + c, a.cols, a.width, v);
    }
  }
}

template <int MODE, int EPI>
__global__ void __launch_bounds__(kTileThreads, 1) k_tiles(const __grid_constant__ TileArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 5];
  __shared__ uint32_t tmem_base;
  __shared__ uint32_t gave_up_word;
  volatile uint32_t* gave_up = &gave_up_word;
  const uint32_t smem = (tc::smem_addr(smem_raw) + 1023) & ~1023u;
  const uint32_t full = tc::smem_addr(bars), empty = full + 8 * kStages;
  const uint32_t acc_full = empty + 8 * kStages, acc_empty = acc_full + 16;
  const uint32_t drained = acc_empty + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::bar_init(full + 8 * s, 1);
      tc::bar_init(empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::bar_init(acc_full + 8 * b, 1);
      tc::bar_init(acc_empty + 8 * b, 128);
    }
    tc::bar_init(drained, 1);
    *gave_up = 0;
    tc::bar_init_fence();
  }
  if (warp == 1) tc::tmem_alloc(tc::smem_addr(&tmem_base), 2 * kN);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  pdl_enter();
  const uint32_t tmem = tmem_base;

  if (warp == 0 && lane == 0) {
    uint32_t it = 0;
    bool live = true;
    for (uint32_t t = blockIdx.x; t < a.tiles && live; t += gridDim.x) {
      uint32_t which, tm, tn;
      tile_at(a, t, &which, &tm, &tn);
      for (uint32_t k = 0; k < a.blocks; ++k, ++it) {
        const uint32_t s = it % kStages, bar = full + 8 * s;
        if (!tc::bar_wait(empty + 8 * s, (it / kStages & 1) ^ 1, gave_up)) {
          live = false;
          break;
        }
        const uint32_t seg = k >= a.seg_blocks;
        const int k0 = (int)((k - seg * a.seg_blocks) * kK);
        const uint32_t sa = smem + s * kStageBytes, sb = sa + kABytes;
        tc::bar_expect(bar, kStageBytes);
        if constexpr (MODE == kGlu) {
          tc::tma_load(sa, &a.a[0], k0, (int)(tm * kM), bar);
          tc::tma_load(sb, &a.b[0], k0, (int)(tn * (kN / 2)), bar);
          tc::tma_load(sb + kBBytes / 2, &a.b[1], k0, (int)(tn * (kN / 2)), bar);
        } else {
          if constexpr (MODE == kDx) {
            tc::tma_load(sa, &a.a[seg], k0, (int)(tm * kM), bar);
          } else {
#pragma unroll
            for (int j = 0; j < kM / 64; ++j)
              tc::tma_load(sa + j * 8192, &a.a[which], (int)(tm * kM) + j * 64, k0, bar);
          }
#pragma unroll
          for (int j = 0; j < kN / 64; ++j)
            tc::tma_load(sb + j * 8192, &a.b[seg], (int)(tn * kN) + j * 64, k0, bar);
        }
      }
    }
    if (!live) {
      // leave no copy in flight behind: the last kStages blocks issued
      const uint32_t first = it > kStages ? it - kStages : 0;
      for (uint32_t i = first; i < it; ++i) tc::bar_poll(full + 8 * (i % kStages), i / kStages & 1);
    }
  } else if (warp == 1 && lane == 0) {
    constexpr bool a_mn = MODE == kDw, b_mn = MODE != kGlu;
    constexpr uint32_t desc = tc::product_desc(kM, kN, a_mn, b_mn);
    uint32_t it = 0, n = 0;
    bool live = true;
    for (uint32_t t = blockIdx.x; t < a.tiles && live; t += gridDim.x, ++n) {
      const uint32_t buf = n & 1, acc = tmem + buf * kN;
      if (!tc::bar_wait(acc_empty + 8 * buf, (n >> 1 & 1) ^ 1, gave_up)) {
        live = false;
        break;
      }
      tc::fence_after();
      for (uint32_t k = 0; k < a.blocks; ++k, ++it) {
        const uint32_t s = it % kStages;
        if (!tc::bar_wait(full + 8 * s, it / kStages & 1, gave_up)) {
          live = false;
          break;
        }
        tc::fence_after();
        const uint32_t sa = smem + s * kStageBytes, sb = sa + kABytes;
#pragma unroll
        for (int j = 0; j < kK / 16; ++j) {
          // 16 K: 32 bytes along a row, or 16 rows
          const uint64_t da = a_mn ? tc::operand(sa + j * 2048, 8192, 1024) : tc::operand(sa + j * 32, 16, 1024);
          const uint64_t db = b_mn ? tc::operand(sb + j * 2048, 8192, 1024) : tc::operand(sb + j * 32, 16, 1024);
          tc::mma(acc, da, db, desc, k || j);
        }
        tc::mma_commit(empty + 8 * s);
      }
      if (live) tc::mma_commit(acc_full + 8 * buf);
    }
    if (!live) {  // leave no product in flight behind
      tc::mma_commit(drained);
      tc::bar_poll(drained, 0);
    }
  } else if (warp >= 2) {
    uint32_t n = 0;
    for (uint32_t t = blockIdx.x; t < a.tiles; t += gridDim.x, ++n) {
      const uint32_t buf = n & 1;
      uint32_t which, tm, tn;
      tile_at(a, t, &which, &tm, &tn);
      // one lane polls, so that the warp stays whole for the tensor memory loads
      bool got = true;
      if (lane == 0) got = tc::bar_wait(acc_full + 8 * buf, n >> 1 & 1, gave_up);
      if (!__shfl_sync(~0u, got, 0)) break;
      tc::fence_after();
      epilogue<MODE, EPI>(a, tmem + buf * kN, which, tm, tn, warp & 3, lane);
      tc::fence_before();
      tc::bar_arrive(acc_empty + 8 * buf);
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (threadIdx.x == 0 && *gave_up) atomicOr(&g_wait_word, 1u);
  if (warp == 1) tc::tmem_free(tmem, 2 * kN);
}

// ---- host side ------------------------------------------------------------------------

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once (nullptr without a driver).
EncodeFn encoder() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// rows x cols bf16 at m, read in boxes of 64 columns x box_rows.  An empty
// matrix is never loaded from: its map stays unset.
cudaError_t encode(CUtensorMap* map, const Mat& m, uint32_t rows, uint32_t cols, uint32_t box_rows) {
  if (!m.p || !rows || !cols) return cudaSuccess;
  const EncodeFn fn = encoder();
  if (!fn) return cudaErrorNotSupported;
  const uint64_t ld = rows > 1 ? m.ld : ((uint64_t)cols + 7) / 8 * 8;
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {ld * 2};
  const cuuint32_t box[2] = {kK, box_rows}, steps[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, m.p, dims, strides, box, steps,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

int store_width(const void* p, uint64_t pitch) {
  const uint64_t bits = reinterpret_cast<uintptr_t>(p) | pitch;
  return bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : 0;
}

uint32_t ceil_div(uint32_t a, uint32_t b) { return (uint32_t)(((uint64_t)a + b - 1) / b); }

// Bytes all rows of the outputs allow.
int out_width(const Mat& m, uint32_t rows, size_t es) { return store_width(m.p, rows > 1 ? m.ld * es : 0); }

template <int MODE, int EPI>
cudaError_t run_tiles(TileArgs& a, cudaStream_t s) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(k_tiles<MODE, EPI>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.tiles < (uint32_t)sms ? a.tiles : (uint32_t)sms);
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = kTileSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_tiles<MODE, EPI>, a);
}

// Tiles of `outputs` outputs of rows x cols, `width` columns a tile.
cudaError_t shape(TileArgs& a, uint32_t rows, uint32_t cols, uint32_t width, uint32_t k,
                  uint32_t products, uint32_t outputs) {
  a.rows = rows, a.cols = cols;
  a.tiles_m = ceil_div(rows, kM), a.tiles_n = ceil_div(cols, width);
  const uint64_t tiles = (uint64_t)a.tiles_m * a.tiles_n * outputs;
  const uint64_t blocks = (uint64_t)ceil_div(k, kK) * products;
  if (tiles >= 1ull << 31 || blocks >= 1ull << 31) return cudaErrorInvalidValue;
  a.tiles = (uint32_t)tiles;
  a.seg_blocks = ceil_div(k, kK);
  a.blocks = (uint32_t)blocks;
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_glu(cr_act act, const GluArgs& g, cudaStream_t s) {
  TileArgs a = {};
  cudaError_t e = shape(a, g.tokens, g.ffn, kN / 2, g.dim, 1, 1);
  if (e == cudaSuccess) e = encode(&a.a[0], g.x, g.tokens, g.dim, kM);
  if (e == cudaSuccess) e = encode(&a.b[0], g.wg, g.ffn, g.dim, kN / 2);
  if (e == cudaSuccess) e = encode(&a.b[1], g.wu, g.ffn, g.dim, kN / 2);
  if (e != cudaSuccess) return e;
  a.out[0] = g.a;
  a.g8 = g.g8, a.u8 = g.u8;
  a.width = out_width(g.a, g.tokens, 2);
  a.width8 = 32;
  for (const Q8* q : {&g.g8, &g.u8})
    if (q->codes) a.width8 = std::min(a.width8, store_width(q->codes, g.tokens > 1 ? q->ld : 0));
  return act == CR_ACT_SILU ? run_tiles<kGlu, CR_ACT_SILU>(a, s) : run_tiles<kGlu, CR_ACT_GELU>(a, s);
}

cudaError_t launch_glu_back(cr_dtype dw, const GluBackArgs& g, cudaStream_t s) {
  if (g.dx.p) {
    TileArgs a = {};
    cudaError_t e = shape(a, g.tokens, g.dim, kN, g.ffn, 2, 1);
    const Mat left[2] = {g.dg, g.du}, right[2] = {g.wg, g.wu};
    for (int k = 0; k < 2 && e == cudaSuccess; ++k) {
      e = encode(&a.a[k], left[k], g.tokens, g.ffn, kM);
      if (e == cudaSuccess) e = encode(&a.b[k], right[k], g.ffn, g.dim, kK);
    }
    if (e != cudaSuccess) return e;
    a.out[0] = g.dx;
    a.width = out_width(g.dx, g.tokens, 2);
    if ((e = run_tiles<kDx, CR_BF16>(a, s)) != cudaSuccess) return e;
  }
  if (!g.dwg && !g.dwu) return cudaSuccess;
  TileArgs a = {};
  const uint32_t outputs = g.dwg && g.dwu ? 2 : 1;
  cudaError_t e = shape(a, g.ffn, g.dim, kN, g.tokens, g.x_lo.p ? 2 : 1, outputs);
  if (e != cudaSuccess) return e;
  a.width = 32;
  uint32_t n = 0;
  for (int k = 0; k < 2; ++k) {
    void* out = k ? g.dwu : g.dwg;
    if (!out) continue;
    a.out[n] = Mat{out, g.dim};
    a.width = std::min(a.width, out_width(a.out[n], g.ffn, dw == CR_BF16 ? 2 : 4));
    if ((e = encode(&a.a[n++], k ? g.du : g.dg, g.tokens, g.ffn, kK)) != cudaSuccess) return e;
  }
  if ((e = encode(&a.b[0], g.x, g.tokens, g.dim, kK)) != cudaSuccess) return e;
  if ((e = encode(&a.b[1], g.x_lo, g.tokens, g.dim, kK)) != cudaSuccess) return e;
  return dw == CR_BF16 ? run_tiles<kDw, CR_BF16>(a, s) : run_tiles<kDw, CR_F32>(a, s);
}

cudaError_t glu_wait_word(bool clear, unsigned int* word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_wait_word, sizeof(*word));
  const unsigned int zero = 0;
  if (e == cudaSuccess && clear) e = cudaMemcpyToSymbol(g_wait_word, &zero, sizeof(zero));
  return e;
}

}  // namespace cr
