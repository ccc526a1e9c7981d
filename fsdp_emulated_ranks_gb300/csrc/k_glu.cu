// k_glu.cu -- the gated feed-forward block: both projections, the activation
// and the product in one kernel, and the products of its backward pass.
//
// One kernel, three uses (T tokens, D dim, F ffn; K in blocks of 64):
//   kGlu  a = act(x Wg^T) * (x Wu^T): a tile's 256 accumulator columns are the
//         same 128 columns of g and of u, so the epilogue has both in one
//         thread's row, and a tile's width is the 8-bit checkpoints' group.
//   kDx   dx = dg Wg + du Wu: one accumulator over both products.
//   kDw   dWg = dg^T x and dWu = du^T x: tiles of both in one launch.
// Operands are read as they lie in memory: rows of K (x, W of kGlu, dg and du
// of kDx) or rows of M or N (W of kDx, everything of kDw), which the tensor
// cores take directly, so nothing is transposed.
//
// k_tiles, for many tiles: persistent blocks, a tile 128 x 256.  Warp 0 loads by
// TMA into a ring of kStages buffers, warp 1 issues the products into one of
// two accumulators in tensor memory, warps 2-9 read the other one out and write
// the results.  TMA fills rows and columns outside a matrix with zeros, so
// ragged sizes need no masks before the epilogue.  Where K is long and the tiles
// are many, two tiles one below the other share their B as one tall tile, which
// loads 64 KB in place of 96 and fills tensor memory: its epilogue runs alone.
//
// k_split, where the tiles are too few for the SMs, and for the tiles that
// would leave most SMs idle in the last turn of k_tiles: the blocks of a
// cluster share one tile.  Each takes a range of its K, leaves its partial
// sums in its own shared memory, and then finishes a range of the tile's rows,
// reading the partials of all in rank order.  k_split_back runs the tiles of dx
// and of dW in one launch.
//
// Both let the next kernel's blocks onto their SMs only when their last products
// are loaded: a waiting block beside them would have nothing to do before.
//
// Measured, 8192 tokens, 2048 x 8192, three seconds on end under the power cap:
// forward 361 us (1.52 PFLOP/s), with codes 393; the backward pass 794, of which
// the products 688 (1.60 PFLOP/s; cuBLAS's four products of these sizes 707 on
// the same card), and 1105 from an 8-bit x, whose second part makes dW's
// products twice as many.  In short bursts forward 329 and 371, backward 734.
// A tile's K block takes 0.27 to 0.34 us, of which the products are 0.25: an SM
// takes 48 KB of it at 62 bytes a cycle from L2.  Tall tiles take 32 KB a tile:
// on one card the backward pass took 765 us with them and 825 without,
// forward over 4096 x 4096 342 and 357, 8192 x 2048 337 and 372.
//
// Every wait is bounded (tc.cuh); a block that gives up sets g_wait_word and
// leaves.  A wait for a tile's sums may last longer the longer K is.
#include <algorithm>
#include <map>
#include <mutex>
#include <type_traits>
#include <utility>

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
constexpr int kTileThreads = 320;

// A tall tile is two tiles, one below the other, that share their B.
constexpr int stages_of(bool tall) { return tall ? 3 : kStages; }
constexpr uint32_t stage_bytes(bool tall) { return (tall ? 2 : 1) * kABytes + kBBytes; }
constexpr uint32_t kTallSmem = stages_of(true) * stage_bytes(true) + 1024;

struct TileArgs {
  CUtensorMap a[4], b[2];     // kDw: a[2], a[3] are what a[0], a[1] were rounded by
  Mat out[2];
  Q8 g8, u8;
  uint32_t rows, cols;        // of an output
  uint32_t seg_blocks;        // K blocks of one product
  uint32_t blocks;            // K blocks of a tile: one to three products
  uint32_t a_lo;              // kDw: the second product takes a[2 + output]
  uint32_t tiles_m, tiles_n;  // of an output
  uint32_t tiles;             // k_tiles: tiles 0 .. tiles - 1 of all outputs
  uint32_t first;             // k_split: its first tile
  uint32_t pairs;             // tall tiles of an output's column of tiles; 0: none are used
  uint32_t skip;              // tall tiles of all outputs that come before tile 0
  uint32_t splits;            // k_split: blocks that share a tile, a power of two
  int width;                  // bytes of the output stores all rows allow: 32, 16 or 0
  int width8;                 // the same for the codes
};

template <int WORDS>
__device__ __forceinline__ void st_run(void* p, const uint32_t* w, int width) {
  uint32_t* out = static_cast<uint32_t*>(p);
#pragma unroll
  for (int i = 0; i < WORDS; i += 8)
    width == 32 ? st_words<2>(out + i, w + i) : st_words<1>(out + i, w + i);
}

constexpr int kSlab = 32 * 17;  // words of a warp's staging slab

// A warp's 32 rows x 32 columns of results, row `row0 + lane` in this
// thread's w, 4 / sizeof(T) results a word; columns c .. c + 31.  Whole rows
// go out as vectors, a thread its own row (full 32-byte sectors).  Where the
// row stride or the pointer does not allow that, or columns are missing, the
// warp turns the square round in shared memory, 16 words of a row at a time,
// and stores consecutive columns from consecutive lanes: the scattered element
// stores this replaces made the epilogue longer than the products.
template <typename T>
__device__ __forceinline__ void st_square(T* out, uint64_t ld, uint64_t row0, uint32_t c,
                                          uint32_t rows, uint32_t cols, int width, int lane,
                                          const uint32_t* w, uint32_t* slab) {
  constexpr int per = 4 / sizeof(T), words = 32 / per;
  if (width && c + 32 <= cols) {
    if (row0 + lane < rows) st_run<words>(out + (row0 + lane) * ld + c, w, width);
    return;
  }
  constexpr int part = words < 16 ? words : 16;          // words of a row a turn
  constexpr int wide = part * per, high = 32 / wide;      // columns and rows a store covers
  const uint32_t height = rows - row0 < 32 ? (uint32_t)(rows - row0) : 32u;
  const int x = lane % wide, y = lane / wide;
#pragma unroll
  for (int p = 0; p < words / part; ++p) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < part; ++i) slab[lane * 17 + i] = w[p * part + i];
    __syncwarp();
    const uint32_t col = c + p * wide + x;
    T* to = out + (row0 + y) * ld + col;
    const uint32_t* from = slab + y * 17 + x / per;
    const int shift = 8 * sizeof(T) * (x % per);
    if (col >= cols) continue;
    if (height == 32) {
#pragma unroll
      for (int r = 0; r < 32; r += high) to[r * ld] = (T)(from[r * 17] >> shift);
    } else {
      for (uint32_t r = 0; r + y < height; r += high) to[r * ld] = (T)(from[r * 17] >> shift);
    }
  }
}

template <int DT>
__device__ __forceinline__ void st_values(const Mat& m, uint64_t row0, uint32_t c, uint32_t rows,
                                          uint32_t cols, int width, int lane, const float* v,
                                          uint32_t* slab) {
  if constexpr (DT == CR_BF16) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = ffn_bf16x2(v[2 * i], v[2 * i + 1]);
    st_square(static_cast<uint16_t*>(m.p), m.ld, row0, c, rows, cols, width, lane, w, slab);
  } else {
    uint32_t w[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(v[i]);
    st_square(static_cast<uint32_t*>(m.p), m.ld, row0, c, rows, cols, width, lane, w, slab);
  }
}

// INF: the warp's rows hold infinities, which the codes make NaN.
template <bool INF>
__device__ __forceinline__ float code_value(float v, float inv) {
  if (INF && fabsf(v) > kFloatMax) return __int_as_float(0x7fc00000);
  return v * inv;
}

template <bool INF>
__device__ __forceinline__ void st_codes(const Q8& q, uint64_t row0, uint32_t c, uint32_t rows,
                                         uint32_t cols, int width, int lane, const float* v,
                                         float inv, uint32_t* slab) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i] = e4m3x2(code_value<INF>(v[4 * i], inv), code_value<INF>(v[4 * i + 1], inv)) |
           e4m3x2(code_value<INF>(v[4 * i + 2], inv), code_value<INF>(v[4 * i + 3], inv)) << 16;
  st_square(q.codes, q.ld, row0, c, rows, cols, width, lane, w, slab);
}

// Tile `t`: its output, first row and tile column.  Tile rows are walked 8 at a
// time, so that their operands stay in L2; 16 in kGlu, whose short K changes
// tiles often.  Forward at 8, 16 and 32 rows, on one card: 8192 x 2048 x 8192
// with codes 375, 355 and 343 us, 4096 x 2048 x 8192 with codes 204, 197 and 194,
// 8192 x 1024 x 16384 390, 371 and 359, 8192 x 1024 x 4096 99.6, 98.4 and 97.1,
// 16384 x 512 x 4096 107.1, 107.3 and 107.5: 32 would be up to 3 % faster than
// 16 where there are many tiles.  The backward pass of 8192 x 2048 x 8192,
// before it had tall tiles: 877, 880 and 895.
// Where some tiles are tall, the others are the halves of the tall tiles that
// come after them.
template <int MODE, bool TALL>
__device__ __forceinline__ void tile_at(const TileArgs& a, uint32_t t, uint32_t* which,
                                        uint32_t* row, uint32_t* tn) {
  const bool pairs = TALL || a.pairs;
  const uint32_t walk = (MODE == kGlu ? 16 : 8) / (pairs ? 2 : 1), lower = TALL || !pairs ? 0 : t & 1;
  const uint32_t high = pairs ? a.pairs : a.tiles_m;
  if (!TALL && pairs) t = a.skip + (t >> 1);
  const uint32_t per_out = high * a.tiles_n;
  *which = t / per_out;
  t -= *which * per_out;
  const uint32_t group = t / (walk * a.tiles_n), first = group * walk;
  const uint32_t height = min(walk, high - first);
  t -= group * walk * a.tiles_n;
  *row = ((first + t % height) * (pairs ? 2 : 1) + lower) * kM;
  *tn = t / height;
}

// Zeros where a tile has no K at all (its accumulator was never written).
__device__ __forceinline__ void ld_acc(uint32_t addr, bool any, float* v) {
  if (any) return tc::tmem_ld32(addr, v);
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = 0.0f;
}

__device__ __forceinline__ void ld_acc2(uint32_t addr, uint32_t addr2, bool any, float* v, float* v2) {
  if (any) return tc::tmem_ld32x2(addr, addr2, v, v2);
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = v2[i] = 0.0f;
}

// What the two warps that share 32 rows of a tile tell each other: each
// row's maxima over the 64 columns of g and of u that each has seen.  The
// turns alternate between two places, so one barrier a turn is enough.
struct Maxima {
  float2 seen[2][2][kM];  // turn & 1, half, row of the tile
  uint64_t bar[4];        // one for each 32 rows, an arrival of each warp
};

// Largest magnitudes of a row's 128 columns of g and of u, NaN passed over; with
// FINITE, infinities too.  Columns past the matrix hold zeros, which no
// magnitude is below.
template <bool FINITE>
__device__ __forceinline__ void row_maxima(uint32_t acc, bool any, Maxima* m, uint32_t* turn,
                                           volatile uint32_t* gave_up, int quarter, int half,
                                           int lane, float* mg, float* mu) {
  const int row = quarter * 32 + lane;
  const uint32_t bar = tc::smem_addr(&m->bar[quarter]);
  *mg = *mu = 0.0f;
#pragma unroll 1
  for (int c = half * 64; c < half * 64 + 64; c += 32) {
    float g[32], u[32];
    ld_acc2(acc + c, acc + kN / 2 + c, any, g, u);
    float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // short chains
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float a = fabsf(g[i + j]), b = fabsf(u[i + j]);
        x[j] = fmaxf(x[j], FINITE && a > kFloatMax ? 0.0f : a);
        x[2 + j] = fmaxf(x[2 + j], FINITE && b > kFloatMax ? 0.0f : b);
      }
    }
    *mg = fmaxf(*mg, fmaxf(x[0], x[1])), *mu = fmaxf(*mu, fmaxf(x[2], x[3]));
  }
  const uint32_t at = *turn & 1;
  m->seen[at][half][row] = make_float2(*mg, *mu);
  __syncwarp();
  if (lane == 0) {
    tc::bar_arrive(bar);
    tc::bar_wait(bar, at, gave_up);  // if it gives up, the next tile's wait ends the warp
  }
  __syncwarp();
  ++*turn;
  const float2 other = m->seen[at][half ^ 1][row];
  *mg = fmaxf(*mg, other.x), *mu = fmaxf(*mu, other.y);
}

// The same among finite values; only where some row of the warp holds an
// infinity (returned) are the columns looked at again.  Both warps of a row
// hold the same maxima, and so decide alike.
__device__ __forceinline__ bool row_magnitudes(uint32_t acc, bool any, Maxima* m, uint32_t* turn,
                                               volatile uint32_t* gave_up, int quarter, int half,
                                               int lane, float* mg, float* mu) {
  row_maxima<false>(acc, any, m, turn, gave_up, quarter, half, lane, mg, mu);
  const bool inf = __any_sync(~0u, *mg > kFloatMax || *mu > kFloatMax);
  if (inf) row_maxima<true>(acc, any, m, turn, gave_up, quarter, half, lane, mg, mu);
  return inf;
}

// Half `half` of the columns of a tile's rows `row0` .. + 31, which are lanes
// 32 * quarter .. + 31 of the accumulator.  EPI: the activation (kGlu) or the
// output's dtype.
template <int MODE, int EPI>
__device__ __forceinline__ void epilogue(const TileArgs& a, uint32_t acc, uint32_t which,
                                         uint64_t row0, uint32_t tn, int quarter, int half,
                                         int lane, uint32_t* slab, Maxima* maxima, uint32_t* turn,
                                         volatile uint32_t* gave_up) {
  if (row0 >= a.rows) return;
  const bool live = row0 + lane < a.rows;
  const bool any = a.blocks != 0;
  acc += (uint32_t)(quarter * 32) << 16;
  if constexpr (MODE == kGlu) {
    const uint32_t c0 = tn * (kN / 2);
    float inv_g = 0.0f, inv_u = 0.0f;
    bool inf = false;
    if (a.g8.codes || a.u8.codes) {
      float mg, mu;
      inf = row_magnitudes(acc, any, maxima, turn, gave_up, quarter, half, lane, &mg, &mu);
      const float sg = q8_scale(mg), su = q8_scale(mu);
      inv_g = 1.0f / sg, inv_u = 1.0f / su;
      if (live && half == 0) {
        if (a.g8.codes) a.g8.scales[(row0 + lane) * a.g8.lds + tn] = sg;
        if (a.u8.codes) a.u8.scales[(row0 + lane) * a.u8.lds + tn] = su;
      }
    }
#pragma unroll 1
    for (uint32_t c = half * 64; c < half * 64u + 64 && c0 + c < a.cols; c += 32) {
      float g[32], u[32];
      __syncwarp();  // the last square's stores leave rows past the matrix out
      ld_acc2(acc + c, acc + kN / 2 + c, any, g, u);
      const auto codes = [&](auto infinite) {
        constexpr bool kInf = decltype(infinite)::value;
        if (a.g8.codes)
          st_codes<kInf>(a.g8, row0, c0 + c, a.rows, a.cols, a.width8, lane, g, inv_g, slab);
        if (a.u8.codes)
          st_codes<kInf>(a.u8, row0, c0 + c, a.rows, a.cols, a.width8, lane, u, inv_u, slab);
      };
      if (inf)
        codes(std::true_type());
      else
        codes(std::false_type());
#pragma unroll
      for (int i = 0; i < 32; ++i) g[i] = act_gate<EPI>(g[i]) * u[i];
      st_values<CR_BF16>(a.out[0], row0, c0 + c, a.rows, a.cols, a.width, lane, g, slab);
    }
  } else {
    const uint32_t c0 = tn * kN;
#pragma unroll 1
    for (uint32_t c = half * 128; c < half * 128u + 128 && c0 + c < a.cols; c += 32) {
      float v[32];
      __syncwarp();
      ld_acc(acc + c, any, v);
      st_values<EPI>(a.out[which], row0, c0 + c, a.rows, a.cols, a.width, lane, v, slab);
    }
  }
  __syncwarp();
}

// Turns (tc.cuh) that the wait for the sums over so many K blocks may take
// beyond those of any wait: 16384 cycles a block, of which the products are 512
// and the loads at most some 2000 where all SMs wait for memory.  If the products
// stop, the warps that issue them and load for them give up first.  (Blocks
// counted as they go would make it exact, but a store each in the loop that
// issues the products made 8192 x 2048 x 8192 with codes 14 us longer.)
constexpr uint32_t kTurnBlocks = tc::kTurnCycles / 16384;

__device__ __forceinline__ int sum_turns(uint32_t blocks) { return (int)(blocks / kTurnBlocks); }

// The products of one K block, A at sa and B at sb: one thread.
template <int MODE>
__device__ __forceinline__ void multiply_block(uint32_t acc, uint32_t sa, uint32_t sb, bool first) {
  constexpr bool a_mn = MODE == kDw, b_mn = MODE != kGlu;
  constexpr uint32_t desc = tc::product_desc(kM, kN, a_mn, b_mn);
#pragma unroll
  for (int j = 0; j < kK / 16; ++j) {
    // 16 K: 32 bytes along a row, or 16 rows
    const uint64_t da = a_mn ? tc::operand(sa + j * 2048, 8192, 1024) : tc::operand(sa + j * 32, 16, 1024);
    const uint64_t db = b_mn ? tc::operand(sb + j * 2048, 8192, 1024) : tc::operand(sb + j * 32, 16, 1024);
    tc::mma(acc, da, db, desc, !first || j);
  }
}

// One K block of the tile at `row` into buffer `sa`, arriving on `bar`: one
// thread.
template <int MODE, bool TALL>
__device__ __forceinline__ void load_block(const TileArgs& a, uint32_t which, uint32_t row,
                                           uint32_t tn, uint32_t k, uint32_t sa, uint32_t bar) {
  constexpr int kHalves = TALL ? 2 : 1;
  const uint32_t seg = (k >= a.seg_blocks) + (k >= 2 * a.seg_blocks), sb = sa + kHalves * kABytes;
  const int k0 = (int)((k - seg * a.seg_blocks) * kK), m0 = (int)row;
  tc::bar_expect(bar, stage_bytes(TALL));
  if constexpr (MODE == kGlu) {
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
      tc::tma_load(sa + h * kABytes, &a.a[0], k0, m0 + h * kM, bar);
    tc::tma_load(sb, &a.b[0], k0, (int)(tn * (kN / 2)), bar);
    tc::tma_load(sb + kBBytes / 2, &a.b[1], k0, (int)(tn * (kN / 2)), bar);
  } else {
    if constexpr (MODE == kDx) {
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
        tc::tma_load(sa + h * kABytes, &a.a[seg], k0, m0 + h * kM, bar);
    } else {
      // (dg, x), then (rest of dg, x), then (dg, rest of x): those there are
      const CUtensorMap* left = &a.a[which + (a.a_lo && seg == 1 ? 2 : 0)];
#pragma unroll
      for (int j = 0; j < 2 * kHalves; ++j) tc::tma_load(sa + j * 8192, left, m0 + j * 64, k0, bar);
    }
    const CUtensorMap* right = &a.b[MODE == kDx ? seg : seg == a.a_lo + 1];
#pragma unroll
    for (int j = 0; j < kN / 64; ++j)
      tc::tma_load(sb + j * 8192, right, (int)(tn * kN) + j * 64, k0, bar);
  }
}

// ---- many tiles: persistent blocks ------------------------------------------------------

template <int MODE, int EPI, bool TALL>
__global__ void __launch_bounds__(kTileThreads, 1) k_tiles(const __grid_constant__ TileArgs a) {
  constexpr int kRing = stages_of(TALL);
  constexpr uint32_t kBytes = stage_bytes(TALL);
  constexpr int kHalves = TALL ? 2 : 1, kAccs = TALL ? 1 : 2;  // of an accumulator; accumulators
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kRing + 5];
  __shared__ Maxima maxima;
  __shared__ uint32_t tmem_base, slab[8 * kSlab];
  __shared__ uint32_t gave_up_word;
  volatile uint32_t* gave_up = &gave_up_word;
  const uint32_t smem = (tc::smem_addr(smem_raw) + 1023) & ~1023u;
  const uint32_t full = tc::smem_addr(bars), empty = full + 8 * kRing;
  const uint32_t acc_full = empty + 8 * kRing, acc_empty = acc_full + 16;
  const uint32_t drained = acc_empty + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kRing; ++s) {
      tc::bar_init(full + 8 * s, 1);
      tc::bar_init(empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::bar_init(acc_full + 8 * b, 1);
      tc::bar_init(acc_empty + 8 * b, 8);  // a lane of each epilogue warp
    }
    for (int q = 0; q < 4; ++q) tc::bar_init(tc::smem_addr(&maxima.bar[q]), 2);
    tc::bar_init(drained, 1);
    *gave_up = 0;
    tc::bar_init_fence();
  }
  if (warp == 1) tc::tmem_alloc(tc::smem_addr(&tmem_base), 2 * kN);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  pdl_wait_prerequisites();
  const uint32_t tmem = tmem_base;

  if (warp == 0 && lane == 0) {
    uint32_t it = 0;
    bool live = true;
    for (uint32_t t = blockIdx.x; t < a.tiles && live; t += gridDim.x) {
      uint32_t which, row, tn;
      tile_at<MODE, TALL>(a, t, &which, &row, &tn);
      for (uint32_t k = 0; k < a.blocks; ++k, ++it) {
        const uint32_t s = it % kRing;
        if (!(live = tc::bar_wait(empty + 8 * s, (it / kRing & 1) ^ 1, gave_up))) break;
        load_block<MODE, TALL>(a, which, row, tn, k, smem + s * kBytes, full + 8 * s);
      }
    }
    pdl_launch_dependents();
    if (!live) {
      // leave no copy in flight behind: the last kRing blocks issued
      const uint32_t first = it > kRing ? it - kRing : 0;
      for (uint32_t i = first; i < it; ++i) tc::bar_poll(full + 8 * (i % kRing), i / kRing & 1);
    }
  } else if (warp == 1 && lane == 0) {
    uint32_t it = 0, n = 0;
    bool live = true;
    for (uint32_t t = blockIdx.x; t < a.tiles && live; t += gridDim.x, ++n) {
      const uint32_t buf = n % kAccs, acc = tmem + buf * kN;
      if (!(live = tc::bar_wait(acc_empty + 8 * buf, (n / kAccs & 1) ^ 1, gave_up))) break;
      tc::fence_after();
      for (uint32_t k = 0; k < a.blocks; ++k, ++it) {
        const uint32_t s = it % kRing;
        if (!(live = tc::bar_wait(full + 8 * s, it / kRing & 1, gave_up))) break;
        tc::fence_after();
        const uint32_t sa = smem + s * kBytes;
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
          multiply_block<MODE>(acc + h * kN, sa + h * kABytes, sa + kHalves * kABytes, k == 0);
        tc::mma_commit(empty + 8 * s);
      }
      if (live) tc::mma_commit(acc_full + 8 * buf);
    }
    if (!live) {  // leave no product in flight behind
      tc::mma_commit(drained);
      tc::bar_poll(drained, 0);
    }
  } else if (warp >= 2) {
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    uint32_t n = 0, turn = 0;
    for (uint32_t t = blockIdx.x; t < a.tiles; t += gridDim.x, ++n) {
      const uint32_t buf = n % kAccs;
      uint32_t which, row, tn;
      tile_at<MODE, TALL>(a, t, &which, &row, &tn);
      // one lane polls, so that the warp stays whole for the tensor memory loads
      bool got = true;
      if (lane == 0) got = tc::bar_wait(acc_full + 8 * buf, n / kAccs & 1, gave_up, sum_turns(a.blocks));
      if (!__shfl_sync(~0u, got, 0)) break;
      tc::fence_after();
#pragma unroll 1
      for (int h = 0; h < kHalves; ++h)
        epilogue<MODE, EPI>(a, tmem + (buf + h) * kN, which, (uint64_t)row + h * kM + quarter * 32,
                            tn, quarter, half, lane, slab + (warp - 2) * kSlab, &maxima, &turn,
                            gave_up);
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(acc_empty + 8 * buf);
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (threadIdx.x == 0 && *gave_up) atomicOr(&g_wait_word, 1u);
  if (warp == 1) tc::tmem_free(tmem, 2 * kN);
}

// ---- few tiles: a cluster for each ------------------------------------------------------

constexpr int kPartStride = kN + 4;  // floats: rows 16 bytes apart in the banks
static_assert(kM * kPartStride * 4 <= kStages * kStageBytes, "partials reuse the buffers");

// One row of a tile, columns 4 * lane .. + 3 of each half (for kGlu, of g and
// of u): whole warp.
template <int MODE, int EPI>
__device__ __forceinline__ void finish_row(const TileArgs& a, uint32_t which, uint64_t row,
                                           uint32_t tn, int lane, const float* lo, const float* hi) {
  if constexpr (MODE == kGlu) {
    const uint32_t c = tn * (kN / 2) + 4 * lane;
    float act[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) act[i] = act_gate<EPI>(lo[i]) * hi[i];
    uint16_t* p = static_cast<uint16_t*>(a.out[0].p) + row * a.out[0].ld + c;
    if (a.width && c + 4 <= a.cols) {
      *reinterpret_cast<uint2*>(p) = make_uint2(ffn_bf16x2(act[0], act[1]), ffn_bf16x2(act[2], act[3]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < a.cols) p[i] = (uint16_t)ffn_bf16x2(act[i], 0.0f);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const Q8& q = k ? a.u8 : a.g8;
      if (!q.codes) continue;
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = k ? hi[i] : lo[i];
      const float m = q8_magnitude<4>(v, [](float x) {
#pragma unroll
        for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, o));
        return x;
      });
      const float s = q8_scale(m), inv = 1.0f / s;
      if (lane == 0) q.scales[row * q.lds + tn] = s;
      const uint32_t w = e4m3x2(v[0] * inv, v[1] * inv) | e4m3x2(v[2] * inv, v[3] * inv) << 16;
      uint8_t* codes = q.codes + row * q.ld + c;
      if (a.width8 && c + 4 <= a.cols) {
        *reinterpret_cast<uint32_t*>(codes) = w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c + i < a.cols) codes[i] = (uint8_t)(w >> (8 * i));
      }
    }
  } else {
    const Mat& m = a.out[which];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t c = tn * kN + k * (kN / 2) + 4 * lane;
      const float* v = k ? hi : lo;
      if constexpr (EPI == CR_BF16) {
        uint16_t* p = static_cast<uint16_t*>(m.p) + row * m.ld + c;
        if (a.width && c + 4 <= a.cols) {
          *reinterpret_cast<uint2*>(p) = make_uint2(ffn_bf16x2(v[0], v[1]), ffn_bf16x2(v[2], v[3]));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c + i < a.cols) p[i] = (uint16_t)ffn_bf16x2(v[i], 0.0f);
        }
      } else {
        float* p = static_cast<float*>(m.p) + row * m.ld + c;
        if (a.width && c + 4 <= a.cols) {
          *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c + i < a.cols) p[i] = v[i];
        }
      }
    }
  }
}

// What every kernel of split tiles keeps in shared memory beside its buffers.
struct SplitShared {
  uint64_t bars[2 * kStages + 1];
  uint32_t tmem_base;
  uint32_t gave_up;
};

// Block `rank` of the a.splits that share tile a.first + `unit`: the rank-th part of its K blocks, then the rank-th part of its rows.  They are
// blocks `peer` .. + splits - 1 of the cluster.  A unit past the last (`units`)
// only takes part in the cluster's barriers.
template <int MODE, int EPI>
__device__ __forceinline__ void split_tile(const TileArgs& a, SplitShared* sh, uint32_t unit,
                                           uint32_t units, uint32_t rank, uint32_t peer) {
  extern __shared__ uint8_t smem_raw[];
  volatile uint32_t* gave_up = &sh->gave_up;
  const uint32_t smem = (tc::smem_addr(smem_raw) + 1023) & ~1023u;
  float* part = reinterpret_cast<float*>(smem_raw + (smem - tc::smem_addr(smem_raw)));
  const uint32_t full = tc::smem_addr(sh->bars), empty = full + 8 * kStages;
  const uint32_t acc_full = empty + 8 * kStages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t tmem = sh->tmem_base;
  const bool mine = unit < units;
  uint32_t which = 0, row0 = 0, tn = 0, k0 = 0, k1 = 0;
  if (mine) {
    tile_at<MODE, false>(a, a.first + unit, &which, &row0, &tn);
    k0 = (uint32_t)((uint64_t)a.blocks * rank / a.splits);
    k1 = (uint32_t)((uint64_t)a.blocks * (rank + 1) / a.splits);
  }

  if (warp == 0 && lane == 0) {
    uint32_t it = 0;
    bool live = true;
    for (uint32_t k = k0; k < k1; ++k, ++it) {
      const uint32_t s = it % kStages;
      if (!(live = tc::bar_wait(empty + 8 * s, (it / kStages & 1) ^ 1, gave_up))) break;
      load_block<MODE, false>(a, which, row0, tn, k, smem + s * kStageBytes, full + 8 * s);
    }
    pdl_launch_dependents();
    if (!live) {
      // leave no copy in flight behind: the last kStages blocks issued
      const uint32_t first = it > kStages ? it - kStages : 0;
      for (uint32_t i = first; i < it; ++i) tc::bar_poll(full + 8 * (i % kStages), i / kStages & 1);
    }
  } else if (warp == 1 && lane == 0) {
    uint32_t it = 0;
    for (uint32_t k = k0; k < k1; ++k, ++it) {
      const uint32_t s = it % kStages;
      if (!tc::bar_wait(full + 8 * s, it / kStages & 1, gave_up)) break;
      tc::fence_after();
      const uint32_t sa = smem + s * kStageBytes;
      multiply_block<MODE>(tmem, sa, sa + kABytes, k == k0);
      tc::mma_commit(empty + 8 * s);
    }
    // every product issued: the buffers are free and the sums complete
    tc::mma_commit(acc_full);
    tc::bar_poll(acc_full, 0);
  }
  __syncwarp();
  if (warp >= 2 && mine) {
    if (lane == 0) tc::bar_wait(acc_full, 0, gave_up, sum_turns(k1 - k0));
    __syncwarp();
    tc::fence_after();
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    float* row = part + (quarter * 32 + lane) * kPartStride;
    const bool any = k1 > k0;
#pragma unroll 1
    for (int c = half * 128; c < half * 128 + 128; c += 32) {
      float v[32];
      ld_acc(tmem + ((uint32_t)(quarter * 32) << 16) + c, any, v);
#pragma unroll
      for (int i = 0; i < 32; i += 4)
        *reinterpret_cast<float4*>(row + c + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
    tc::fence_before();
  }
  __syncwarp();
  tc::cluster_sync();
  if (mine) {
    // kRows rows a warp at a time, so that as many reads are in flight
    constexpr int kRows = 4, kWarps = kTileThreads / 32;
    const int height = kM / (int)a.splits, at0 = (int)rank * height;
    for (int r = warp; r < height; r += kRows * kWarps) {
      float4 lo[kRows], hi[kRows];
#pragma unroll
      for (int j = 0; j < kRows; ++j) lo[j] = hi[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (uint32_t p = 0; p < a.splits; ++p) {
        const uint32_t from = tc::cluster_addr(smem, peer + p) + 16 * lane;
        float4 x[kRows], y[kRows];
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          // rows past this block's part are read again from its last, and dropped
          const int at = at0 + min(r + j * kWarps, height - 1);
          x[j] = tc::cluster_ld4(from + (uint32_t)(at * kPartStride) * 4);
          y[j] = tc::cluster_ld4(from + (uint32_t)(at * kPartStride + kN / 2) * 4);
        }
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          lo[j].x += x[j].x, lo[j].y += x[j].y, lo[j].z += x[j].z, lo[j].w += x[j].w;
          hi[j].x += y[j].x, hi[j].y += y[j].y, hi[j].z += y[j].z, hi[j].w += y[j].w;
        }
      }
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const uint64_t row = (uint64_t)row0 + at0 + r + j * kWarps;
        if (r + j * kWarps < height && row < a.rows)
          finish_row<MODE, EPI>(a, which, row, tn, lane, &lo[j].x, &hi[j].x);
      }
    }
  }
  __syncwarp();
  tc::cluster_sync();  // no block leaves while another reads its partials
}

__device__ __forceinline__ void split_begin(SplitShared* sh) {
  if (threadIdx.x == 0) {
    const uint32_t bars = tc::smem_addr(sh->bars);
    for (int b = 0; b < 2 * kStages + 1; ++b) tc::bar_init(bars + 8 * b, 1);
    sh->gave_up = 0;
    tc::bar_init_fence();
  }
  if (threadIdx.x >> 5 == 1) tc::tmem_alloc(tc::smem_addr(&sh->tmem_base), kN);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  pdl_wait_prerequisites();
}

__device__ __forceinline__ void split_end(SplitShared* sh) {
  tc::fence_after();
  if (threadIdx.x == 0 && sh->gave_up) atomicOr(&g_wait_word, 1u);
  if (threadIdx.x >> 5 == 1) tc::tmem_free(sh->tmem_base, kN);
}

// A cluster of a.splits blocks for each tile from a.first on.
template <int MODE, int EPI>
__global__ void __launch_bounds__(kTileThreads, 1) k_split(const __grid_constant__ TileArgs a) {
  __shared__ __align__(8) SplitShared sh;
  split_begin(&sh);
  split_tile<MODE, EPI>(a, &sh, blockIdx.x / a.splits, ~0u, tc::cluster_rank(), 0);
  split_end(&sh);
}

// dx and dW at once, where both together have few tiles: blocks 0 ..
// dx_blocks - 1 work on dx, the others on dW.  The cluster is as large as the
// larger of the two splits.
struct BackArgs {
  TileArgs dx, dw;
  uint32_t dx_blocks, dx_units, dw_units;
};

template <int DW>
__global__ void __launch_bounds__(kTileThreads, 1) k_split_back(const __grid_constant__ BackArgs b) {
  __shared__ __align__(8) SplitShared sh;
  split_begin(&sh);
  const uint32_t crank = tc::cluster_rank();
  if (blockIdx.x < b.dx_blocks) {
    const uint32_t rank = crank % b.dx.splits;
    split_tile<kDx, CR_BF16>(b.dx, &sh, blockIdx.x / b.dx.splits, b.dx_units, rank, crank - rank);
  } else {
    const uint32_t rank = crank % b.dw.splits, at = blockIdx.x - b.dx_blocks;
    split_tile<kDw, DW>(b.dw, &sh, at / b.dw.splits, b.dw_units, rank, crank - rank);
  }
  split_end(&sh);
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

using Kernel = void (*)(const TileArgs);

struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];

  Launch(uint32_t grid, uint32_t threads, uint32_t smem, uint32_t cluster, cudaStream_t s) {
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
};

// Blocks of these kernels the device holds at once (an SM holds one), by log2
// of the cluster, whose SMs lie in one part of the chip.
constexpr int kClusterLogs = 3;
struct Capacity {
  uint32_t blocks[kClusterLogs];
};

// Cached per device.  Every kernel is allowed its shared memory here.
cudaError_t capacity(Capacity* out) {
  static std::mutex mu;
  static std::map<int, Capacity> cache;
  int dev = 0, n = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  const auto it = cache.find(dev);
  if (it != cache.end()) {
    *out = it->second;
    return cudaSuccess;
  }
  for (Kernel k : {k_tiles<kGlu, CR_ACT_SILU, false>, k_tiles<kGlu, CR_ACT_GELU, false>, k_tiles<kDx, CR_BF16, false>,
                   k_tiles<kDw, CR_BF16, false>, k_tiles<kDw, CR_F32, false>, k_split<kGlu, CR_ACT_SILU>,
                   k_split<kGlu, CR_ACT_GELU>, k_split<kDx, CR_BF16>, k_split<kDw, CR_BF16>,
                   k_split<kDw, CR_F32>}) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileSmem);
    if (e != cudaSuccess) return e;
  }
  for (Kernel k : {k_tiles<kGlu, CR_ACT_SILU, true>, k_tiles<kGlu, CR_ACT_GELU, true>, k_tiles<kDx, CR_BF16, true>, k_tiles<kDw, CR_BF16, true>, k_tiles<kDw, CR_F32, true>}) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kTallSmem);
    if (e != cudaSuccess) return e;
  }
  for (auto k : {k_split_back<CR_BF16>, k_split_back<CR_F32>}) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileSmem);
    if (e != cudaSuccess) return e;
  }
  Capacity c;
  for (int log = 0; log < kClusterLogs; ++log) {
    Launch split(1u << log, kTileThreads, kTileSmem, 1u << log, nullptr);
    split.cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&n, k_split<kGlu, CR_ACT_SILU>, &split.cfg);
    if (e != cudaSuccess) return e;
    c.blocks[log] = (uint32_t)std::max(n, 1) << log;
  }
  *out = cache[dev] = c;
  return cudaSuccess;
}

// Blocks to share a tile: as many as find an SM each, all units at once, and
// have at least `least` K blocks; 4 at most.  Clusters of 8 wait long for 8
// free SMs in one part of the chip: 6 tiles of dx and 64 of dW (257 x 512 x
// 2048) took 31.1 us in clusters of 8, 19.6 of 4, 19.3 of 2 and 26.6 unsplit; 8
// tiles of dx alone (64 x 2048 x 8192 backward) 66 us in all in clusters of 8,
// 61 of 4.
uint32_t splits_of(uint32_t units, uint32_t blocks, const Capacity& c, uint32_t least) {
  int log = 0;
  while (log + 1 < kClusterLogs && (uint64_t)units << (log + 1) <= c.blocks[log + 1] &&
         blocks >= (least << (log + 1)))
    ++log;
  return 1u << log;
}

constexpr uint32_t kMinBlocks = 4;    // K blocks worth a block of a cluster
// K blocks from which tall tiles are the faster: dW of 2048 x 8192 over 2048
// tokens (32) 216 us against 216 with the rest of its backward pass, over 1024
// 130 against 125; kGlu over 8192 tokens and 8192 columns, no codes, 2048 (32)
// 349 against 353, 1024 187 against 176.  With codes (read back after it) the
// epilogue, which a tall tile does not overlap with products, is longer: 2048 443 against 430, 2560 504
// against 503, 2816 558 against 553, 4096 x 4096 392 against 405.  Rows that do
// not start on 128 bytes cost more L2 traffic, which tall tiles save: 2040 with
// codes 497 against 587.
constexpr uint32_t kTallBlocks = 32, kTallBlocksCodes = 48;
constexpr uint32_t kTailBlocks = 32;  // K blocks for which splitting the last turn is worth a launch

// Clusters for a tile each if several blocks find SMs for every tile; else
// persistent blocks, the last turn's tiles split where they would leave most
// SMs idle.
template <int MODE, int EPI>
cudaError_t run_tiles(TileArgs& a, uint32_t outputs, cudaStream_t s, uint32_t least = kTallBlocks) {
  Capacity cap;
  cudaError_t e = capacity(&cap);
  if (e != cudaSuccess) return e;
  uint64_t n = (uint64_t)a.tiles_m * a.tiles_n * outputs;
  if (n >= 1ull << 31) return cudaErrorInvalidValue;
  const uint32_t sms = cap.blocks[0];
  if (n > sms && a.blocks >= least) {
    // as many tall tiles as make whole turns, or fill more than half the SMs in
    // the last: two tiles on an SM in turn take longer than the tall one
    a.pairs = ceil_div(a.tiles_m, 2);
    const uint32_t all = a.pairs * a.tiles_n * outputs, rest = all % sms;
    a.tiles = a.skip = 2 * rest > sms ? all : all - rest;
    const Launch l(std::min(a.tiles, sms), kTileThreads, kTallSmem, 1, s);
    if ((e = cudaLaunchKernelEx(&l.cfg, k_tiles<MODE, EPI, true>, a)) != cudaSuccess) return e;
    n = 2 * (all - a.skip);
    if (!n) return cudaSuccess;
  }
  const uint32_t rest = (uint32_t)(n % sms);
  uint32_t units = 0;
  a.tiles = (uint32_t)n;
  if (n <= sms) {
    units = (uint32_t)n;
    a.splits = splits_of(units, a.blocks, cap, kMinBlocks);
    if (a.splits == 1) units = 0;  // k_tiles ends sooner after its products: 11.5 against 13.7 us
  } else if (rest) {
    a.splits = splits_of(rest, a.blocks, cap, kTailBlocks);
    if (a.splits > 1) units = rest;
  }
  a.tiles -= units;
  if (a.tiles) {
    const Launch l(std::min(a.tiles, sms), kTileThreads, kTileSmem, 1, s);
    if ((e = cudaLaunchKernelEx(&l.cfg, k_tiles<MODE, EPI, false>, a)) != cudaSuccess) return e;
  }
  if (!units) return cudaSuccess;
  a.first = a.tiles;
  const Launch l(units * a.splits, kTileThreads, kTileSmem, a.splits, s);
  return cudaLaunchKernelEx(&l.cfg, k_split<MODE, EPI>, a);
}

// dx and dW in one launch, if their tiles together leave an SM for each.  The blocks left over go to whichever has the more K blocks a block.
template <int DW>
cudaError_t run_split_back(BackArgs& b, uint32_t outputs, bool* done, cudaStream_t s) {
  Capacity cap;
  cudaError_t e = capacity(&cap);
  if (e != cudaSuccess) return e;
  TileArgs* const both[2] = {&b.dx, &b.dw};
  uint64_t units[2];
  for (int k = 0; k < 2; ++k) {
    TileArgs& a = *both[k];
    a.splits = 1;
    units[k] = (uint64_t)a.tiles_m * a.tiles_n * (k ? outputs : 1);
  }
  if (units[0] + units[1] > cap.blocks[0]) return cudaSuccess;
  b.dx_units = (uint32_t)units[0], b.dw_units = (uint32_t)units[1];
  const auto blocks = [&](int k, uint32_t cluster) {  // whole clusters of them
    return ceil_div((uint32_t)units[k] * both[k]->splits, cluster) * cluster;
  };
  uint32_t cluster = 1;
  const auto log2 = [](uint32_t c) { return c == 4 ? 2 : c == 2 ? 1 : 0; };
  for (;;) {
    int k = both[0]->blocks / both[0]->splits >= both[1]->blocks / both[1]->splits ? 0 : 1;
    bool grown = false;
    for (int look = 0; look < 2 && !grown; ++look, k ^= 1) {
      TileArgs& a = *both[k];
      if (a.splits == 1u << (kClusterLogs - 1) || a.blocks < a.splits * 2 * kMinBlocks) continue;
      a.splits *= 2;
      const uint32_t c = std::max(cluster, a.splits);
      if (blocks(0, c) + blocks(1, c) <= cap.blocks[log2(c)]) {
        cluster = c;
        grown = true;
      } else {
        a.splits /= 2;
      }
    }
    if (!grown) break;
  }
  b.dx_blocks = blocks(0, cluster);
  *done = true;
  const Launch l(b.dx_blocks + blocks(1, cluster), kTileThreads, kTileSmem, cluster, s);
  return cudaLaunchKernelEx(&l.cfg, k_split_back<DW>, b);
}

// An output of rows x cols, `width` columns a tile, of `products` products
// over k.
cudaError_t shape(TileArgs& a, uint32_t rows, uint32_t cols, uint32_t width, uint32_t k,
                  uint32_t products) {
  a.rows = rows, a.cols = cols;
  a.tiles_m = ceil_div(rows, kM), a.tiles_n = ceil_div(cols, width);
  const uint64_t blocks = (uint64_t)ceil_div(k, kK) * products;
  if (blocks >= 1ull << 31) return cudaErrorInvalidValue;
  a.seg_blocks = ceil_div(k, kK);
  a.blocks = (uint32_t)blocks;
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_glu(cr_act act, const GluArgs& g, cudaStream_t s) {
  TileArgs a = {};
  cudaError_t e = shape(a, g.tokens, g.ffn, kN / 2, g.dim, 1);
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
  bool apart = false;  // rows of 128 bytes start in the middle of one
  for (const Mat* m : {&g.x, &g.wg, &g.wu})
    apart = apart || (reinterpret_cast<uintptr_t>(m->p) | m->ld * 2) % 128;
  const uint32_t least = (g.g8.codes || g.u8.codes) && !apart ? kTallBlocksCodes : kTallBlocks;
  return act == CR_ACT_SILU ? run_tiles<kGlu, CR_ACT_SILU>(a, 1, s, least)
                            : run_tiles<kGlu, CR_ACT_GELU>(a, 1, s, least);
}

cudaError_t launch_glu_back(cr_dtype dw, const GluBackArgs& g, cudaStream_t s) {
  BackArgs b = {};
  cudaError_t e = cudaSuccess;
  if (g.dx.p) {
    TileArgs& a = b.dx;
    e = shape(a, g.tokens, g.dim, kN, g.ffn, 2);
    const Mat left[2] = {g.dg, g.du}, right[2] = {g.wg, g.wu};
    for (int k = 0; k < 2 && e == cudaSuccess; ++k) {
      e = encode(&a.a[k], left[k], g.tokens, g.ffn, kM);
      if (e == cudaSuccess) e = encode(&a.b[k], right[k], g.ffn, g.dim, kK);
    }
    if (e != cudaSuccess) return e;
    a.out[0] = g.dx;
    a.width = out_width(g.dx, g.tokens, 2);
  }
  const uint32_t outputs = (g.dwg ? 1 : 0) + (g.dwu ? 1 : 0);
  if (outputs) {
    TileArgs& a = b.dw;
    a.a_lo = g.dg_lo.p != nullptr;
    e = shape(a, g.ffn, g.dim, kN, g.tokens, 1 + a.a_lo + (g.x_lo.p != nullptr));
    a.width = 32;
    uint32_t n = 0;
    for (int k = 0; k < 2 && e == cudaSuccess; ++k) {
      void* out = k ? g.dwu : g.dwg;
      if (!out) continue;
      a.out[n] = Mat{out, g.dim};
      a.width = std::min(a.width, out_width(a.out[n], g.ffn, dw == CR_BF16 ? 2 : 4));
      e = encode(&a.a[n], k ? g.du : g.dg, g.tokens, g.ffn, kK);
      if (e == cudaSuccess) e = encode(&a.a[2 + n], k ? g.du_lo : g.dg_lo, g.tokens, g.ffn, kK);
      ++n;
    }
    if (e == cudaSuccess) e = encode(&a.b[0], g.x, g.tokens, g.dim, kK);
    if (e == cudaSuccess) e = encode(&a.b[1], g.x_lo, g.tokens, g.dim, kK);
    if (e != cudaSuccess) return e;
  }
  if (g.dx.p && outputs) {
    bool done = false;
    e = dw == CR_BF16 ? run_split_back<CR_BF16>(b, outputs, &done, s)
                      : run_split_back<CR_F32>(b, outputs, &done, s);
    if (e != cudaSuccess || done) return e;
  }
  if (g.dx.p && (e = run_tiles<kDx, CR_BF16>(b.dx, 1, s)) != cudaSuccess) return e;
  if (!outputs) return cudaSuccess;
  return dw == CR_BF16 ? run_tiles<kDw, CR_BF16>(b.dw, outputs, s)
                       : run_tiles<kDw, CR_F32>(b.dw, outputs, s);
}

cudaError_t glu_wait_word(bool clear, unsigned int* word) {
  // the default stream, which the copies go by, does not wait for every stream
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(word, g_wait_word, sizeof(*word));
  const unsigned int zero = 0;
  // a word that was 0 is left alone: it may have been set since
  if (e == cudaSuccess && clear && *word) e = cudaMemcpyToSymbol(g_wait_word, &zero, sizeof(zero));
  return e;
}

}  // namespace cr
