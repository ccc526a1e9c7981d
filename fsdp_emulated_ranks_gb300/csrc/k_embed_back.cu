// k_embed_back.cu -- the embedding's gradient: for each row of the table, the sum of the
// gradients of the tokens that name it.
//
// Tokens are sorted by id first, so that a row's sum has a fixed order and every row is
// written once, by whoever adds it up:
//   1. k_group  A block takes a bucket, the ids that share their low bits.  It reads all ids
//               twice: to count its ids' tokens (and all tokens of earlier buckets, which is where
//               its own begin), and to put its tokens in order of id, then of token.
//   2. k_sum    A warp takes a chunk of the columns of a tile of tokens next to each other in that
//               order, and adds up rows until the id changes: the work of a warp does not depend on
//               how often an id occurs.  A table row that lies in one tile is written at once; of one in
//               several, each warp leaves an fp32 sum in the workspace, and the last to finish adds
//               them up in order.
//   3. k_free   Writes the rows that no token names.  It starts when k_sum's blocks have
//               started, not when they have ended: the table's zeros fill the time in which k_sum waits for
//               dout.
// Reading the ids once for each bucket costs little: they stay in L2, and are 8 bytes to a row of dout's
// thousands.  Bound by memory: dout is read and the table written once.
//
// Measured, 8192 x 2048 bf16 into 32000 rows (165 MB): 36.6 us a call in a loop, 4.5 TB/s; 27.4 with no
// token at all, of which 8 are the sort and the launches' starts; 29.0 in place (60 MB).  With k_free's work at the end of k_sum's launch
// (80 registers a thread for stores) 43.
#include <algorithm>

#include "lm_internal.cuh"
#include "pdl.cuh"

namespace cr {

namespace {

constexpr int kThreads = 1024;        // of a block of k_group
constexpr int kEach = 8;              // ids of a thread at a time
constexpr uint32_t kStepBits = 13, kStep = 1u << kStepBits;
static_assert(kStep == kThreads * kEach, "a step is every thread's ids");
constexpr uint32_t kLocals = 2048;    // ids of a bucket at most
constexpr uint32_t kLeastBuckets = 128;

// The workspace.
struct Sorted {
  uint2* order;      // [tokens] id and token, by bucket, id, token
  uint2* rows;       // [vocab] first place of the row's tokens in that order, and how many
  uint32_t* total;   // places in use
  // Of rows in several tiles: a part's slot is 2 * tile for a row that began in an earlier tile, and one
  // more for a row that goes on in the next.  kGroup parts are a group, at its first part's slot.
  float* sums;       // [slots][pitch] a part's sum, then its group's
  uint32_t* ticks;   // [slots][slices] parts of a group that are done
  uint32_t* groups;  // [slots][slices] groups of a row that are done, at its first part's slot
  uint32_t buckets, bucket_bits, tile_bits, tiles, slices;
  uint64_t pitch;
};

constexpr uint32_t kGroup = 8;  // parts that one warp adds up, one after another

// The slot of part p of a row that begins in tile `from`.
__device__ __forceinline__ uint64_t slot_of(uint32_t from, uint32_t p) {
  return 2 * ((uint64_t)from + p) + (p ? 0 : 1);
}

uint64_t up(uint64_t v, uint64_t m) { return (v + m - 1) / m * m; }

// Tokens of a tile: few where there are few tokens, so that warps are enough; more where there are
// many, so that the sums left in the workspace (and the time to add up those of one row) stay small.
uint32_t tile_bits(uint64_t tokens) { return tokens <= 16384 ? 4 : 5; }  // a lane a token

// Everything but the addresses, then the addresses from `p` on; returns the bytes.
uint64_t layout(Sorted* w, void* p, uint64_t tokens, uint64_t vocab, uint64_t dim, uint32_t slices) {
  w->bucket_bits = 0;
  while ((1u << w->bucket_bits) < kLeastBuckets || ((uint64_t)kLocals << w->bucket_bits) < vocab)
    ++w->bucket_bits;
  w->buckets = 1u << w->bucket_bits;
  w->tile_bits = tile_bits(tokens);
  w->tiles = (uint32_t)((tokens + (1u << w->tile_bits) - 1) >> w->tile_bits);
  w->slices = slices;
  w->pitch = up(dim + 7, 512);  // spans may lead by 7 columns
  char* at = static_cast<char*>(p);
  const auto take = [&](uint64_t bytes) {
    char* q = at;
    at += up(bytes, 128);
    return q;
  };
  w->sums = reinterpret_cast<float*>(take((uint64_t)w->tiles * 2 * w->pitch * 4));
  w->order = reinterpret_cast<uint2*>(take(tokens * 8));
  w->rows = reinterpret_cast<uint2*>(take(vocab * 8));
  w->ticks = reinterpret_cast<uint32_t*>(take((uint64_t)w->tiles * 2 * slices * 4));
  w->groups = reinterpret_cast<uint32_t*>(take((uint64_t)w->tiles * 2 * slices * 4));
  w->total = reinterpret_cast<uint32_t*>(take(4));
  return (uint64_t)(at - static_cast<char*>(p));
}

// ---- 1: group -------------------------------------------------------------------------------

// Exclusive sum over the block's threads, and the total; `s` holds a word a warp and one more.
__device__ __forceinline__ uint32_t block_scan(uint32_t n, uint32_t* s, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  uint32_t sum = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(~0u, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) s[warp] = sum;
  __syncthreads();
  if (warp == 0) {
    uint32_t w = s[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(~0u, w, o);
      if (lane >= o) w += v;
    }
    s[lane] = w;
  }
  __syncthreads();
  *total = s[31];
  const uint32_t before = warp ? s[warp - 1] : 0;
  __syncthreads();
  return before + sum - n;
}

// dout as bytes, for the blocks of k_group beyond the buckets: they ask for its rows while the others
// sort, so that k_sum finds them in L2.
struct Ahead {
  const char* p;
  uint64_t pitch;
  uint32_t width;
};
constexpr uint32_t kAheadBlocks = 32;
// Where dout is more, it would not stay in L2.  Without and with the blocks, bf16 into 8192 rows: 4 MB 23.0 and 21.5 us, 32 MB
// 30.7 and 26.5, 64 MB 49.1 and 43.9; 128 MB (16384 x 4096) 76.2 and 84.6, 256 MB 125 and 167.  The lower limit
// is on the safe side: 1 MB 21.3 and 19.5.
constexpr uint64_t kAheadLeast = 4 << 20, kAheadMost = 64 << 20;

// A warp a token's row, 128 bytes a lane.
__device__ __forceinline__ void bring(const Ids& ids, uint32_t tokens, uint32_t vocab, const Ahead& dout,
                                      uint32_t block) {
  constexpr uint32_t warps = kThreads / 32;
  for (uint64_t k = (uint64_t)block * warps + threadIdx.x / 32; k < tokens; k += kAheadBlocks * warps) {
    if (token_id(ids, k, vocab) < 0) continue;
    const char* row = dout.p + k * dout.pitch;
    for (uint32_t at = (threadIdx.x & 31) * 128; at < dout.width; at += 32 * 128)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(row + at));
  }
}

__global__ void __launch_bounds__(kThreads) k_group(const __grid_constant__ Ids ids, uint32_t tokens,
                                                    uint32_t vocab,
                                                    const __grid_constant__ Sorted w,
                                                    const __grid_constant__ Ahead dout) {
  __shared__ uint32_t next[kLocals];  // counts, then where an id's next token goes
  __shared__ uint32_t list[kStep];    // a step's tokens of this bucket, in order: id in the bucket, place in the step
  __shared__ uint32_t scan[32];
  __shared__ uint32_t earlier_all, valid_all;
  // tokens of this bucket among the 32 of a warp at j, then in all such cells before
  __shared__ __align__(16) uint32_t cells[kEach * (kThreads / 32)];
  __shared__ uint32_t in_step;
  pdl_enter();
  const uint32_t t = threadIdx.x, lane = t & 31, warp = t / 32, b = blockIdx.x;
  if (b >= w.buckets) return bring(ids, tokens, vocab, dout, b - w.buckets);
  const uint32_t mask = w.buckets - 1;
  for (uint32_t k = t; k < kLocals; k += kThreads) next[k] = 0;
  if (t == 0) earlier_all = valid_all = 0;
  __syncthreads();
  int32_t id[kEach];  // of tokens i0 + j * kThreads + t
  const auto read = [&](uint64_t i0) {
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const uint64_t i = i0 + j * kThreads + t;
      id[j] = i < tokens ? token_id(ids, i, vocab) : -1;
    }
  };
  // an id's tokens, and the tokens of earlier buckets
  uint32_t earlier = 0, valid = 0;
  for (uint64_t i0 = 0; i0 < tokens; i0 += kStep) {
    read(i0);
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      if (id[j] < 0) continue;
      ++valid;
      earlier += (id[j] & mask) < b;
      if ((id[j] & mask) == b) atomicAdd(&next[id[j] >> w.bucket_bits], 1u);
    }
  }
  earlier = __reduce_add_sync(~0u, earlier);
  valid = __reduce_add_sync(~0u, valid);
  if (lane == 0) atomicAdd(&earlier_all, earlier), atomicAdd(&valid_all, valid);
  __syncthreads();
  // each id's first place: a thread takes two ids next to each other
  const uint32_t first = earlier_all;
  static_assert(kLocals == 2 * kThreads, "two ids a thread");
  const uint32_t n0 = next[2 * t], n1 = next[2 * t + 1];
  uint32_t all;
  const uint32_t at = first + block_scan(n0 + n1, scan, &all);
  next[2 * t] = at, next[2 * t + 1] = at + n0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint64_t id = (uint64_t)(2 * t + k) << w.bucket_bits | b;
    const uint32_t n = k ? n1 : n0, start = k ? at + n0 : at;
    if (id >= vocab) continue;
    w.rows[id] = make_uint2(start, n);
    if (n == 0) continue;
    const uint32_t tile = start >> w.tile_bits, parts = ((start + n - 1) >> w.tile_bits) - tile + 1;
    if (parts == 1) continue;
    for (uint32_t q = 0; q < w.slices; ++q) w.groups[slot_of(tile, 0) * w.slices + q] = 0;
    for (uint32_t p = 0; p < parts; p += kGroup)
      for (uint32_t q = 0; q < w.slices; ++q) w.ticks[slot_of(tile, p) * w.slices + q] = 0;
  }
  if (b == 0 && t == 0) *w.total = valid_all;
  if (all == 0) return;
  __syncthreads();
  // tokens to their places
  for (uint64_t i0 = 0; i0 < tokens; i0 += kStep) {
    if (tokens > kStep) read(i0);  // else they are still there
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const uint32_t at = __ballot_sync(~0u, id[j] >= 0 && (id[j] & mask) == b);
      if (lane == 0) cells[j * (kThreads / 32) + warp] = __popc(at);
    }
    __syncthreads();
    if (warp == 0) {
      static_assert(kEach == 8 && kThreads == 1024, "eight cells a lane");
      uint4* mine = reinterpret_cast<uint4*>(cells) + 2 * lane;
      uint4 p = mine[0], q = mine[1];
      const uint32_t n = p.x + p.y + p.z + p.w + q.x + q.y + q.z + q.w;
      uint32_t sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(~0u, sum, o);
        if (lane >= o) sum += v;
      }
      if (lane == 31) in_step = sum;
      uint32_t before = sum - n;
      const auto turn = [&](uint32_t& c) { const uint32_t k = c; c = before, before += k; };
      turn(p.x), turn(p.y), turn(p.z), turn(p.w), turn(q.x), turn(q.y), turn(q.z), turn(q.w);
      mine[0] = p, mine[1] = q;
    }
    __syncthreads();
    const uint32_t m = in_step;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const bool own = id[j] >= 0 && (id[j] & mask) == b;
      const uint32_t at = __ballot_sync(~0u, own);
      if (own)
        list[cells[j * (kThreads / 32) + warp] + __popc(at & ((1u << lane) - 1))] =
            (uint32_t)id[j] >> w.bucket_bits << kStepBits | (j * kThreads + t);
    }
    __syncthreads();
    // a warp places its share of the ids, so that it alone moves their `next`
    for (uint32_t s = 0; s < m; s += 32) {
      const uint32_t e = s + lane < m ? list[s + lane] : 0, local = e >> kStepBits;
      const bool own = s + lane < m && local % 32 == warp;
      if (!__any_sync(~0u, own)) continue;
      const uint32_t same = __match_any_sync(~0u, own ? local : ~0u);
      if (own) {
        const uint32_t place = next[local] + __popc(same & ((1u << lane) - 1));
        w.order[place] = make_uint2(local << w.bucket_bits | b, (uint32_t)i0 + (e & (kStep - 1)));
      }
      __syncwarp();
      if (own && (same >> lane) == 1) next[local] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
  }
}

// ---- 2: sum ---------------------------------------------------------------------------------

// Table row `id`: base + scale * acc.
template <int OT, int MODE>
__device__ __forceinline__ void finish(const EmbedBackArgs& a, uint32_t id, uint32_t col, int lane,
                                       float* acc) {
  constexpr int vals = place_vals(MODE);
  char* out = row_at<OT>(a.dtable, id);
  const Place<MODE> at(col, a.dim, lane, out);
#pragma unroll
  for (int e = 0; e < vals; ++e) acc[e] = __fmul_rn(acc[e], a.scale);
  if (a.base.p) {
    Loaded<OT, MODE> base;
    base.load(row_at<OT>(a.base, id), at);
    base.ready();
#pragma unroll
    for (int e = 0; e < vals; ++e) acc[e] += base.value(e);
  }
  st_place<OT, MODE>(out, at, acc);
}

// acc at a slot of the workspace: a lane's values 16 bytes each, next to its neighbours'.
template <int MODE>
__device__ __forceinline__ void put_sum(const Sorted& w, uint64_t slot, uint32_t col, int lane,
                                        const float* acc) {
  float* to = w.sums + slot * w.pitch + col + 4 * lane;
#pragma unroll
  for (int e = 0; e < place_vals(MODE); e += 4)
    __stcg(reinterpret_cast<float4*>(to + 32 * e), make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]));
}

// Whether this warp, whose sum is written, is the last of n to come here; if so, it sees the others'.
__device__ __forceinline__ bool last_of(uint32_t* tick, uint32_t n, int lane) {
  __threadfence();
  __syncwarp();
  uint32_t before = 0;
  if (lane == 0) before = atomicAdd(tick, 1u);
  const bool last = __shfl_sync(~0u, before, 0) == n - 1;
  if (last) __threadfence();
  return last;
}

// acc = the sums of parts p, p + step, ... below `end`, in order.
template <int MODE>
__device__ __forceinline__ void get_sums(const Sorted& w, uint32_t from, uint32_t p, uint32_t end,
                                         uint32_t step, uint32_t col, int lane, float* acc) {
  constexpr int vals = place_vals(MODE);
#pragma unroll
  for (int e = 0; e < vals; ++e) acc[e] = 0.0f;
#pragma unroll 4
  for (; p < end; p += step) {
    const float* at = w.sums + slot_of(from, p) * w.pitch + col + 4 * lane;
#pragma unroll
    for (int e = 0; e < vals; e += 4) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(at + 32 * e));
      acc[e] += v.x, acc[e + 1] += v.y, acc[e + 2] += v.z, acc[e + 3] += v.w;
    }
  }
}

// A warp a tile and chunk of columns.
template <int DT, int OT, int MODE>
__global__ void __launch_bounds__(kBlock, 2) k_sum(const __grid_constant__ EmbedBackArgs a,
                                                const __grid_constant__ Sorted w,
                                                const __grid_constant__ FastDiv slices) {
  constexpr int vals = place_vals(MODE);
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const uint64_t k = (uint64_t)blockIdx.x * (kBlock / 32) + (threadIdx.x >> 5);
  const uint64_t n = fastdiv_div(slices, k);
  const uint32_t slice = (uint32_t)(k - n * w.slices), col = slice * place_cols(MODE);
  float acc[vals];
#pragma unroll
  for (int e = 0; e < vals; ++e) acc[e] = 0.0f;
  const uint32_t tile = (uint32_t)n;
  if (tile >= w.tiles) return;
  const uint32_t total = *w.total, begin = tile << w.tile_bits;
  if (begin >= total) return;
  const uint32_t end = min(total, begin + (1u << w.tile_bits));
  const uint32_t after = end < total ? w.order[end].x : ~0u;
  const uint32_t before = begin ? w.order[begin - 1].x : ~0u;
  const uint2 entry = begin + lane < end ? w.order[begin + lane] : make_uint2(~0u, 0);
  // rows in flight: as many as make 128 bytes of a lane
  constexpr int ahead = 128 / (place_vals(MODE) * (DT == CR_BF16 ? 2 : 4));
  Loaded<DT, MODE> in[ahead];
  const auto load = [&](Loaded<DT, MODE>& to, uint32_t i) {
    const uint32_t id = __shfl_sync(~0u, entry.x, i & 31), token = __shfl_sync(~0u, entry.y, i & 31);
    if (i < end - begin)
      to.load(row_at<DT>(a.dout, token), Place<MODE>(col, a.dim, lane, row_at<OT>(a.dtable, id)));
  };
#pragma unroll
  for (int j = 0; j < ahead; ++j) load(in[j], j);
  bool joined = __shfl_sync(~0u, entry.x, 0) == before;  // the row at work began in an earlier tile
#pragma unroll 1
  for (uint32_t i = 0; i < end - begin; ++i) {
    const uint32_t id = __shfl_sync(~0u, entry.x, i), next = __shfl_sync(~0u, entry.x, (i + 1) & 31);
    in[0].ready();
#pragma unroll
    for (int e = 0; e < vals; ++e) acc[e] += in[0].value(e);
#pragma unroll
    for (int j = 1; j < ahead; ++j) in[j - 1] = in[j];
    load(in[ahead - 1], i + ahead);
    const bool ends = i + 1 == end - begin, goes_on = ends && after == id;
    if (!ends && next == id) continue;
    bool whole = true;
    if (joined || goes_on) {
      const uint2 row = w.rows[id];
      const uint32_t from = row.x >> w.tile_bits, parts = ((row.x + row.y - 1) >> w.tile_bits) - from + 1;
      const uint32_t part = tile - from, first = part / kGroup * kGroup;
      // parts to groups, groups to the row
      put_sum<MODE>(w, slot_of(from, part), col, lane, acc);
      whole = last_of(&w.ticks[slot_of(from, first) * w.slices + slice], min(kGroup, parts - first), lane);
      if (whole) {
        get_sums<MODE>(w, from, first, min(parts, first + kGroup), 1, col, lane, acc);
        if (parts > kGroup) {
          put_sum<MODE>(w, slot_of(from, first), col, lane, acc);
          whole = last_of(&w.groups[slot_of(from, 0) * w.slices + slice], (parts + kGroup - 1) / kGroup, lane);
          if (whole) get_sums<MODE>(w, from, 0, parts, kGroup, col, lane, acc);
        }
      }
      joined = false;
    }
    if (whole) finish<OT, MODE>(a, id, col, lane, acc);
#pragma unroll
    for (int e = 0; e < vals; ++e) acc[e] = 0.0f;
  }
}

// ---- 3: rows without tokens ---------------------------------------------------------------------

constexpr uint32_t kFree = 16;  // chunks of the table that a warp looks at at a time

// base, or zeros.  chained: launched after k_sum, and started when each of its blocks has returned from its
// wait for k_group (pdl.cuh): k_group, and with it all that came before this call, has ended, and what they
// wrote is in L2.  Without a wait of this launch's own nothing says that L1 holds no older lines of it (a workspace
// is used by call after call): rows are read by way of L2, and a fence comes before loads of base (where there
// is none it would cost 0.9 of the 36.6 us above).  It is k_sum that one block waits for at its end, so that this
// launch ends after it.
template <int OT, int MODE>
__global__ void __launch_bounds__(kBlock) k_free(const __grid_constant__ EmbedBackArgs a,
                                                 const __grid_constant__ Sorted w,
                                                 const __grid_constant__ FastDiv slices, bool chained) {
  constexpr int vals = place_vals(MODE), ahead = 4;  // of a warp in flight
  if (!chained)
    pdl_wait_prerequisites();
  else if (a.base.p)
    __threadfence();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const uint64_t all = (uint64_t)a.vocab * w.slices, stride = (uint64_t)gridDim.x * (kBlock / 32) * kFree;
  for (uint64_t first = ((uint64_t)blockIdx.x * (kBlock / 32) + (threadIdx.x >> 5)) * kFree; first < all;
       first += stride) {
    // a lane a chunk
    const uint64_t mine = first + lane;
    uint32_t id = 0, slice = 0;
    bool is_free = false;
    if (lane < kFree && mine < all) {
      id = (uint32_t)fastdiv_div(slices, mine);
      slice = (uint32_t)(mine - (uint64_t)id * w.slices);
      is_free = __ldcg(&w.rows[id].y) == 0;
    }
    uint32_t left = __ballot_sync(~0u, is_free);
    while (left) {
      Loaded<OT, MODE> base[ahead];
      uint32_t row[ahead], col[ahead];
      int n_here = 0;
#pragma unroll
      for (int j = 0; j < ahead; ++j) {
        if (!left) break;
        const int at = __ffs(left) - 1;
        left &= left - 1;
        row[j] = __shfl_sync(~0u, id, at), col[j] = __shfl_sync(~0u, slice, at) * place_cols(MODE);
        n_here = j + 1;
        if (a.base.p)
          base[j].load(row_at<OT>(a.base, row[j]),
                       Place<MODE>(col[j], a.dim, lane, row_at<OT>(a.dtable, row[j])));
      }
#pragma unroll
      for (int j = 0; j < ahead; ++j) {
        if (j >= n_here) break;
        char* out = row_at<OT>(a.dtable, row[j]);
        float v[vals];
        if (a.base.p) base[j].ready();
#pragma unroll
        for (int e = 0; e < vals; ++e) v[e] = a.base.p ? base[j].value(e) : 0.0f;
        st_place<OT, MODE>(out, Place<MODE>(col[j], a.dim, lane, out), v);
      }
    }
  }
  if (chained && blockIdx.x == 0) pdl_wait_prerequisites();
}

template <int DT, int OT, int MODE>
cudaError_t run(const EmbedBackArgs& a, void* workspace, cudaStream_t s) {
  Sorted w;
  layout(&w, workspace, a.tokens, a.vocab, a.dim, place_chunks(a.dim, MODE));
  constexpr uint64_t es = DT == CR_BF16 ? 2 : 4;
  const Ahead dout = {static_cast<const char*>(a.dout.p), a.dout.ld * es, (uint32_t)(a.dim * es)};
  const uint64_t bytes = a.tokens * a.dim * es;
  const bool ahead = bytes >= kAheadLeast && bytes <= kAheadMost;
  cudaError_t e = launch_pdl(k_group, dim3(w.buckets + (ahead ? kAheadBlocks : 0)), kThreads, s, a.ids,
                             (uint32_t)a.tokens, a.vocab, w, dout);
  const uint64_t warps = (uint64_t)w.tiles * w.slices, chunks = (uint64_t)a.vocab * w.slices;
  const FastDiv slices = fastdiv_make(w.slices, std::max(warps + kBlock / 32, chunks));
  if (e == cudaSuccess && warps)
    e = launch_pdl(k_sum<DT, OT, MODE>, dim3((unsigned)((warps + kBlock / 32 - 1) / (kBlock / 32))), kBlock,
                   s, a, w, slices);
  if (e != cudaSuccess || a.in_place) return e;
  const uint64_t blocks = (chunks + kFree * (kBlock / 32) - 1) / (kFree * (kBlock / 32));
  return launch_pdl(k_free<OT, MODE>, dim3((unsigned)std::min(blocks, (uint64_t)1 << 30)), kBlock, s, a, w,
                    slices, warps != 0);
}

template <int DT, int OT>
cudaError_t by_mode(const EmbedBackArgs& a, void* workspace, int vec, cudaStream_t s) {
  if (vec == 2) return run<DT, OT, 2>(a, workspace, s);
  if (vec == 1) return run<DT, OT, 1>(a, workspace, s);
  if constexpr (DT == CR_BF16 && OT == CR_BF16) return run<DT, OT, kSpan>(a, workspace, s);
  return run<DT, OT, 0>(a, workspace, s);
}

}  // namespace

uint64_t embed_back_workspace(uint64_t tokens, uint64_t vocab, uint64_t dim) {
  Sorted w;
  return layout(&w, nullptr, tokens, vocab, dim, place_chunks((uint32_t)dim, kSpan));
}

cudaError_t launch_embed_back(cr_dtype d, cr_dtype out, const EmbedBackArgs& a, void* workspace,
                              int vec, cudaStream_t s) {
  if (d == CR_BF16)
    return out == CR_BF16 ? by_mode<CR_BF16, CR_BF16>(a, workspace, vec, s)
                          : by_mode<CR_BF16, CR_F32>(a, workspace, vec, s);
  return out == CR_BF16 ? by_mode<CR_F32, CR_BF16>(a, workspace, vec, s)
                        : by_mode<CR_F32, CR_F32>(a, workspace, vec, s);
}

}  // namespace cr
