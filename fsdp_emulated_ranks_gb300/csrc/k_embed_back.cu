// k_embed_back.cu -- the embedding's gradient: for each row of the table, the sum of the
// gradients of the tokens that name it.
//
// Tokens are sorted by id first, so that a row's sum has a fixed order and every row is
// written once, by whoever adds it up:
//   1. k_sort   a block sorts 1024 tokens by (bucket, id, token), where an id's bucket is its
//               low bits, and notes where each bucket begins
//   2. k_group  a block takes a bucket: its part of every sorted 1024, in order, gives the
//               tokens of each of its ids (256 at most), in order
//   3. k_sum    a warp takes a chunk of a table row and adds up its tokens' rows; where more
//               than kLong tokens name it, a warp each kPart of them, and the last to finish
//               adds the parts' fp32 sums, in order
// Few tokens leave most of the table without any: then the call is bound by writing it,
// else by reading the tokens' gradients and writing the table.
#include <algorithm>

#include "lm_internal.cuh"
#include "pdl.cuh"

namespace cr {

namespace {

constexpr uint32_t kChunk = 1024;      // tokens a block sorts
constexpr uint32_t kLocals = 256;      // ids of a bucket at most
constexpr uint32_t kLong = 64;         // tokens of a row that one warp adds up at most
constexpr uint32_t kPart = 64;         // tokens of a part of a longer row
constexpr uint32_t kNone = 1u << 21;   // the sort key's id of what is no token

struct Item {  // a part of a long row
  uint32_t id, part, first, parts;  // first: the row's first item
};

// The workspace.
struct Sorted {
  uint32_t* keys;     // [chunks][kChunk] (bucket, id within it) << 10 | token, sorted
  uint16_t* ranks;    // [chunks][kChunk] place among the chunk's tokens of that id; the last one's | kLast
  uint16_t* begins;   // [chunks][buckets + 1] where buckets begin
  uint32_t* tokens;   // [tokens] by bucket, id, token
  uint2* rows;        // [vocab] first of the row's tokens, and how many
  Item* items;        // [cap]
  uint32_t* ticks;    // [cap][slices] parts of a long row that are done (at its first item)
  float* sums;        // [cap][pitch]
  uint32_t* count;    // items in use
  uint32_t chunks, buckets, bucket_bits, local_bits, cap, slices;
  uint64_t pitch;
};

constexpr uint16_t kLast = 0x8000;

uint64_t up(uint64_t v, uint64_t m) { return (v + m - 1) / m * m; }

// Everything but the addresses, then the addresses from `p` on; returns the bytes.
uint64_t layout(Sorted* w, void* p, uint64_t tokens, uint64_t vocab, uint64_t dim, uint32_t slices) {
  w->bucket_bits = 5;
  while (((uint64_t)kLocals << w->bucket_bits) < vocab) ++w->bucket_bits;
  w->buckets = 1u << w->bucket_bits;
  w->local_bits = 0;
  while (vocab && ((vocab - 1) >> w->bucket_bits) >> w->local_bits) ++w->local_bits;
  w->chunks = (uint32_t)std::max<uint64_t>(1, (tokens + kChunk - 1) / kChunk);
  // a row of n > kLong tokens has ceil(n / kPart) parts
  w->cap = (uint32_t)(tokens / kPart + tokens / (kLong + 1));
  w->slices = slices;
  w->pitch = up(dim + 7, 512);  // spans may lead by 7 columns
  char* at = static_cast<char*>(p);
  const auto take = [&](uint64_t bytes) {
    char* q = at;
    at += up(bytes, 128);
    return q;
  };
  w->sums = reinterpret_cast<float*>(take(w->cap * w->pitch * 4));
  w->keys = reinterpret_cast<uint32_t*>(take((uint64_t)w->chunks * kChunk * 4));
  w->ranks = reinterpret_cast<uint16_t*>(take((uint64_t)w->chunks * kChunk * 2));
  w->begins = reinterpret_cast<uint16_t*>(take((uint64_t)w->chunks * (w->buckets + 1) * 2));
  w->tokens = reinterpret_cast<uint32_t*>(take(tokens * 4));
  w->rows = reinterpret_cast<uint2*>(take(vocab * 8));
  w->items = reinterpret_cast<Item*>(take((uint64_t)w->cap * sizeof(Item)));
  w->ticks = reinterpret_cast<uint32_t*>(take((uint64_t)w->cap * slices * 4));
  w->count = reinterpret_cast<uint32_t*>(take(4));
  return (uint64_t)(at - static_cast<char*>(p));
}

// ---- 1: sort ------------------------------------------------------------------------------

__global__ void __launch_bounds__(kChunk) k_sort(const __grid_constant__ Ids ids, uint64_t tokens,
                                                 uint32_t vocab, const __grid_constant__ Sorted w) {
  __shared__ uint32_t s[2][kChunk];
  pdl_enter();
  const uint32_t t = threadIdx.x;
  const uint64_t token = (uint64_t)blockIdx.x * kChunk + t;
  const int32_t id = token < tokens ? token_id(ids, token, vocab) : -1;
  uint32_t key = id < 0 ? kNone : (id & (w.buckets - 1)) << w.local_bits | (uint32_t)id >> w.bucket_bits;
  key = key << 10 | t;
  // bitonic: within a warp by shuffles, beyond it through shared memory
  int side = 0;
#pragma unroll
  for (uint32_t size = 2; size <= kChunk; size <<= 1) {
#pragma unroll
    for (uint32_t step = size / 2; step; step >>= 1) {
      uint32_t other;
      if (step >= 32) {
        s[side][t] = key;
        __syncthreads();
        other = s[side][t ^ step];
        side ^= 1;
      } else {
        other = __shfl_xor_sync(~0u, key, step);
      }
      const bool low = ((t & step) == 0) == ((t & size) == 0);
      key = low ? min(key, other) : max(key, other);
    }
  }
  __syncthreads();
  s[0][t] = key;
  __syncthreads();
  const auto bucket_of = [&](uint32_t k) { return min(k >> 10 >> w.local_bits, w.buckets); };
  uint16_t* begins = w.begins + (uint64_t)blockIdx.x * (w.buckets + 1);
  const uint32_t mine = bucket_of(key), before = t ? bucket_of(s[0][t - 1]) + 1 : 0;
  for (uint32_t b = before; b <= mine; ++b) begins[b] = (uint16_t)t;
  if (t == kChunk - 1)
    for (uint32_t b = mine + 1; b <= w.buckets; ++b) begins[b] = kChunk;
  // the first of the keys with this id
  const uint32_t least = key & ~1023u;
  uint32_t lo = 0, hi = t;
  while (lo < hi) {
    const uint32_t mid = (lo + hi) / 2;
    if (s[0][mid] < least)
      lo = mid + 1;
    else
      hi = mid;
  }
  const bool last = t == kChunk - 1 || s[0][t + 1] >> 10 != key >> 10;
  w.keys[(uint64_t)blockIdx.x * kChunk + t] = key;
  w.ranks[(uint64_t)blockIdx.x * kChunk + t] = (uint16_t)((t - lo) | (last ? kLast : 0));
  if (blockIdx.x == 0 && t == 0) *w.count = 0;
}

// ---- 2: group ------------------------------------------------------------------------------

__global__ void __launch_bounds__(kLocals) k_group(uint32_t vocab, const __grid_constant__ Sorted w) {
  __shared__ uint32_t count[kLocals], next[kLocals], warp_sum[kLocals / 32 + 1];
  __shared__ unsigned long long first_sum;
  pdl_enter();
  const uint32_t t = threadIdx.x, lane = t & 31, warp = t / 32, b = blockIdx.x;
  const uint64_t pitch = w.buckets + 1;
  const uint32_t local_mask = (1u << w.local_bits) - 1;
  count[t] = 0;
  if (t == 0) first_sum = 0;
  __syncthreads();
  // tokens of earlier buckets, and of each id of this one
  uint64_t earlier = 0;
  for (uint32_t c = t; c < w.chunks; c += kLocals) earlier += w.begins[c * pitch + b];
  if (earlier) atomicAdd(&first_sum, (unsigned long long)earlier);
  for (uint32_t c = warp; c < w.chunks; c += kLocals / 32) {
    const uint32_t lo = w.begins[c * pitch + b], hi = w.begins[c * pitch + b + 1];
    for (uint32_t i = lo + lane; i < hi; i += 32) {
      const uint32_t rank = w.ranks[(uint64_t)c * kChunk + i];
      if (rank & kLast)
        atomicAdd(&count[w.keys[(uint64_t)c * kChunk + i] >> 10 & local_mask], (rank & ~kLast) + 1);
    }
  }
  __syncthreads();
  // where each id's tokens begin
  const uint32_t n = count[t];
  uint32_t sum = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(~0u, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) warp_sum[warp] = sum;
  __syncthreads();
  uint32_t start = sum - n;
  for (uint32_t k = 0; k < warp; ++k) start += warp_sum[k];
  const uint32_t first = (uint32_t)first_sum;
  next[t] = first + start;
  const uint64_t id = (uint64_t)t << w.bucket_bits | b;
  if (id < vocab) {
    w.rows[id] = make_uint2(first + start, n);
    if (n > kLong) {
      const uint32_t parts = (n + kPart - 1) / kPart, at = atomicAdd(w.count, parts);
      for (uint32_t k = 0; k < parts; ++k) w.items[at + k] = Item{(uint32_t)id, k, at, parts};
      for (uint32_t k = 0; k < w.slices; ++k) w.ticks[(uint64_t)at * w.slices + k] = 0;
    }
  }
  __syncthreads();
  // Tokens to their places.  A warp goes through all of the bucket's tokens in order but
  // places those of its share of the ids alone, so that warps need not wait for each other.
  constexpr uint32_t warps = kLocals / 32;
  for (uint32_t c = 0; c < w.chunks; ++c) {
    const uint32_t lo = w.begins[c * pitch + b], hi = w.begins[c * pitch + b + 1];
    for (uint32_t i0 = lo; i0 < hi; i0 += 32) {
      const uint32_t i = i0 + lane;
      uint32_t key = 0, rank = 0;
      bool mine = i < hi;
      if (mine) {
        key = w.keys[(uint64_t)c * kChunk + i];
        rank = w.ranks[(uint64_t)c * kChunk + i];
        mine = (key >> 10) % warps == warp;
      }
      const uint32_t local = key >> 10 & local_mask;
      if (mine) w.tokens[next[local] + (rank & ~kLast)] = c * kChunk + (key & 1023);
      __syncwarp();
      if (mine && (rank & kLast)) next[local] += (rank & ~kLast) + 1;
      __syncwarp();
    }
  }
}

// ---- 3: sum ---------------------------------------------------------------------------------

constexpr int kAhead = 4;  // rows of a warp in flight

// acc += rows tokens[0 .. n - 1] of dout, in order.
template <int DT, int MODE>
__device__ __forceinline__ void add_rows(const Mat& dout, const uint32_t* tokens, uint32_t n,
                                         const Place<MODE>& at, float* acc) {
  for (uint32_t i0 = 0; i0 < n; i0 += 32) {
    const uint32_t here = min(n - i0, 32u);
    const uint32_t token = (uint32_t)at.lane < here ? tokens[i0 + at.lane] : 0;
    for (uint32_t i = 0; i < here; i += kAhead) {
      Loaded<DT, MODE> in[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const uint32_t row = __shfl_sync(~0u, token, (i + j) & 31);
        if (i + j < here) in[j].load(row_at<DT>(dout, row), at);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (i + j >= here) break;
        in[j].ready();
#pragma unroll
        for (int e = 0; e < place_vals(MODE); ++e) acc[e] += in[j].value(e);
      }
    }
  }
}

// Table row `id`: base + scale * acc.
template <int OT, int MODE>
__device__ __forceinline__ void finish(const EmbedBackArgs& a, uint32_t id, const Place<MODE>& at,
                                       float* acc) {
#pragma unroll
  for (int e = 0; e < place_vals(MODE); ++e) acc[e] *= a.scale;
  if (a.base.p) {
    Loaded<OT, MODE> base;
    base.load(row_at<OT>(a.base, id), at);
    base.ready();
#pragma unroll
    for (int e = 0; e < place_vals(MODE); ++e) acc[e] += base.value(e);
  }
  st_place<OT, MODE>(row_at<OT>(a.dtable, id), at, acc);
}

// Warps [0, cap * slices) take the parts of long rows, the others a chunk of a row each.
template <int DT, int OT, int MODE>
__global__ void __launch_bounds__(kBlock) k_sum(const __grid_constant__ EmbedBackArgs a,
                                                const __grid_constant__ Sorted w,
                                                const __grid_constant__ FastDiv slices) {
  constexpr int vals = place_vals(MODE);
  pdl_enter();
  const int lane = threadIdx.x & 31;
  uint64_t k = (uint64_t)blockIdx.x * (kBlock / 32) + (threadIdx.x >> 5);
  const uint64_t part_warps = (uint64_t)w.cap * w.slices;
  float acc[vals];
#pragma unroll
  for (int e = 0; e < vals; ++e) acc[e] = 0.0f;
  if (k >= part_warps) {
    k -= part_warps;
    const uint64_t id = fastdiv_div(slices, k);
    if (id >= a.vocab) return;
    const uint2 row = w.rows[id];
    if (row.y > kLong || (row.y == 0 && a.in_place)) return;
    const uint32_t base = (uint32_t)(k - id * w.slices) * place_cols(MODE);
    const Place<MODE> at(base, a.dim, lane, row_at<OT>(a.dtable, id));
    add_rows<DT, MODE>(a.dout, w.tokens + row.x, row.y, at, acc);
    finish<OT, MODE>(a, (uint32_t)id, at, acc);
    return;
  }
  const uint64_t n = fastdiv_div(slices, k);
  if (n >= *w.count) return;
  const Item item = w.items[n];
  const uint2 row = w.rows[item.id];
  const uint32_t slice = (uint32_t)(k - n * w.slices), base = slice * place_cols(MODE);
  const Place<MODE> at(base, a.dim, lane, row_at<OT>(a.dtable, item.id));
  const uint32_t from = item.part * kPart;
  add_rows<DT, MODE>(a.dout, w.tokens + row.x + from, min(kPart, row.y - from), at, acc);
  // a lane's sums, 16 bytes apart: the place of lane `lane` of slice `slice`
  float* sums = w.sums + (uint64_t)item.first * w.pitch + base + 4 * lane;
#pragma unroll
  for (int e = 0; e < vals; e += 4)
    *reinterpret_cast<float4*>(sums + item.part * w.pitch + 32 * e) =
        make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
  __threadfence();
  __syncwarp();
  uint32_t done = 0;
  if (lane == 0) done = atomicAdd(&w.ticks[(uint64_t)item.first * w.slices + slice], 1u);
  if (__shfl_sync(~0u, done, 0) != item.parts - 1) return;
  __threadfence();  // the last part: the others' sums are there
#pragma unroll
  for (int e = 0; e < vals; ++e) acc[e] = 0.0f;
  for (uint32_t p = 0; p < item.parts; ++p) {
#pragma unroll
    for (int e = 0; e < vals; e += 4) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(sums + p * w.pitch + 32 * e));
      acc[e] += v.x, acc[e + 1] += v.y, acc[e + 2] += v.z, acc[e + 3] += v.w;
    }
  }
  finish<OT, MODE>(a, item.id, at, acc);
}

template <int DT, int OT, int MODE>
cudaError_t run(const EmbedBackArgs& a, void* workspace, cudaStream_t s) {
  Sorted w;
  layout(&w, workspace, a.tokens, a.vocab, a.dim, place_chunks(a.dim, MODE));
  cudaError_t e = launch_pdl(k_sort, dim3(w.chunks), kChunk, s, a.ids, a.tokens, a.vocab, w);
  if (e == cudaSuccess) e = launch_pdl(k_group, dim3(w.buckets), kLocals, s, a.vocab, w);
  if (e != cudaSuccess) return e;
  const uint64_t warps = ((uint64_t)w.cap + a.vocab) * w.slices;
  return launch_pdl(k_sum<DT, OT, MODE>, dim3((unsigned)((warps + kBlock / 32 - 1) / (kBlock / 32))),
                    kBlock, s, a, w, fastdiv_make(w.slices, warps));
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
