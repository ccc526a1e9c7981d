// k_logp.cu -- log probabilities of given tokens, entropy, log-sum-exp and the most
// likely tokens, in one read of the logits.
//
// Running softmax: with m the largest logit so far and t = (x - m) scale log2(e), a thread
// keeps s = sum of 2^t and w = sum of 2^t t, and when m grows so that its own t is d
//     w -> 2^d (w + d s),   s -> 2^d s.
// Then lse = scale m + ln2 log2 s, logp = scale (x_target - m) - ln2 log2 s and
// entropy = ln2 (log2 s - w / s): differences of small numbers, not of lse and z.  x - m comes
// first (a product more than one fma with m scaled) because a row masked with the type's lowest
// value has no scaled m.
//
// Most likely tokens.  A thread also keeps its columns' largest logit, which the sum
// needs anyway.  Of 64 groups of four threads (or 32 lanes) the top-th largest maximum
// is a lower bound of the top-th largest logit, so only columns at or above it can be
// wanted, and only threads whose maximum reaches it can hold one: these columns are
// looked at again (from L2) and those that reach the bound ranked by counting.  Where
// too many reach it (equal logits: a masked row, a row of zeros), the bound is taken
// once more over (logit, column) pairs, which are all different.
//
// A row is read by a warp, by a block, or by a cluster of blocks where rows are few.
#include <cooperative_groups.h>

#include <algorithm>

#include "lm_internal.cuh"
#include "pdl.cuh"

namespace cr {

namespace {

namespace cg = cooperative_groups;

constexpr float kInf = __builtin_huge_valf();
constexpr float kFar = -1e30f;  // 2^kFar = 0
constexpr int kUnroll = 4;      // 16-byte vectors of a thread in flight
constexpr int kWarpMaxCl = 8;   // blocks of a cluster at most

// Sums over some columns of a row: see above.  s = 0: none, or all -infinity.
struct Stat {
  float m, s, w;
};

__device__ __forceinline__ Stat merge(const Stat& a, const Stat& b, float c) {
  const float m = fmaxf(a.m, b.m);
  const float da = a.m == -kInf ? 0.0f : (a.m - m) * c, db = b.m == -kInf ? 0.0f : (b.m - m) * c;
  const float fa = fast_exp2(da), fb = fast_exp2(db);
  // what is far below adds nothing, and 0 times -infinity is not to be formed
  return {m, fmaf(fa, a.s, fb * b.s),
          fmaf(fa, fmaf(fmaxf(da, kFar), a.s, a.w), fb * fmaf(fmaxf(db, kFar), b.s, b.w))};
}

__device__ __forceinline__ Stat warp_merge(Stat v, float c) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
    v = merge(v, Stat{__shfl_xor_sync(~0u, v.m, o), __shfl_xor_sync(~0u, v.s, o),
                      __shfl_xor_sync(~0u, v.w, o)},
              c);
  return v;
}

// Order of logits as integers: rising with the value, -0 equal to 0, NaN below all
// numbers, 0 for no logit at all.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 1;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A logit and its column as one number: larger for what comes first.
__device__ __forceinline__ uint64_t pair_key(float x, uint32_t col) {
  return (uint64_t)order_key(x) << 32 | (0xffffffffu - col);
}

// Part of a row: its vectors (16-byte aligned), and the single columns before and
// behind them, fewer than a vector each.
template <int DT>
struct RowPart {
  static constexpr int kVec = DT == CR_BF16 ? 8 : 4;  // columns of a vector
  const char* p;
  uint32_t begin;  // its first column in the row
  uint32_t head, vectors, tail;

  __device__ __forceinline__ RowPart(const void* row, uint32_t b, uint32_t n) : begin(b) {
    constexpr uint32_t es = 16 / kVec;
    p = static_cast<const char*>(row) + (uint64_t)b * es;
    head = (uint32_t)(-reinterpret_cast<intptr_t>(p) & 15) / es;
    if (head > n) head = n;
    vectors = (n - head) / kVec;
    tail = n - head - vectors * kVec;
  }
  __device__ __forceinline__ float one(uint32_t col) const {
    if constexpr (DT == CR_BF16)
      return ffn_bf16(reinterpret_cast<const uint16_t*>(p)[col]);
    else
      return reinterpret_cast<const float*>(p)[col];
  }
  __device__ __forceinline__ uint4 vec(uint32_t j) const {
    return reinterpret_cast<const uint4*>(p + head * (16 / kVec))[j];
  }
  static __device__ __forceinline__ float value(const uint4& v, int i) {
    if constexpr (DT == CR_BF16) {
      const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
      return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
    } else {
      return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
    }
  }
  static __device__ __forceinline__ uint4 none() {
    const uint32_t w = DT == CR_BF16 ? 0xff80ff80u : 0xff800000u;  // -infinity
    return make_uint4(w, w, w, w);
  }
  // Columns of the thread t of n: single(column) of the head and the tail, many(first
  // column, vector) of the rest.
  template <typename F>
  __device__ __forceinline__ void each_of(uint32_t t, uint32_t n, F f) const {
    if (t < head) f(t, one(t));
    for (uint32_t j = t; j < vectors; j += n) {
      const uint4 v = vec(j);
#pragma unroll
      for (int i = 0; i < kVec; ++i) f(head + j * kVec + i, value(v, i));
    }
    if (t < tail) f(head + vectors * kVec + t, one(head + vectors * kVec + t));
  }
};

// The largest of two packed bf16 pairs (NaN passed over).
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int DT, int N>
__device__ __forceinline__ float largest(const uint4 (&v)[N]) {
  if constexpr (DT == CR_BF16) {
    uint32_t m = v[0].x;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i) m = max_bf16x2(m, v[i].x);
      m = max_bf16x2(max_bf16x2(m, v[i].y), max_bf16x2(v[i].z, v[i].w));
    }
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  } else {
    float m = -kInf;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      m = fmaxf(m, fmaxf(__uint_as_float(v[i].x), __uint_as_float(v[i].y)));
      m = fmaxf(m, fmaxf(__uint_as_float(v[i].z), __uint_as_float(v[i].w)));
    }
    return m;
  }
}

// A thread's running sums.
template <bool ENT>
struct Running {
  Stat v = {-kInf, 0.0f, 0.0f};

  __device__ __forceinline__ void reach(float x, float c) {
    if (!(x > v.m)) return;
    if (v.m != -kInf) {
      const float d = (v.m - x) * c, f = fast_exp2(d);
      if constexpr (ENT) v.w = f * fmaf(fmaxf(d, kFar), v.s, v.w);
      v.s *= f;
    }
    v.m = x;
  }
  __device__ __forceinline__ void add(float x, float c, float m) {
    const float t = (x - m) * c, e = fast_exp2(t);
    v.s += e;
    if constexpr (ENT) v.w = fmaf(e, fmaxf(t, kFar), v.w);  // 0 times -infinity is 0 here
  }
  // What add() subtracts: -infinity less -infinity is not to be formed.
  __device__ __forceinline__ float reference() const { return v.m == -kInf ? 0.0f : v.m; }
};

// What the threads of a team (a warp, or a block) share for the most likely tokens.
template <int TEAM>
struct TopShared {
  static constexpr int kGroups = TEAM == 32 ? 32 : 64;
  static constexpr int kCands = TEAM == 32 ? 256 : 1024;
  uint64_t keys[kGroups];
  uint64_t cand[kCands];
  uint64_t best[CR_MAX_TOP];
  uint64_t bound;
  uint32_t count, threads;
  uint16_t thread[TEAM];
};

template <int TEAM>
__device__ __forceinline__ void team_sync() {
  if constexpr (TEAM == 32)
    __syncwarp();
  else
    __syncthreads();
}

// sh.bound = the k-th largest of the groups' largest keys.
template <int TEAM>
__device__ __forceinline__ void find_bound(TopShared<TEAM>& sh, uint64_t key, int k, int t) {
  constexpr int per = TEAM / TopShared<TEAM>::kGroups;
#pragma unroll
  for (int o = 1; o < per; o <<= 1) {
    const uint64_t other = __shfl_xor_sync(~0u, key, o);
    key = other > key ? other : key;
  }
  if (t % per == 0) sh.keys[t / per] = key;
  if (t == 0) sh.count = sh.threads = 0;
  team_sync<TEAM>();
  if (t < TopShared<TEAM>::kGroups) {
    const uint64_t mine = sh.keys[t];
    int rank = 0;
    for (int i = 0; i < TopShared<TEAM>::kGroups; ++i) {
      const uint64_t other = sh.keys[i];
      rank += other > mine || (other == mine && i < t);
    }
    if (rank == k - 1) sh.bound = mine;
  }
  team_sync<TEAM>();
}

// sh.cand = the pairs at or above sh.bound, of the threads whose key reaches it.
template <int DT, int TEAM>
__device__ __forceinline__ void collect(TopShared<TEAM>& sh, const RowPart<DT>& row, uint64_t key,
                                        int t) {
  const uint64_t bound = sh.bound;
  if (key >= bound) sh.thread[atomicAdd(&sh.threads, 1u)] = (uint16_t)t;
  team_sync<TEAM>();
  const uint32_t n = sh.threads;
  const auto look = [&](uint32_t col, float x) {
    const uint64_t pair = pair_key(x, row.begin + col);
    if (pair < bound) return;
    const uint32_t slot = atomicAdd(&sh.count, 1u);
    if (slot < TopShared<TEAM>::kCands) sh.cand[slot] = pair;
  };
  const int lane = t & 31;
  for (uint32_t i = t / 32; i < n; i += TEAM / 32) {  // a warp takes a thread's columns
    const uint32_t who = sh.thread[i];
    if (lane == 0 && who < row.head) look(who, row.one(who));
    if (lane == 0 && who < row.tail)
      look(row.head + row.vectors * RowPart<DT>::kVec + who,
           row.one(row.head + row.vectors * RowPart<DT>::kVec + who));
    for (uint64_t j = who + (uint64_t)lane * TEAM; j < row.vectors; j += 32 * TEAM) {
      const uint4 v = row.vec((uint32_t)j);
#pragma unroll
      for (int e = 0; e < RowPart<DT>::kVec; ++e)
        look(row.head + (uint32_t)j * RowPart<DT>::kVec + e, RowPart<DT>::value(v, e));
    }
  }
  team_sync<TEAM>();
}

// sh.best[0 .. k - 1] = the k largest pairs of the row part, which has at least k columns,
// in falling order.  `most`: the thread's largest logit.
template <int DT, int TEAM>
__device__ __forceinline__ void find_top(TopShared<TEAM>& sh, const RowPart<DT>& row, float most,
                                         bool any, int k, int t) {
  constexpr uint32_t cands = TopShared<TEAM>::kCands;
  // a pair of the thread's largest logit is at least this
  uint64_t key = any ? (uint64_t)order_key(most) << 32 : 0;
  find_bound<TEAM>(sh, key, k, t);
  collect<DT, TEAM>(sh, row, any ? key | 0xffffffffu : 0, t);
  if (sh.count > cands) {
    key = 0;
    row.each_of(t, TEAM, [&](uint32_t col, float x) {
      const uint64_t pair = pair_key(x, row.begin + col);
      key = pair > key ? pair : key;
    });
    team_sync<TEAM>();  // sh.count has been read
    find_bound<TEAM>(sh, key, k, t);
    collect<DT, TEAM>(sh, row, key, t);
  }
  const uint32_t n = sh.count;
  if (n <= cands) {
    for (uint32_t i = t; i < n; i += TEAM) {
      const uint64_t mine = sh.cand[i];
      int rank = 0;
      for (uint32_t j = 0; j < n && rank < k; ++j) rank += sh.cand[j] > mine;
      if (rank < k) sh.best[rank] = mine;
    }
  } else {
    // the wanted pairs crowd in few threads' columns: one after another
    uint64_t last = ~0ull;
    for (int i = 0; i < k; ++i) {
      uint64_t mine = 0;
      row.each_of(t, TEAM, [&](uint32_t col, float x) {
        const uint64_t pair = pair_key(x, row.begin + col);
        if (pair < last && pair > mine) mine = pair;
      });
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const uint64_t other = __shfl_xor_sync(~0u, mine, o);
        mine = other > mine ? other : mine;
      }
      team_sync<TEAM>();
      if (t % 32 == 0) sh.keys[t / 32] = mine;
      team_sync<TEAM>();
      for (int w = 0; w < TEAM / 32; ++w) mine = sh.keys[w] > mine ? sh.keys[w] : mine;
      if (t == 0) sh.best[i] = mine;
      last = mine;
    }
  }
  team_sync<TEAM>();
}

// Sums and most likely tokens of a part of a row, by the threads of a team.  Every
// thread returns the sums.  `stats`: TEAM / 32 of them in shared memory.
template <int DT, int TEAM, bool ENT, bool TOP>
__device__ __forceinline__ Stat read_part(const RowPart<DT>& row, float c, int k, int t,
                                          TopShared<TEAM>* sh, Stat* stats) {
  using Part = RowPart<DT>;
  Running<ENT> run;
  for (uint64_t j = t; j < row.vectors; j += (uint64_t)TEAM * kUnroll) {
    uint4 v[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i)
      v[i] = j + i * TEAM < row.vectors ? row.vec((uint32_t)(j + i * TEAM)) : Part::none();
    run.reach(largest<DT>(v), c);
    const float m = run.reference();
#pragma unroll
    for (int i = 0; i < kUnroll; ++i)
#pragma unroll
      for (int e = 0; e < Part::kVec; ++e) run.add(Part::value(v[i], e), c, m);
  }
#pragma unroll
  for (int end = 0; end < 2; ++end) {
    if ((uint32_t)t >= (end ? row.tail : row.head)) continue;
    const float x = row.one(end ? row.head + row.vectors * Part::kVec + t : t);
    run.reach(x, c);
    run.add(x, c, run.reference());
  }
  Stat all = warp_merge(run.v, c);
  if constexpr (TEAM > 32) {
    if (t % 32 == 0) stats[t / 32] = all;
    __syncthreads();
    all = stats[0];
#pragma unroll
    for (int w = 1; w < TEAM / 32; ++w) all = merge(all, stats[w], c);
  }
  if constexpr (TOP) {
    const bool any = (uint32_t)t < row.vectors || (uint32_t)t < row.head || (uint32_t)t < row.tail;
    // a largest logit of -infinity may stand for NaN alone, which is below it
    uint32_t has = 0;
    if (any && run.v.m == -kInf)
      row.each_of(t, TEAM, [&](uint32_t, float x) { has |= x == -kInf; });
    const float most = any && run.v.m == -kInf && !has ? __int_as_float(0x7fc00000) : run.v.m;
    find_top<DT, TEAM>(*sh, row, most, any, k, t);
  }
  return all;
}

template <int DT>
__device__ __forceinline__ void write_row(const LogProbArgs& a, uint64_t row, const Stat& v,
                                          const char* logits) {
  const float total = log2f(v.s);
  if (a.lse) a.lse[row] = v.s == 0.0f ? -kInf : fmaf(v.m, a.scale, kLn2 * total);
  if (a.entropy) {
    const float e = v.s == 0.0f ? 0.0f : kLn2 * (total - v.w / v.s);
    a.entropy[row] = e < 0.0f ? 0.0f : e;
  }
  if (a.logp) {
    const int32_t id = token_id(a.targets, row, a.vocab);
    float lp = 0.0f;
    if (id >= 0) {
      const float x = DT == CR_BF16 ? ffn_bf16(reinterpret_cast<const uint16_t*>(logits)[id])
                                    : reinterpret_cast<const float*>(logits)[id];
      lp = v.s == 0.0f ? -kInf : fmaf(x - v.m, a.scale, -kLn2 * total);
    }
    a.logp[row] = lp;
  }
}

template <int DT>
__device__ __forceinline__ void write_top(const LogProbArgs& a, uint64_t row, int i, uint64_t pair,
                                          const Stat& v, const char* logits) {
  const uint32_t col = 0xffffffffu - (uint32_t)pair;
  if (a.top_ids) a.top_ids[row * a.top + i] = (int32_t)col;
  if (a.top_logp) {
    const float x = DT == CR_BF16 ? ffn_bf16(reinterpret_cast<const uint16_t*>(logits)[col])
                                  : reinterpret_cast<const float*>(logits)[col];
    a.top_logp[row * a.top + i] =
        v.s == 0.0f ? -kInf : fmaf(x - v.m, a.scale, -kLn2 * log2f(v.s));
  }
}

// A warp a row.
template <int DT, bool ENT, bool TOP>
__global__ void __launch_bounds__(kBlock) k_logp_warp(const __grid_constant__ LogProbArgs a) {
  __shared__ TopShared<32> top[TOP ? kBlock / 32 : 1];
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float c = a.scale * kLog2E;
  for (uint64_t row = (uint64_t)blockIdx.x * (kBlock / 32) + warp; row < a.rows;
       row += (uint64_t)gridDim.x * (kBlock / 32)) {
    const char* logits = row_at<DT>(a.logits, row);
    const RowPart<DT> part(logits, 0, a.vocab);
    TopShared<32>* sh = TOP ? &top[warp] : nullptr;
    const Stat v = read_part<DT, 32, ENT, TOP>(part, c, a.top, lane, sh, nullptr);
    if (lane == 0) write_row<DT>(a, row, v, logits);
    if constexpr (TOP) {
      if (lane < a.top) write_top<DT>(a, row, lane, sh->best[lane], v, logits);
      __syncwarp();
    }
  }
}

// A block a row, or a cluster a row (gridDim.x a multiple of the cluster).
template <int DT, bool ENT, bool TOP>
__global__ void __launch_bounds__(kBlock) k_logp_block(const __grid_constant__ LogProbArgs a,
                                                       uint32_t per) {
  __shared__ TopShared<kBlock> top[1];
  __shared__ Stat stats[kBlock / 32];
  __shared__ Stat shared_stat;
  pdl_enter();
  const float c = a.scale * kLog2E;
  const int t = threadIdx.x;
  const cg::cluster_group cluster = cg::this_cluster();
  const uint32_t parts = cluster.num_blocks(), part_no = cluster.block_rank();
  for (uint64_t row = blockIdx.x / parts; row < a.rows; row += gridDim.x / parts) {
    const char* logits = row_at<DT>(a.logits, row);
    const uint32_t begin = min(part_no * per, a.vocab);
    const RowPart<DT> part(logits, begin, min(per, a.vocab - begin));
    Stat v = read_part<DT, kBlock, ENT, TOP>(part, c, a.top, t, top, stats);
    if (parts == 1) {
      if (t == 0) write_row<DT>(a, row, v, logits);
      if constexpr (TOP) {
        if (t < a.top) write_top<DT>(a, row, t, top->best[t], v, logits);
      }
      __syncthreads();
      continue;
    }
    if (t == 0) shared_stat = v;
    cluster.sync();
    if (part_no == 0) {
      for (uint32_t q = 1; q < parts; ++q) v = merge(v, *cluster.map_shared_rank(&shared_stat, q), c);
      if (t == 0) write_row<DT>(a, row, v, logits);
      if constexpr (TOP) {
        // rank the parts' best among each other
        const int n = (int)parts * a.top;
        static_assert(kWarpMaxCl * CR_MAX_TOP <= kBlock, "a thread for every pair");
        uint64_t mine = 0;
        if (t < n) {
          mine = cluster.map_shared_rank(top, t / a.top)->best[t % a.top];
          top->cand[t] = mine;
        }
        __syncthreads();
        if (t < n) {
          int rank = 0;
          for (int i = 0; i < n; ++i) rank += top->cand[i] > mine;
          if (rank < a.top) write_top<DT>(a, row, rank, mine, v, logits);
        }
      }
    }
    cluster.sync();
  }
}

template <int DT, bool ENT, bool TOP>
cudaError_t run(const LogProbArgs& a, cudaStream_t s) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  if (a.vocab <= 2048 && a.rows >= (uint64_t)sms)
    return launch_pdl(k_logp_warp<DT, ENT, TOP>, dim3(flat_grid(a.rows * 32)), kBlock, s, a);
  // Parts of a row: while rows are too few to fill the SMs, and parts keep two vectors a
  // thread (and more columns than are wanted of them).
  uint32_t parts = 1;
  while (parts < kWarpMaxCl && a.rows * parts < 4 * (uint64_t)sms &&
         a.vocab / (2 * parts) >= 2 * kBlock * RowPart<DT>::kVec)
    parts *= 2;
  const uint32_t per = (uint32_t)((((uint64_t)a.vocab + parts - 1) / parts + 63) / 64 * 64);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(std::min<uint64_t>(a.rows, 1u << 27) * parts));
  cfg.blockDim = dim3(kBlock);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = parts;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = parts > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_logp_block<DT, ENT, TOP>, a, per);
}

template <int DT>
cudaError_t by_outputs(const LogProbArgs& a, cudaStream_t s) {
  if (a.top) return a.entropy ? run<DT, true, true>(a, s) : run<DT, false, true>(a, s);
  return a.entropy ? run<DT, true, false>(a, s) : run<DT, false, false>(a, s);
}

}  // namespace

cudaError_t launch_log_probs(cr_dtype d, const LogProbArgs& a, cudaStream_t s) {
  return d == CR_BF16 ? by_outputs<CR_BF16>(a, s) : by_outputs<CR_F32>(a, s);
}

}  // namespace cr
