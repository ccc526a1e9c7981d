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
// Most likely tokens.  Of its lanes' largest logits so far, which the sums need anyway, each warp notes
// the share-th largest.  Where `need` warps' notes are at or above a value, and share * need is at least the
// wanted number, so are as many logits: one below that value is not wanted.  Vectors whose
// largest may be wanted go to a list, few, and are read again at the end (from L2): what is at or
// above the last such value is ranked by counting.  (Testing every logit on the way instead took
// 283 us for 8192 x 32000 against 81 without: that much code runs out of the instruction cache.)  Where a
// list overflows (equal logits: a masked row, a row of zeros) or NaN leaves it short, the row is
// looked at again with a bound over (logit, column) pairs, which are all different.
//
// A row is read by a warp, by a block, or by a cluster of blocks where rows are few.
//
// Measured, a call in a loop: 8192 x 32000 bf16 (525 MB) 81 us, 6.5 TB/s, top 8 114, top 32 146;
// 6124 x 50304 fp32 (1.23 GB) 179, 6.9 TB/s, top 8 215; 1 x 32000 5.7, top 20 8.5.  (With a step of a thread
// listed in place of a vector: 111, 174, 226, 7.9.)
#include <cooperative_groups.h>

#include <algorithm>

#include "lm_internal.cuh"
#include "pdl.cuh"

namespace cr {

namespace {

namespace cg = cooperative_groups;

constexpr float kInf = __builtin_huge_valf();
constexpr float kFar = -1e30f;  // 2^kFar = 0
constexpr int kUnroll = 8;        // 16-byte vectors of a thread in flight
constexpr int kThreadsPerSm = 1024;  // at 64 registers
constexpr uint32_t kMostParts = 8;  // blocks of a cluster at most

// Sums over some columns of a row: see above.  s = 0: none, or all -infinity.
struct Stat {
  float m, s, w;
};

// v's sums with the reference m >= v.m.  What is far below adds nothing, and 0 times
// -infinity is not to be formed.
__device__ __forceinline__ Stat moved(const Stat& v, float m, float c) {
  const float d = v.m == -kInf ? 0.0f : (v.m - m) * c, f = fast_exp2(d);
  return {m, f * v.s, f * fmaf(fmaxf(d, kFar), v.s, v.w)};
}

// The sums of N neighbouring lanes, for all of them.
template <int N>
__device__ __forceinline__ Stat lanes_merge(Stat v, float c) {
  float m = v.m;
#pragma unroll
  for (int o = N / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  v = moved(v, m, c);
#pragma unroll
  for (int o = N / 2; o; o >>= 1) {
    v.s += __shfl_xor_sync(~0u, v.s, o);
    v.w += __shfl_xor_sync(~0u, v.w, o);
  }
  return v;
}

// Order of logits as integers: rising with the value, -0 equal to 0, NaN below all
// numbers, 0 for no logit at all.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 1;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The logit of such a key (0 for -0).
__device__ __forceinline__ float key_logit(uint32_t key) {
  if (key == 1) return __int_as_float(0x7fc00000);
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// A logit and its column as one number: larger for what comes first.
__device__ __forceinline__ uint64_t pair_key(float x, uint32_t col) {
  return (uint64_t)order_key(x) << 32 | (0xffffffffu - col);
}

// Part of a row: its vectors, and the single columns before and behind them, fewer than 32 each.
// Vectors start where the row passes kAlign bytes, so that a warp's 512 bytes are whole sectors.
template <int DT>
struct RowPart {
  static constexpr int kVec = DT == CR_BF16 ? 8 : 4;  // columns of a vector
  static constexpr uintptr_t kAlign = 32 * 16 / kVec;   // 32 columns
  const char* p;
  uint32_t begin;  // its first column in the row
  uint32_t head, vectors, tail;

  __device__ __forceinline__ RowPart(const void* row, uint32_t b, uint32_t n) : begin(b) {
    constexpr uint32_t es = 16 / kVec;
    p = static_cast<const char*>(row) + (uint64_t)b * es;
    head = (uint32_t)(-reinterpret_cast<intptr_t>(p) & (kAlign - 1)) / es;
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

// Largest and smallest of packed bf16 pairs, NaN passed over.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Largest (x) and smallest (y) logit of N vectors, NaN passed over.
template <int DT, int N>
__device__ __forceinline__ float2 extremes(const uint4 (&v)[N]) {
  if constexpr (DT == CR_BF16) {
    uint32_t hi = v[0].x, lo = v[0].x;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int e = i ? 0 : 1; e < 4; ++e) hi = max_bf16x2(hi, w[e]), lo = min_bf16x2(lo, w[e]);
    }
    return make_float2(fmaxf(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)),
                       fminf(__uint_as_float(lo << 16), __uint_as_float(lo & 0xffff0000u)));
  } else {
    float hi = -kInf, lo = kInf;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float x = __uint_as_float(v[i].x), y = __uint_as_float(v[i].y);
      const float z = __uint_as_float(v[i].z), w = __uint_as_float(v[i].w);
      hi = fmaxf(fmaxf(hi, x), y), lo = fminf(fminf(lo, x), y);
      hi = fmaxf(fmaxf(hi, z), w), lo = fminf(fminf(lo, z), w);
    }
    return make_float2(hi, lo);
  }
}

template <int DT, int N>
__device__ __forceinline__ float largest(const uint4 (&v)[N]) {
  return extremes<DT>(v).x;
}

// Two floats in a 64-bit register, and the operations on both at once.
using Two = unsigned long long;
__device__ __forceinline__ Two two(float a, float b) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 both(Two a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// A thread's running sums, of two columns at a time: fp32 instructions are what bounds
// the sum, and packed ones do two columns' work.
struct Running {
  float m = -kInf;  // largest logit
  Two s = 0, w = 0;

  __device__ __forceinline__ void reach(float x, float c) {
    if (!(x > m)) return;
    if (m != -kInf) {
      const float d = (m - x) * c, f = fast_exp2(d), far = fmaxf(d, kFar);
      w = mul2(two(f, f), fma2(two(far, far), s, w));
      s = mul2(two(f, f), s);
    }
    m = x;
  }
  // What is subtracted of a logit: -infinity less -infinity is not to be formed.
  __device__ __forceinline__ float reference() const { return m == -kInf ? 0.0f : m; }

  // x less the reference, times c.  FAR: some x may be -infinity, and 0 times that is 0 here.
  template <bool FAR>
  __device__ __forceinline__ void add(Two x, Two minus, Two c) {
    const Two t = mul2(add2(x, minus), c);
    float2 u = both(t);
    const Two e = two(fast_exp2(u.x), fast_exp2(u.y));
    s = add2(s, e);
    w = fma2(e, FAR ? two(fmaxf(u.x, kFar), fmaxf(u.y, kFar)) : t, w);
  }
  template <int DT, bool FAR, int N>
  __device__ __forceinline__ void add_vectors(const uint4 (&v)[N], float c) {
    const float r = reference();
    const Two minus = two(-r, -r), cc = two(c, c);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < RowPart<DT>::kVec; e += 2)
        add<FAR>(two(RowPart<DT>::value(v[i], e), RowPart<DT>::value(v[i], e + 1)), minus, cc);
  }
  template <int DT, int N>
  __device__ __forceinline__ float take(const uint4 (&v)[N], float c) {  // returns their largest
    const float2 ends = extremes<DT>(v);
    reach(ends.x, c);
    if ((ends.y - reference()) * c >= kFar)
      add_vectors<DT, false>(v, c);
    else
      add_vectors<DT, true>(v, c);
    return ends.x;
  }
  __device__ __forceinline__ Stat stat() const {
    const float2 a = both(s), b = both(w);
    return {m, a.x + a.y, b.x + b.y};
  }
};

// What the threads of a team (a warp, or a block) share for the most likely tokens.
template <int TEAM>
struct TopShared {
  static constexpr int kGroups = 64;
  static constexpr int kCands = TEAM == 32 ? 384 : 1024;  // eight warps' stay below 48 KB
  alignas(16) uint64_t keys[kGroups];
  alignas(16) uint64_t cand[kCands];
  uint64_t best[CR_MAX_TOP];
  uint64_t bound;
  alignas(16) float notes[TEAM / 32];
  uint32_t count, threads, listed;
  uint32_t vector[kCands];
  uint16_t thread[TEAM];

  __device__ __forceinline__ void push(uint64_t pair) {
    const uint32_t slot = atomicAdd(&count, 1u);
    if (slot < kCands) cand[slot] = pair;
  }
};

template <int TEAM>
__device__ __forceinline__ void team_sync() {
  if constexpr (TEAM == 32)
    __syncwarp();
  else
    __syncthreads();
}

// A value that at least k of the warp's are not below (k up to 32): the k-th largest where all
// differ.  NaN counts as -infinity.
__device__ __forceinline__ float warp_bound(float x, int k) {
  uint32_t key = order_key(x), most = 0;
  for (int i = 0; i < k;) {
    most = __reduce_max_sync(~0u, key);
    i += __popc(__ballot_sync(~0u, key == most));
    if (key == most) key = 0;
  }
  return most > 1 ? key_logit(most) : -kInf;
}

// A value that at least share * need of the team's logits are not below: the need-th largest note.
template <int TEAM>
__device__ __forceinline__ float least_wanted(const TopShared<TEAM>& sh, int need) {
  constexpr int warps = TEAM / 32;
  if constexpr (warps == 1) return sh.notes[0];
  const volatile float* notes = sh.notes;
  const int lane = threadIdx.x & 31;
  const float mine = notes[lane % warps];
  int rank = 0;  // above it, or equal and of an earlier warp
#pragma unroll
  for (int w = 0; w < warps; ++w) {
    const float other = __shfl_sync(~0u, mine, w);
    rank += other > mine || (other == mine && w < lane % warps);
  }
  return __shfl_sync(~0u, mine, __ffs(__ballot_sync(~0u, rank == need - 1)) - 1);
}

// sh.bound = the k-th largest of the groups' largest pairs; no candidates yet.  Groups are neighbouring
// threads, or halves of a lane's columns: `key` and `other` are the thread's largest pairs of two
// halves.
template <int TEAM>
__device__ __forceinline__ void find_bound(TopShared<TEAM>& sh, uint64_t key, uint64_t other, int k, int t) {
  constexpr int groups = TopShared<TEAM>::kGroups;
  if constexpr (TEAM == 32) {
    sh.keys[t] = key, sh.keys[t + 32] = other;
  } else {
    constexpr int per = TEAM / groups;
    key = other > key ? other : key;
#pragma unroll
    for (int o = 1; o < per; o <<= 1) {
      const uint64_t near = __shfl_xor_sync(~0u, key, o);
      key = near > key ? near : key;
    }
    if (t % per == 0) sh.keys[t / per] = key;
  }
  if (t == 0) sh.count = sh.threads = 0;
  team_sync<TEAM>();
  for (int g = t; g < groups; g += TEAM) {
    const uint64_t mine = sh.keys[g];
    int rank = 0;
#pragma unroll 4
    for (int i = 0; i < groups; i += 2) {
      const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(sh.keys + i);
      rank += (v.x > mine || (v.x == mine && i < g)) + (v.y > mine || (v.y == mine && i + 1 < g));
    }
    if (rank == k - 1) sh.bound = mine;
  }
  team_sync<TEAM>();
}

// sh.cand = the pairs at or above `bound`, of the threads whose key reaches it.
template <int DT, int TEAM>
__device__ __forceinline__ void collect(TopShared<TEAM>& sh, const RowPart<DT>& row, uint64_t bound,
                                        uint64_t key, int t) {
  if (key >= bound) sh.thread[atomicAdd(&sh.threads, 1u)] = (uint16_t)t;
  team_sync<TEAM>();
  const uint32_t n = sh.threads;
  const auto look = [&](uint32_t col, float x) {
    const uint64_t pair = pair_key(x, row.begin + col);
    if (pair < bound) return;
    sh.push(pair);
  };
  // Eight lanes take a thread's columns, so that a step of the team usually reads all there are.
  const int sub = t % 8;
  for (uint32_t i = t / 8; i < n; i += TEAM / 8) {
    const uint32_t who = sh.thread[i];
    if (sub == 0 && who < row.head) look(who, row.one(who));
    if (sub == 1 && who < row.tail)
      look(row.head + row.vectors * RowPart<DT>::kVec + who,
           row.one(row.head + row.vectors * RowPart<DT>::kVec + who));
    for (uint64_t j = who + (uint64_t)sub * TEAM; j < row.vectors; j += 16 * TEAM) {
      uint4 v[2];
#pragma unroll
      for (int q = 0; q < 2; ++q)
        v[q] = j + q * 8 * TEAM < row.vectors ? row.vec((uint32_t)j + q * 8 * TEAM) : RowPart<DT>::none();
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (q && j + 8 * TEAM >= row.vectors) break;
#pragma unroll
        for (int e = 0; e < RowPart<DT>::kVec; ++e)
          look(row.head + ((uint32_t)j + q * 8 * TEAM) * RowPart<DT>::kVec + e, RowPart<DT>::value(v[q], e));
      }
    }
  }
  team_sync<TEAM>();
}

// How many of the n pairs are above `mine`.
__device__ __forceinline__ int rank_of(const uint64_t* pairs, int n, uint64_t mine) {
  int rank = 0, j = 0;
#pragma unroll 4
  for (; j + 1 < n; j += 2) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(pairs + j);
    rank += (v.x > mine) + (v.y > mine);
  }
  if (j < n) rank += pairs[j] > mine;
  return rank;
}

// put(i, pair) for the k largest pairs of the row part, which has at least k columns: i-th in
// falling order.  sh.cand holds sh.count pairs, or lacks some.
template <int DT, int TEAM, typename Put>
__device__ __forceinline__ void find_top(TopShared<TEAM>& sh, const RowPart<DT>& row, int k, int t,
                                         Put put) {
  constexpr uint32_t cands = TopShared<TEAM>::kCands;
  if (sh.count > cands || sh.count < k) {
    uint64_t key = 0, other = 0;
    row.each_of(t, TEAM, [&](uint32_t col, float x) {
      const uint64_t pair = pair_key(x, row.begin + col);
      uint64_t& most = (col - row.head) / (TEAM * RowPart<DT>::kVec) % 2 ? other : key;
      if (pair > most) most = pair;
    });
    team_sync<TEAM>();  // sh.count has been read
    find_bound<TEAM>(sh, key, other, k, t);
    collect<DT, TEAM>(sh, row, sh.bound, other > key ? other : key, t);
  }
  const uint32_t n = sh.count;
  if (n <= cands) {
    for (uint32_t i = t; i < n; i += TEAM) {
      const uint64_t mine = sh.cand[i];
      const int rank = rank_of(sh.cand, n, mine);
      if (rank < k) put(rank, mine);
    }
    return;
  }
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
    if (t == 0) put(i, mine);
    last = mine;
  }
}

// Sums of a part of a row, by the threads of a team, for all of them; find_top may follow where
// TOP.  `stats`: TEAM / 32 of them in shared memory.
template <int DT, int TEAM, bool TOP>
__device__ __forceinline__ Stat read_part(const RowPart<DT>& row, float c, int k, int t,
                                          TopShared<TEAM>* sh, Stat* stats) {
  using Part = RowPart<DT>;
  constexpr int unroll = kUnroll, warps = TEAM / 32;
  constexpr uint64_t step = (uint64_t)TEAM * unroll;
  Running run;
  // twice the average share, of which half the warps are needed: the better half
  const int share = min(k, (2 * k + warps - 1) / warps), need = TOP ? (k + share - 1) / share : 0;
  float least = -kInf;
  const auto note = [&] {
    const float bound = warp_bound(run.m, share);
    if (t % 32 == 0) *const_cast<volatile float*>(&sh->notes[t / 32]) = bound;
  };
  // A warp's own lanes bound a few wanted ones only: of 32 the smallest lane's largest logit would be
  // the bound.  Without a list find_top looks again, at 64 groups (8192 x 2000 bf16, top 20: 21 us with the
  // list, 51 without; top 32 89 and 58; top 28 31 with it).
  const bool lists = TEAM > 32 || k <= 28;
  // notes after 1, 2, 4, ... steps: all warps take as many
  const uint32_t steps = (uint32_t)max((uint64_t)1, (row.vectors + step - 1) / step);
  for (uint32_t b = 0; b < steps; ++b) {
    const uint64_t j = b * step + t;
    uint4 v[unroll];
#pragma unroll
    for (int i = 0; i < unroll; ++i)
      v[i] = j + i * TEAM < row.vectors ? row.vec((uint32_t)(j + i * TEAM)) : Part::none();
    const float most = run.take<DT>(v, c);
    if constexpr (TOP) {
      if ((b & (b + 1)) == 0) {
        if (lists) note();
        if (b == 0) {
          if (t == 0) sh->count = sh->threads = sh->listed = 0;
          team_sync<TEAM>();
        } else {
          __syncwarp();
        }
        if (lists) least = least_wanted(*sh, need);
      }
      if (lists && most >= least) {
        uint32_t some = 0;  // bit i: vector i has one that may be wanted
#pragma unroll
        for (int i = 0; i < unroll; ++i) {
          const uint4 one[1] = {v[i]};
          some |= (largest<DT>(one) >= least ? 1u : 0u) << i;
        }
        for (uint32_t at = atomicAdd(&sh->listed, (uint32_t)__popc(some)); some; some &= some - 1, ++at)
          if (at < TopShared<TEAM>::kCands) sh->vector[at] = (uint32_t)j + (__ffs(some) - 1) * TEAM;
      }
    }
  }
  const bool single = (uint32_t)t < row.head, behind = (uint32_t)t < row.tail;
  const uint32_t col = row.head + row.vectors * Part::kVec + t;
  const float x = single ? row.one(t) : -kInf, y = behind ? row.one(col) : -kInf;
  if (single || behind) {
    run.reach(fmaxf(x, y), c);
    const float r = run.reference();
    run.add<true>(two(x, y), two(-r, -r), two(c, c));
  }
  Stat sums = lanes_merge<32>(run.stat(), c);
  if constexpr (TOP) {
    if (lists && steps & (steps - 1)) note();  // else the last step did
  }
  if constexpr (TEAM > 32) {
    if (t % 32 == 0) stats[t / 32] = sums;
    __syncthreads();
    sums = lanes_merge<warps>(stats[t % warps], c);
  } else if constexpr (TOP) {
    __syncwarp();
  }
  if (TOP && lists) {
    least = least_wanted(*sh, need);
    if (single && x >= least) sh->push(pair_key(x, row.begin + t));
    if (behind && y >= least) sh->push(pair_key(y, row.begin + col));
    const bool all = sh->listed <= TopShared<TEAM>::kCands;
    const uint32_t n = all ? sh->listed : 0;
    if (t == 0 && !all) sh->count = TopShared<TEAM>::kCands + 1;
    for (uint32_t i = t; i < n; i += TEAM) {
      const uint32_t vec = sh->vector[i];
      if (vec >= row.vectors) continue;  // past the end: -infinity, where all may be wanted
      const uint4 one[1] = {row.vec(vec)};
      if (!(largest<DT>(one) >= least)) continue;
#pragma unroll
      for (int e = 0; e < Part::kVec; ++e) {
        const float z = Part::value(one[0], e);
        if (z >= least) sh->push(pair_key(z, row.begin + row.head + vec * Part::kVec + e));
      }
    }
    team_sync<TEAM>();
  }
  return sums;
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

__device__ __forceinline__ void write_top(const LogProbArgs& a, uint64_t row, int i, uint64_t pair,
                                          const Stat& v) {
  if (a.top_ids) a.top_ids[row * a.top + i] = (int32_t)(0xffffffffu - (uint32_t)pair);
  if (a.top_logp) {
    const float x = key_logit((uint32_t)(pair >> 32));
    a.top_logp[row * a.top + i] =
        v.s == 0.0f ? -kInf : fmaf(x - v.m, a.scale, -kLn2 * log2f(v.s));
  }
}

// A warp a row.
template <int DT, bool TOP>
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
    const Stat v = read_part<DT, 32, TOP>(part, c, a.top, lane, sh, nullptr);
    if (lane == 0) write_row<DT>(a, row, v, logits);
    if constexpr (TOP) {
      find_top<DT, 32>(*sh, part, a.top, lane,
                       [&](int i, uint64_t pair) { write_top(a, row, i, pair, v); });
      __syncwarp();
    }
  }
}

// A block of TEAM threads a row, or a cluster a row (gridDim.x a multiple of the cluster).
template <int DT, int TEAM, bool TOP>
__global__ void __launch_bounds__(TEAM, kThreadsPerSm / TEAM) k_logp_block(const __grid_constant__ LogProbArgs a,
                                                     uint32_t per) {
  __shared__ TopShared<TOP ? TEAM : 32> top[1];
  __shared__ Stat stats[TEAM / 32];
  __shared__ Stat sums;
  pdl_enter();
  const float c = a.scale * kLog2E;
  const int t = threadIdx.x;
  const cg::cluster_group cluster = cg::this_cluster();
  const uint32_t parts = cluster.num_blocks(), part_no = cluster.block_rank();
  for (uint64_t row = blockIdx.x / parts; row < a.rows; row += gridDim.x / parts) {
    const char* logits = row_at<DT>(a.logits, row);
    const uint32_t begin = min(part_no * per, a.vocab);
    const RowPart<DT> part(logits, begin, min(per, a.vocab - begin));
    TopShared<TEAM>* sh = nullptr;
    if constexpr (TOP) sh = top;
    Stat v = read_part<DT, TEAM, TOP>(part, c, a.top, t, sh, stats);
    if (parts == 1) {
      if (t == 0) write_row<DT>(a, row, v, logits);
      if constexpr (TOP)
        find_top<DT, TEAM>(*sh, part, a.top, t,
                           [&](int i, uint64_t pair) { write_top(a, row, i, pair, v); });
      __syncthreads();
      continue;
    }
    if (t == 0) sums = v;
    if constexpr (TOP)
      find_top<DT, TEAM>(*sh, part, a.top, t, [&](int i, uint64_t pair) { sh->best[i] = pair; });
    cluster.sync();
    if (part_no == 0) {
      v = lanes_merge<kMostParts>(t % kMostParts < parts ? *cluster.map_shared_rank(&sums, t % kMostParts)
                                                         : Stat{-kInf, 0.0f, 0.0f}, c);
      if (t == 0) write_row<DT>(a, row, v, logits);
      if constexpr (TOP) {
        // rank the parts' best among each other
        const int n = (int)parts * a.top;
        for (int i = t; i < n; i += TEAM)
          top->cand[i] = cluster.map_shared_rank(top, i / a.top)->best[i % a.top];
        __syncthreads();
        for (int i = t; i < n; i += TEAM) {
          const uint64_t mine = top->cand[i];
          const int rank = rank_of(top->cand, n, mine);
          if (rank < a.top) write_top(a, row, rank, mine, v);
        }
      }
    }
    cluster.sync();
  }
}

template <int DT, int TEAM, bool TOP>
cudaError_t run_block(const LogProbArgs& a, uint32_t parts, cudaStream_t s) {
  const uint32_t per = (uint32_t)((((uint64_t)a.vocab + parts - 1) / parts + 63) / 64 * 64);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(std::min<uint64_t>(a.rows, 1u << 27) * parts));
  cfg.blockDim = dim3(TEAM);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = parts;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = parts > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_logp_block<DT, TEAM, TOP>, a, per);
}

template <int DT, bool TOP>
cudaError_t run(const LogProbArgs& a, cudaStream_t s) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  if (a.vocab <= 2048)
    return launch_pdl(k_logp_warp<DT, TOP>, dim3(flat_grid(a.rows * 32)), kBlock, s, a);
  // Parts of a row: while rows are too few to give each SM two, and parts keep a step of loads a
  // thread (200 x 32000 bf16: 5.6 us so, 10.5 with parts of a quarter step; 400 rows: 7.6 so, 10.4 with parts up to four
  // an SM).
  uint32_t parts = 1;
  while (parts < kMostParts && a.rows * parts < 2 * (uint64_t)sms &&
         a.vocab / (2 * parts) >= kUnroll * kBlock * RowPart<DT>::kVec)
    parts *= 2;
  // Many short rows: fewer threads each, so that a row's end costs less of it.  With 128 threads and with
  // 256: 8192 x 32000 bf16 81.5 and 88.1 us, top 8 114 and 148; 4096 x 64000 (125 KB a row) 82.6 and 83.6, top 8
  // 104 and 119; 4096 x 90000 (176 KB) 113 and 116, top 8 137 and 157; 1531 x 50257 fp32 (196 KB) 55.5
  // and 52.1, top 8 64.1 and 63.0.  The limit is below where the two meet.
  constexpr uint64_t kShort = 128 << 10;
  if (a.rows >= 4 * (uint64_t)sms && a.vocab * (16 / RowPart<DT>::kVec) <= kShort)
    return run_block<DT, 128, TOP>(a, 1, s);
  return run_block<DT, kBlock, TOP>(a, parts, s);
}

}  // namespace

cudaError_t launch_log_probs(cr_dtype d, const LogProbArgs& a, cudaStream_t s) {
  if (d == CR_BF16) return a.top ? run<CR_BF16, true>(a, s) : run<CR_BF16, false>(a, s);
  return a.top ? run<CR_F32, true>(a, s) : run<CR_F32, false>(a, s);
}

}  // namespace cr
