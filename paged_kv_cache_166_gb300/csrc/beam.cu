// Beam search's selection over beams and vocabulary.
//
// For every request s, from the logits of its K live beams and their scores so far:
//   candidate (b, v): score = beam_scores[s, b] + logits[s, b, v] - lse[s, b],
//   lse[s, b] = log sum_v exp(logits[s, b, v]),
// the N best candidates in order: by score, equal scores by beam, and within a beam by
// logit and then by token, lower first.
//
// One pass over the logits, one launch.  A CTA streams a part of one row and reduces it to
// its maximum, its sum of exponentials and its best N logits (a row's candidates are
// ordered by their logits alone, so its lse is not needed for that); the CTA that finishes
// a request's last part merges them all (many of them: the one that finishes a row's last
// part merges that row first).  Nobody waits: tickets say who is last.
//
// Best N of a set spread over a block's threads: with t the N-th best of the best entries
// of small groups of threads, at least N entries are as good as t, and those that are lie
// in N groups: few, so they are collected in shared memory and each counts the entries
// better than itself.  Entries are compared as integer keys and no two are equal (equal
// values are told apart by their position), so the order of collection does not matter.
//
// What bounds it: many rows of large vocabularies the memory (64 x 8 rows of 131,072 fp32
// logits, 268 MB: 53.5 us, 5.0 TB/s), small calls the chain of steps of which each waits for
// the one before: a tile's loads, its threshold, the list and its ranking, a ticket, the merge
// (4 rows of 32,000: 9.5 us; 32 x 4 of 65,537 fp16: 20.2 us, 17 MB).
//
// Precision: candidates of different beams may lie next to each other, so a thread's sums
// carry their rounding errors, sums across threads are 64-bit integers, and lse and the
// scores are pairs of fp32 values (48 bits).  Only the score handed out is rounded to fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxBeams = 64;
constexpr int kMaxOut = 128;
constexpr int kMaxRows = 65535;    // num_seqs * num_beams
constexpr int kMaxEntries = 8192;  // entries a merge takes: parts * N, beams * N
// Entries of a request that are merged at once, not row by row before (4,096 entries at once:
// 41.4 us against 37.7; fewer than 2,048 are no faster row by row).
constexpr int kOneMerge = 2048;
constexpr int kElements = 16;      // logits of a tile a thread holds
constexpr int kTile = kElements * kThreads;
constexpr int kMaxSmem = 128 << 10;  // the most is 96 KB: kMaxOut x 32 entries of 24 bytes, dealt from 64 lists
constexpr int kList = kMaxOut + kMaxOut * kElements;  // entries of the list

struct BeamArgs {
  const void* logits;
  int64_t seq_stride, beam_stride;  // elements
  const float* beam_scores;
  float* scores;
  int32_t* beams;
  int32_t* tokens;
  // workspace: the tickets, zero between launches, then per (row, part) and per row
  int32_t* row_ticket;
  int32_t* seq_ticket;
  float* part_max;
  uint64_t* part_sum;  // in units of 2^-32 exp(part_max)
  uint64_t* part_top;  // keys of a part's best N
  uint64_t* row_top;   // keys of a row's best N (by_row)
  int32_t K, V, N, parts;
  int32_t tiles;       // of a part
  int32_t by_row;
};

// A value of about 48 bits as the unevaluated sum of two fp32 ones, |lo| at most half a step
// of hi: fp64 operations run at a 64th of the rate of fp32 ones and take as much longer.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {  // exactly a + b
  const float s = __fadd_rn(a, b), z = __fsub_rn(s, a);
  return Two{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, z)), __fsub_rn(b, z))};
}
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 as 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}

// Keys: larger is better, 0 is no entry, and no two entries of a set have the same one.
// A token of a row: its logit's bits in the order of the values (-0 as 0), then the token,
// lower first.
__device__ __forceinline__ uint64_t token_key(float x, int token) {
  return (static_cast<uint64_t>(ordered(x)) << 32) | static_cast<uint32_t>(~token);
}
__device__ __forceinline__ int key_token(uint64_t key) {
  return static_cast<int>(~static_cast<uint32_t>(key));
}
__device__ __forceinline__ float key_logit(uint64_t key) {
  return unordered(static_cast<uint32_t>(key >> 32));
}
// A candidate of a request: its score's bits in the order of the values, then the beam, lower
// first, then its key in the beam's row.
struct ScoreKey {
  uint64_t score, token;
  uint32_t beam;  // ~beam
  __device__ __forceinline__ bool operator>(const ScoreKey& o) const {
    // no branches: rankings compare many
    return (score > o.score) |
           ((score == o.score) & ((beam > o.beam) | ((beam == o.beam) & (token > o.token))));
  }
  __device__ __forceinline__ bool none() const { return score == 0; }
};
__device__ __forceinline__ ScoreKey score_key(Two x, int beam, uint64_t token) {
  return ScoreKey{(static_cast<uint64_t>(ordered(x.hi)) << 32) | ordered(x.lo), token,
                  ~static_cast<uint32_t>(beam)};
}
// beam score + logit - lse; -infinity beyond fp32's range.
__device__ __forceinline__ Two score_of(float beam_score, float x, Two lse) {
  const Two a = two_sum(beam_score, x), b = two_sum(a.hi, -lse.hi);
  const Two c = two_sum(b.hi, (a.lo + b.lo) - lse.lo);
  return isfinite(c.hi) && isfinite(c.lo) ? c : Two{-INFINITY, 0.f};
}
// m + log(2^-32 sum), sum > 0.  sum = f 2^e with f in (0.7, 1.42); log f = 2 atanh z with
// z = (f - 1) / (f + 1), its series from the third power on in fp32 (|z| < 0.172), and e
// log 2 with log 2 in two parts, the first of 16 bits: off by some 2^-31.
__device__ __forceinline__ Two log_sum(float m, uint64_t sum) {
  const int lead = __clzll(static_cast<long long>(sum));
  const uint64_t u = sum << lead;
  int e = 63 - lead - 32;
  float f = static_cast<float>(static_cast<uint32_t>(u >> 40)) * 0x1p-23f;
  float g = static_cast<float>(static_cast<uint32_t>(u >> 16) & 0xffffffu) * 0x1p-47f;
  if (f > 1.41421356f) {
    f *= 0.5f;
    g *= 0.5f;
    ++e;
  }
  const float n = f - 1.f, d = f + 1.f, d_lo = (f - (d - 1.f)) + g;
  const float z = __fdiv_rn(n, d);
  const float z_lo = __fdividef(fmaf(-z, d, n) + (g - z * d_lo), d);
  const float y = z * z;
  const float tail =
      y * (1.f / 3.f + y * (1.f / 5.f + y * (1.f / 7.f + y * (1.f / 9.f + y * (1.f / 11.f)))));
  const float k = static_cast<float>(e);
  const Two a = two_sum(m, k * 0.693145751953125f), b = two_sum(a.hi, 2.f * z);
  return two_sum(b.hi, (a.lo + b.lo) + (k * 1.42860682e-6f + 2.f * (z_lo + z * tail)));
}
__device__ __forceinline__ bool none(uint64_t k) { return k == 0; }
__device__ __forceinline__ bool none(const ScoreKey& k) { return k.none(); }

__device__ __forceinline__ uint64_t shfl_xor(uint64_t k, int o) {
  return __shfl_xor_sync(0xffffffffu, static_cast<unsigned long long>(k), o);
}
__device__ __forceinline__ ScoreKey shfl_xor(const ScoreKey& k, int o) {
  return ScoreKey{shfl_xor(k.score, o), shfl_xor(k.token, o),
                  __shfl_xor_sync(0xffffffffu, k.beam, o)};
}

// Threads whose best entries are merged before the threshold is sought: about four
// groups of them for each entry wanted, in 32 to 256 groups.  (Ranking all 256 threads' best
// for 8 wanted of one request: 19.1 us a call against 9.5.)
__host__ __device__ constexpr int group_of(int n) {
  return n <= 8 ? 8 : (n <= 16 ? 4 : (n <= 32 ? 2 : 1));
}

template <typename Key>
struct TopShared {
  int count;
  Key threshold;
  Key best[kThreads];
};

// Threshold of the block's entries, `mine` the thread's best: the n-th best of the groups'
// best, so that at least n entries are as good as it and those that are lie in n groups;
// an empty key ("everything") if fewer groups have an entry.
template <typename Key>
__device__ __forceinline__ Key threshold_of(Key mine, int n, TopShared<Key>& sh) {
  const int g = group_of(n), groups = kThreads / g;
  for (int o = 1; o < g; o <<= 1) {
    const Key other = shfl_xor(mine, o);
    if (other > mine) mine = other;
  }
  __syncthreads();
  if (threadIdx.x % g == 0) sh.best[threadIdx.x / g] = mine;
  if (threadIdx.x == 0) {
    sh.count = 0;
    sh.threshold = Key{};
  }
  __syncthreads();
  // a group's threads share the ranking of its best: their number is the group's size
  const Key k = sh.best[threadIdx.x / g];
  int rank = 0;
#pragma unroll 4
  for (int i = threadIdx.x % g; i < groups; i += g) rank += sh.best[i] > k;
  for (int o = 1; o < g; o <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
  if (rank == n - 1 && !none(k) && threadIdx.x % g == 0) sh.threshold = k;
  __syncthreads();
  return sh.threshold;
}

// The entries of a list by rank: put(rank, key) for rank < n, eight threads an entry.
template <typename Key, typename Put>
__device__ __forceinline__ void by_rank(const Key* list, int count, int n, Put put) {
  const int sub = threadIdx.x & 7;
  for (int i0 = 0; i0 < count; i0 += kThreads / 8) {
    const int i = i0 + (threadIdx.x >> 3);
    const Key k = list[i < count ? i : 0];
    int rank = 0;
#pragma unroll 4
    for (int j = sub; j < count; j += 8) rank += list[j] > k;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (sub == 0 && i < count && rank < n) put(rank, k);
  }
}

// The collected entries in their order, empty keys behind them.
template <typename Key, typename Put>
__device__ __forceinline__ void ranked(const Key* list, int n, const TopShared<Key>& sh, Put put) {
  __syncthreads();
  const int count = sh.count;
  by_rank(list, count, n, put);
  for (int i = count + threadIdx.x; i < n; i += kThreads) put(i, Key{});
}

// log2 of the places a list of n entries takes when lists are dealt to threads.
__host__ __device__ constexpr int places_log2(int n) {
  int k = 0;
  while (1 << k < n) ++k;
  return k;
}

// The best n of L lists in order, of n entries each: get(l, r) is the r-th of list l.
// The threshold is a tight one if the best entries lie with many threads, whether they are
// the first few of every list or most of a single one's.  So a list is dealt to the threads
// side by side, and where it begins is moved on from round to round (by the golden section,
// so that few first entries meet).  Where it was not, the first entries of 32 lists of 128
// lay with few threads and 2,000 entries were left to be ranked: 157 us a call of one beam of
// 128,256 tokens, 128 wanted, and 38 now; 64 beams of 32,000: 119 and 91, and 319 with the
// lists dealt entry by entry, all first ones and then all second ones.
template <typename Key, typename Get, typename Put>
__device__ __forceinline__ void merge_top(int L, int n, Get get, Key* list, TopShared<Key>& sh,
                                          Put put) {
  const int tid = threadIdx.x, k = places_log2(n), places = 1 << k;
  const int step = (places * 79 >> 7) | 1, M = L << k;
  auto entry = [&](int i) {  // i = tid + j * kThreads
    const int l = i >> k, r = (i + i / kThreads * step) & (places - 1);
    return l < L && r < n ? get(l, r) : Key{};
  };
  const Key first = tid < M ? entry(tid) : Key{};
  Key best = first, t{};
  if (M > 32) {
    for (int i = tid + kThreads; i < M; i += kThreads) {
      const Key x = entry(i);
      if (x > best) best = x;
    }
    t = threshold_of(best, n, sh);
  } else {  // few enough to be ranked as they are
    __syncthreads();
    if (tid == 0) sh.count = 0;
    __syncthreads();
  }
  for (int i = tid; i < M; i += kThreads) {
    const Key x = i == tid ? first : entry(i);
    if (!none(x) && !(t > x)) list[atomicAdd(&sh.count, 1)] = x;
  }
  ranked(list, n, sh, put);
}

// One tile's logits of a thread, as they were loaded: pieces of 16 bytes, piece j the
// tokens first + (j * kThreads + thread) * W onwards.  A row may start at any element, and
// which tokens a thread has does not depend on where, so equal rows have equal lse, bit
// for bit: of a row that starts off a 16-byte boundary, 32-bit pieces are loaded element by
// element (the lines are shared), 16-bit ones as the two aligned pieces around them, shifted
// together when they are used.
template <typename T>
struct Tile {
  static constexpr int W = 16 / static_cast<int>(sizeof(T));
  static constexpr int kPieces = kElements / W;
  static constexpr bool kWide = sizeof(T) == 4;
  uint4 lo[kPieces], hi[kWide ? 1 : kPieces];
  uint32_t shifted;  // pieces to be shifted

  __device__ __forceinline__ void load(const T* x, int first, int V, uint32_t skew) {
    shifted = 0;
    if (skew == 0 && first + kTile <= V) {  // the usual tile
      const uint4* at = reinterpret_cast<const uint4*>(x + first) + threadIdx.x;
#pragma unroll
      for (int j = 0; j < kPieces; ++j) lo[j] = __ldcs(at + j * kThreads);
      return;
    }
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int p = first + (j * kThreads + static_cast<int>(threadIdx.x)) * W;
      if (skew == 0 && p + W <= V) {
        lo[j] = __ldcs(reinterpret_cast<const uint4*>(x + p));
      } else if (!kWide && skew != 0 && p >= W && p + 2 * W <= V) {
        const uint4* at =
            reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(x + p) - skew);
        lo[j] = __ldg(at);
        hi[kWide ? 0 : j] = __ldg(at + 1);
        shifted |= 1u << j;
      } else {
        T e[W];
#pragma unroll
        for (int w = 0; w < W; ++w)
          e[w] = p + w < V ? x[p + w] : ptx::from_float<T>(-INFINITY);
        lo[j] = *reinterpret_cast<const uint4*>(e);
      }
    }
  }

  __device__ __forceinline__ void values(uint32_t skew, float (&v)[kElements]) const {
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      uint4 u = lo[j];
      if constexpr (!kWide) {
        if (shifted & (1u << j)) u = joined(lo[j], hi[j], skew);
      }
      const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        if constexpr (kWide) v[j * W + w] = e[w];
        else v[j * W + w] = ptx::to_float(e[w]);
      }
    }
  }

  // 16 bytes from byte `skew` of two pieces on.
  static __device__ __forceinline__ uint4 joined(const uint4& a, const uint4& b, uint32_t skew) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (skew & 4) {
#pragma unroll
      for (int i = 0; i < 7; ++i) w[i] = w[i + 1];
    }
    if (skew & 8) {
#pragma unroll
      for (int i = 0; i < 5; ++i) w[i] = w[i + 2];
    }
    const uint32_t bits = 8 * (skew & 3);
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                      __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
  }

  static __device__ __forceinline__ int token(int first, int i) {
    return first + ((i / W) * kThreads + static_cast<int>(threadIdx.x)) * W + i % W;
  }
};

// What is seldom done with a thread's logits is done in loops over bits: a kernel of few
// microseconds waits for its instructions too.
__device__ __forceinline__ uint32_t at_least(const float (&v)[kElements], float x) {
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < kElements; ++i) bits |= v[i] >= x ? 1u << i : 0u;
  return bits;
}
__device__ __forceinline__ float element(const float (&v)[kElements], int i) {
  float x = v[0];  // v stays in registers: no index at run time
#pragma unroll
  for (int j = 1; j < kElements; ++j) x = i == j ? v[j] : x;
  return x;
}

// A thread's running sum of exponentials: sum_i 2^(x_i log2 e - ref), ref the rounded
// product of log2 e and a logit `base` no further below the largest one so far than kLag.  A
// term is one multiply-add, one ex2 and one addition; what the rounding of ref leaves out is
// put right at the end.  The terms of a tile are added in fp32, and the tiles' sums with
// their rounding errors carried along.  Beyond 2^20, where ref could be off by more than
// 1/16, a term goes by the difference of its logit and base.
struct ExpSum {
  static constexpr float kLog2e = 1.4426950408889634f;
  static constexpr float kHuge = 1048576.f;
  static constexpr float kLag = 16.f;
  float base = -INFINITY, ref = 0.f, sum = 0.f, carry = 0.f;

  static __device__ __forceinline__ bool huge(float x) { return fabsf(x) > kHuge; }
  // What a sum's unit is short of 2^(x log2 e), as an exponent: exact.
  static __device__ __forceinline__ float lost(float x, float r) {
    return huge(x) ? 0.f : fmaf(x, kLog2e, -r);
  }

  __device__ __forceinline__ void add(const float (&v)[kElements], float most) {
    if (most > base + kLag && most < INFINITY) {  // seldom but for the first finite logit
      const float r = most * kLog2e;
      const float f = ptx::ex2((base - most) * kLog2e + (lost(most, r) - lost(base, ref)));
      sum *= f;  // 0 before the first finite logit
      carry *= f;
      base = most;
      ref = r;
    }
    float part = 0.f;
    if (base > -INFINITY) {
      if (!huge(base)) {
        // two terms at a time
        const uint64_t l = ptx::pair(kLog2e, kLog2e), r = ptx::pair(-ref, -ref);
        uint64_t sums = ptx::pair(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kElements; i += 2) {
          float x, y;
          ptx::unpair(ptx::fma2(ptx::pair(v[i], v[i + 1]), l, r), x, y);
          sums = ptx::add2(sums, ptx::pair(ptx::ex2(x), ptx::ex2(y)));
        }
        float x, y;
        ptx::unpair(sums, x, y);
        part = x + y;
      }
      if (huge(base) || part != part) {  // or a NaN among them: a banned token
        part = 0.f;
#pragma unroll 1
        for (int i = 0; i < kElements; ++i) {
          const float x = element(v, i);
          const float y = huge(base) ? (x - base) * kLog2e : fmaf(x, kLog2e, -ref);
          part += x == x ? ptx::ex2(y) : 0.f;
        }
      }
    }
    const float t = sum + part, z = t - sum;
    carry += (sum - (t - z)) + (part - z);
    sum = t;
  }

  // The sum in units of exp(m), m at least the largest logit: at most 1 a term.
  __device__ __forceinline__ float total(float m) const {
    if (base == -INFINITY) return 0.f;
    return (sum + carry) * exp2f(fmaf(base - m, kLog2e, -lost(base, ref)));
  }
};

// Sums across threads are integers, multiples of 2^-32: their order does not matter, and
// fp64 additions run at a 64th of their rate.  A row's sum stays below 2^31.
constexpr float kFixed = 4294967296.f;
__device__ __forceinline__ uint64_t warp_sum_of(uint64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += shfl_xor(x, o);
  return x;
}

// x w, w in [0, 1] with its 24 bits as an integer: both halves of the product count.
__device__ __forceinline__ uint64_t scaled(uint64_t x, float w) {
  if (w == 1.f) return x;
  const uint64_t q = static_cast<uint64_t>(w * 0x1p32f);
  return __umul64hi(x, q << 32);
}

__device__ __forceinline__ uint64_t load_key(const uint64_t* p) {
  return static_cast<uint64_t>(__ldcg(reinterpret_cast<const unsigned long long*>(p)));
}

// True for the block that is the last of `of` to come here; it sees what the others wrote.
__device__ __forceinline__ bool last_to_come(int32_t* ticket, int of, int* flag) {
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const int t = atomicAdd(ticket, 1);
    if (t == of - 1) *ticket = 0;  // ready for the next launch
    *flag = t == of - 1;
  }
  __syncthreads();
  const bool last = *flag != 0;
  if (last) __threadfence();
  __syncthreads();
  return last;
}

// A CTA per (part, row): it streams the part's tiles, the next one loading while this one is
// worked on.  The list holds the candidates so far: the best N of the first tile (found by
// a threshold), then whatever beats the N-th best of the list when it was last cut down.
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) beam_select_kernel(const BeamArgs a) {
  extern __shared__ __align__(16) unsigned char buf[];
  __shared__ union {
    TopShared<uint64_t> row;
    TopShared<ScoreKey> seq;
  } sh;
  __shared__ uint64_t cut[kMaxOut];
  __shared__ uint64_t warp_sums[kThreads / 32];
  __shared__ Two lse_s[kMaxBeams];
  __shared__ float largest_s;
  __shared__ int listed, flag;
  const int tid = threadIdx.x, part = blockIdx.x;
  const int row = blockIdx.y, N = a.N, V = a.V;
  const int s = row / a.K, b = row - s * a.K;
  uint64_t* const list = reinterpret_cast<uint64_t*>(buf);

  const bool alive = isfinite(a.beam_scores[row]);  // a dead beam's logits are not read
  const int64_t slot = static_cast<int64_t>(row) * a.parts + part;
  if (alive) {
    const T* const x = static_cast<const T*>(a.logits) + s * a.seq_stride + b * a.beam_stride;
    const uint32_t skew = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(x) & 15);
    const int64_t begin = static_cast<int64_t>(part) * a.tiles * kTile;
    const int64_t behind = begin + static_cast<int64_t>(a.tiles) * kTile;
    const int first = static_cast<int>(begin < V ? begin : V);
    const int end = static_cast<int>(behind < V ? behind : V);
    // The N-th best of the list when it was last cut down (0: none yet), and the least logit
    // that beats it: later tokens lose to earlier equal ones, so a larger one.
    uint64_t least = 0;
    float bar = -INFINITY;
    ExpSum es;
    Tile<T> tile;
    if (tid == 0) listed = 0;
    if (first < end) tile.load(x, first, V, skew);
    __syncthreads();
    // The first tile is worked on with care: however many candidates it has, those that reach
    // a threshold are listed, and the list is cut down to the best N.  Then come groups of
    // three times the tiles seen so far, of which a few N logits are expected to beat the
    // N-th best: those are listed as they come, and the list is cut down at the group's end.
    // Logits that keep growing overflow it: then the group is gone through once more, with
    // care.
    int stop = first + kTile, start = first;  // the group's tiles
    int summed = first;                       // tiles before are in the sum
    bool care = true;
    for (int at = first; at < end;) {
      float v[kElements];
      tile.values(skew, v);
      if (at + kTile < end) tile.load(x, at + kTile, V, skew);
      float most = -INFINITY;
#pragma unroll
      for (int i = 0; i < kElements; ++i) most = fmaxf(most, v[i]);
      if (at == summed) {
        es.add(v, most);
        summed += kTile;
      }
      bool lists = most >= bar;
      float floor = bar;
      uint64_t t = 0;
      if (care) {
#pragma unroll
        for (int i = 0; i < kElements; ++i) v[i] = fmaxf(v[i], -INFINITY);  // NaN: banned
        // the thread's best: the lowest token of its largest logit
        const uint32_t same = lists ? at_least(v, most) : 0u;
        const int token = Tile<T>::token(at, __ffs(same) - 1);
        t = threshold_of(same != 0 && token < V ? token_key(most, token) : 0, N, sh.row);
        if (t != 0) floor = fmaxf(floor, key_logit(t));
      }
      if (lists) {
        for (uint32_t left = at_least(v, floor); left != 0; left &= left - 1) {
          const int i = __ffs(left) - 1;
          const int token = Tile<T>::token(at, i);
          const uint64_t k = token_key(element(v, i), token);
          if (token < V && !(t > k)) {
            const int n = atomicAdd(&listed, 1);
            if (n < kList) list[n] = k;
          }
        }
      }
      at += kTile;
      if (!care && at < stop && at < end) continue;
      __syncthreads();
      const int count = listed;
      __syncthreads();  // every thread has read it before the next one is listed
      if (count > kList) {  // only without care
        if (tid == 0) listed = N;
        care = true;
        at = start;
        tile.load(x, at, V, skew);
        __syncthreads();
        continue;
      }
      if (count >= N && at < end && (count > N || least == 0)) {
        by_rank(list, count, N, [&](int rank, uint64_t k) { cut[rank] = k; });
        __syncthreads();
        if (tid < N) list[tid] = cut[tid];
        if (tid == 0) listed = N;
        least = cut[N - 1];
        bar = nextafterf(key_logit(least), INFINITY);
        __syncthreads();
      }
      if (at >= stop) {  // the next group; a list that is not full yet needs care
        start = at;
        care = least == 0;
        stop = care ? at + kTile : ((end - at) / 3 <= at - first ? end : at + 3 * (at - first));
      }
    }
    // the part's list in order, its maximum and its sum
    uint64_t* const out = a.part_top + slot * N;
    if (tid == 0) {
      sh.row.count = listed;
      largest_s = -INFINITY;
    }
    ranked(list, N, sh.row, [&](int rank, uint64_t k) {
      out[rank] = k;
      if (rank == 0 && k != 0) largest_s = key_logit(k);
    });
    __syncthreads();
    const float m = largest_s;
    const uint64_t mine =
        warp_sum_of(isfinite(m) ? __float2ull_rn(es.total(m) * kFixed) : 0);
    if ((tid & 31) == 0) warp_sums[tid >> 5] = mine;
    __syncthreads();
    if (tid == 0) {
      uint64_t sum = 0;
#pragma unroll
      for (int i = 0; i < kThreads / 32; ++i) sum += warp_sums[i];
      a.part_max[slot] = m;
      a.part_sum[slot] = sum;
    }
  }

  // Many entries (a.by_row): a row's lists are merged by the CTA that finishes it last.
  const int64_t r0 = static_cast<int64_t>(s) * a.K;
  const uint64_t* in = a.part_top + r0 * a.parts * N;
  int lists = a.parts;  // of a beam, N entries each
  if (a.by_row) {
    if (!last_to_come(a.row_ticket + row, a.parts, &flag)) return;
    if (alive) {
      const uint64_t* const mine = a.part_top + static_cast<int64_t>(row) * a.parts * N;
      uint64_t* const out = a.row_top + static_cast<int64_t>(row) * N;
      merge_top<uint64_t>(
          a.parts, N, [&](int l, int r) { return load_key(mine + l * N + r); }, list, sh.row,
          [&](int rank, uint64_t k) { out[rank] = k; });
    }
    in = a.row_top + r0 * N;
    lists = 1;
  }
  if (!last_to_come(a.seq_ticket + s, a.by_row ? a.K : a.K * a.parts, &flag)) return;

  // The request, by the CTA that finishes it last: the rows' lse, a warp each, from their
  // parts' maxima and sums (+infinity: a beam without a finite score or largest logit,
  // whose candidates are its first tokens at -infinity), then the best of all lists.
  for (int bb = tid >> 5; bb < a.K; bb += kThreads / 32) {
    const int64_t first = (r0 + bb) * a.parts;
    float m = -INFINITY;
    uint64_t sum = 0;
    const bool lives = isfinite(a.beam_scores[r0 + bb]);
    if (lives) {
      for (int c = tid & 31; c < a.parts; c += 32) m = fmaxf(m, __ldcg(a.part_max + first + c));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (isfinite(m))
        for (int c = tid & 31; c < a.parts; c += 32) {
          const float w = exp2f((__ldcg(a.part_max + first + c) - m) * ExpSum::kLog2e);
          sum += scaled(load_key(a.part_sum + first + c), w);
        }
      sum = warp_sum_of(sum);
    }
    if ((tid & 31) == 0)
      lse_s[bb] = lives && isfinite(m) ? log_sum(m, sum) : Two{INFINITY, 0.f};
  }
  __syncthreads();
  merge_top<ScoreKey>(
      a.K * lists, N,
      [&](int l, int r) {
        const int bb = l / lists;
        const Two lse = lse_s[bb];
        const Two none{-INFINITY, 0.f};
        if (lse.hi == INFINITY)
          return l == bb * lists && r < V ? score_key(none, bb, token_key(0.f, r)) : ScoreKey{};
        const uint64_t k = load_key(in + l * N + r);
        if (k == 0) return ScoreKey{};
        const float x = key_logit(k);
        return score_key(x == -INFINITY ? none : score_of(a.beam_scores[r0 + bb], x, lse), bb, k);
      },
      reinterpret_cast<ScoreKey*>(buf), sh.seq,
      [&](int rank, const ScoreKey& k) {
        const int64_t at = static_cast<int64_t>(s) * N + rank;
        a.scores[at] = unordered(static_cast<uint32_t>(k.score >> 32));  // rounded to nearest
        a.beams[at] = static_cast<int>(~k.beam);
        a.tokens[at] = key_token(k.token);
      });
}

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct BeamLayout {
  size_t row_ticket, seq_ticket, part_max, part_sum, part_top, row_top, total;
};

// Parts a row is cut into: as many as fill the SMs once, at three CTAs each.  Two, three, four:
// 50 x 4 rows of 128,256 fp32 logits 33.3, 27.6, 27.1 us (too few CTAs to hide their steps from
// one another); 64 x 4 of 32,000 bf16 17.1, 17.1, 19.2 and 32 x 4 of 65,537 fp16 19.8, 20.2,
// 22.0 (every part has its first tile, its list and its place in the merge).
int parts_of(int64_t rows, int32_t V, int32_t N, int sms) {
  const int64_t tiles = (static_cast<int64_t>(V) + kTile - 1) / kTile;
  int64_t parts = rows > 0 ? 3 * static_cast<int64_t>(sms) / rows : 1;
  parts = parts < kMaxEntries / N ? parts : kMaxEntries / N;
  parts = parts < tiles ? parts : tiles;
  parts = parts > 1 ? parts : 1;
  const int64_t each = (tiles + parts - 1) / parts;
  return static_cast<int>((tiles + each - 1) / each);  // none of them empty
}

// The tickets lie where they are whatever the sizes, so one workspace serves every call.
BeamLayout beam_layout(int32_t S, int32_t K, int32_t N, int parts) {
  BeamLayout L;
  const size_t rows = static_cast<size_t>(S) * K, slots = rows * parts;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += round256(bytes);
    return at;
  };
  L.row_ticket = take(PKV_BEAM_TICKET_BYTES / 2);
  L.seq_ticket = take(PKV_BEAM_TICKET_BYTES / 2);
  L.part_max = take(slots * 4);
  L.part_sum = take(slots * 8);
  L.part_top = take(slots * N * 8);
  L.row_top = take(rows * N * 8);
  L.total = off;
  return L;
}
static_assert(PKV_BEAM_TICKET_BYTES / 2 >= (kMaxRows + 1) * 4, "a ticket for every row");

int beam_check(int32_t S, int32_t K, int32_t V, int32_t N, int32_t dtype) {
  PKV_REQUIRE(dtype == PKV_F32 || dtype == PKV_F16 || dtype == PKV_BF16, PKV_ERR_DTYPE,
              "dtype %d is not f32, f16 or bf16", dtype);
  PKV_REQUIRE(S >= 0 && K > 0 && V > 0 && N > 0, PKV_ERR_INVALID_ARG,
              "sizes must be positive (num_seqs >= 0)");
  PKV_REQUIRE(K <= kMaxBeams && N <= kMaxOut, PKV_ERR_UNSUPPORTED,
              "num_beams %d above %d or num_out %d above %d", K, kMaxBeams, N, kMaxOut);
  PKV_REQUIRE(static_cast<int64_t>(N) <= static_cast<int64_t>(K) * V, PKV_ERR_INVALID_ARG,
              "num_out %d above num_beams * vocab", N);
  PKV_REQUIRE(static_cast<int64_t>(S) * K <= kMaxRows, PKV_ERR_UNSUPPORTED,
              "num_seqs * num_beams above %d", kMaxRows);
  PKV_REQUIRE(V <= INT_MAX - 2 * kTile, PKV_ERR_UNSUPPORTED, "vocab %d above %d", V,
              INT_MAX - 2 * kTile);
  return PKV_OK;
}

int beam_sizes(int32_t S, int32_t K, int32_t V, int32_t N, int* parts, BeamLayout* L) {
  int sms = 0, dev = 0;
  const int rc = device_sm_count(&sms, &dev);
  if (rc != PKV_OK) return rc;
  *parts = parts_of(static_cast<int64_t>(S) * K, V, N, sms);
  *L = beam_layout(S, K, N, *parts);
  return PKV_OK;
}

template <typename T>
int launch_beam(const BeamArgs& a, int32_t S, cudaStream_t st) {
  // the list of a part, or those of the merges: the entries of the N groups of threads that
  // reach a threshold, or all of a small set
  auto merged = [&](int lists) {
    const int rounds = ((lists << places_log2(a.N)) + kThreads - 1) / kThreads;
    const size_t n = static_cast<size_t>(a.N) * group_of(a.N) * rounds;
    return n < kThreads ? static_cast<size_t>(kThreads) : n;
  };
  size_t smem = kList * sizeof(uint64_t);
  const size_t rows = a.by_row ? merged(a.parts) * sizeof(uint64_t) : 0;
  const size_t seqs = merged(a.K * (a.by_row ? 1 : a.parts)) * sizeof(ScoreKey);
  smem = smem < rows ? rows : smem;
  smem = smem < seqs ? seqs : smem;
  static SmemOnce once;
  const int rc = allow_dynamic_smem(once, reinterpret_cast<const void*>(beam_select_kernel<T>),
                                    kMaxSmem);
  if (rc != PKV_OK) return rc;
  beam_select_kernel<T><<<dim3(a.parts, S * a.K), kThreads, smem, st>>>(a);
  PKV_CUDA(cudaGetLastError());
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_beam_workspace_size(int32_t num_seqs, int32_t num_beams, int32_t vocab, int32_t num_out,
                            int32_t dtype, size_t* bytes) {
  PKV_REQUIRE(bytes != nullptr, PKV_ERR_INVALID_ARG, "bytes is NULL");
  int rc = beam_check(num_seqs, num_beams, vocab, num_out, dtype);
  if (rc != PKV_OK) return rc;
  int parts = 0;
  BeamLayout L;
  rc = beam_sizes(num_seqs, num_beams, vocab, num_out, &parts, &L);
  if (rc != PKV_OK) return rc;
  *bytes = L.total;
  return ok();
}

int pkv_beam_select(const void* logits, int64_t seq_stride, int64_t beam_stride,
                    const float* beam_scores, int32_t num_seqs, int32_t num_beams, int32_t vocab,
                    int32_t num_out, float* scores, int32_t* beams, int32_t* tokens,
                    void* workspace, size_t workspace_bytes, int32_t dtype, void* stream) {
  int rc = beam_check(num_seqs, num_beams, vocab, num_out, dtype);
  if (rc != PKV_OK) return rc;
  PKV_REQUIRE(seq_stride >= 0 && beam_stride >= 0, PKV_ERR_INVALID_ARG, "negative stride");
  if (num_seqs == 0) return ok();
  const int elt = element_bytes(dtype);
  PKV_REQUIRE(logits && beam_scores && scores && beams && tokens, PKV_ERR_INVALID_ARG,
              "NULL pointer");
  PKV_REQUIRE(aligned(logits, elt) && aligned(beam_scores, 4) && aligned(scores, 4) &&
                  aligned(beams, 4) && aligned(tokens, 4),
              PKV_ERR_INVALID_ARG, "a pointer is not aligned to its element");
  PKV_REQUIRE(workspace != nullptr && aligned(workspace, 256), PKV_ERR_INVALID_ARG,
              "workspace must be non-NULL and 256-byte aligned");
  PKV_REQUIRE(scores != beam_scores && beams != tokens, PKV_ERR_INVALID_ARG,
              "scores must not be beam_scores, nor beams tokens");
  int parts = 0;
  BeamLayout L;
  rc = beam_sizes(num_seqs, num_beams, vocab, num_out, &parts, &L);
  if (rc != PKV_OK) return rc;
  PKV_REQUIRE(workspace_bytes >= L.total, PKV_ERR_INVALID_ARG, "workspace of %zu bytes < %zu needed",
              workspace_bytes, L.total);
  char* ws = static_cast<char*>(workspace);
  BeamArgs a{};
  a.logits = logits;
  a.seq_stride = seq_stride;
  a.beam_stride = beam_stride;
  a.beam_scores = beam_scores;
  a.scores = scores;
  a.beams = beams;
  a.tokens = tokens;
  a.row_ticket = reinterpret_cast<int32_t*>(ws + L.row_ticket);
  a.seq_ticket = reinterpret_cast<int32_t*>(ws + L.seq_ticket);
  a.part_max = reinterpret_cast<float*>(ws + L.part_max);
  a.part_sum = reinterpret_cast<uint64_t*>(ws + L.part_sum);
  a.part_top = reinterpret_cast<uint64_t*>(ws + L.part_top);
  a.row_top = reinterpret_cast<uint64_t*>(ws + L.row_top);
  a.K = num_beams;
  a.V = vocab;
  a.N = num_out;
  a.parts = parts;
  a.by_row = parts > 1 && static_cast<int64_t>(num_beams) * parts * num_out > kOneMerge;
  const int64_t tiles = (static_cast<int64_t>(vocab) + kTile - 1) / kTile;
  a.tiles = static_cast<int32_t>((tiles + parts - 1) / parts);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  rc = dtype == PKV_F32   ? launch_beam<float>(a, num_seqs, st)
       : dtype == PKV_F16 ? launch_beam<__half>(a, num_seqs, st)
                          : launch_beam<__nv_bfloat16>(a, num_seqs, st);
  return rc == PKV_OK ? ok() : rc;
}

}  // extern "C"
