// Beam search's selection over beams and vocabulary.
//
// For every request s, from the logits of its K live beams and their scores so far:
//   candidate (b, v): score = beam_scores[s, b] + logits[s, b, v] - lse[s, b],
//   lse[s, b] = log sum_v exp(logits[s, b, v]),
// the N best candidates in order: by score, equal scores by beam, and within a beam by
// logit and then by token, lower first.
//
// One pass over the logits, one launch.  A CTA holds a chunk of one row in registers and
// reduces it to its maximum, its sum of exponentials and its best N logits (a row's
// candidates are ordered by their logits alone, so its lse is not needed for that); the
// CTA that finishes a row last merges the row's chunks, and the one that finishes a
// request's rows last merges its beams.  Nobody waits: tickets say who is last.
//
// Best N of a set spread over a block's threads: with t the N-th best of the best entries
// of small groups of threads, at least N entries are as good as t, and those that are lie
// in N groups: few, so they are collected in shared memory and each counts the entries
// better than itself.  Entries are compared as integer keys and no two are equal (equal
// values are told apart by their position), so the order of collection does not matter.
//
// Precision: candidates of different beams may lie next to each other, so lse and the
// scores are 64-bit: an fp32 exponential per logit, 32 of a thread's terms summed in fp32,
// everything across threads in fp64.  Only the score handed out is rounded to fp32.
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
constexpr int kMaxEntries = 8192;  // entries a merge takes: chunks * N, beams * N
constexpr int kLargeChunk = 32;    // elements a thread holds
constexpr int kSmallChunk = 8;

struct BeamArgs {
  const void* logits;
  int64_t seq_stride, beam_stride;  // elements
  const float* beam_scores;
  float* scores;
  int32_t* beams;
  int32_t* tokens;
  // workspace: the tickets, zero between launches, then per (row, chunk) and per row
  int32_t* row_ticket;
  int32_t* seq_ticket;
  float* chunk_max;
  double* chunk_sum;
  uint64_t* chunk_top;  // keys of a chunk's best N
  double* row_lse;
  uint64_t* row_top;    // keys of a row's best N
  int32_t K, V, N, chunks;
};

// Keys: larger is better, 0 is no entry, and no two entries of a set have the same one.
// A token of a row: its logit's bits in the order of the values (-0 as 0), then the token,
// lower first.
__device__ __forceinline__ uint64_t token_key(float x, int token) {
  uint32_t u = __float_as_uint(x + 0.f);
  u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return (static_cast<uint64_t>(u) << 32) | static_cast<uint32_t>(~token);
}
__device__ __forceinline__ int key_token(uint64_t key) {
  return static_cast<int>(~static_cast<uint32_t>(key));
}
__device__ __forceinline__ float key_logit(uint64_t key) {
  const uint32_t u = static_cast<uint32_t>(key >> 32);
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}
// A candidate of a request: its 64-bit score's bits in the order of the values, then its
// place in the list of beams' lists.  (Compared as integers: fp64 comparisons run at a
// 64th of their rate.)
struct ScoreKey {
  uint64_t score;
  uint32_t at;  // ~place
  __device__ __forceinline__ bool operator>(const ScoreKey& o) const {
    return score > o.score || (score == o.score && at > o.at);
  }
  __device__ __forceinline__ bool none() const { return score == 0; }
};
__device__ __forceinline__ ScoreKey score_key(double x, int place) {
  uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  u = (u >> 63) ? ~u : (u | (uint64_t(1) << 63));
  return ScoreKey{u, ~static_cast<uint32_t>(place)};
}
__device__ __forceinline__ double key_score(const ScoreKey& k) {
  const uint64_t u = k.score;
  return __longlong_as_double(static_cast<long long>((u >> 63) ? (u & ~(uint64_t(1) << 63)) : ~u));
}
__device__ __forceinline__ bool none(uint64_t k) { return k == 0; }
__device__ __forceinline__ bool none(const ScoreKey& k) { return k.none(); }

__device__ __forceinline__ uint64_t shfl_xor(uint64_t k, int o) {
  return __shfl_xor_sync(0xffffffffu, static_cast<unsigned long long>(k), o);
}
__device__ __forceinline__ ScoreKey shfl_xor(const ScoreKey& k, int o) {
  return ScoreKey{shfl_xor(k.score, o), __shfl_xor_sync(0xffffffffu, k.at, o)};
}

// Threads whose best entries are merged before the threshold is sought: about four
// groups of them for each entry wanted, in 32 to 256 groups.
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
  if (static_cast<int>(threadIdx.x) < groups) {
    const Key k = sh.best[threadIdx.x];
    int rank = 0;
#pragma unroll 8
    for (int i = 0; i < groups; ++i) rank += sh.best[i] > k;
    if (rank == n - 1 && !none(k)) sh.threshold = k;
  }
  __syncthreads();
  return sh.threshold;
}

// The collected entries in their order: put(rank, key) for rank < n, empty keys behind them.
template <typename Key, typename Put>
__device__ __forceinline__ void ranked(const Key* list, int n, const TopShared<Key>& sh, Put put) {
  __syncthreads();
  const int count = sh.count;
  for (int i = threadIdx.x; i < count; i += kThreads) {
    const Key k = list[i];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < count; ++j) rank += list[j] > k;
    if (rank < n) put(rank, k);
  }
  for (int i = count + threadIdx.x; i < n; i += kThreads) put(i, Key{});
}

// The best n of the entries get(i), i < M, M <= kMaxEntries.
template <typename Key, typename Get, typename Put>
__device__ __forceinline__ void merge_top(int M, int n, Get get, Key* list, TopShared<Key>& sh,
                                          Put put) {
  Key best{}, t{};
  if (M > kThreads) {
    for (int i = threadIdx.x; i < M; i += kThreads) {
      const Key k = get(i);
      if (k > best) best = k;
    }
    t = threshold_of(best, n, sh);
  } else {  // few enough to be ranked as they are
    __syncthreads();
    if (threadIdx.x == 0) sh.count = 0;
    __syncthreads();
  }
  for (int i = threadIdx.x; i < M; i += kThreads) {
    const Key k = get(i);
    if (!none(k) && !(t > k)) list[atomicAdd(&sh.count, 1)] = k;
  }
  ranked(list, n, sh, put);
}

__device__ __forceinline__ double block_sum(double x, double* warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warp[threadIdx.x >> 5] = x;
  __syncthreads();
  double y = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) y += warp[i];
  return y;
}

__device__ __forceinline__ float block_max(float x, float* warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warp[threadIdx.x >> 5] = x;
  __syncthreads();
  float y = -INFINITY;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) y = fmaxf(y, warp[i]);
  return y;
}

template <typename T>
__device__ __forceinline__ float logit(T x) {
  float y;
  if constexpr (std::is_same<T, float>::value) y = x;
  else y = ptx::to_float(x);
  return fmaxf(y, -INFINITY);  // NaN: a banned token
}

// The 16 bytes at p, which lies `skew` bytes past a 16-byte boundary: the two aligned
// pieces around them, shifted together.
__device__ __forceinline__ uint4 load_piece(const void* p, uint32_t skew) {
  const uint4* a = reinterpret_cast<const uint4*>(static_cast<const char*>(p) - skew);
  const uint4 lo = __ldcs(a);
  if (skew == 0) return lo;
  const uint4 hi = __ldcs(a + 1);
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
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

// A CTA per (chunk, row); E elements a thread.
template <typename T, int E>
__global__ void __launch_bounds__(kThreads) beam_select_kernel(const BeamArgs a) {
  extern __shared__ __align__(16) unsigned char buf[];
  __shared__ union {
    TopShared<uint64_t> row;
    TopShared<ScoreKey> seq;
  } sh;
  __shared__ double warp_sum[kThreads / 32];
  __shared__ float warp_max[kThreads / 32];
  __shared__ int flag;
  constexpr int W = 16 / static_cast<int>(sizeof(T));
  constexpr int kVecs = E / W;
  constexpr int kChunk = E * kThreads;
  const int tid = threadIdx.x, chunk = blockIdx.x;
  const int row = blockIdx.y, N = a.N, V = a.V;
  const int s = row / a.K, b = row - s * a.K;
  uint64_t* const list = reinterpret_cast<uint64_t*>(buf);

  const float bs = a.beam_scores[row];
  const bool alive = isfinite(bs);  // a dead beam's logits are not read
  const int64_t slot = static_cast<int64_t>(row) * a.chunks + chunk;
  if (alive) {
    const T* const x = static_cast<const T*>(a.logits) + s * a.seq_stride + b * a.beam_stride;
    // Which tokens a thread sums does not depend on where the row starts, so equal rows
    // have equal lse, bit for bit.
    const uint32_t skew = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(x) & 15);
    const int base = chunk * kChunk;
    float v[E];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int p = base + (j * kThreads + tid) * W;
      if (skew == 0 ? p + W <= V : p >= W && p + 2 * W <= V) {
        const uint4 u = load_piece(x + p, skew);
        const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
        for (int w = 0; w < W; ++w) v[j * W + w] = logit(e[w]);
      } else {
#pragma unroll
        for (int w = 0; w < W; ++w) v[j * W + w] = p + w < V ? logit(x[p + w]) : -INFINITY;
      }
    }
    // element j * W + w of the thread is token base + (j * kThreads + tid) * W + w: ascending,
    // so the first of the largest is the best
    auto token = [&](int i) { return base + ((i / W) * kThreads + tid) * W + i % W; };
    float best = v[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < E; ++i) {
      if (v[i] > best) {
        best = v[i];
        at = i;
      }
    }
    const float top = block_max(best, warp_max);
    float part = 0.f;
    if (isfinite(top)) {
      // e^d as 2^(d log2 e): the product is off by 2^-24 |d| log2 e, a term by 2^-20 of
      // itself where it counts (d > -17)
#pragma unroll
      for (int i = 0; i < E; ++i) part += ptx::ex2((v[i] - top) * 1.4426950408889634f);
    }
    const double sum = block_sum(static_cast<double>(part), warp_sum);
    const uint64_t mine = token(0) < V ? token_key(best, token(at)) : 0;
    const uint64_t t = threshold_of(mine, N, sh.row);
    if (mine != 0 && !(t > mine)) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const uint64_t k = token_key(v[i], token(i));
        if (token(i) < V && !(t > k)) list[atomicAdd(&sh.row.count, 1)] = k;
      }
    }
    uint64_t* const out = a.chunk_top + slot * N;
    ranked(list, N, sh.row, [&](int rank, uint64_t k) { out[rank] = k; });
    if (tid == 0) {
      a.chunk_max[slot] = top;
      a.chunk_sum[slot] = sum;
    }
  }
  if (!last_to_come(a.row_ticket + row, a.chunks, &flag)) return;

  // The row: its lse and its best N, from its chunks'.
  if (alive) {
    const int64_t first = static_cast<int64_t>(row) * a.chunks;
    float m = -INFINITY;
    for (int c = tid; c < a.chunks; c += kThreads) m = fmaxf(m, __ldcg(a.chunk_max + first + c));
    m = block_max(m, warp_max);
    double sum = 0.0;
    if (isfinite(m))
      for (int c = tid; c < a.chunks; c += kThreads)
        sum += __ldcg(a.chunk_sum + first + c) *
               exp(static_cast<double>(__ldcg(a.chunk_max + first + c)) - m);
    sum = block_sum(sum, warp_sum);
    if (tid == 0) a.row_lse[row] = isfinite(m) ? m + log(sum) : INFINITY;
    const uint64_t* const in = a.chunk_top + first * N;
    uint64_t* const out = a.row_top + static_cast<int64_t>(row) * N;
    merge_top<uint64_t>(
        a.chunks * N, N,
        [&](int i) {
          return static_cast<uint64_t>(__ldcg(reinterpret_cast<const unsigned long long*>(in + i)));
        },
        list, sh.row, [&](int rank, uint64_t k) { out[rank] = k; });
  } else if (tid == 0) {
    a.row_lse[row] = INFINITY;
  }
  if (!last_to_come(a.seq_ticket + s, a.K, &flag)) return;

  // The request: candidate j of beam b has place b * N + j, so equal scores go by beam and
  // then by the beam's own order.  A beam without a finite score or lse has candidates of
  // score -infinity, its first tokens in order.
  const int64_t r0 = static_cast<int64_t>(s) * a.K;
  auto row_key = [&](int i) {
    return static_cast<uint64_t>(
        __ldcg(reinterpret_cast<const unsigned long long*>(a.row_top + r0 * N + i)));
  };
  merge_top<ScoreKey>(
      a.K * N, N,
      [&](int i) {
        const int bb = i / N;
        const double lse = __ldcg(a.row_lse + r0 + bb);
        if (lse == INFINITY) return i - bb * N < V ? score_key(-INFINITY, i) : ScoreKey{};
        const uint64_t k = row_key(i);
        if (k == 0) return ScoreKey{};
        const double x = key_logit(k);
        return score_key(static_cast<double>(__ldg(a.beam_scores + r0 + bb)) + (x - lse), i);
      },
      reinterpret_cast<ScoreKey*>(buf), sh.seq,
      [&](int rank, const ScoreKey& k) {
        const int i = static_cast<int>(~k.at), bb = i / N;
        const int64_t at = static_cast<int64_t>(s) * N + rank;
        a.scores[at] = static_cast<float>(key_score(k));
        a.beams[at] = bb;
        a.tokens[at] = __ldcg(a.row_lse + r0 + bb) == INFINITY ? i - bb * N : key_token(row_key(i));
      });
}

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct BeamLayout {
  size_t row_ticket, seq_ticket, chunk_max, chunk_sum, chunk_top, row_lse, row_top, total;
};

// Chunks of E * kThreads elements that cover a row.
int chunks_of(int32_t V, int E) {
  const int64_t n = static_cast<int64_t>(E) * kThreads;
  return static_cast<int>((V + n - 1) / n);
}

// Elements a thread holds: 8,192-element chunks, or for batches that would leave SMs
// without work 2,048-element ones.
int elements_per_thread(int64_t rows, int32_t V, int32_t N, int sms) {
  const int small = chunks_of(V, kSmallChunk);
  if (rows * chunks_of(V, kLargeChunk) < 2 * sms &&
      static_cast<int64_t>(small) * N <= kMaxEntries)
    return kSmallChunk;
  return kLargeChunk;
}

// The tickets lie where they are whatever the sizes, so one workspace serves every call.
BeamLayout beam_layout(int32_t S, int32_t K, int32_t N, int chunks) {
  BeamLayout L;
  const size_t rows = static_cast<size_t>(S) * K, slots = rows * chunks;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += round256(bytes);
    return at;
  };
  L.row_ticket = take(PKV_BEAM_TICKET_BYTES / 2);
  L.seq_ticket = take(PKV_BEAM_TICKET_BYTES / 2);
  L.chunk_max = take(slots * 4);
  L.chunk_sum = take(slots * 8);
  L.chunk_top = take(slots * N * 8);
  L.row_lse = take(rows * 8);
  L.row_top = take(rows * N * 8);
  L.total = off;
  return L;
}
static_assert(PKV_BEAM_TICKET_BYTES / 2 >= (kMaxRows + 1) * 4, "a ticket for every row");

int beam_sizes(int32_t S, int32_t K, int32_t V, int32_t N, int32_t dtype, int* elements,
               BeamLayout* L) {
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
  PKV_REQUIRE(V <= INT_MAX - 65536 &&
                  static_cast<int64_t>(chunks_of(V, kLargeChunk)) * N <= kMaxEntries,
              PKV_ERR_UNSUPPORTED, "vocab %d with num_out %d: more than %d candidates of a row", V,
              N, kMaxEntries);
  int sms = 0, dev = 0;
  const int rc = device_sm_count(&sms, &dev);
  if (rc != PKV_OK) return rc;
  *elements = elements_per_thread(static_cast<int64_t>(S) * K, V, N, sms);
  *L = beam_layout(S, K, N, chunks_of(V, *elements));
  return PKV_OK;
}

template <typename T, int E>
int launch_beam(const BeamArgs& a, int32_t S, cudaStream_t st) {
  // a list holds the entries of the N groups that reach a threshold, or all of a small set
  auto listed = [&](int per_thread) {
    const size_t n = static_cast<size_t>(a.N) * group_of(a.N) * per_thread;
    return n < kThreads ? static_cast<size_t>(kThreads) : n;
  };
  auto per_thread = [](int m) { return (m + kThreads - 1) / kThreads; };
  size_t smem = listed(E) * sizeof(uint64_t);
  const size_t rows = listed(per_thread(a.chunks * a.N)) * sizeof(uint64_t);
  const size_t seqs = listed(per_thread(a.K * a.N)) * sizeof(ScoreKey);
  smem = smem < rows ? rows : smem;
  smem = smem < seqs ? seqs : smem;
  PKV_CUDA(cudaFuncSetAttribute(beam_select_kernel<T, E>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(smem)));
  beam_select_kernel<T, E><<<dim3(a.chunks, S * a.K), kThreads, smem, st>>>(a);
  PKV_CUDA(cudaGetLastError());
  return PKV_OK;
}

template <typename T>
int launch_beam_as(const BeamArgs& a, int32_t S, int elements, cudaStream_t st) {
  return elements == kLargeChunk ? launch_beam<T, kLargeChunk>(a, S, st)
                                 : launch_beam<T, kSmallChunk>(a, S, st);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_beam_workspace_size(int32_t num_seqs, int32_t num_beams, int32_t vocab, int32_t num_out,
                            int32_t dtype, size_t* bytes) {
  PKV_REQUIRE(bytes != nullptr, PKV_ERR_INVALID_ARG, "bytes is NULL");
  int elements = 0;
  BeamLayout L;
  const int rc = beam_sizes(num_seqs, num_beams, vocab, num_out, dtype, &elements, &L);
  if (rc != PKV_OK) return rc;
  *bytes = L.total;
  return ok();
}

int pkv_beam_select(const void* logits, int64_t seq_stride, int64_t beam_stride,
                    const float* beam_scores, int32_t num_seqs, int32_t num_beams, int32_t vocab,
                    int32_t num_out, float* scores, int32_t* beams, int32_t* tokens,
                    void* workspace, size_t workspace_bytes, int32_t dtype, void* stream) {
  int elements = 0;
  BeamLayout L;
  int rc = beam_sizes(num_seqs, num_beams, vocab, num_out, dtype, &elements, &L);
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
  a.chunk_max = reinterpret_cast<float*>(ws + L.chunk_max);
  a.chunk_sum = reinterpret_cast<double*>(ws + L.chunk_sum);
  a.chunk_top = reinterpret_cast<uint64_t*>(ws + L.chunk_top);
  a.row_lse = reinterpret_cast<double*>(ws + L.row_lse);
  a.row_top = reinterpret_cast<uint64_t*>(ws + L.row_top);
  a.K = num_beams;
  a.V = vocab;
  a.N = num_out;
  a.chunks = chunks_of(vocab, elements);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  rc = dtype == PKV_F32   ? launch_beam_as<float>(a, num_seqs, elements, st)
       : dtype == PKV_F16 ? launch_beam_as<__half>(a, num_seqs, elements, st)
                          : launch_beam_as<__nv_bfloat16>(a, num_seqs, elements, st);
  return rc == PKV_OK ? ok() : rc;
}

}  // extern "C"
