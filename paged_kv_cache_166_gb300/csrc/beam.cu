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
// Best N of a set spread over a block's threads: with t the N-th best of the threads' own
// best entries, at least N entries are as good as t, and those that are lie in N threads:
// few, so they are collected in shared memory and each counts the entries better than
// itself.  The order has no ties (equal values are told apart by their position), so the
// result does not depend on the order of collection.
//
// Precision: candidates of different beams may lie next to each other, so lse and the
// scores are 64-bit: expf per logit, 32 of a thread's terms summed in fp32, everything
// across threads in fp64.  Only the score handed out is rounded to fp32.
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
  // workspace: per (row, chunk), then per row, then the tickets
  float* chunk_max;
  double* chunk_sum;
  float* chunk_val;
  int32_t* chunk_tok;
  double* row_lse;
  float* row_val;
  int32_t* row_tok;
  int32_t* row_ticket;
  int32_t* seq_ticket;
  int32_t K, V, N, chunks;
};

// a before b: larger value, equal values by position.  Position INT_MAX: no entry.
template <typename V>
__device__ __forceinline__ bool better(V av, int ai, V bv, int bi) {
  return av > bv || (av == bv && ai < bi);
}

struct TopShared {
  int count;
  int thr_id;
  double thr_val;
  int best_id[kThreads];
  alignas(8) unsigned char best_val[kThreads * sizeof(double)];
};

// Threshold: the n-th best of the threads' best entries (v, id), or "everything" if
// fewer threads have one.
template <typename V>
__device__ __forceinline__ void threshold(V v, int id, int n, TopShared& sh, V* tv, int* ti) {
  V* const bv = reinterpret_cast<V*>(sh.best_val);
  __syncthreads();
  bv[threadIdx.x] = v;
  sh.best_id[threadIdx.x] = id;
  if (threadIdx.x == 0) {
    sh.count = 0;
    sh.thr_val = -INFINITY;
    sh.thr_id = INT_MAX;
  }
  __syncthreads();
  int rank = 0;
#pragma unroll 8
  for (int i = 0; i < kThreads; ++i) rank += better(bv[i], sh.best_id[i], v, id);
  if (rank == n - 1 && id != INT_MAX) {
    sh.thr_val = static_cast<double>(v);
    sh.thr_id = id;
  }
  __syncthreads();
  *tv = static_cast<V>(sh.thr_val);
  *ti = sh.thr_id;
}

// The collected entries in their order: put(rank, value, position) for rank < n.
template <typename V, typename Put>
__device__ __forceinline__ void ranked(const V* cv, const int* ci, int n, const TopShared& sh,
                                       Put put) {
  __syncthreads();
  const int count = sh.count;
  for (int i = threadIdx.x; i < count; i += kThreads) {
    const V v = cv[i];
    const int id = ci[i];
    int rank = 0;
    for (int j = 0; j < count; ++j) rank += better(cv[j], ci[j], v, id);
    if (rank < n) put(rank, v, id);
  }
  for (int i = count + threadIdx.x; i < n; i += kThreads)
    put(i, static_cast<V>(-INFINITY), INT_MAX);
}

// The best n of entries get(i), i < M (value and position), M <= kMaxEntries; buf holds
// n * ceil(M / kThreads) entries.
template <typename V, typename Get, typename Put>
__device__ __forceinline__ void merge_top(int M, int n, Get get, unsigned char* buf, int cap,
                                          TopShared& sh, Put put) {
  V best = static_cast<V>(-INFINITY), v;
  int best_id = INT_MAX, id;
  for (int i = threadIdx.x; i < M; i += kThreads) {
    get(i, &v, &id);
    if (id != INT_MAX && better(v, id, best, best_id)) {
      best = v;
      best_id = id;
    }
  }
  V tv;
  int ti;
  threshold(best, best_id, n, sh, &tv, &ti);
  V* const cv = reinterpret_cast<V*>(buf);
  int* const ci = reinterpret_cast<int*>(cv + cap);
  for (int i = threadIdx.x; i < M; i += kThreads) {
    get(i, &v, &id);
    if (id != INT_MAX && !better(tv, ti, v, id)) {
      const int at = atomicAdd(&sh.count, 1);
      cv[at] = v;
      ci[at] = id;
    }
  }
  ranked(cv, ci, n, sh, put);
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

__device__ __forceinline__ float block_max(float x, double* warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warp[threadIdx.x >> 5] = static_cast<double>(x);
  __syncthreads();
  float y = -INFINITY;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) y = fmaxf(y, static_cast<float>(warp[i]));
  return y;
}

template <typename T>
__device__ __forceinline__ float logit(T x) {
  float y;
  if constexpr (std::is_same<T, float>::value) y = x;
  else y = ptx::to_float(x);
  return y != y ? -INFINITY : y;  // NaN: a banned token
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
  __shared__ TopShared sh;
  __shared__ double warp[kThreads / 32];
  __shared__ int flag;
  constexpr int W = 16 / static_cast<int>(sizeof(T));
  constexpr int kVecs = E / W;
  constexpr int kChunk = E * kThreads;
  const int tid = threadIdx.x, chunk = blockIdx.x;
  const int row = blockIdx.y, N = a.N, V = a.V;
  const int s = row / a.K, b = row - s * a.K;

  const float bs = a.beam_scores[row];
  const bool alive = isfinite(bs);  // a dead beam's logits are not read
  float top = -INFINITY;
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
    // element j * W + w of the thread: its token, INT_MAX past the row
    auto token = [&](int i) {
      const int p = base + ((i / W) * kThreads + tid) * W + i % W;
      return p < V ? p : INT_MAX;
    };
    float best = -INFINITY;
    int best_id = INT_MAX;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if (better(v[i], token(i), best, best_id)) {
        best = v[i];
        best_id = token(i);
      }
    }
    top = block_max(best, warp);
    float part = 0.f;
    if (isfinite(top)) {
#pragma unroll
      for (int i = 0; i < E; ++i) part += expf(v[i] - top);
    }
    const double sum = block_sum(static_cast<double>(part), warp);
    float tv;
    int ti;
    threshold(best, best_id, N, sh, &tv, &ti);
    float* const cv = reinterpret_cast<float*>(buf);
    int* const ci = reinterpret_cast<int*>(cv + N * E);
    if (!better(tv, ti, best, best_id)) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int id = token(i);
        if (id != INT_MAX && !better(tv, ti, v[i], id)) {
          const int at = atomicAdd(&sh.count, 1);
          cv[at] = v[i];
          ci[at] = id;
        }
      }
    }
    float* const ov = a.chunk_val + slot * N;
    int32_t* const ot = a.chunk_tok + slot * N;
    ranked(cv, ci, N, sh, [&](int rank, float val, int id) {
      ov[rank] = val;
      ot[rank] = id;
    });
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
    m = block_max(m, warp);
    double sum = 0.0;
    if (isfinite(m))
      for (int c = tid; c < a.chunks; c += kThreads)
        sum += __ldcg(a.chunk_sum + first + c) *
               exp(static_cast<double>(__ldcg(a.chunk_max + first + c)) - m);
    sum = block_sum(sum, warp);
    if (tid == 0) a.row_lse[row] = isfinite(m) ? m + log(sum) : INFINITY;
    const int M = a.chunks * N;
    float* const ov = a.row_val + static_cast<int64_t>(row) * N;
    int32_t* const ot = a.row_tok + static_cast<int64_t>(row) * N;
    merge_top<float>(
        M, N,
        [&](int i, float* v, int* id) {
          *v = __ldcg(a.chunk_val + first * N + i);
          *id = __ldcg(a.chunk_tok + first * N + i);
        },
        buf, N * ((M + kThreads - 1) / kThreads), sh,
        [&](int rank, float val, int id) {
          ov[rank] = val;
          ot[rank] = id;
        });
  } else if (tid == 0) {
    a.row_lse[row] = INFINITY;
  }
  if (!last_to_come(a.seq_ticket + s, a.K, &flag)) return;

  // The request: candidate j of beam b is entry b * N + j, so equal scores go by beam and
  // then by the beam's own order.  A beam without a finite score or lse has candidates of
  // score -infinity, its first tokens in order.
  const int M = a.K * N;
  const int64_t r0 = static_cast<int64_t>(s) * a.K;
  merge_top<double>(
      M, N,
      [&](int i, double* v, int* id) {
        const int bb = i / N, j = i - bb * N;
        const double lse = __ldcg(a.row_lse + r0 + bb);
        *id = i;
        if (lse == INFINITY) {
          *v = -INFINITY;
          if (j >= V) *id = INT_MAX;
          return;
        }
        if (__ldcg(a.row_tok + r0 * N + i) == INT_MAX) {
          *v = -INFINITY;
          *id = INT_MAX;
          return;
        }
        *v = static_cast<double>(__ldg(a.beam_scores + r0 + bb)) +
             (static_cast<double>(__ldcg(a.row_val + r0 * N + i)) - lse);
      },
      buf, N * ((M + kThreads - 1) / kThreads), sh,
      [&](int rank, double val, int i) {
        const int bb = i / N, j = i - bb * N;
        const int64_t at = static_cast<int64_t>(s) * N + rank;
        a.scores[at] = static_cast<float>(val);
        a.beams[at] = bb;
        a.tokens[at] =
            __ldcg(a.row_lse + r0 + bb) == INFINITY ? j : __ldcg(a.row_tok + r0 * N + i);
      });
}

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct BeamLayout {
  size_t row_ticket, seq_ticket, tickets_end, chunk_max, chunk_sum, chunk_val, chunk_tok, row_lse,
      row_val, row_tok, total;
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

BeamLayout beam_layout(int32_t S, int32_t K, int32_t N, int chunks) {
  BeamLayout L;
  const size_t rows = static_cast<size_t>(S) * K, slots = rows * chunks;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += round256(bytes);
    return at;
  };
  L.row_ticket = take(rows * 4);
  L.seq_ticket = take(static_cast<size_t>(S) * 4);
  L.tickets_end = off;
  L.chunk_max = take(slots * 4);
  L.chunk_sum = take(slots * 8);
  L.chunk_val = take(slots * N * 4);
  L.chunk_tok = take(slots * N * 4);
  L.row_lse = take(rows * 8);
  L.row_val = take(rows * N * 4);
  L.row_tok = take(rows * N * 4);
  L.total = off;
  return L;
}

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
  PKV_REQUIRE(static_cast<int64_t>(S) * K <= 65535, PKV_ERR_UNSUPPORTED,
              "num_seqs * num_beams above 65535");
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
  const int N = a.N;
  auto entries = [&](int m) { return static_cast<size_t>(N) * ((m + kThreads - 1) / kThreads); };
  size_t smem = static_cast<size_t>(N) * E * 8;  // a chunk's: value and token
  const size_t rows = entries(a.chunks * N) * 8, seqs = entries(a.K * N) * 12;
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
  a.chunk_val = reinterpret_cast<float*>(ws + L.chunk_val);
  a.chunk_tok = reinterpret_cast<int32_t*>(ws + L.chunk_tok);
  a.row_lse = reinterpret_cast<double*>(ws + L.row_lse);
  a.row_val = reinterpret_cast<float*>(ws + L.row_val);
  a.row_tok = reinterpret_cast<int32_t*>(ws + L.row_tok);
  a.K = num_beams;
  a.V = vocab;
  a.N = num_out;
  a.chunks = chunks_of(vocab, elements);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // the tickets start each call at zero, so no layout of an earlier call matters
  PKV_CUDA(cudaMemsetAsync(ws, 0, L.tickets_end, st));
  rc = dtype == PKV_F32   ? launch_beam_as<float>(a, num_seqs, elements, st)
       : dtype == PKV_F16 ? launch_beam_as<__half>(a, num_seqs, elements, st)
                          : launch_beam_as<__nv_bfloat16>(a, num_seqs, elements, st);
  return rc == PKV_OK ? ok() : rc;
}

}  // extern "C"
