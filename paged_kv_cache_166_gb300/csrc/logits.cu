// Penalties for repeated tokens, biases and masks of allowed tokens on logits.
//
// Row r of request s, token v, with n the times that v came in what the request has written so
// far and in the row's path, and `seen` true if v came there or in the prompt:
//   x = logits[r, v];
//   seen:  x = x > 0 ? x / repetition_s : x * repetition_s;
//   n > 0:  x = (x - frequency_s * n) - presence_s;   x = x + bias_s(v);
//   not allowed:  x = -infinity;
// in fp32, each operation rounded, then rounded to the type.
//
// What the mask bans, or everything if out is not logits, goes through a first kernel: a warp
// takes 1,024 tokens of a row, writes 16 bytes of banned ones without reading them and, in
// place, leaves allowed ones alone.  The second kernel, whose counting overlaps the first, puts
// the adjusted logits over that: a CTA takes every NP-th segment of 256 tokens of the
// vocabulary for one request (the low numbers, which most texts use most, are spread over all
// CTAs).  The CTAs of a cluster share the request's tokens out and count each in the shared
// memory of the CTA that has it (integers, so their order does not matter); then each goes
// through the rows with those that came.  Without a mask a row thus costs, in place, as much as
// the request has tokens, not the vocabulary.
//
// Bound by memory latency for small calls (lengths, history, logits one after the other), else
// by the bytes of the mask and of the logits that change (32 for each adjusted one alone).
// Measured: 32 requests of 8 rows of 131,072 bf16 logits and histories up to 8,192, under a mask 42
// us (the mask 18), without one 27; 4 rows of 32,000 fp32 5.1.  One kernel over the whole
// vocabulary took 50 and 7.8.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kAdjThreads = 256;
constexpr int kAdjSegment = 256;              // tokens next to each other that one CTA has
constexpr int kAdjSegments = 32;              // at most so many segments of a CTA
constexpr int kAdjCluster = 8;                // at most so many CTAs count together
constexpr int kAdjSpan = 1024;                // tokens of a row that a warp looks at together
constexpr int kAdjSpans = 4;                  // such spans of a warp, their masks loaded at once
constexpr uint32_t kAdjPrompt = 0x80000000u;  // beside a token's count: it is in the prompt

struct AdjustArgs {
  const void* logits;
  void* out;
  int64_t in_stride, out_stride;  // elements from row to row
  const int32_t* history;         // [S, L]
  const int32_t* history_lens;    // [S]
  const int32_t* prompt_lens;     // [S] or NULL: 0
  const int32_t* row_start;       // [S + 1], or NULL: row s is request s's
  const float* repetition;        // [S] each, or NULL: 1, 0, 0
  const float* frequency;
  const float* presence;
  const int32_t* path;            // [T, P] or NULL
  const int32_t* bias_tokens;     // [S, NBias] or NULL
  const float* bias_values;
  const uint32_t* allowed;        // [T, W] or NULL
  int32_t S, T, V, L, P, NBias, W;
  int32_t segments;               // of a CTA
  int32_t log_ctas;               // log2 of the CTAs that share a request's vocabulary (NP)
};

template <typename T>
__device__ __forceinline__ float logit_of(T x) {
  if constexpr (std::is_same<T, float>::value) return x;
  else return ptx::to_float(x);
}

template <typename T>
struct alignas(16) AdjPiece {
  T x[16 / sizeof(T)];
};

// ---- what the mask bans, and what is copied ------------------------------------------------
// A warp a span of a row; the mask's words are loaded by a lane each and handed round.
template <typename T>
__global__ void __launch_bounds__(kAdjThreads, 4) adjust_mask_kernel(const AdjustArgs a) {
  // the second kernel may start to count; it waits for this grid before it touches a logit
  asm volatile("griddepcontrol.launch_dependents;");
  constexpr int VEC = 16 / sizeof(T);
  constexpr uint32_t all = (1u << VEC) - 1u;
  constexpr int kSteps = kAdjSpan / VEC / 32;  // pieces of a lane (one more if they are shifted)
  const int lane = threadIdx.x & 31;
  const int64_t r = blockIdx.y + static_cast<int64_t>(blockIdx.z) * 65535;
  if (r >= a.T) return;
  if (a.row_start != nullptr && (r < __ldg(a.row_start) || r >= __ldg(a.row_start + a.S))) return;
  const int64_t first =
      (static_cast<int64_t>(blockIdx.x) * (kAdjThreads / 32) + (threadIdx.x >> 5)) * kAdjSpans * kAdjSpan;
  const bool in_place = a.logits == a.out && a.in_stride == a.out_stride;
  uint32_t word4[kAdjSpans];
#pragma unroll
  for (int q = 0; q < kAdjSpans; ++q) {
    const int64_t w = first / 32 + q * 32 + lane;
    word4[q] = a.allowed == nullptr ? 0xffffffffu : (w < a.W ? __ldg(a.allowed + r * a.W + w) : 0u);
  }
  const T* const in_row = static_cast<const T*>(a.logits) + r * a.in_stride;
  T* const out_row = static_cast<T*>(a.out) + r * a.out_stride;
  const uintptr_t off = reinterpret_cast<uintptr_t>(out_row) & 15;  // (spans are whole 16 bytes)
  const int before = static_cast<int>(off) / static_cast<int>(sizeof(T));
  const bool wide = (reinterpret_cast<uintptr_t>(in_row) & 15) == off;
  AdjPiece<T> ban;
#pragma unroll
  for (int e = 0; e < VEC; ++e) ban.x[e] = ptx::from_float<T>(-INFINITY);
  constexpr int U = 4;
  static_assert(kSteps % U == 0, "spans");
#pragma unroll 1
  for (int q = 0; q < kAdjSpans; ++q) {
    const int64_t c0 = first + q * kAdjSpan;
    if (c0 >= a.V) break;
    const int most = static_cast<int>(min(static_cast<int64_t>(kAdjSpan), a.V - c0));  // tokens of the span
    const T* const in = in_row + c0;
    T* const out = out_row + c0;
    const uint32_t word = q == 0 ? word4[0] : (q == 1 ? word4[1] : (q == 2 ? word4[2] : word4[3]));
#pragma unroll 1
    for (int x0 = 0; x0 < kSteps + (before != 0 ? 1 : 0); x0 += U) {
      uint32_t good[U];
      bool whole[U], read[U];
      AdjPiece<T> p[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = ((x0 + u) * 32 + lane) * VEC - before;  // the piece's first token
        const uint32_t lo = __shfl_sync(0xffffffffu, word, (t >> 5) & 31);
        const uint32_t hi = __shfl_sync(0xffffffffu, word, ((t >> 5) + 1) & 31);
        good[u] = __funnelshift_r(lo, hi, t & 31) & all;
        whole[u] = wide && t >= 0 && t + VEC <= most;
        read[u] = whole[u] && good[u] != 0 && !(in_place && good[u] == all);
        if (read[u]) p[u] = *reinterpret_cast<const AdjPiece<T>*>(in + t);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = ((x0 + u) * 32 + lane) * VEC - before;
        if (whole[u]) {
          if (good[u] != 0 && !read[u]) continue;
          AdjPiece<T> y = ban;
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if ((good[u] >> e) & 1u) y.x[e] = p[u].x[e];
          *reinterpret_cast<AdjPiece<T>*>(out + t) = y;
        } else {  // the ends of the span, or rows that do not share the boundaries
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            if (t + e < 0 || t + e >= most) continue;
            // (t < 0: the bits below the span's first come out of the last word; token t + e >= 0
            // is bit e + t of the first)
            const bool ok = (good[u] >> e) & 1u;
            if (!ok) out[t + e] = ban.x[0];
            else if (!in_place) out[t + e] = in[t + e];
          }
        }
      }
    }
  }
}

// ---- the tokens that came, or have a bias ----------------------------------------------------
// Shared memory words: counts [chunk], bias entries [chunk] (with biases), marks of the tokens in
// any row's path [chunk / 32], the list of tokens that something touches, 16 bits each [chunk];
// chunk = 256 * segments.
__host__ __device__ constexpr int adjust_words(int segments, bool biases) {
  const int chunk = segments * kAdjSegment;
  return chunk * (biases ? 2 : 1) + chunk / 32 + chunk / 2;
}

// Grid: CTAs of a request's vocabulary (a power of two), requests, shares of a request's rows.
template <typename T>
__global__ void __launch_bounds__(kAdjThreads, 5) adjust_tokens_kernel(const AdjustArgs a) {
  extern __shared__ __align__(16) uint32_t adj_smem[];  // (read four words at a time)
  __shared__ int listed;
  const int tid = threadIdx.x, s = blockIdx.y, first = blockIdx.x;
  const int CH = a.segments * kAdjSegment;
  uint32_t* const count = adj_smem;
  uint32_t* const entry = count + CH;  // 1 + the bias entry of a token (0: none)
  uint32_t* const marks = entry + (a.bias_tokens != nullptr ? CH : 0);
  uint16_t* const list = reinterpret_cast<uint16_t*>(marks + CH / 32);
  const int words = static_cast<int>(marks - adj_smem) + CH / 32;
  const int r_first = a.row_start != nullptr ? max(0, __ldg(a.row_start + s)) : s;
  const int r_end = a.row_start != nullptr ? min(a.T, __ldg(a.row_start + s + 1)) : s + 1;
  const int held = min(max(__ldg(a.history_lens + s), 0), a.L);
  const int prompt = a.prompt_lens != nullptr ? __ldg(a.prompt_lens + s) : 0;
  if (r_first + static_cast<int64_t>(blockIdx.z) >= r_end) {
    // (what is queued behind this grid relies on the first kernel being done, too)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int shares = gridDim.z, row0 = r_first + blockIdx.z;
  const int rows = (r_end - row0 - 1) / shares + 1;  // row0, row0 + shares, ...
  auto row = [&](int k) { return row0 + static_cast<int64_t>(k) * shares; };
  // CTAs of the cluster: numbers c0 .. c0 + cluster - 1 of the request's
  const int cluster = min(kAdjCluster, static_cast<int>(gridDim.x)), c0 = first & ~(cluster - 1);
  const int rank = first - c0;
  // place of token v in its CTA's segments (-1: in none of this cluster's), and the token at a
  // place of this CTA's
  int owner = 0;  // that CTA's rank in the cluster
  auto place = [&](int v) {
    const int seg = v >> 8;
    owner = (seg & ((1 << a.log_ctas) - 1)) - c0;
    if (static_cast<uint32_t>(v) >= static_cast<uint32_t>(a.V) ||
        static_cast<uint32_t>(owner) >= static_cast<uint32_t>(cluster))
      return -1;
    return (seg >> a.log_ctas) << 8 | (v & 255);
  };
  auto token = [&](int i) { return (((i >> 8) << a.log_ctas) + first) << 8 | (i & 255); };
  static_assert(kAdjSegment == 256, "places");
  for (int i = tid; i < words; i += kAdjThreads) adj_smem[i] = 0u;
  if (tid == 0) listed = 0;
  cg::cluster_group together = cg::this_cluster();
  together.sync();  // every table of the cluster is cleared
  {
    const int32_t* const tokens = a.history + static_cast<int64_t>(s) * a.L;
    auto one = [&](int at, int tok) {
      const int i = place(tok);
      if (i < 0) return;
      uint32_t* const c = together.map_shared_rank(count + i, owner);
      if (at >= prompt) atomicAdd(c, 1u);
      else atomicOr(c, kAdjPrompt);
    };
    // four tokens at once from the first 16-byte boundary on, four such loads on their way
    const int head =
        min(held, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(tokens) & 15)) & 15) / 4);
    const int quads = (held - head) / 4;
    const int4* const body = reinterpret_cast<const int4*>(tokens + head);
    const int threads = cluster * kAdjThreads, me = rank * kAdjThreads + tid;
    for (int i0 = me; i0 < quads; i0 += 4 * threads) {
      int4 q[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i0 + u * threads < quads) q[u] = __ldg(body + i0 + u * threads);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int at = head + 4 * (i0 + u * threads);
        if (i0 + u * threads >= quads) continue;
        one(at, q[u].x);
        one(at + 1, q[u].y);
        one(at + 2, q[u].z);
        one(at + 3, q[u].w);
      }
    }
    if (me < head) one(me, __ldg(tokens + me));
    const int rest = head + 4 * quads + me;
    if (rest < held) one(rest, __ldg(tokens + rest));
    if (a.bias_tokens != nullptr) {  // of entries for one token the last counts
      const int32_t* const ids = a.bias_tokens + static_cast<int64_t>(s) * a.NBias;
      for (int e = me; e < a.NBias; e += threads) {
        const int i = place(__ldg(ids + e));
        if (i >= 0) atomicMax(together.map_shared_rank(entry + i, owner), static_cast<uint32_t>(e) + 1u);
      }
    }
    if (a.path != nullptr) {
      for (int k = me / 32; k < rows; k += threads / 32) {  // a warp a row
        for (int p = me % 32; p < a.P; p += 32) {
          const int i = place(__ldg(a.path + row(k) * a.P + p));
          if (i >= 0)
            atomicOr(together.map_shared_rank(marks + (i >> 5), owner), 1u << (i & 31));
        }
      }
    }
  }
  const float rep = a.repetition != nullptr ? __ldg(a.repetition + s) : 1.f;
  const float freq = a.frequency != nullptr ? __ldg(a.frequency + s) : 0.f;
  const float pres = a.presence != nullptr ? __ldg(a.presence + s) : 0.f;
  const float* const values =
      a.bias_tokens != nullptr ? a.bias_values + static_cast<int64_t>(s) * a.NBias : nullptr;
  together.sync();  // everything is counted: no CTA looks into another one's tables from here on
  // the places that something touches, in any order (each is dealt with by itself): four
  // neighbours a thread
  for (int i0 = 0; i0 < CH; i0 += 4 * kAdjThreads) {
    const int i = i0 + 4 * tid;
    uint32_t on = 0;
    if (i < CH) {
      const uint4 c = *reinterpret_cast<const uint4*>(count + i);
      on = (c.x != 0 ? 1u : 0u) | (c.y != 0 ? 2u : 0u) | (c.z != 0 ? 4u : 0u) | (c.w != 0 ? 8u : 0u);
      on |= (marks[i >> 5] >> (i & 31)) & 15u;
      if (values != nullptr) {
        const uint4 e = *reinterpret_cast<const uint4*>(entry + i);
        on |= (e.x != 0 ? 1u : 0u) | (e.y != 0 ? 2u : 0u) | (e.z != 0 ? 4u : 0u) | (e.w != 0 ? 8u : 0u);
      }
    }
    const int own = __popc(on);
    int upto = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if ((tid & 31) >= o) upto += y;
    }
    int at = 0;
    if ((tid & 31) == 31 && upto != 0) at = atomicAdd(&listed, upto);
    at = __shfl_sync(0xffffffffu, at, 31) + upto - own;
    for (; on != 0; on &= on - 1) list[at++] = static_cast<uint16_t>(i + __ffs(on) - 1);
  }
  __syncthreads();
  // the first kernel's logits, and whatever was queued before
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = listed;
  int sh = 0;  // log2 of the threads that share a token's rows, if there are few tokens
  while (sh < 5 && (n << (sh + 1)) <= kAdjThreads) ++sh;
  const int step = 1 << sh;
  const T* const in = static_cast<const T*>(a.logits);
  T* const out = static_cast<T*>(a.out);
  for (int e = tid >> sh; e < n; e += kAdjThreads >> sh) {
    const int i = list[e], v = token(i);
    const uint32_t held_count = count[i];
    const uint32_t be = values != nullptr ? entry[i] : 0u;
    const float bias = be != 0 ? __ldg(values + be - 1) : 0.f;
    const bool in_path = (marks[i >> 5] >> (i & 31)) & 1u;
    for (int k = tid & (step - 1); k < rows; k += 4 * step) {
      T x[4];
      bool on[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        on[u] = k + u * step < rows;
        if (on[u] && a.allowed != nullptr)
          on[u] = (__ldg(a.allowed + row(k + u * step) * a.W + (v >> 5)) >> (v & 31)) & 1u;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (on[u]) x[u] = in[row(k + u * step) * a.in_stride + v];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (!on[u]) continue;
        const int64_t r = row(k + u * step);
        uint32_t c = held_count;
        if (in_path) {
          const int32_t* const path = a.path + r * a.P;
          for (int p = 0; p < a.P; ++p) c += __ldg(path + p) == v ? 1u : 0u;
        }
        if (c == 0 && be == 0) continue;  // of another row's path
        float y = logit_of(x[u]);
        if (c != 0) y = y > 0.f ? __fdiv_rn(y, rep) : __fmul_rn(y, rep);
        if ((c & ~kAdjPrompt) != 0)
          y = __fsub_rn(__fsub_rn(y, __fmul_rn(freq, static_cast<float>(c & ~kAdjPrompt))), pres);
        if (be != 0) y = __fadd_rn(y, bias);
        out[r * a.out_stride + v] = ptx::from_float<T>(y);
      }
    }
  }
}

template <typename T>
int launch_adjust(const AdjustArgs& a, int shares, cudaStream_t st) {
  static SmemOnce once;
  const int rc = allow_dynamic_smem(once, reinterpret_cast<const void*>(adjust_tokens_kernel<T>),
                                    adjust_words(kAdjSegments, true) * 4);
  if (rc != PKV_OK) return rc;
  const bool masks = a.allowed != nullptr || a.logits != a.out;
  if (masks) {
    const int spans = (a.V - 1) / (kAdjSpan * kAdjSpans) + 1, warps = kAdjThreads / 32;
    const int deep = (a.T - 1) / 65535 + 1;
    adjust_mask_kernel<T>
        <<<dim3((spans - 1) / warps + 1, deep > 1 ? 65535 : a.T, deep), kAdjThreads, 0, st>>>(a);
    PKV_CUDA(cudaGetLastError());
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(1u << a.log_ctas, a.S, shares);
  cfg.blockDim = dim3(kAdjThreads);
  cfg.dynamicSmemBytes = adjust_words(a.segments, a.bias_tokens != nullptr) * sizeof(uint32_t);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = std::min(kAdjCluster, 1 << a.log_ctas);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = masks ? 2 : 1;
  PKV_CUDA(cudaLaunchKernelEx(&cfg, adjust_tokens_kernel<T>, a));
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_adjust_logits(
    const void* logits, int64_t row_stride, void* out, int64_t out_stride, int32_t num_rows,
    int32_t vocab, const int32_t* row_start, int32_t num_requests, const int32_t* history,
    int32_t history_cols, const int32_t* history_lens, const int32_t* prompt_lens,
    const float* repetition, const float* frequency, const float* presence, const int32_t* path,
    int32_t path_cols, const int32_t* bias_tokens, const float* bias_values, int32_t bias_cols,
    const int32_t* allowed, int32_t allowed_words, int32_t dtype, void* stream) {
  PKV_REQUIRE(dtype == PKV_F32 || dtype == PKV_F16 || dtype == PKV_BF16, PKV_ERR_DTYPE,
              "dtype %d is not f32, f16 or bf16", dtype);
  PKV_REQUIRE(num_rows >= 0 && num_requests >= 0 && vocab > 0 && history_cols >= 0 &&
                  path_cols >= 0 && bias_cols >= 0 && allowed_words >= 0,
              PKV_ERR_INVALID_ARG, "sizes must not be negative (vocab positive)");
  PKV_REQUIRE(vocab <= (1 << 30) && num_requests <= 65535 && history_cols < (1 << 24) &&
                  path_cols < (1 << 24),
              PKV_ERR_UNSUPPORTED,
              "vocab above 2^30, over 65535 requests or 2^24 tokens of one request");
  PKV_REQUIRE(row_start != nullptr || num_rows == num_requests, PKV_ERR_INVALID_ARG,
              "without row_start every row is a request of its own (%d rows, %d requests)", num_rows,
              num_requests);
  PKV_REQUIRE(row_stride >= vocab && out_stride >= vocab, PKV_ERR_INVALID_ARG,
              "a row stride is smaller than the vocabulary");
  PKV_REQUIRE((bias_tokens != nullptr) == (bias_values != nullptr), PKV_ERR_INVALID_ARG,
              "bias_tokens and bias_values come together");
  PKV_REQUIRE(allowed == nullptr || static_cast<int64_t>(allowed_words) * 32 >= vocab,
              PKV_ERR_INVALID_ARG, "a row of allowed has %d words for a vocabulary of %d",
              allowed_words, vocab);
  if (num_rows == 0 || num_requests == 0) return ok();
  PKV_REQUIRE(logits && out && history_lens && (history || history_cols == 0),
              PKV_ERR_INVALID_ARG, "NULL pointer");
  PKV_REQUIRE(logits != out || row_stride == out_stride, PKV_ERR_INVALID_ARG,
              "out at logits with another row stride");
  const int elt = element_bytes(dtype);
  PKV_REQUIRE(aligned(logits, elt) && aligned(out, elt) && aligned(history, 4) &&
                  aligned(history_lens, 4) && aligned(prompt_lens, 4) && aligned(row_start, 4) &&
                  aligned(repetition, 4) && aligned(frequency, 4) && aligned(presence, 4) &&
                  aligned(path, 4) && aligned(bias_tokens, 4) && aligned(bias_values, 4) &&
                  aligned(allowed, 4),
              PKV_ERR_INVALID_ARG, "a pointer is not aligned to its element");
  int sms = 0, dev = 0;
  int rc = device_sm_count(&sms, &dev);
  if (rc != PKV_OK) return rc;
  AdjustArgs a{};
  a.logits = logits;
  a.out = out;
  a.in_stride = row_stride;
  a.out_stride = out_stride;
  a.history = history;
  a.history_lens = history_lens;
  a.prompt_lens = prompt_lens;
  a.row_start = row_start;
  a.repetition = repetition;
  a.frequency = frequency;
  a.presence = presence;
  a.path = path_cols > 0 ? path : nullptr;
  a.bias_tokens = bias_cols > 0 ? bias_tokens : nullptr;
  a.bias_values = bias_values;
  a.allowed = reinterpret_cast<const uint32_t*>(allowed);
  a.S = num_requests;
  a.T = num_rows;
  a.V = vocab;
  a.L = history_cols;
  a.P = path_cols;
  a.NBias = bias_cols;
  a.W = allowed_words;
  // A power of two of CTAs, as few as hold the vocabulary (256 rows of 65,537 under a mask: 104
  // us with at most 16 segments a CTA, 82 with 32); of those of over 16 more until the SMs have
  // eight (32 requests of 8 rows of 131,072: 42 us with 16 segments, 48 with 32), and of those of
  // over 4 until they have three.
  const int total = (vocab + kAdjSegment - 1) / kAdjSegment;
  auto more = [&](int segments, int each) {
    return (int64_t(segments) << a.log_ctas) < total &&
           (int64_t(num_requests) << a.log_ctas) < int64_t(each) * sms;
  };
  while ((int64_t(kAdjSegments) << a.log_ctas) < total) ++a.log_ctas;
  while (more(16, 8) || more(4, 3)) ++a.log_ctas;
  a.segments = (total - 1) / (1 << a.log_ctas) + 1;
  // a request's rows are shared out until the SMs have two CTAs each
  const int per = (num_rows - 1) / num_requests + 1;
  int shares = 1;
  while (shares < per && shares < 64 &&
         (int64_t(num_requests) << a.log_ctas) * shares < 2 * sms)
    shares *= 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  rc = dtype == PKV_F32   ? launch_adjust<float>(a, shares, st)
       : dtype == PKV_F16 ? launch_adjust<__half>(a, shares, st)
                          : launch_adjust<__nv_bfloat16>(a, shares, st);
  return rc == PKV_OK ? ok() : rc;
}
