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
// A CTA takes a piece of the vocabulary for one request: it counts the request's tokens that
// fall there in shared memory (integers, so their order does not matter) and marks them in a
// bit map, then goes through the request's rows.  In place, only tokens that are marked or
// banned are touched: without a mask a row costs as much as the request has tokens, not the
// vocabulary, and 16 bytes of banned tokens are written without being read.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kAdjThreads = 512;
constexpr int kAdjChunk = 8192;                // tokens of the largest piece of the vocabulary
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
  int32_t chunk;                  // tokens of a CTA's piece of the vocabulary, a multiple of 32
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

// Grid: pieces of the vocabulary, requests, shares of a request's rows.  Shared memory: counts
// [chunk], bias entries [chunk] (with biases), marks [chunk / 32 + 1].
template <typename T>
__global__ void __launch_bounds__(kAdjThreads) adjust_logits_kernel(const AdjustArgs a) {
  constexpr int VEC = 16 / sizeof(T);
  extern __shared__ uint32_t adj_smem[];
  const int CH = a.chunk, tid = threadIdx.x;
  const int s = blockIdx.y;
  const int v0 = blockIdx.x * CH, v1 = min(a.V, v0 + CH);
  uint32_t* const count = adj_smem;
  uint32_t* const entry = count + CH;  // 1 + the bias entry of a token (0: none)
  uint32_t* const marks = entry + (a.bias_tokens != nullptr ? CH : 0);
  const int words = static_cast<int>(marks - adj_smem) + CH / 32 + 1;
  const int r_first = a.row_start != nullptr ? max(0, __ldg(a.row_start + s)) : s;
  const int r_end = a.row_start != nullptr ? min(a.T, __ldg(a.row_start + s + 1)) : s + 1;
  if (r_first + static_cast<int64_t>(blockIdx.z) >= r_end) return;
  for (int i = tid; i < words; i += kAdjThreads) adj_smem[i] = 0u;
  __syncthreads();
  auto mark = [&](int i) { atomicOr(marks + (i >> 5), 1u << (i & 31)); };
  {
    const int n = min(max(__ldg(a.history_lens + s), 0), a.L);
    const int prompt = a.prompt_lens != nullptr ? __ldg(a.prompt_lens + s) : 0;
    const int32_t* const tokens = a.history + static_cast<int64_t>(s) * a.L;
    auto one = [&](int at, int tok) {
      if (tok < v0 || tok >= v1) return;
      if (at < prompt) atomicOr(count + (tok - v0), kAdjPrompt);
      else atomicAdd(count + (tok - v0), 1u);
      mark(tok - v0);
    };
    // four tokens at once from the first 16-byte boundary on
    const int head =
        min(n, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(tokens) & 15)) & 15) / 4);
    const int quads = (n - head) / 4;
    if (tid < head) one(tid, __ldg(tokens + tid));
    for (int i = tid; i < quads; i += kAdjThreads) {
      const int4 q = __ldg(reinterpret_cast<const int4*>(tokens + head) + i);
      const int at = head + 4 * i;
      one(at, q.x);
      one(at + 1, q.y);
      one(at + 2, q.z);
      one(at + 3, q.w);
    }
    const int rest = head + 4 * quads + tid;
    if (rest < n) one(rest, __ldg(tokens + rest));
    if (a.bias_tokens != nullptr) {  // of entries for one token the last counts
      const int32_t* const ids = a.bias_tokens + static_cast<int64_t>(s) * a.NBias;
      for (int i = tid; i < a.NBias; i += kAdjThreads) {
        const int tok = __ldg(ids + i);
        if (tok < v0 || tok >= v1) continue;
        atomicMax(entry + (tok - v0), static_cast<uint32_t>(i) + 1u);
        mark(tok - v0);
      }
    }
  }
  const float rep = a.repetition != nullptr ? __ldg(a.repetition + s) : 1.f;
  const float freq = a.frequency != nullptr ? __ldg(a.frequency + s) : 0.f;
  const float pres = a.presence != nullptr ? __ldg(a.presence + s) : 0.f;
  const float* const values =
      a.bias_tokens != nullptr ? a.bias_values + static_cast<int64_t>(s) * a.NBias : nullptr;
  // a marked token's logit (token v0 + i)
  auto adjusted = [&](float x, int i) {
    const uint32_t c = count[i];
    const uint32_t n = c & ~kAdjPrompt;
    if (c != 0) x = x > 0.f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
    if (n != 0) x = __fsub_rn(__fsub_rn(x, __fmul_rn(freq, static_cast<float>(n))), pres);
    if (values != nullptr) {
      const uint32_t e = entry[i];
      if (e != 0) x = __fadd_rn(x, __ldg(values + e - 1));
    }
    return x;
  };
  const bool in_place = a.logits == a.out && a.in_stride == a.out_stride;
  for (int r = r_first + blockIdx.z; r < r_end; r += gridDim.z) {
    const int32_t* const path =
        a.path != nullptr ? a.path + static_cast<int64_t>(r) * a.P : nullptr;
    __syncthreads();  // counts complete; the row before is done
    if (path != nullptr) {
      for (int i = tid; i < a.P; i += kAdjThreads) {
        const int tok = __ldg(path + i);
        if (tok < v0 || tok >= v1) continue;
        atomicAdd(count + (tok - v0), 1u);
        mark(tok - v0);
      }
      __syncthreads();
    }
    const T* const src = static_cast<const T*>(a.logits) + r * a.in_stride;
    T* const dst = static_cast<T*>(a.out) + r * a.out_stride;
    const uint32_t* const ok =
        a.allowed != nullptr ? a.allowed + static_cast<int64_t>(r) * a.W : nullptr;
    // a mark may be of another row's path: only a token that something touches changes
    auto touched = [&](int i) {
      return count[i] != 0 || (values != nullptr && entry[i] != 0);
    };
    if (in_place && ok == nullptr) {
      for (int w = tid; w < CH / 32; w += kAdjThreads) {
        for (uint32_t m = marks[w]; m != 0; m &= m - 1) {
          const int i = 32 * w + __ffs(m) - 1;
          if (touched(i)) dst[v0 + i] = ptx::from_float<T>(adjusted(logit_of(src[v0 + i]), i));
        }
      }
    } else {
      // bits of tokens v .. v + 31 of a bit row of n words, the first being token 0's
      auto bits = [](const uint32_t* row, int n, int v) {
        const int w = v >> 5;
        const uint32_t lo = w < n ? row[w] : 0u;
        const uint32_t hi = (v & 31) != 0 && w + 1 < n ? row[w + 1] : 0u;
        return __funnelshift_r(lo, hi, v & 31);
      };
      auto one = [&](int v) {  // a token by itself
        const int i = v - v0;
        if (ok != nullptr && !((__ldg(ok + (v >> 5)) >> (v & 31)) & 1u))
          dst[v] = ptx::from_float<T>(-INFINITY);
        else if (touched(i)) dst[v] = ptx::from_float<T>(adjusted(logit_of(src[v]), i));
        else if (!in_place) dst[v] = src[v];
      };
      // 16 bytes at a time from the first boundary of the row on (if logits and out share it)
      const uintptr_t off = reinterpret_cast<uintptr_t>(dst) & 15;
      const bool wide = (reinterpret_cast<uintptr_t>(src) & 15) == off;
      const int head = static_cast<int>((16 - off) & 15) / static_cast<int>(sizeof(T));
      // whole pieces inside [v0, v1): n of them from token p0 on
      int p0 = v0 <= head ? head : head + (v0 - head + VEC - 1) / VEC * VEC;
      const int n = wide && v1 > p0 ? (v1 - p0) / VEC : 0;
      if (n == 0) p0 = v1;
      for (int v = v0 + tid; v < p0; v += kAdjThreads) one(v);
      for (int v = p0 + n * VEC + tid; v < v1; v += kAdjThreads) one(v);
      const uint32_t all = (1u << VEC) - 1u;
      AdjPiece<T> ban;
#pragma unroll
      for (int e = 0; e < VEC; ++e) ban.x[e] = ptx::from_float<T>(-INFINITY);
      for (int i = tid; i < n; i += kAdjThreads) {
        const int v = p0 + i * VEC;
        const uint32_t good = ok == nullptr ? all : bits(ok, a.W, v) & all;
        const uint32_t mk = bits(marks, CH / 32 + 1, v - v0) & all;
        if (good == 0) {
          *reinterpret_cast<AdjPiece<T>*>(dst + v) = ban;
          continue;
        }
        if (in_place && good == all && mk == 0) continue;
        AdjPiece<T> p = *reinterpret_cast<const AdjPiece<T>*>(src + v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          if (!((good >> e) & 1u)) p.x[e] = ban.x[e];
          else if (((mk >> e) & 1u) && touched(v - v0 + e))
            p.x[e] = ptx::from_float<T>(adjusted(logit_of(p.x[e]), v - v0 + e));
        }
        *reinterpret_cast<AdjPiece<T>*>(dst + v) = p;
      }
    }
    if (path != nullptr) {  // the row's own tokens are taken out again
      __syncthreads();
      for (int i = tid; i < a.P; i += kAdjThreads) {
        const int tok = __ldg(path + i);
        if (tok >= v0 && tok < v1) atomicSub(count + (tok - v0), 1u);
      }
    }
  }
}

template <typename T>
int launch_adjust(const AdjustArgs& a, int pieces, int shares, size_t smem, cudaStream_t st) {
  static SmemOnce once;
  const int rc = allow_dynamic_smem(once, reinterpret_cast<const void*>(adjust_logits_kernel<T>),
                                    (2 * kAdjChunk + kAdjChunk / 32 + 1) * 4);
  if (rc != PKV_OK) return rc;
  adjust_logits_kernel<T><<<dim3(pieces, a.S, shares), kAdjThreads, smem, st>>>(a);
  PKV_CUDA(cudaGetLastError());
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
  // pieces of the vocabulary small enough for every SM to have one, up to 8,192 tokens
  a.chunk = kAdjChunk;
  while (a.chunk > 1024 &&
         static_cast<int64_t>((vocab + a.chunk - 1) / a.chunk) * num_requests < sms)
    a.chunk /= 2;
  const int pieces = (vocab + a.chunk - 1) / a.chunk;
  // a request's rows are shared out until the SMs have two CTAs each
  const int per = (num_rows - 1) / num_requests + 1;
  int shares = 1;
  while (shares < per && shares < 64 &&
         static_cast<int64_t>(pieces) * num_requests * shares < 2 * sms)
    shares *= 2;
  const size_t smem =
      (static_cast<size_t>(a.chunk) * (a.bias_tokens != nullptr ? 2 : 1) + a.chunk / 32 + 1) * 4;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  rc = dtype == PKV_F32   ? launch_adjust<float>(a, pieces, shares, smem, st)
       : dtype == PKV_F16 ? launch_adjust<__half>(a, pieces, shares, smem, st)
                          : launch_adjust<__nv_bfloat16>(a, pieces, shares, smem, st);
  return rc == PKV_OK ? ok() : rc;
}
