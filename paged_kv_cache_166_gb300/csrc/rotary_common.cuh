// What the kernels that turn q and k to their positions and write the paged cache share:
// their arguments, the turning of pairs, the codes of 8-bit caches.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"
#include "quant8.cuh"

namespace pkv {

constexpr int kMaxRotaryPairs = 128;  // rotary_dim <= 256

struct RotaryArgs {
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  const int32_t* positions;
  const float* table;  // [P, rot]: cos of the rot / 2 angles, then their sin
  const int32_t* slots;
  void* kc;
  void* vc;
  const float* ks;  // 8-bit caches: per-KV-head scales
  const float* vs;
  int32_t* status;  // or NULL
  int64_t q_stride, k_stride, v_stride, qo_stride;  // elements from token to token
  int32_t T, Hq, Hkv, D, rot, B, NB, P;
  int32_t v_parts;  // 8-bit caches: CTAs of one window of V
};

// Checks the arguments that every rotary write has and fills `a` (rotary.cu).  `codes`: 0,
// PKV_FP8_E4M3 or PKV_INT8.
int rotary_args(int32_t codes, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                const void* v, int64_t v_stride, const int32_t* positions, const float* table,
                int32_t max_positions, int32_t rotary_dim, int32_t interleaved,
                const int32_t* slot_mapping, int32_t num_tokens, void* k_cache, void* v_cache,
                const float* k_scale, const float* v_scale, int32_t num_blocks,
                int32_t num_q_heads, int32_t num_kv_heads, int32_t block_size, int32_t head_dim,
                void* q_out, int64_t q_out_stride, int32_t* status, int32_t dtype, RotaryArgs& a);

namespace {

// N consecutive elements, moved at once.
template <typename T, int N>
struct alignas(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Pack {
  T x[N];
};

template <typename T>
__device__ __forceinline__ float widen(T x) {
  if constexpr (std::is_same<T, float>::value) return x;
  else return ptx::to_float(x);
}

// N consecutive values, each rounded once to T.
template <typename T, int N>
__device__ __forceinline__ void store_as(T* dst, const float (&y)[N]) {
  if constexpr (sizeof(T) == 2 && N % 2 == 0) {
    Pack<uint32_t, N / 2> o;
#pragma unroll
    for (int i = 0; i < N; i += 2) o.x[i / 2] = ptx::pack2<T>(y[i], y[i + 1]);
    *reinterpret_cast<Pack<uint32_t, N / 2>*>(dst) = o;
  } else {
    Pack<T, N> o;
#pragma unroll
    for (int i = 0; i < N; ++i) o.x[i] = ptx::from_float<T>(y[i]);
    *reinterpret_cast<Pack<T, N>*>(dst) = o;
  }
}

// Codes of two elements (kCodes 1: E4M3, 2: int8), the first in the low byte.
template <int kCodes>
__device__ __forceinline__ uint32_t codes_of(float x, float y, const Quotients& by) {
  if constexpr (kCodes == 1) return e4m3_codes(by(x), by(y));
  return (static_cast<uint32_t>(int8_code_of(by(x))) & 0xffu) |
         (static_cast<uint32_t>(int8_code_of(by(y))) & 0xffu) << 8;
}

// Codes of N consecutive elements, to dst.
template <int kCodes, int N>
__device__ __forceinline__ void store_codes(uint8_t* dst, const float (&x)[N], const Quotients& by) {
  if constexpr (N == 1) {
    *dst = static_cast<uint8_t>(codes_of<kCodes>(x[0], x[0], by));
  } else {
    Pack<uint16_t, N / 2> c;
#pragma unroll
    for (int i = 0; i < N; i += 2)
      c.x[i / 2] = static_cast<uint16_t>(codes_of<kCodes>(x[i], x[i + 1], by));
    *reinterpret_cast<Pack<uint16_t, N / 2>*>(dst) = c;
  }
}

// The turned pieces: y1 = x1 c - x2 s, y2 = x2 c + x1 s (half layout: x1 and x2 are a piece
// of either half; interleaved: elements 2i and 2i + 1 of x1).  One pair at a time: products
// and sums of two pairs packed in 64-bit registers (mul and add .f32x2) come out fused, so that
// a token's bits would depend on the path that its alignment allows.  They were little
// faster: a step of 256 tokens 3.6 us against 3.7, an fp8 prompt 25.8 against 26.0.
template <typename T, int VEC, bool kInter>
__device__ __forceinline__ void turn(const Pack<T, VEC>& x1, const Pack<T, VEC>& x2,
                                     const float (&c)[kInter ? VEC / 2 : VEC],
                                     const float (&s)[kInter ? VEC / 2 : VEC], float (&y1)[VEC],
                                     float (&y2)[VEC]) {
  constexpr int kAng = kInter ? VEC / 2 : VEC;
  auto a = [&](int i) { return widen(kInter ? x1.x[2 * i] : x1.x[i]); };
  auto b = [&](int i) { return widen(kInter ? x1.x[2 * i + 1] : x2.x[i]); };
  auto first = [&](int i) -> float& { return kInter ? y1[2 * i] : y1[i]; };
  auto second = [&](int i) -> float& { return kInter ? y1[2 * i + 1] : y2[i]; };
#pragma unroll
  for (int i = 0; i < kAng; ++i) {
    const float p = a(i), r = b(i);
    first(i) = __fsub_rn(__fmul_rn(p, c[i]), __fmul_rn(r, s[i]));
    second(i) = __fadd_rn(__fmul_rn(r, c[i]), __fmul_rn(p, s[i]));
  }
}

// V of 8-bit caches: a token is one byte of each 16-byte row of its transposed tile.  A
// run of consecutive tokens in consecutive slots of one block is written as a whole, a
// thread two rows: 32 contiguous bytes if the run fills the block (a prompt's usual case),
// else byte pairs and bytes.  The CTAs of window w own the runs that begin in tokens
// 16 w .. 16 w + 15, and take their work items (run, head, two rows) in turn.
template <typename T, bool kPairs, int kCodes>
__device__ __forceinline__ void write_v8(const RotaryArgs& a, int window, int part, int parts) {
  __shared__ int slot_s[48];  // tokens 16 (w - 1) .. 16 (w + 2) - 1; -1: nothing to write
  __shared__ int run_first[16], run_len[16], run_count;
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
  const int64_t t0 = static_cast<int64_t>(window) * 16 - 16;
  if (tid < 48) {
    int slot = -1;
    if (t0 + tid >= 0 && t0 + tid < a.T) slot = __ldg(a.slots + t0 + tid);
    if (slot < 0 || slot >= a.NB * 16) slot = -1;
    slot_s[tid] = slot;
  }
  __syncthreads();
  if (tid < 32) {
    const int i = 16 + tid, slot = slot_s[i];
    // a token that goes on its predecessor's run
    const bool goes_on = slot > 0 && slot % 16 != 0 && slot_s[i - 1] == slot - 1;
    const bool begins = tid < 16 && slot >= 0 && !goes_on;
    const uint32_t on = __ballot_sync(0xffffffffu, goes_on);
    const uint32_t all = __ballot_sync(0xffffffffu, begins);
    if (begins) {  // at most 16 tokens, so in the 32 looked at: a run ends with its block
      const int at = __popc(all & ((1u << tid) - 1));
      run_first[at] = i;
      run_len[at] = __ffs(~(on >> (tid + 1)));
    }
    if (tid == 0) run_count = __popc(all);
  }
  __syncthreads();
  const int pairs = a.D / 2, per_run = a.Hkv * pairs;
  const int items = run_count * per_run;
  for (int it = part * threads + tid; it < items; it += parts * threads) {
    const int run = it / per_run, g = (it - run * per_run) / pairs;
    const int d = 2 * (it - run * per_run - g * pairs);
    const int first = run_first[run], n = run_len[run], slot = slot_s[first];
    const int off = slot % 16;
    const Quotients by = quotients_by(__ldg(a.vs + g));
    const T* const src = static_cast<const T*>(a.v) + (t0 + first - off) * a.v_stride +
                         static_cast<int64_t>(g) * a.D + d;  // row of the block's token 0
    // two elements a token, packed as they are loaded
    Pack<T, 2> x[16];
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      x[t].x[0] = x[t].x[1] = ptx::from_float<T>(0.f);
      if (t >= off && t < off + n) {
        const T* const at = src + t * a.v_stride;
        if constexpr (kPairs) {
          x[t] = *reinterpret_cast<const Pack<T, 2>*>(at);
        } else {
          x[t].x[0] = at[0];
          x[t].x[1] = at[1];
        }
      }
    }
    // word j of a row: tokens 2j, 2j + 1, 2j + 8 and 2j + 9
    uint32_t w[2][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
        w[r][j] = codes_of<kCodes>(widen(x[2 * j].x[r]), widen(x[2 * j + 1].x[r]), by) |
                  codes_of<kCodes>(widen(x[2 * j + 8].x[r]), widen(x[2 * j + 9].x[r]), by) << 16;
    }
    uint8_t* const dst = static_cast<uint8_t*>(a.vc) +
                         ((static_cast<int64_t>(slot / 16) * a.Hkv + g) * a.D + d) * 16;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      uint8_t* const to = dst + 16 * r;
      if (n == 16) {
        *reinterpret_cast<uint4*>(to) = make_uint4(w[r][0], w[r][1], w[r][2], w[r][3]);
        continue;
      }
#pragma unroll
      for (int p = 0; p < 8; ++p) {  // byte pairs: tokens t and t + 1
        const int t = p % 2 == 0 ? p : p + 7;
        const uint32_t c = w[r][p / 2] >> (16 * (p % 2));
        const bool one = t >= off && t < off + n, two = t + 1 >= off && t + 1 < off + n;
        if (one && two) *reinterpret_cast<uint16_t*>(to + 2 * p) = static_cast<uint16_t>(c);
        else if (one) to[2 * p] = static_cast<uint8_t>(c);
        else if (two) to[2 * p + 1] = static_cast<uint8_t>(c >> 8);
      }
    }
  }
}

}  // namespace
}  // namespace pkv
