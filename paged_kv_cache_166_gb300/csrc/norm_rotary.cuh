// Norms of q and k for each head, rotary positions on one or several axes, and the write of k
// and v into the paged cache, in one pass: the kernels.
//
// A head x of D elements is first normed (unless the call asks for none),
//   y_d = (x_d * r) * w_d,   r = 1 / sqrt(sum_e x_e^2 / D + eps),
// then its first rotary_dim elements are turned in pairs as rotary.cu does, pair i by the row
// of the table at the token's position on the pair's axis.  q goes to q_out, k and v to their
// slots, so q, k and v are read once and nothing between is written.
//
// Arithmetic: fp32; squares are added as they are formed, the mean is a product with 1 / D, the
// root an approximate one corrected by a Newton step, the two products of the norm are rounded
// each, and of a turn (x1 c - x2 s) the second product is rounded, the first and the sum together.
// (Without a norm each product and sum is rounded by itself: the bits of rotary.cu.)  Then one
// rounding to the type, or one quantisation straight from fp32.  Two elements go through packed
// instructions where a lane has them, which round as single ones do.  A head's squares are
// summed in an order that depends on its layout alone (D, rotary_dim, pairing, type), so a token's
// bits depend neither on strides or alignment nor on how many tokens come with it.
//
// A group of up to 32 lanes takes a head: a lane's pieces of 16 bytes (both halves' ones of a
// turned pair), the sum of squares by shuffles; then the next head with the cos, sin and
// weights that the lane has loaded once.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "rotary_common.cuh"

namespace pkv {

constexpr int kMaxAxes = 4;

struct NormArgs : RotaryArgs {
  const void* qw;  // weights [D] or [heads, D], or NULL: ones
  const void* kw;
  float eps, inv_d;
  int32_t norm, axes, per_head, w_f32;
  int32_t wide, w_wide, v_pairs;  // addresses that allow 16 bytes (or a pair) at once
  uint32_t axis_bits[kMaxRotaryPairs / 16];  // two bits a pair
};

// Caches of 8-bit codes (a translation unit of their own: they compile beside the others).
int norm_rotary_8bit(const NormArgs& a, int32_t codes, int32_t dtype, bool interleaved,
                     cudaStream_t st);

namespace {

constexpr int kNormThreads = 128;

// What a kernel is compiled for: pieces at 16-byte boundaries and a norm, the same without a norm
// (caches of q's type), or anything.  (One for all: a step of 256 tokens of 64 + 8 heads of 128 7.5
// us, this 5.8; with the branches for single elements out of line 7.3.)
enum NormForm { kAlignedNorm, kAligned, kAnyNorm };

template <typename T, int N>
__device__ __forceinline__ Pack<T, N> load_piece(const T* p, bool wide) {
  Pack<T, N> x;
  if (wide) {
    x = *reinterpret_cast<const Pack<T, N>*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x.x[i] = p[i];
  }
  return x;
}

template <typename T, int N>
__device__ __forceinline__ void store_piece(T* p, const float (&y)[N], bool wide) {
  if (wide) {
    store_as<T, N>(p, y);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = ptx::from_float<T>(y[i]);
  }
}

// Squares of a piece added to (even, odd) elements' sums.
template <int VEC>
__device__ __forceinline__ void add_squares(const float (&x)[VEC], float& even, float& odd) {
  if constexpr (VEC == 1) {
    even = __fmaf_rn(x[0], x[0], even);
  } else {
    uint64_t sum = ptx::pair(even, odd);
#pragma unroll
    for (int i = 0; i < VEC; i += 2) {
      const uint64_t p = ptx::pair(x[i], x[i + 1]);
      sum = ptx::fma2(p, p, sum);
    }
    ptx::unpair(sum, even, odd);
  }
}

// 1 / sqrt(sum / D + eps).
__device__ __forceinline__ float inverse_root(float sum, float inv_d, float eps) {
  const float m = __fmaf_rn(sum, inv_d, eps);
  const float y = rsqrtf(m);
  if (!(m >= 0x1p-100f && m <= 0x1p100f)) return __frsqrt_rn(m);  // the step's squares need room
  const float e = __fmaf_rn(__fmul_rn(m, y), -y, 1.f);
  return __fmaf_rn(__fmul_rn(0.5f, y), e, y);
}

// x = (x * r) * w.
template <int VEC>
__device__ __forceinline__ void apply_norm(float (&x)[VEC], float r, const float (&w)[VEC]) {
  if constexpr (VEC == 1) {
    x[0] = __fmul_rn(__fmul_rn(x[0], r), w[0]);
  } else {
    const uint64_t rr = ptx::pair(r, r);
#pragma unroll
    for (int i = 0; i < VEC; i += 2)
      ptx::unpair(ptx::mul2(ptx::mul2(ptx::pair(x[i], x[i + 1]), rr), ptx::pair(w[i], w[i + 1])),
                  x[i], x[i + 1]);
  }
}

// z1 = a c - b s, z2 = b c + a s for N pairs.  fused: the first product and the sum together.
template <int N>
__device__ __forceinline__ void turn_pairs(const float (&a)[N], const float (&b)[N],
                                           const float (&c)[N], const float (&s)[N], bool fused,
                                           float (&z1)[N], float (&z2)[N]) {
  if (!fused) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      z1[i] = __fsub_rn(__fmul_rn(a[i], c[i]), __fmul_rn(b[i], s[i]));
      z2[i] = __fadd_rn(__fmul_rn(b[i], c[i]), __fmul_rn(a[i], s[i]));
    }
  } else if constexpr (N == 1) {
    z1[0] = __fmaf_rn(a[0], c[0], __fmul_rn(b[0], -s[0]));
    z2[0] = __fmaf_rn(b[0], c[0], __fmul_rn(a[0], s[0]));
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint64_t pa = ptx::pair(a[i], a[i + 1]), pb = ptx::pair(b[i], b[i + 1]);
      const uint64_t pc = ptx::pair(c[i], c[i + 1]);
      ptx::unpair(ptx::fma2(pa, pc, ptx::mul2(pb, ptx::pair(-s[i], -s[i + 1]))), z1[i], z1[i + 1]);
      ptx::unpair(ptx::fma2(pb, pc, ptx::mul2(pa, ptx::pair(s[i], s[i + 1]))), z2[i], z2[i + 1]);
    }
  }
}

// A piece of a head normed (x1, x2 its halves' ones) and turned: f(0, z1) and, half layout,
// f(half, z2).
template <int VEC, bool kInter, typename F>
__device__ __forceinline__ void turn_piece(const float (&x1)[VEC], const float (&x2)[VEC],
                                           const float (&c)[kInter ? VEC / 2 : VEC],
                                           const float (&s)[kInter ? VEC / 2 : VEC], bool fused,
                                           int half, F f) {
  if constexpr (kInter) {
    constexpr int N = VEC / 2;
    float a[N], b[N], z1[N], z2[N], z[VEC];
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] = x1[2 * i], b[i] = x1[2 * i + 1];
    turn_pairs<N>(a, b, c, s, fused, z1, z2);
#pragma unroll
    for (int i = 0; i < N; ++i) z[2 * i] = z1[i], z[2 * i + 1] = z2[i];
    f(0, z);
  } else {
    float z1[VEC], z2[VEC];
    turn_pairs<VEC>(x1, x2, c, s, fused, z1, z2);
    f(0, z1);
    f(half, z2);
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void widen_piece(const Pack<T, VEC>& p, float (&x)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) x[i] = widen(p.x[i]);
}

// A lane's pieces of one head.
template <typename T, int VEC, int NU>
struct Pieces {
  Pack<T, VEC> one[NU], two[NU];  // two: the second half's, of turned pieces (half layout)
};

// blockIdx.x < T: a token, its heads split over gridDim.y CTAs and the CTA's groups of lanes;
// 8-bit caches: then V's windows, a.v_parts CTAs each.  Bound by how many loads are on their
// way: with seven CTAs an SM a prompt keeps DRAM at 50% and the SM at 38% of their peaks, its warps
// waiting for loads (into fp8 the SM at 57%).  CTAs an SM: 8,191 tokens of 40 + 40 heads of 128, f16, half
// layout, 114 us with six, 105 with seven (4.8 TB/s), 101 with eight; 1,000 of 64 + 8 heads 12.9,
// 10.2, 12.1; 640 of them 7.8, 8.6, 9.8: seven.  Interleaved, 4,099 tokens of 32 + 8 heads into fp8
// 32.7 with eight, 31.8 with nine, 34.4 with ten.  (Most forms with a norm spill for it, 16-bit caches
// 8 to 44 bytes; the other types' numbers were not measured one by one.)  Two heads' loads in flight pay where a head is
// one piece a lane (37.8 us there with two, 44.6 with four).
template <typename T, int VEC, bool kInter, int kCodes, int NU, NormForm kForm>
__global__ void __launch_bounds__(kNormThreads, kInter ? 9 : 7)
    norm_rotary_kernel(const __grid_constant__ NormArgs a) {
  // as rotary_write_kernel: a launch queued behind reads and writes nothing of this one's
  // before this grid has completed
  asm volatile("griddepcontrol.launch_dependents;");
  using P = Pack<T, VEC>;
  constexpr int kAng = kInter ? VEC / 2 : VEC;  // pairs of a piece
  const int64_t t = blockIdx.x;
  if constexpr (kCodes != 0) {
    if (t >= a.T) {
      const int64_t i = (t - a.T) * gridDim.y + blockIdx.y;
      const int64_t window = i / a.v_parts;
      if (window * 16 < a.T) {
        const int part = static_cast<int>(i - window * a.v_parts);
        if (a.v_pairs) write_v8<T, true, kCodes>(a, static_cast<int>(window), part, a.v_parts);
        else write_v8<T, false, kCodes>(a, static_cast<int>(window), part, a.v_parts);
      }
      return;
    }
  }
  const int half = a.rot >> 1;
  const int nturn = kInter ? a.rot / VEC : half / VEC;
  const int units = nturn + (a.D - a.rot) / VEC;
  const int L = blockDim.x;  // lanes of a head: a power of two
  const int lane = (threadIdx.y * L + threadIdx.x) & 31;
  const uint32_t group = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << (lane & ~(L - 1));

  const int32_t slot = __ldg(a.slots + t);
  const bool write = slot >= 0 && static_cast<int64_t>(slot) < static_cast<int64_t>(a.NB) * a.B;
  int32_t pos[kMaxAxes];
#pragma unroll
  for (int x = 0; x < kMaxAxes; ++x) {
    pos[x] = 0;
    if (x < a.axes) {
      pos[x] = __ldg(a.positions + static_cast<int64_t>(x) * a.T + t);
      if (pos[x] < 0 || pos[x] >= a.P) {
        if (a.status != nullptr && threadIdx.x == 0 && threadIdx.y == 0 && blockIdx.y == 0)
          atomicOr(a.status, PKV_DEV_BAD_POSITION);
        pos[x] = pos[x] < 0 ? 0 : a.P - 1;
      }
    }
  }
  int at[NU];  // first element of the lane's unit; D: none
  float c[NU][kAng], s[NU][kAng];
#pragma unroll
  for (int j = 0; j < NU; ++j) {
    const int u = threadIdx.x + j * L;
    at[j] = u < nturn ? u * VEC : (u < units ? a.rot + (u - nturn) * VEC : a.D);
    if (u >= nturn) {
#pragma unroll
      for (int i = 0; i < kAng; ++i) c[j][i] = s[j][i] = 0.f;  // (not used)
      continue;
    }
    const int i0 = u * kAng;
    // a piece whose pairs all turn by one axis loads its angles at once
    uint32_t x0 = 0;
    bool one = true;
    if (a.axes > 1) {
      constexpr uint32_t mask = (1u << (2 * kAng)) - 1u;
      const uint32_t bits = (a.axis_bits[i0 >> 4] >> (2 * (i0 & 15))) & mask;
      x0 = bits & 3u;
      one = bits == (mask / 3u) * x0;
    }
    if (one) {
      const int32_t p = x0 == 0 ? pos[0] : (x0 == 1 ? pos[1] : (x0 == 2 ? pos[2] : pos[3]));
      const float* const row = a.table + static_cast<int64_t>(p) * a.rot + i0;
      const Pack<float, kAng> pc = *reinterpret_cast<const Pack<float, kAng>*>(row);
      const Pack<float, kAng> ps = *reinterpret_cast<const Pack<float, kAng>*>(row + half);
#pragma unroll
      for (int i = 0; i < kAng; ++i) {
        c[j][i] = pc.x[i];
        s[j][i] = ps.x[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kAng; ++i) {
        const uint32_t x = (a.axis_bits[(i0 + i) >> 4] >> (2 * ((i0 + i) & 15))) & 3u;
        const int32_t p = x == 0 ? pos[0] : (x == 1 ? pos[1] : (x == 2 ? pos[2] : pos[3]));
        const float* const row = a.table + static_cast<int64_t>(p) * a.rot + i0 + i;
        c[j][i] = __ldg(row);
        s[j][i] = __ldg(row + half);
      }
    }
  }
  auto turns = [&](int j) { return static_cast<int>(threadIdx.x) + j * L < nturn; };
  const bool wide = kForm != kAnyNorm || a.wide != 0, w_wide = kForm != kAnyNorm || a.w_wide != 0;
  const bool norm = kForm == kAlignedNorm || (kForm == kAnyNorm && a.norm != 0);

  float w1[NU][VEC], w2[NU][VEC];
  auto weights = [&](const void* w, int h) {  // of head h, or of all
#pragma unroll
    for (int j = 0; j < NU; ++j) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) w1[j][i] = w2[j][i] = 1.f;
      if (w == nullptr || !norm || at[j] >= a.D) continue;
      const int64_t d = (a.per_head ? static_cast<int64_t>(h) * a.D : 0) + at[j];
      const bool second = !kInter && turns(j);
      if (a.w_f32) {
        const float* const p = static_cast<const float*>(w) + d;
        const Pack<float, VEC> x = load_piece<float, VEC>(p, w_wide);
#pragma unroll
        for (int i = 0; i < VEC; ++i) w1[j][i] = x.x[i];
        if (second) {
          const Pack<float, VEC> y = load_piece<float, VEC>(p + half, w_wide);
#pragma unroll
          for (int i = 0; i < VEC; ++i) w2[j][i] = y.x[i];
        }
      } else {
        const T* const p = static_cast<const T*>(w) + d;
        const P x = load_piece<T, VEC>(p, w_wide);
#pragma unroll
        for (int i = 0; i < VEC; ++i) w1[j][i] = widen(x.x[i]);
        if (second) {
          const P y = load_piece<T, VEC>(p + half, w_wide);
#pragma unroll
          for (int i = 0; i < VEC; ++i) w2[j][i] = widen(y.x[i]);
        }
      }
    }
  };
  using Own = Pieces<T, VEC, NU>;
  auto load = [&](const T* src, Own& x) {
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      if (at[j] >= a.D) continue;
      x.one[j] = load_piece<T, VEC>(src + at[j], wide);
      if (!kInter && turns(j)) x.two[j] = load_piece<T, VEC>(src + at[j] + half, wide);
    }
  };
  // norm and turn of a head; put(j, element, values) for each of the lane's pieces
  auto work = [&](const Own& x, auto put) {
    float r = 1.f;
    if (norm) {
      float even = 0.f, odd = 0.f;
#pragma unroll
      for (int j = 0; j < NU; ++j) {
        if (at[j] >= a.D) continue;
        float y[VEC];
        widen_piece(x.one[j], y);
        add_squares<VEC>(y, even, odd);
        if (!kInter && turns(j)) {
          widen_piece(x.two[j], y);
          add_squares<VEC>(y, even, odd);
        }
      }
      float sum = __fadd_rn(even, odd);
      for (int o = L >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(group, sum, o);
      r = inverse_root(sum, a.inv_d, a.eps);
    }
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      if (at[j] >= a.D) continue;
      float x1[VEC], x2[VEC] = {};
      widen_piece(x.one[j], x1);
      if (norm) apply_norm<VEC>(x1, r, w1[j]);
      if constexpr (kInter) {  // lanes that turn and lanes that don't side by side
        turn_piece<VEC, true>(x1, x2, c[j], s[j], norm, half,
                              [&](int, const float (&z)[VEC]) {
#pragma unroll
                                for (int i = 0; i < VEC; ++i) x1[i] = turns(j) ? z[i] : x1[i];
                              });
        put(j, at[j], x1);
        continue;
      }
      if (!turns(j)) {
        put(j, at[j], x1);
        continue;
      }
      widen_piece(x.two[j], x2);
      if (norm) apply_norm<VEC>(x2, r, w2[j]);
      turn_piece<VEC, kInter>(x1, x2, c[j], s[j], norm, half,
                              [&](int d, const float (&z)[VEC]) { put(j, at[j] + d, z); });
    }
  };
  const int h0 = threadIdx.y + blockDim.y * blockIdx.y, step = blockDim.y * gridDim.y;
  constexpr int U = NU == 1 && kInter ? 2 : 1;  // heads whose loads go out together
  auto each = [&](const T* src, int H, auto put) {
    for (int h = h0; h < H; h += U * step) {
      Own x[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h + u * step < H) load(src + static_cast<int64_t>(h + u * step) * a.D, x[u]);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (h + u * step < H) put(h + u * step, x[u]);
    }
  };
  // a piece that neither norm nor turn touches keeps its bits (a NaN's too)
  auto put_same = [&](T* row, int j, int d, const float (&y)[VEC], const Own& x, bool w) {
    if (!norm && !turns(j)) {
      if (w) {
        *reinterpret_cast<P*>(row + d) = x.one[j];
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) row[d + i] = x.one[j].x[i];
      }
    } else {
      store_piece<T, VEC>(row + d, y, w);
    }
  };
  if (!a.per_head) weights(a.qw, 0);
  T* const qo = static_cast<T*>(a.q_out) + t * a.qo_stride;
  each(static_cast<const T*>(a.q) + t * a.q_stride, a.Hq, [&](int h, const Own& x) {
    if (a.per_head) weights(a.qw, h);
    T* const row = qo + static_cast<int64_t>(h) * a.D;
    work(x, [&](int j, int d, const float (&y)[VEC]) { put_same(row, j, d, y, x, wide); });
  });
  if (!write) return;
  const int32_t block = (a.B & (a.B - 1)) == 0 ? slot >> (31 - __clz(a.B)) : slot / a.B;
  const int32_t off = slot - block * a.B;
  const int64_t row0 = (static_cast<int64_t>(block) * a.Hkv * a.B + off) * a.D;  // of head 0
  const int64_t head = static_cast<int64_t>(a.B) * a.D;
  if (!a.per_head) weights(a.kw, 0);
  each(static_cast<const T*>(a.k) + t * a.k_stride, a.Hkv, [&](int g, const Own& x) {
    if (a.per_head) weights(a.kw, g);
    if constexpr (kCodes == 0) {
      T* const row = static_cast<T*>(a.kc) + row0 + g * head;
      work(x, [&](int j, int d, const float (&y)[VEC]) { put_same(row, j, d, y, x, true); });
    } else {
      uint8_t* const row = static_cast<uint8_t*>(a.kc) + row0 + g * head;
      const Quotients by = quotients_by(__ldg(a.ks + g));
      work(x, [&](int, int d, const float (&y)[VEC]) { store_codes<kCodes, VEC>(row + d, y, by); });
    }
  });
  if constexpr (kCodes == 0) {  // V rows, copied
    each(static_cast<const T*>(a.v) + t * a.v_stride, a.Hkv, [&](int g, const Own& x) {
      T* const row = static_cast<T*>(a.vc) + row0 + g * head;
#pragma unroll
      for (int j = 0; j < NU; ++j) {
        if (at[j] >= a.D) continue;
        *reinterpret_cast<P*>(row + at[j]) = x.one[j];
        if (!kInter && turns(j)) *reinterpret_cast<P*>(row + at[j] + half) = x.two[j];
      }
    });
  }
}

int lanes_of(int units) {
  int l = 1;
  while (l < units && l < 32) l *= 2;
  return l;
}

template <typename T, int kCodes>
int launch_norm(NormArgs a, bool interleaved, cudaStream_t st) {
  constexpr int W = 16 / sizeof(T);
  // pieces of 16 bytes where head_dim and rotary_dim allow them, else the smallest that
  // hold whole pairs
  const bool whole = a.rot % (interleaved ? W : 2 * W) == 0 && a.D % W == 0;
  const int vec = whole ? W : (interleaved ? 2 : 1);
  const bool strides = a.q_stride % W == 0 && a.k_stride % W == 0 && a.v_stride % W == 0 &&
                       a.qo_stride % W == 0 && aligned(a.q, 16) && aligned(a.k, 16) &&
                       aligned(a.v, 16) && aligned(a.q_out, 16);
  // (interleaved pairs are aligned to their two elements, single elements to themselves)
  a.wide = !whole || strides;
  a.w_wide = vec == 1 || (aligned(a.qw, 16) && aligned(a.kw, 16));
  a.v_pairs = (a.v_stride % 2 == 0 && aligned(a.v, 2 * sizeof(T))) ? 1 : 0;
  const int units = (interleaved ? a.rot / vec : a.rot / (2 * vec)) + (a.D - a.rot) / vec;
  const int lanes = lanes_of(units), rows = kNormThreads / lanes;
  int sms = 0, dev = 0;
  const int rc = device_sm_count(&sms, &dev);
  if (rc != PKV_OK) return rc;
  // few tokens: their heads are spread over more CTAs until the SMs have a few each
  int split = 1;
  while (split * rows < a.Hq && static_cast<int64_t>(a.T) * split < 4 * sms) split *= 2;
  int64_t columns = a.T;
  if (kCodes != 0) {  // V's windows: an item a thread if the window is one run
    const int64_t windows = (static_cast<int64_t>(a.T) + 15) / 16;
    const int64_t items = static_cast<int64_t>(a.Hkv) * a.D / 2;
    const int64_t parts = (items + kNormThreads - 1) / kNormThreads;
    a.v_parts = static_cast<int32_t>(parts);
    columns += (windows * parts + split - 1) / split;
  }
  PKV_REQUIRE(columns < (int64_t(1) << 31), PKV_ERR_UNSUPPORTED, "too many tokens");
  const dim3 grid(static_cast<unsigned>(columns), split), threads(lanes, rows);
  constexpr int NU = W == 4 ? 2 : 1;
  auto launch = [&](auto vec_c, auto inter, auto nu, auto form) {
    norm_rotary_kernel<T, decltype(vec_c)::value, decltype(inter)::value, kCodes,
                       decltype(nu)::value, decltype(form)::value><<<grid, threads, 0, st>>>(a);
  };
  using std::integral_constant;
  const auto all = [&](auto inter) {
    const integral_constant<int, W> w{};
    const integral_constant<int, W == 4 ? 2 : 1> nu{};
    if (a.wide && a.w_wide && a.norm)
      return launch(w, inter, nu, integral_constant<NormForm, kAlignedNorm>{});
    if constexpr (kCodes == 0) {
      if (a.wide && !a.norm) return launch(w, inter, nu, integral_constant<NormForm, kAligned>{});
    }
    return launch(w, inter, nu, integral_constant<NormForm, kAnyNorm>{});
  };
  if (whole && interleaved)
    all(std::true_type{});
  else if (whole)
    all(std::false_type{});
  else if (interleaved)
    launch(integral_constant<int, 2>{}, std::true_type{}, integral_constant<int, 4>{},
           integral_constant<NormForm, kAnyNorm>{});
  else
    launch(integral_constant<int, 1>{}, std::false_type{}, integral_constant<int, 8>{},
           integral_constant<NormForm, kAnyNorm>{});
  PKV_CUDA(cudaGetLastError());
  return PKV_OK;
}

template <int kCodes>
int launch_norm_of(const NormArgs& a, int32_t dtype, bool interleaved, cudaStream_t st) {
  return dtype == PKV_F32   ? launch_norm<float, kCodes>(a, interleaved, st)
         : dtype == PKV_F16 ? launch_norm<__half, kCodes>(a, interleaved, st)
                            : launch_norm<__nv_bfloat16, kCodes>(a, interleaved, st);
}

}  // namespace
}  // namespace pkv
