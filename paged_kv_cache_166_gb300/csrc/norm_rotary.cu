// Norms of q and k for each head, rotary positions on one or several axes, and the write of k
// and v into the paged cache, in one pass.
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
// weights that the lane has loaded once.  Bound by memory.
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
namespace {

constexpr int kMaxAxes = 4;
constexpr int kNormThreads = 128;
constexpr int kBulkTokens = 6;  // tokens an SM from which on whole tokens are fetched

struct NormArgs : RotaryArgs {
  const void* qw;  // weights [D] or [heads, D], or NULL: ones
  const void* kw;
  float eps, inv_d;
  int32_t norm, axes, per_head, w_f32;
  int32_t wide, w_wide, v_pairs;  // addresses that allow 16 bytes (or a pair) at once
  uint32_t axis_bits[kMaxRotaryPairs / 16];  // two bits a pair
};

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
// 8-bit caches: then V's windows, a.v_parts CTAs each.  Bound by the instructions of a head and by
// how many warps hide its loads: 4,099 tokens of 32 + 8 heads of 128 into fp8, interleaved,
// 37.8 us with eight CTAs an SM and two heads in flight, 42.3 with six, 43.1 with ten (spills);
// the half layout holds a piece more and wants six (1,000 tokens of 64 + 8 heads 10.1 against
// 11.4).  Loading a token's first rows ahead of its position was no gain (46).
template <typename T, int VEC, bool kInter, int kCodes, int NU>
__global__ void __launch_bounds__(kNormThreads, kInter ? 8 : 6)
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
    if (a.axes == 1) {
      const float* const row = a.table + static_cast<int64_t>(pos[0]) * a.rot + i0;
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
  const bool wide = a.wide != 0;

  float w1[NU][VEC], w2[NU][VEC];
  auto weights = [&](const void* w, int h) {  // of head h, or of all
#pragma unroll
    for (int j = 0; j < NU; ++j) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) w1[j][i] = w2[j][i] = 1.f;
      if (w == nullptr || !a.norm || at[j] >= a.D) continue;
      const int64_t d = (a.per_head ? static_cast<int64_t>(h) * a.D : 0) + at[j];
      const bool second = !kInter && turns(j);
      if (a.w_f32) {
        const float* const p = static_cast<const float*>(w) + d;
        const Pack<float, VEC> x = load_piece<float, VEC>(p, a.w_wide != 0);
#pragma unroll
        for (int i = 0; i < VEC; ++i) w1[j][i] = x.x[i];
        if (second) {
          const Pack<float, VEC> y = load_piece<float, VEC>(p + half, a.w_wide != 0);
#pragma unroll
          for (int i = 0; i < VEC; ++i) w2[j][i] = y.x[i];
        }
      } else {
        const T* const p = static_cast<const T*>(w) + d;
        const P x = load_piece<T, VEC>(p, a.w_wide != 0);
#pragma unroll
        for (int i = 0; i < VEC; ++i) w1[j][i] = widen(x.x[i]);
        if (second) {
          const P y = load_piece<T, VEC>(p + half, a.w_wide != 0);
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
    if (a.norm) {
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
      if (a.norm) apply_norm<VEC>(x1, r, w1[j]);
      if constexpr (kInter) {  // lanes that turn and lanes that don't side by side
        turn_piece<VEC, true>(x1, x2, c[j], s[j], a.norm != 0, half,
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
      if (a.norm) apply_norm<VEC>(x2, r, w2[j]);
      turn_piece<VEC, kInter>(x1, x2, c[j], s[j], a.norm != 0, half,
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
    if (!a.norm && !turns(j)) {
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

// ---- many tokens: rows of whole tokens by bulk copies ------------------------------------------
// One warp fetches: the rows of a token's q, k and v and its rows of the table go to a stage of
// shared memory by cp.async.bulk, several tokens ahead, so that neither positions nor tables nor
// rows are waited for.  Seven warps norm, turn and write a stage's heads (with the eighth a CTA of
// 256 threads: two on an SM leave a thread 128 registers; eight and one spilled, and took 127 us
// where this takes 112); the lanes of a head, and so its bits, are those of the kernel above.
// Measured against it: 8,191 tokens of 40 + 40 heads of 128 on three axes 112 us (4.5 TB/s) to
// 148, on one 107 to 134, without a norm 84 to 115; of 64 + 8 heads 1,000 tokens 15.9 to 17.6,
// 640 tokens 12.3 to 10.1, hence six tokens an SM.  8-bit caches, 32-bit types (121 to 108) and a
// weight for each head (56 to 46) stay with the kernel above.
constexpr int kBulkWarps = 7;
constexpr int kBulkThreads = (kBulkWarps + 1) * 32;
constexpr int kBulkStages = 8;                 // at most
constexpr uint64_t kBulkWaitNs = 1000000000ull;  // 1 s per wait before giving up

struct BulkShape {
  uint32_t q, k, stage;  // bytes of a token's q and k (and v), and of a stage (16 for the slot)
  int32_t stages;
};

template <typename T, bool kInter, bool kNorm>
__global__ void __launch_bounds__(kBulkThreads, 2)
    norm_rotary_bulk_kernel(const __grid_constant__ NormArgs a, const BulkShape sh) {
  asm volatile("griddepcontrol.launch_dependents;");
  constexpr int VEC = 8;  // of 16-bit types
  constexpr int kAng = kInter ? VEC / 2 : VEC;
  using P = Pack<T, VEC>;
  extern __shared__ __align__(128) uint8_t bulk_smem[];
  __shared__ uint64_t bar_mem[2 * kBulkStages];
  const uint32_t bars = ptx::smem_addr(bar_mem);
  auto full = [&](uint32_t st) { return bars + 8 * st; };
  auto empty = [&](uint32_t st) { return bars + 8 * (kBulkStages + st); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kBulkStages; ++i) {
      ptx::mbar_init(full(i), 1);
      ptx::mbar_init(empty(i), kBulkWarps);
    }
    ptx::fence_barrier_init();
  }
  __syncthreads();
  const uint32_t stages = sh.stages;
  const int64_t step = gridDim.x;
  if (warp == kBulkWarps) {
    uint32_t it = 0;
    bool alive = true;
    for (int64_t t0 = blockIdx.x; alive && t0 < a.T; t0 += 32 * step) {
      // a lane looks up a token's slot and positions
      const int64_t t = t0 + lane * step;
      int32_t slot = -1, pos[kMaxAxes] = {0, 0, 0, 0};
      if (t < a.T) {
        slot = __ldg(a.slots + t);
#pragma unroll
        for (int x = 0; x < kMaxAxes; ++x) {
          if (x >= a.axes) continue;
          pos[x] = __ldg(a.positions + static_cast<int64_t>(x) * a.T + t);
          if (pos[x] < 0 || pos[x] >= a.P) {
            if (a.status != nullptr) atomicOr(a.status, PKV_DEV_BAD_POSITION);
            pos[x] = pos[x] < 0 ? 0 : a.P - 1;
          }
        }
      }
      for (int l = 0; l < 32 && t0 + l * step < a.T; ++l, ++it) {
        const int32_t sl = __shfl_sync(0xffffffffu, slot, l);
        int32_t ps[kMaxAxes];
#pragma unroll
        for (int x = 0; x < kMaxAxes; ++x) ps[x] = __shfl_sync(0xffffffffu, pos[x], l);
        const uint32_t st = it % stages;
        if (lane == 0) {
          alive = ptx::mbar_wait(empty(st), ((it / stages) & 1u) ^ 1u, kBulkWaitNs);
          if (alive) {
            uint8_t* const stage = bulk_smem + st * sh.stage;
            const uint32_t at = ptx::smem_addr(stage);
            *reinterpret_cast<int32_t*>(stage + sh.stage - 16) = sl;
            const uint32_t row = static_cast<uint32_t>(a.rot) * 4;
            ptx::mbar_arrive_expect_tx(full(st), sh.q + 2 * sh.k + row * a.axes);
            const int64_t tok = t0 + l * step;
            ptx::bulk_load(at, static_cast<const T*>(a.q) + tok * a.q_stride, sh.q, full(st));
            ptx::bulk_load(at + sh.q, static_cast<const T*>(a.k) + tok * a.k_stride, sh.k, full(st));
            ptx::bulk_load(at + sh.q + sh.k, static_cast<const T*>(a.v) + tok * a.v_stride, sh.k,
                           full(st));
#pragma unroll
            for (int x = 0; x < kMaxAxes; ++x)
              if (x < a.axes)
                ptx::bulk_load(at + sh.q + 2 * sh.k + x * row,
                               a.table + static_cast<int64_t>(ps[x]) * a.rot, row, full(st));
          }
        }
        alive = __shfl_sync(0xffffffffu, alive, 0);
        if (!alive) break;
      }
    }
    if (lane == 0) {
      if (!alive && a.status != nullptr) atomicOr(a.status, PKV_DEV_WAIT_TIMEOUT);
      for (uint32_t i = it > stages ? it - stages : 0; i < it; ++i)  // copies in flight land first
        ptx::mbar_wait(full(i % stages), (i / stages) & 1u, kBulkWaitNs / 8);
    }
    return;
  }
  const int half = a.rot >> 1;
  const int nturn = kInter ? a.rot / VEC : half / VEC;
  const int units = nturn + (a.D - a.rot) / VEC;  // at most 32
  int L = 1;  // lanes of a head
  while (L < units) L *= 2;
  const uint32_t group = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << (lane & ~(L - 1));
  const int u = threadIdx.x & (L - 1), h0 = threadIdx.x / L, hstep = kBulkWarps * 32 / L;
  const bool turns = u < nturn, mine = u < units;
  const int at = turns ? u * VEC : a.rot + (u - nturn) * VEC;  // the lane's piece
  auto weight = [&](const void* w, int d, float (&y)[VEC]) {
    if (a.w_f32) {
      const Pack<float, VEC> x = *reinterpret_cast<const Pack<float, VEC>*>(static_cast<const float*>(w) + d);
#pragma unroll
      for (int i = 0; i < VEC; ++i) y[i] = x.x[i];
    } else {
      widen_piece(*reinterpret_cast<const P*>(static_cast<const T*>(w) + d), y);
    }
  };
  uint32_t it = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += step, ++it) {
    const uint32_t st = it % stages;
    if (!__all_sync(0xffffffffu, ptx::mbar_wait(full(st), (it / stages) & 1u, kBulkWaitNs))) {
      if (lane == 0 && a.status != nullptr) atomicOr(a.status, PKV_DEV_WAIT_TIMEOUT);
      return;
    }
    const uint8_t* const stage = bulk_smem + st * sh.stage;
    const int32_t slot = *reinterpret_cast<const int32_t*>(stage + sh.stage - 16);
    const bool write = slot >= 0 && static_cast<int64_t>(slot) < static_cast<int64_t>(a.NB) * a.B;
    const int32_t block = !write ? 0 : ((a.B & (a.B - 1)) == 0 ? slot >> (31 - __clz(a.B)) : slot / a.B);
    const int64_t row0 =
        (static_cast<int64_t>(block) * a.Hkv * a.B + (write ? slot - block * a.B : 0)) * a.D;
    const int64_t head = static_cast<int64_t>(a.B) * a.D;
    const float* const table = reinterpret_cast<const float*>(stage + sh.q + 2 * sh.k);
    float c[kAng], s[kAng];
    if (turns) {
      const int i0 = u * kAng;
      if (a.axes == 1) {
        const Pack<float, kAng> pc = *reinterpret_cast<const Pack<float, kAng>*>(table + i0);
        const Pack<float, kAng> ps = *reinterpret_cast<const Pack<float, kAng>*>(table + half + i0);
#pragma unroll
        for (int i = 0; i < kAng; ++i) c[i] = pc.x[i], s[i] = ps.x[i];
      } else {
#pragma unroll
        for (int i = 0; i < kAng; ++i) {
          const uint32_t x = (a.axis_bits[(i0 + i) >> 4] >> (2 * ((i0 + i) & 15))) & 3u;
          c[i] = table[x * a.rot + i0 + i];
          s[i] = table[x * a.rot + half + i0 + i];
        }
      }
    }
    auto some_heads = [&](const T* src, int H, T* dst, int64_t apart, const void* w) {
      float w1[VEC], w2[VEC];  // (loaded once a token for all heads; they stay in L1)
#pragma unroll
      for (int i = 0; i < VEC; ++i) w1[i] = w2[i] = 1.f;
      if (kNorm && w != nullptr && mine) {
        weight(w, at, w1);
        if (!kInter && turns) weight(w, at + half, w2);
      }
      for (int h = h0; h < H; h += hstep) {
        const T* const from = src + static_cast<int64_t>(h) * a.D;
        T* const to = dst + h * apart;
        P p1, p2;
        float x1[VEC], x2[VEC] = {};
        if (mine) {
          p1 = *reinterpret_cast<const P*>(from + at);
          widen_piece(p1, x1);
          if (!kInter && turns) {
            p2 = *reinterpret_cast<const P*>(from + at + half);
            widen_piece(p2, x2);
          }
        }
        if constexpr (kNorm) {
          float even = 0.f, odd = 0.f;
          if (mine) {
            add_squares<VEC>(x1, even, odd);
            if (!kInter && turns) add_squares<VEC>(x2, even, odd);
          }
          float sum = __fadd_rn(even, odd);
          for (int o = L >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(group, sum, o);
          const float r = inverse_root(sum, a.inv_d, a.eps);
          if (mine) {
            apply_norm<VEC>(x1, r, w1);
            if (!kInter && turns) apply_norm<VEC>(x2, r, w2);
          }
        }
        if (!mine) continue;
        if (turns)
          turn_piece<VEC, kInter>(x1, x2, c, s, kNorm, half,
                                  [&](int d, const float (&z)[VEC]) { store_as<T, VEC>(to + at + d, z); });
        else if (kNorm)
          store_as<T, VEC>(to + at, x1);
        else  // neither normed nor turned: its bits
          *reinterpret_cast<P*>(to + at) = p1;
      }
    };
    some_heads(reinterpret_cast<const T*>(stage), a.Hq, static_cast<T*>(a.q_out) + t * a.qo_stride,
               a.D, a.qw);
    if (write) {
      some_heads(reinterpret_cast<const T*>(stage + sh.q), a.Hkv, static_cast<T*>(a.kc) + row0, head,
                 a.kw);
      const uint4* const v = reinterpret_cast<const uint4*>(stage + sh.q + sh.k);  // copied
      const int per = a.D * static_cast<int>(sizeof(T)) / 16;
      for (int i = threadIdx.x; i < a.Hkv * per; i += kBulkWarps * 32) {
        const int g = i / per;
        reinterpret_cast<uint4*>(static_cast<T*>(a.vc) + row0 + g * head)[i - g * per] = v[i];
      }
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(empty(st));
  }
}

// Stages of whole tokens, if three or more fit half of an SM's shared memory.
bool bulk_shape(const NormArgs& a, BulkShape& sh) {
  const int64_t q = static_cast<int64_t>(a.Hq) * a.D * 2, k = static_cast<int64_t>(a.Hkv) * a.D * 2;
  const int64_t stage = q + 2 * k + static_cast<int64_t>(a.axes) * a.rot * 4 + 16;
  const int64_t room = 112 << 10;  // of the 227 KB, for two CTAs
  if (stage * 3 > room) return false;
  sh.q = static_cast<uint32_t>(q);
  sh.k = static_cast<uint32_t>(k);
  sh.stage = static_cast<uint32_t>(stage);
  sh.stages = static_cast<int32_t>(std::min<int64_t>(kBulkStages, room / stage));
  return true;
}

template <typename T, bool kInter, bool kNorm>
int launch_bulk(const NormArgs& a, const BulkShape& sh, int sms, cudaStream_t st) {
  static SmemOnce once;
  const int rc = allow_dynamic_smem(
      once, reinterpret_cast<const void*>(norm_rotary_bulk_kernel<T, kInter, kNorm>), 112 << 10);
  if (rc != PKV_OK) return rc;
  const int64_t ctas = std::min<int64_t>(a.T, 2 * sms);
  norm_rotary_bulk_kernel<T, kInter, kNorm>
      <<<static_cast<unsigned>(ctas), kBulkThreads, sh.stage * sh.stages, st>>>(a, sh);
  PKV_CUDA(cudaGetLastError());
  return PKV_OK;
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
  if constexpr (kCodes == 0 && sizeof(T) == 2) {
    BulkShape shape;
    if (whole && strides && a.w_wide && !a.per_head && a.T >= kBulkTokens * sms &&
        bulk_shape(a, shape)) {
      if (interleaved)
        return a.norm ? launch_bulk<T, true, true>(a, shape, sms, st)
                      : launch_bulk<T, true, false>(a, shape, sms, st);
      return a.norm ? launch_bulk<T, false, true>(a, shape, sms, st)
                    : launch_bulk<T, false, false>(a, shape, sms, st);
    }
  }
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
  if (whole && interleaved)
    norm_rotary_kernel<T, W, true, kCodes, W == 4 ? 2 : 1><<<grid, threads, 0, st>>>(a);
  else if (whole)
    norm_rotary_kernel<T, W, false, kCodes, W == 4 ? 2 : 1><<<grid, threads, 0, st>>>(a);
  else if (interleaved)
    norm_rotary_kernel<T, 2, true, kCodes, 4><<<grid, threads, 0, st>>>(a);
  else
    norm_rotary_kernel<T, 1, false, kCodes, 8><<<grid, threads, 0, st>>>(a);
  PKV_CUDA(cudaGetLastError());
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_norm_rotary_write(
    int32_t codes, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
    int64_t v_stride, const void* q_weight, const void* k_weight, int32_t weight_dtype,
    int32_t weight_per_head, float eps, const int32_t* positions, const int32_t* pair_axes,
    int32_t num_axes, const float* table, int32_t max_positions, int32_t rotary_dim,
    int32_t interleaved, const int32_t* slot_mapping, int32_t num_tokens, void* k_cache,
    void* v_cache, const float* k_scale, const float* v_scale, int32_t num_blocks,
    int32_t num_q_heads, int32_t num_kv_heads, int32_t block_size, int32_t head_dim, void* q_out,
    int64_t q_out_stride, int32_t* status, int32_t dtype, void* stream) {
  PKV_REQUIRE(codes == 0 || codes == PKV_FP8_E4M3 || codes == PKV_INT8, PKV_ERR_DTYPE,
              "cache code %d is not 0, PKV_FP8_E4M3 or PKV_INT8", codes);
  RotaryArgs base;
  int rc = rotary_args(codes, q, q_stride, k, k_stride, v, v_stride, positions, table,
                       max_positions, rotary_dim, interleaved, slot_mapping, num_tokens, k_cache,
                       v_cache, k_scale, v_scale, num_blocks, num_q_heads, num_kv_heads,
                       block_size, head_dim, q_out, q_out_stride, status, dtype, base);
  if (rc != PKV_OK) return rc;
  PKV_REQUIRE(std::isfinite(eps), PKV_ERR_INVALID_ARG, "eps must be finite (negative: no norm)");
  const bool norm = eps >= 0.f;
  PKV_REQUIRE(norm || (!q_weight && !k_weight), PKV_ERR_INVALID_ARG,
              "weights without a norm (eps is negative)");
  PKV_REQUIRE(weight_dtype == dtype || weight_dtype == PKV_F32, PKV_ERR_DTYPE,
              "weights have q's dtype or f32 (dtype %d)", weight_dtype);
  PKV_REQUIRE(num_axes >= 1 && num_axes <= kMaxAxes, PKV_ERR_UNSUPPORTED,
              "num_axes %d outside [1, %d]", num_axes, kMaxAxes);
  PKV_REQUIRE(num_axes == 1 || pair_axes != nullptr, PKV_ERR_INVALID_ARG,
              "several axes need pair_axes");
  const int welt = element_bytes(weight_dtype);
  PKV_REQUIRE(aligned(q_weight, welt) && aligned(k_weight, welt), PKV_ERR_INVALID_ARG,
              "a weight is not aligned to its element");
  NormArgs a{};
  static_cast<RotaryArgs&>(a) = base;
  a.qw = q_weight;
  a.kw = k_weight;
  a.eps = eps;
  a.inv_d = 1.f / static_cast<float>(head_dim);
  a.norm = norm;
  a.axes = num_axes;
  a.per_head = weight_per_head != 0;
  a.w_f32 = weight_dtype == PKV_F32;
  if (num_axes > 1) {
    for (int i = 0; i < rotary_dim / 2; ++i) {
      PKV_REQUIRE(pair_axes[i] >= 0 && pair_axes[i] < num_axes, PKV_ERR_INVALID_ARG,
                  "axis %d of pair %d outside [0, %d)", pair_axes[i], i, num_axes);
      a.axis_bits[i / 16] |= static_cast<uint32_t>(pair_axes[i]) << (2 * (i % 16));
    }
  }
  if (num_tokens == 0) return ok();
  cudaStream_t st = static_cast<cudaStream_t>(stream);
#define PKV_NORM(C)                                                            \
  rc = dtype == PKV_F32   ? launch_norm<float, C>(a, interleaved != 0, st)     \
       : dtype == PKV_F16 ? launch_norm<__half, C>(a, interleaved != 0, st)    \
                          : launch_norm<__nv_bfloat16, C>(a, interleaved != 0, st)
  if (codes == 0) PKV_NORM(0);
  else if (codes == PKV_FP8_E4M3) PKV_NORM(1);
  else PKV_NORM(2);
#undef PKV_NORM
  return rc == PKV_OK ? ok() : rc;
}
