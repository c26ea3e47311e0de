// Rotary positions of q and k, with k and v written into the paged cache.
//
// A head's first rotary_dim elements form pairs (x1, x2); pair i of a token at
// position p is turned by the angle p * f_i:
//   y1 = x1 cos - x2 sin,   y2 = x2 cos + x1 sin,
// so the dot product of a turned q and a turned k depends on the distance of their
// positions.  Half layout: pair i is elements i and i + rotary_dim / 2; interleaved
// layout: elements 2i and 2i + 1.  Elements from rotary_dim on pass through.  The
// turned q goes to q_out, the turned k and the v into their slots (the cache write of
// kv_ops.cu, quantised for 8-bit caches), so k is read once and written once.
//
// Arithmetic: fp32 with every product and sum rounded once (no contraction), then one
// rounding to q's type, or one quantisation straight from fp32 for an 8-bit cache: the
// results are those of the written formula, the same bits on every path.  cos and sin
// come from a table of fp32 values computed in 64 bits: an angle p * f_i near 131,072
// has only 2^-7 left of its fraction in fp32.
//
// Bound by memory: q, k, v read once, q_out and the cache rows written once.  A CTA takes a
// token, or some of its heads: a row of threads turns a head, each thread its 16 bytes (both
// halves' ones), and goes on to other heads with the cos and sin it has loaded once.  8,192
// tokens of 64 / 8 heads of 128 in bf16, 340 MB: 65 us, 5.2 TB/s; a 13B-shaped prompt, 505 MB,
// 80 us, 6.3 TB/s.  With an 8-bit cache the codes cost arithmetic: the first 67 us for 323 MB,
// 4,099 tokens of 32 / 8 heads 25.9 us for 94 MB (int8 24.3).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "rotary_common.cuh"

namespace pkv {
namespace {

// A thread's pieces of heads h0, h0 + step, ... < H of src [H, D], a few heads' loads ahead
// of put(h, x1, x2); two: there is a second piece, `half` elements on.
template <typename T, int VEC, bool kInter, typename Put>
__device__ __forceinline__ void each_head(const T* src, int H, int D, int h0, int step, int half,
                                          bool two, Put put) {
  using P = Pack<T, VEC>;
  constexpr int U = kInter ? 4 : 2;
  for (int h = h0; h < H; h += U * step) {
    P x1[U], x2[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h + u * step < H) {
        const T* const at = src + (h + u * step) * D;
        x1[u] = *reinterpret_cast<const P*>(at);
        if (!kInter && two) x2[u] = *reinterpret_cast<const P*>(at + half);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h + u * step < H) put(h + u * step, x1[u], x2[u]);
  }
}

// blockIdx.x < T: a token, its heads split over gridDim.y CTAs and the CTA's rows of threads;
// 8-bit caches: then V's windows, a.v_parts CTAs each.  VEC: elements a thread moves at once.
template <typename T, int VEC, bool kInter, int kCodes>
__global__ void __launch_bounds__(256, kCodes != 0 ? 4 : 3) rotary_write_kernel(const RotaryArgs a) {
  // a decode launch queued behind may start its prologue; it reads the caches and q_out, and
  // writes anything that this grid may still read, only after this grid has completed
  asm volatile("griddepcontrol.launch_dependents;");
  using P = Pack<T, VEC>;
  constexpr int kAng = kInter ? VEC / 2 : VEC;  // pairs a thread turns at once
  const int64_t t = blockIdx.x;
  if constexpr (kCodes != 0) {
    if (t >= a.T) {
      const int64_t i = (t - a.T) * gridDim.y + blockIdx.y;
      const int64_t window = i / a.v_parts;
      if (window * 16 < a.T)
        write_v8<T, VEC != 1, kCodes>(a, static_cast<int>(window),
                                      static_cast<int>(i - window * a.v_parts), a.v_parts);
      return;
    }
  }
  const int half = a.rot >> 1;
  const int nturn = kInter ? a.rot / VEC : half / VEC;  // turning units of a row, then passing ones
  const int u = threadIdx.x;

  const int32_t slot = __ldg(a.slots + t);
  const bool write = slot >= 0 && static_cast<int64_t>(slot) < static_cast<int64_t>(a.NB) * a.B;
  int32_t pos = __ldg(a.positions + t);
  if (pos < 0 || pos >= a.P) {
    if (a.status != nullptr && threadIdx.x == 0 && threadIdx.y == 0 && blockIdx.y == 0)
      atomicOr(a.status, PKV_DEV_BAD_POSITION);
    pos = pos < 0 ? 0 : a.P - 1;
  }
  const bool turns = u < nturn;
  float c[kAng], s[kAng];
  if (turns) {
    const float* row = a.table + static_cast<int64_t>(pos) * a.rot + u * kAng;
    const Pack<float, kAng> pc = *reinterpret_cast<const Pack<float, kAng>*>(row);
    const Pack<float, kAng> ps = *reinterpret_cast<const Pack<float, kAng>*>(row + half);
#pragma unroll
    for (int i = 0; i < kAng; ++i) {
      c[i] = pc.x[i];
      s[i] = ps.x[i];
    }
  }
  const int d = turns ? u * VEC : a.rot + (u - nturn) * VEC;  // first element of the unit
  const bool two = turns && !kInter;
  const int h0 = threadIdx.y + blockDim.y * blockIdx.y, step = blockDim.y * gridDim.y;
  // a turned piece, rounded to the type; a passing one keeps its bits (a NaN's too)
  auto turned = [&](T* dst, const P& x1, const P& x2) {
    if (turns) {
      float y1[VEC], y2[VEC];
      turn<T, VEC, kInter>(x1, x2, c, s, y1, y2);
      store_as<T, VEC>(dst, y1);
      if (!kInter) store_as<T, VEC>(dst + half, y2);
    } else {
      *reinterpret_cast<P*>(dst) = x1;
    }
  };
  T* const qo = static_cast<T*>(a.q_out) + t * a.qo_stride + d;
  each_head<T, VEC, kInter>(static_cast<const T*>(a.q) + t * a.q_stride + d, a.Hq, a.D, h0, step,
                            half, two, [&](int h, const P& x1, const P& x2) {
                              turned(qo + h * a.D, x1, x2);
                            });
  if (!write) return;
  const int32_t block = (a.B & (a.B - 1)) == 0 ? slot >> (31 - __clz(a.B)) : slot / a.B;
  const int32_t off = slot - block * a.B;
  const int64_t at = (static_cast<int64_t>(block) * a.Hkv * a.B + off) * a.D + d;  // head 0
  const int64_t head = static_cast<int64_t>(a.B) * a.D;
  each_head<T, VEC, kInter>(
      static_cast<const T*>(a.k) + t * a.k_stride + d, a.Hkv, a.D, h0, step, half, two,
      [&](int g, const P& x1, const P& x2) {
        if constexpr (kCodes == 0) {
          turned(static_cast<T*>(a.kc) + at + g * head, x1, x2);
        } else {
          float y1[VEC], y2[VEC];
          if (turns) {
            turn<T, VEC, kInter>(x1, x2, c, s, y1, y2);
          } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) y1[i] = widen(x1.x[i]);
          }
          uint8_t* const dst = static_cast<uint8_t*>(a.kc) + at + g * head;
          const Quotients by = quotients_by(__ldg(a.ks + g));
          store_codes<kCodes, VEC>(dst, y1, by);
          if (two) store_codes<kCodes, VEC>(dst + half, y2, by);
        }
      });
  if constexpr (kCodes == 0) {  // V rows, copied
    each_head<T, VEC, kInter>(static_cast<const T*>(a.v) + t * a.v_stride + d, a.Hkv, a.D, h0,
                              step, half, two, [&](int g, const P& x1, const P& x2) {
                                T* const dst = static_cast<T*>(a.vc) + at + g * head;
                                *reinterpret_cast<P*>(dst) = x1;
                                if (two) *reinterpret_cast<P*>(dst + half) = x2;
                              });
  }
}

struct Frequencies {
  double f[kMaxRotaryPairs];
};

// table[p, i] = m cos(p f_i), table[p, rot / 2 + i] = m sin(p f_i), angles in 64 bits.
__global__ void rotary_table_kernel(const __grid_constant__ Frequencies fr, double magnitude,
                                    int32_t half, int64_t total, float* table) {
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += stride) {
    const int64_t p = i / half;
    const int j = static_cast<int>(i - p * half);
    double s, c;
    sincos(static_cast<double>(p) * fr.f[j], &s, &c);
    table[p * 2 * half + j] = static_cast<float>(c * magnitude);
    table[p * 2 * half + half + j] = static_cast<float>(s * magnitude);
  }
}

template <typename T, int VEC, int kCodes>
void launch_layout(const RotaryArgs& a, bool interleaved, dim3 grid, dim3 threads,
                   cudaStream_t st) {
  if (interleaved) {
    // a thread's piece holds whole pairs
    constexpr int V = VEC < 2 ? 2 : VEC;
    rotary_write_kernel<T, V, true, kCodes><<<grid, threads, 0, st>>>(a);
  } else {
    rotary_write_kernel<T, VEC, false, kCodes><<<grid, threads, 0, st>>>(a);
  }
}

template <typename T, int kCodes>
int launch_typed(RotaryArgs a, bool interleaved, cudaStream_t st) {
  // 16-byte pieces where rotary_dim, the strides and the addresses allow them, else the
  // smallest that hold whole pairs (13B-shaped prompt 80 and 99 us, fp8 prompt 26 and 42)
  constexpr int W = 16 / sizeof(T);
  const int unit = interleaved ? W : 2 * W;
  const bool wide = a.rot % unit == 0 && a.D % W == 0 && a.q_stride % W == 0 &&
                    a.k_stride % W == 0 && a.v_stride % W == 0 && a.qo_stride % W == 0 &&
                    aligned(a.q, 16) && aligned(a.k, 16) && aligned(a.v, 16) &&
                    aligned(a.q_out, 16);
  int sms = 0, dev = 0;
  const int rc = device_sm_count(&sms, &dev);
  if (rc != PKV_OK) return rc;
  const int vec = wide ? W : (interleaved ? 2 : 1);
  const int units = (interleaved ? a.rot / vec : a.rot / (2 * vec)) + (a.D - a.rot) / vec;
  // a row's units side by side, as many rows as 128 threads hold (units < head_dim <= 256)
  const int rows = units < 128 ? 128 / units : 1;
  const dim3 threads(units, rows);
  // few tokens: their heads are spread over more CTAs until the SMs have a few each (one
  // token of 64 heads 2.5 us, 3.5 with one CTA; 64 tokens 2.8 and 3.6)
  int split = 1;
  while (split * rows < a.Hq && static_cast<int64_t>(a.T) * split < 4 * sms) split *= 2;
  int64_t columns = a.T;
  if (kCodes != 0) {
    // V's windows: an item a thread if the window is one run (more CTAs, for runs of single
    // tokens, were no faster: 4.4 us against 4.2 for 64 tokens)
    const int64_t windows = (a.T + 15) / 16;
    const int64_t items = static_cast<int64_t>(a.Hkv) * a.D / 2;  // of one run
    const int64_t parts = (items + units * rows - 1) / (units * rows);
    a.v_parts = static_cast<int32_t>(parts);
    columns += (windows * parts + split - 1) / split;
  }
  const dim3 grid(static_cast<unsigned>(columns), split);
  if (wide) launch_layout<T, W, kCodes>(a, interleaved, grid, threads, st);
  else launch_layout<T, 1, kCodes>(a, interleaved, grid, threads, st);
  PKV_CUDA(cudaGetLastError());
  return PKV_OK;
}

int rotary_entry(int32_t codes, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                 const void* v, int64_t v_stride, const int32_t* positions, const float* table,
                 int32_t max_positions, int32_t rotary_dim, int32_t interleaved,
                 const int32_t* slot_mapping, int32_t num_tokens, void* k_cache, void* v_cache,
                 const float* k_scale, const float* v_scale, int32_t num_blocks,
                 int32_t num_q_heads, int32_t num_kv_heads, int32_t block_size, int32_t head_dim,
                 void* q_out, int64_t q_out_stride, int32_t* status, int32_t dtype,
                 void* stream) {
  RotaryArgs a;
  int rc = rotary_args(codes, q, q_stride, k, k_stride, v, v_stride, positions, table,
                       max_positions, rotary_dim, interleaved, slot_mapping, num_tokens, k_cache,
                       v_cache, k_scale, v_scale, num_blocks, num_q_heads, num_kv_heads,
                       block_size, head_dim, q_out, q_out_stride, status, dtype, a);
  if (rc != PKV_OK) return rc;
  if (num_tokens == 0) return ok();
  cudaStream_t st = static_cast<cudaStream_t>(stream);
#define PKV_ROTARY(C)                                                                          \
  rc = dtype == PKV_F32   ? launch_typed<float, C>(a, interleaved != 0, st)         \
       : dtype == PKV_F16 ? launch_typed<__half, C>(a, interleaved != 0, st)        \
                          : launch_typed<__nv_bfloat16, C>(a, interleaved != 0, st)
  if (codes == 0) PKV_ROTARY(0);
  else if (codes == PKV_FP8_E4M3) PKV_ROTARY(1);
  else PKV_ROTARY(2);
#undef PKV_ROTARY
  return rc == PKV_OK ? ok() : rc;
}

}  // namespace

int rotary_args(int32_t codes, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                const void* v, int64_t v_stride, const int32_t* positions, const float* table,
                int32_t max_positions, int32_t rotary_dim, int32_t interleaved,
                const int32_t* slot_mapping, int32_t num_tokens, void* k_cache, void* v_cache,
                const float* k_scale, const float* v_scale, int32_t num_blocks,
                int32_t num_q_heads, int32_t num_kv_heads, int32_t block_size, int32_t head_dim,
                void* q_out, int64_t q_out_stride, int32_t* status, int32_t dtype, RotaryArgs& a) {
  PKV_REQUIRE(dtype == PKV_F32 || dtype == PKV_F16 || dtype == PKV_BF16, PKV_ERR_DTYPE,
              "dtype %d is not f32, f16 or bf16", dtype);
  PKV_REQUIRE(num_tokens >= 0 && num_blocks > 0 && num_q_heads > 0 && num_kv_heads > 0 &&
                  block_size > 0 && head_dim > 0,
              PKV_ERR_INVALID_ARG, "sizes must be positive (num_tokens >= 0)");
  PKV_REQUIRE(rotary_dim > 0 && rotary_dim % 2 == 0 && rotary_dim <= head_dim,
              PKV_ERR_INVALID_ARG, "rotary_dim %d must be even and in [2, head_dim %d]",
              rotary_dim, head_dim);
  PKV_REQUIRE(head_dim <= 2 * kMaxRotaryPairs, PKV_ERR_UNSUPPORTED, "head_dim %d above %d",
              head_dim, 2 * kMaxRotaryPairs);
  PKV_REQUIRE(num_q_heads <= 65535 && num_kv_heads <= 65535, PKV_ERR_UNSUPPORTED,
              "num_q_heads %d or num_kv_heads %d above 65535", num_q_heads, num_kv_heads);
  PKV_REQUIRE(max_positions > 0, PKV_ERR_INVALID_ARG, "max_positions must be positive");
  const int elt = element_bytes(dtype);
  if (codes != 0) {
    PKV_REQUIRE(block_size == 16, PKV_ERR_UNSUPPORTED, "8-bit caches use block_size 16, not %d",
                block_size);
    PKV_REQUIRE(head_dim % 16 == 0, PKV_ERR_INVALID_ARG, "head_dim must be a multiple of 16");
  }
  PKV_REQUIRE((static_cast<int64_t>(head_dim) * elt) % 16 == 0, PKV_ERR_INVALID_ARG,
              "head_dim * element size must be a multiple of 16 bytes");
  PKV_REQUIRE(static_cast<int64_t>(num_blocks) * block_size < (int64_t(1) << 31),
              PKV_ERR_INVALID_ARG, "num_blocks * block_size must be < 2^31");
  PKV_REQUIRE(q_stride >= static_cast<int64_t>(num_q_heads) * head_dim &&
                  k_stride >= static_cast<int64_t>(num_kv_heads) * head_dim &&
                  v_stride >= static_cast<int64_t>(num_kv_heads) * head_dim &&
                  q_out_stride >= static_cast<int64_t>(num_q_heads) * head_dim,
              PKV_ERR_INVALID_ARG, "a token stride is smaller than the token's row");
  a = RotaryArgs{};
  if (num_tokens == 0) return PKV_OK;
  PKV_REQUIRE(q && k && v && positions && table && slot_mapping && k_cache && v_cache && q_out &&
                  (codes == 0 || (k_scale && v_scale)),
              PKV_ERR_INVALID_ARG, "NULL pointer");
  PKV_REQUIRE(aligned(k_cache, 16) && aligned(v_cache, 16) && aligned(table, 16),
              PKV_ERR_INVALID_ARG, "caches and table must be 16-byte aligned");
  PKV_REQUIRE(aligned(q, elt) && aligned(k, elt) && aligned(v, elt) && aligned(q_out, elt) &&
                  aligned(positions, 4) && aligned(slot_mapping, 4) && aligned(status, 4) &&
                  aligned(k_scale, 4) && aligned(v_scale, 4),
              PKV_ERR_INVALID_ARG, "a pointer is not aligned to its element");
  // a pair of interleaved elements is moved at once
  PKV_REQUIRE(!interleaved || (q_stride % 2 == 0 && k_stride % 2 == 0 && v_stride % 2 == 0 &&
                               q_out_stride % 2 == 0 && aligned(q, 2 * elt) &&
                               aligned(k, 2 * elt) && aligned(v, 2 * elt) &&
                               aligned(q_out, 2 * elt)),
              PKV_ERR_INVALID_ARG, "interleaved pairs must be aligned to their two elements");
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  a.positions = positions;
  a.table = table;
  a.slots = slot_mapping;
  a.kc = k_cache;
  a.vc = v_cache;
  a.ks = k_scale;
  a.vs = v_scale;
  a.status = status;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.qo_stride = q_out_stride;
  a.T = num_tokens;
  a.Hq = num_q_heads;
  a.Hkv = num_kv_heads;
  a.D = head_dim;
  a.rot = rotary_dim;
  a.B = block_size;
  a.NB = num_blocks;
  a.P = max_positions;
  return PKV_OK;
}

}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_rotary_frequencies(int32_t rotary_dim, float base, int32_t scaling, float factor,
                           int32_t original_length, float low_turns, float high_turns,
                           double* inv_freq) {
  const double settings[4] = {base, factor, low_turns, high_turns};
  return pkv_rotary_frequencies_f64(rotary_dim, settings, scaling, original_length, inv_freq);
}

int pkv_rotary_frequencies_f64(int32_t rotary_dim, const double* settings, int32_t scaling,
                               int32_t original_length, double* inv_freq) {
  PKV_REQUIRE(settings != nullptr, PKV_ERR_INVALID_ARG, "settings is NULL");
  const double base = settings[0], factor = settings[1];
  const double low_turns = settings[2], high_turns = settings[3];
  PKV_REQUIRE(rotary_dim > 0 && rotary_dim % 2 == 0 && rotary_dim <= 2 * kMaxRotaryPairs,
              PKV_ERR_INVALID_ARG, "rotary_dim %d must be even and in [2, %d]", rotary_dim,
              2 * kMaxRotaryPairs);
  PKV_REQUIRE(inv_freq != nullptr, PKV_ERR_INVALID_ARG, "inv_freq is NULL");
  PKV_REQUIRE(std::isfinite(base) && base > 1.0, PKV_ERR_INVALID_ARG, "base must be above 1");
  PKV_REQUIRE(scaling >= PKV_ROTARY_PLAIN && scaling <= PKV_ROTARY_BANDS, PKV_ERR_INVALID_ARG,
              "unknown scaling %d", scaling);
  PKV_REQUIRE(scaling == PKV_ROTARY_PLAIN || (std::isfinite(factor) && factor >= 1.0),
              PKV_ERR_INVALID_ARG, "factor must be finite and at least 1");
  PKV_REQUIRE(scaling != PKV_ROTARY_BANDS ||
                  (original_length > 0 && std::isfinite(low_turns) && std::isfinite(high_turns) &&
                   low_turns >= 0.0 && high_turns > low_turns),
              PKV_ERR_INVALID_ARG,
              "bands need original_length > 0 and 0 <= low_turns < high_turns");
  const double pi = 3.14159265358979323846;
  double b = base;
  if (scaling == PKV_ROTARY_NTK && rotary_dim > 2)
    b *= std::pow(factor, rotary_dim / (rotary_dim - 2.0));
  for (int32_t i = 0; i < rotary_dim / 2; ++i) {
    double f = std::pow(b, -2.0 * i / rotary_dim);
    if (scaling == PKV_ROTARY_LINEAR) f /= factor;
    if (scaling == PKV_ROTARY_BANDS) {
      const double turns = original_length * f / (2.0 * pi);
      double t = (turns - low_turns) / (high_turns - low_turns);
      t = t < 0.0 ? 0.0 : (t > 1.0 ? 1.0 : t);
      f *= (1.0 - t) / factor + t;
    }
    inv_freq[i] = f;
  }
  return ok();
}

int pkv_rotary_table(const double* inv_freq, int32_t rotary_dim, float magnitude,
                     int32_t max_positions, float* table, void* stream) {
  PKV_REQUIRE(rotary_dim > 0 && rotary_dim % 2 == 0 && rotary_dim <= 2 * kMaxRotaryPairs,
              PKV_ERR_INVALID_ARG, "rotary_dim %d must be even and in [2, %d]", rotary_dim,
              2 * kMaxRotaryPairs);
  PKV_REQUIRE(max_positions > 0, PKV_ERR_INVALID_ARG, "max_positions must be positive");
  PKV_REQUIRE(inv_freq && table, PKV_ERR_INVALID_ARG, "NULL pointer");
  PKV_REQUIRE(aligned(table, 16), PKV_ERR_INVALID_ARG, "table must be 16-byte aligned");
  Frequencies fr{};
  const int32_t half = rotary_dim / 2;
  for (int32_t i = 0; i < half; ++i) fr.f[i] = inv_freq[i];
  const int64_t total = static_cast<int64_t>(max_positions) * half;
  int sms = 0, dev = 0;
  const int rc = device_sm_count(&sms, &dev);
  if (rc != PKV_OK) return rc;
  const int64_t want = (total + 255) / 256, cap = static_cast<int64_t>(sms) * 8;
  rotary_table_kernel<<<static_cast<int>(want < cap ? want : cap), 256, 0,
                        static_cast<cudaStream_t>(stream)>>>(
      fr, static_cast<double>(magnitude), half, total, table);
  PKV_CUDA(cudaGetLastError());
  return ok();
}

int pkv_rotary_write(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                     const void* v, int64_t v_stride, const int32_t* positions,
                     const float* table, int32_t max_positions, int32_t rotary_dim,
                     int32_t interleaved, const int32_t* slot_mapping, int32_t num_tokens,
                     void* k_cache, void* v_cache, int32_t num_blocks, int32_t num_q_heads,
                     int32_t num_kv_heads, int32_t block_size, int32_t head_dim, void* q_out,
                     int64_t q_out_stride, int32_t* status, int32_t dtype, void* stream) {
  return rotary_entry(0, q, q_stride, k, k_stride, v, v_stride, positions, table, max_positions,
                      rotary_dim, interleaved, slot_mapping, num_tokens, k_cache, v_cache,
                      nullptr, nullptr, num_blocks, num_q_heads, num_kv_heads, block_size,
                      head_dim, q_out, q_out_stride, status, dtype, stream);
}

int pkv_rotary_write_fp8(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                         const void* v, int64_t v_stride, const int32_t* positions,
                         const float* table, int32_t max_positions, int32_t rotary_dim,
                         int32_t interleaved, const int32_t* slot_mapping, int32_t num_tokens,
                         void* k_cache, void* v_cache, const float* k_scale,
                         const float* v_scale, int32_t num_blocks, int32_t num_q_heads,
                         int32_t num_kv_heads, int32_t block_size, int32_t head_dim, void* q_out,
                         int64_t q_out_stride, int32_t* status, int32_t dtype, void* stream) {
  return rotary_entry(PKV_FP8_E4M3, q, q_stride, k, k_stride, v, v_stride, positions, table,
                      max_positions, rotary_dim, interleaved, slot_mapping, num_tokens, k_cache,
                      v_cache, k_scale, v_scale, num_blocks, num_q_heads, num_kv_heads,
                      block_size, head_dim, q_out, q_out_stride, status, dtype, stream);
}

int pkv_rotary_write_int8(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                          const void* v, int64_t v_stride, const int32_t* positions,
                          const float* table, int32_t max_positions, int32_t rotary_dim,
                          int32_t interleaved, const int32_t* slot_mapping, int32_t num_tokens,
                          void* k_cache, void* v_cache, const float* k_scale,
                          const float* v_scale, int32_t num_blocks, int32_t num_q_heads,
                          int32_t num_kv_heads, int32_t block_size, int32_t head_dim,
                          void* q_out, int64_t q_out_stride, int32_t* status, int32_t dtype,
                          void* stream) {
  return rotary_entry(PKV_INT8, q, q_stride, k, k_stride, v, v_stride, positions, table,
                      max_positions, rotary_dim, interleaved, slot_mapping, num_tokens, k_cache,
                      v_cache, k_scale, v_scale, num_blocks, num_q_heads, num_kv_heads,
                      block_size, head_dim, q_out, q_out_stride, status, dtype, stream);
}

}  // extern "C"
