// Norms of q and k for each head, rotary positions and the cache write: the entry point, and the
// kernels of caches of q's own type.
#include <cmath>

#include "norm_rotary.cuh"

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
  rc = codes == 0 ? launch_norm_of<0>(a, dtype, interleaved != 0, st)
                  : norm_rotary_8bit(a, codes, dtype, interleaved != 0, st);
  return rc == PKV_OK ? ok() : rc;
}
