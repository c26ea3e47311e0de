// Decode attention that also accumulates attention weights, for eviction by use.
//
// Besides out[s, h, :], every cached token's weight, summed over the query heads of its
// KV group, is added to a running sum:
//   sums[s, g, p] += sum_{h of group g} softmax_p(scale * q[s, h] . K[slot(p), g]),  p < t.
// A weight needs the log-sum-exp of its whole context, which the attention's single pass
// over K and V knows only at its end.  So that pass (decode_attention.cu, kWeights) leaves
// the fp32 scores behind, 4 bytes per token and query head beside the 4 * head_dim bytes
// (16-bit caches) of the token's K and V per KV head, and the kernel here turns them into
// weights: w = 2^(x - lse), x and lse in log2 units.  Reading K a second time instead
// would cost half of the K and V bytes again; the scores cost 4 G bytes twice, an eighth
// of them at G = 8 and head_dim 128.
//
// The kernel below reads the scores once, and reads and writes the sums once.  Most scores come
// from L2, where the attention's stores ask to be kept ahead of the K and V that stream
// through, and a line that has been read is dropped: nothing of it need go to memory.  70B
// shape (256 sequences, 451,896 tokens, 1.85 GB of K and V, 116 MB of scores): both kernels 332
// us, of which the attention without the weights takes 286; 13B shape (509 MB, 4 MB) 95 of 87;
// 8 sequences to 131,072 tokens over an fp8 cache (1.75 GB, 219 MB of scores, more than L2
// holds) 384 of 281.
// Every sum belongs to one thread and its heads are added in order: no atomics, the same
// bits on every run.
#include <mutex>

#define PKV_DECODE_TEMPLATES_ONLY
#include "decode_attention.cu"

namespace pkv {
namespace {

constexpr int kSumThreads = 256;
constexpr int kSumUnroll = 4;  // tokens a lane has in flight

struct SumArgs {
  const float* scores;
  const float* lse;
  const int32_t* steps;
  const int32_t* context_lens;
  float* sums;
  int32_t* status;
  int32_t S, Hkv, limit, cols;  // limit: positions a block table holds
  int32_t score_steps;          // steps that scores has room for
};

// cursor_at, by a warp: the sequence is looked for among 32 places a round, one a lane.
__device__ __forceinline__ Cursor warp_cursor_at(const int32_t* pre, int S, int Hkv, int f) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = S;  // pre[lo] <= f < pre[hi]
  while (hi - lo > 1) {
    const int stride = (hi - lo + 31) / 32, at = lo + lane * stride;
    const bool below = at < hi && pre[at] <= f;  // true for lanes 0 .. n - 1
    const int n = __popc(__ballot_sync(0xffffffffu, below));
    lo += (n - 1) * stride;
    hi = min(hi, lo + stride);
  }
  Cursor c;
  c.s = lo;
  const int r = f - pre[lo];
  c.nb = (pre[lo + 1] - pre[lo]) / Hkv;
  c.g = r / c.nb;
  c.j = r - c.g * c.nb;
  return c;
}

// A warp walks its run of the flat step list unit by unit: a unit's tokens, scores and sums
// are contiguous, its G log-sum-exps stay in registers.
template <int G>
__global__ void __launch_bounds__(kSumThreads) weight_sums_kernel(const SumArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int warps = gridDim.x * (kSumThreads / 32);
  const int gw = blockIdx.x * (kSumThreads / 32) + (threadIdx.x >> 5);
  const int total = a.steps[a.S];
  if (total > a.score_steps) return;  // reported by the attention, which left no scores
  const int per = (total + warps - 1) / warps;
  if (static_cast<int64_t>(gw) * per >= total) return;
  int f = gw * per;
  const int f1 = total - f < per ? total : f + per;
  Cursor c = warp_cursor_at(a.steps, a.S, a.Hkv, f);
  while (f < f1) {
    const int j1 = min(c.nb, c.j + (f1 - f));  // steps c.j .. j1 - 1 of unit (c.s, c.g)
    int end = j1 * kTok;                       // positions in the context
    if (j1 == c.nb) {
      end = min(a.context_lens[c.s], a.limit);
      if (end > a.cols && lane == 0) atomicOr(a.status, PKV_DEV_BAD_CONTEXT_LEN);
    }
    const int n = min(end, a.cols) - c.j * kTok;
    const int64_t unit = static_cast<int64_t>(c.s) * a.Hkv + c.g;
    const float* const x = a.scores + static_cast<int64_t>(f) * (kTok * G);
    float* const sums = a.sums + unit * a.cols + c.j * kTok;
    float lse[G];
#pragma unroll
    for (int h = 0; h < G; ++h) lse[h] = a.lse[unit * G + h];
    for (int t = lane; t < n; t += 32 * kSumUnroll) {
      float v[kSumUnroll][G], old[kSumUnroll];
#pragma unroll
      for (int u = 0; u < kSumUnroll; ++u) {
        if (t + 32 * u < n) {
          const float* const row = x + static_cast<int64_t>(t + 32 * u) * G;
          if constexpr (G % 4 == 0) {
#pragma unroll
            for (int h = 0; h < G; h += 4) {
              const float4 y = __ldcs(reinterpret_cast<const float4*>(row + h));
              v[u][h] = y.x;
              v[u][h + 1] = y.y;
              v[u][h + 2] = y.z;
              v[u][h + 3] = y.w;
            }
          } else {
#pragma unroll
            for (int h = 0; h < G; ++h) v[u][h] = __ldcs(row + h);
          }
          old[u] = sums[t + 32 * u];
        }
      }
#pragma unroll
      for (int u = 0; u < kSumUnroll; ++u) {
        if (t + 32 * u < n) {
          float w = 0.f;
#pragma unroll
          for (int h = 0; h < G; ++h) w += exp2f(v[u][h] - lse[h]);
          sums[t + 32 * u] = old[u] + w;
        }
      }
    }
    // The scores are not read again: lines still in L2 need not be written to memory.
    __syncwarp();
    const uintptr_t s0 = reinterpret_cast<uintptr_t>(x);
    const uintptr_t s1 = s0 + static_cast<uintptr_t>(j1 - c.j) * (kTok * G * sizeof(float));
    for (uintptr_t l = ((s0 + 127) & ~uintptr_t(127)) + 128 * lane; l + 128 <= s1; l += 128 * 32)
      ptx::discard_line(reinterpret_cast<const void*>(l));
    f += j1 - c.j;
    c.j = j1 - 1;
    advance(c, a.steps, a.S, a.Hkv);
  }
}

struct WeightsLayout {
  size_t steps, lse, scores, total;
  int32_t score_steps;
};

// The decode workspace, then what the weights need.  A sequence has at most ceil(max_blocks *
// block_size / 16) steps per KV head, and S of at most max_tokens (if not negative) together
// no more than max_tokens / 16 + S.
WeightsLayout weights_layout(int32_t S, int32_t MAXB, int32_t B, int32_t Hq, int32_t Hkv,
                             int32_t D, int32_t W, int64_t max_tokens) {
  WeightsLayout L;
  L.steps = round256(workspace_bytes_for(Hq / Hkv, D, W));
  L.lse = L.steps + round256((static_cast<size_t>(S) + 1) * sizeof(int32_t));
  L.scores = L.lse + round256(static_cast<size_t>(S) * Hq * sizeof(float));
  int64_t steps = S * ((static_cast<int64_t>(MAXB) * B + kTok - 1) / kTok);
  if (max_tokens >= 0 && max_tokens / kTok < steps - S) steps = max_tokens / kTok + S;
  L.total = L.scores + static_cast<size_t>(steps) * Hq * kTok * sizeof(float);
  steps *= Hkv;
  L.score_steps = steps < INT32_MAX ? static_cast<int32_t>(steps) : INT32_MAX;
  return L;
}

int weights_entry(HostArgs h, float* weight_sums, int32_t sums_cols, int64_t max_tokens = -1) {
  int W = 0;
  int rc = validate(h, &W);
  if (rc != PKV_OK) return rc;
  PKV_REQUIRE(sums_cols > 0, PKV_ERR_INVALID_ARG, "weight_sums must have columns");
  const WeightsLayout L =
      weights_layout(h.S, h.MAXB, h.block_size, h.Hq, h.Hkv, h.D, W, max_tokens);
  PKV_REQUIRE(h.workspace_bytes >= L.total, PKV_ERR_INVALID_ARG,
              "workspace of %zu bytes < %zu needed", h.workspace_bytes, L.total);
  if (h.S == 0) return ok();
  PKV_REQUIRE(weight_sums && aligned(weight_sums, 4), PKV_ERR_INVALID_ARG,
              "weight_sums is NULL or misaligned");
  char* ws = static_cast<char*>(h.workspace);
  h.steps = reinterpret_cast<int32_t*>(ws + L.steps);
  h.lse = reinterpret_cast<float*>(ws + L.lse);
  h.scores = reinterpret_cast<float*>(ws + L.scores);
  h.score_steps = L.score_steps;
  SumArgs a{};
  a.scores = h.scores;
  a.lse = h.lse;
  a.steps = h.steps;
  a.context_lens = h.context_lens;
  a.sums = weight_sums;
  a.status = reinterpret_cast<int32_t*>(ws);
  a.S = h.S;
  a.Hkv = h.Hkv;
  a.limit = h.MAXB * h.block_size;
  a.cols = sums_cols;
  a.score_steps = L.score_steps;
  int sms = 0, dev = 0;
  rc = device_sm_count(&sms, &dev);
  if (rc != PKV_OK) return rc;
  // eight CTAs on an SM (four: 70B shape 338 us, then 336 with eight), but no more warps than a batch
  // this wide can have steps
  const int64_t most = (static_cast<int64_t>(h.S) * h.Hkv *
                            ((static_cast<int64_t>(h.MAXB) * h.block_size + kTok - 1) / kTok) +
                        kSumThreads / 32 - 1) / (kSumThreads / 32);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(most < 8 * sms ? most : 8 * sms));
  cfg.blockDim = dim3(kSumThreads);
  cfg.stream = h.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // The two launches hand the scores over through the workspace: they are queued one behind
  // the other, whatever other host threads queue on the stream with the same workspace.
  static std::mutex queue;
  const std::lock_guard<std::mutex> both(queue);
  rc = dispatch<true>(h, W);
  if (rc != PKV_OK) return rc;
  switch (h.Hq / h.Hkv) {
    case 1: PKV_CUDA(cudaLaunchKernelEx(&cfg, weight_sums_kernel<1>, a)); break;
    case 2: PKV_CUDA(cudaLaunchKernelEx(&cfg, weight_sums_kernel<2>, a)); break;
    case 4: PKV_CUDA(cudaLaunchKernelEx(&cfg, weight_sums_kernel<4>, a)); break;
    default: PKV_CUDA(cudaLaunchKernelEx(&cfg, weight_sums_kernel<8>, a)); break;
  }
  return ok();
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_decode_weights_workspace_size_tokens(int32_t num_seqs, int32_t max_blocks_per_seq,
                                             int32_t block_size, int32_t num_q_heads,
                                             int32_t num_kv_heads, int32_t head_dim,
                                             int32_t dtype, int32_t num_warps,
                                             int64_t max_tokens, size_t* bytes) {
  PKV_REQUIRE(bytes != nullptr, PKV_ERR_INVALID_ARG, "bytes is NULL");
  PKV_REQUIRE(element_bytes(dtype) != 0, PKV_ERR_DTYPE, "unknown dtype %d", dtype);
  PKV_REQUIRE(num_seqs >= 0 && max_blocks_per_seq > 0 && block_size > 0, PKV_ERR_INVALID_ARG,
              "sizes must be positive (num_seqs >= 0)");
  PKV_REQUIRE(num_q_heads > 0 && num_kv_heads > 0 && num_q_heads % num_kv_heads == 0,
              PKV_ERR_INVALID_ARG, "bad head counts %d / %d", num_q_heads, num_kv_heads);
  PKV_REQUIRE(supported_head_dim(dtype, head_dim), PKV_ERR_UNSUPPORTED,
              "head_dim %d unsupported for dtype %d", head_dim, dtype);
  PKV_REQUIRE(num_warps >= 0, PKV_ERR_INVALID_ARG, "negative num_warps");
  int W = num_warps;
  if (W == 0) {
    W = default_warps(dtype, head_dim);
    if (W < 0) return W;
  }
  *bytes = weights_layout(num_seqs, max_blocks_per_seq, block_size, num_q_heads, num_kv_heads,
                          head_dim, W, max_tokens).total;
  return ok();
}

int pkv_decode_weights_workspace_size(int32_t num_seqs, int32_t max_blocks_per_seq,
                                      int32_t block_size, int32_t num_q_heads,
                                      int32_t num_kv_heads, int32_t head_dim, int32_t dtype,
                                      int32_t num_warps, size_t* bytes) {
  return pkv_decode_weights_workspace_size_tokens(num_seqs, max_blocks_per_seq, block_size,
                                                  num_q_heads, num_kv_heads, head_dim, dtype,
                                                  num_warps, -1, bytes);
}

int pkv_decode_attention_weights(const void* q, const void* k_cache, const void* v_cache,
                                 const int32_t* block_tables, int32_t max_blocks_per_seq,
                                 const int32_t* context_lens, int32_t num_seqs,
                                 int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                 int32_t block_size, int32_t num_blocks, float scale, void* out,
                                 float* weight_sums, int32_t sums_cols, void* workspace,
                                 size_t workspace_bytes, int32_t num_warps, int32_t dtype,
                                 void* stream) {
  return weights_entry(host_args(q, k_cache, v_cache, block_tables, max_blocks_per_seq,
                                 context_lens, num_seqs, num_q_heads, num_kv_heads, head_dim,
                                 block_size, num_blocks, scale, out, workspace, workspace_bytes,
                                 num_warps, dtype, stream),
                       weight_sums, sums_cols);
}

int pkv_decode_attention_weights_fp8(const void* q, const void* k_cache, const void* v_cache,
                                     const float* k_scale, const float* v_scale,
                                     const int32_t* block_tables, int32_t max_blocks_per_seq,
                                     const int32_t* context_lens, int32_t num_seqs,
                                     int32_t num_q_heads, int32_t num_kv_heads,
                                     int32_t head_dim, int32_t block_size, int32_t num_blocks,
                                     float scale, void* out, float* weight_sums,
                                     int32_t sums_cols, void* workspace, size_t workspace_bytes,
                                     int32_t num_warps, int32_t dtype, void* stream) {
  HostArgs h = host_args(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                         num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                         scale, out, workspace, workspace_bytes, num_warps, dtype, stream);
  h.codes = PKV_FP8_E4M3;
  h.k_scale = k_scale;
  h.v_scale = v_scale;
  return weights_entry(h, weight_sums, sums_cols);
}

int pkv_decode_attention_weights_int8(const void* q, const void* k_cache, const void* v_cache,
                                      const float* k_scale, const float* v_scale,
                                      const int32_t* block_tables, int32_t max_blocks_per_seq,
                                      const int32_t* context_lens, int32_t num_seqs,
                                      int32_t num_q_heads, int32_t num_kv_heads,
                                      int32_t head_dim, int32_t block_size, int32_t num_blocks,
                                      float scale, void* out, float* weight_sums,
                                      int32_t sums_cols, void* workspace,
                                      size_t workspace_bytes, int32_t num_warps, int32_t dtype,
                                      void* stream) {
  HostArgs h = host_args(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                         num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                         scale, out, workspace, workspace_bytes, num_warps, dtype, stream);
  h.codes = PKV_INT8;
  h.k_scale = k_scale;
  h.v_scale = v_scale;
  return weights_entry(h, weight_sums, sums_cols);
}

int pkv_decode_attention_weights_tokens(int32_t codes, const void* q, const void* k_cache,
                                        const void* v_cache, const float* k_scale,
                                        const float* v_scale, const int32_t* block_tables,
                                        int32_t max_blocks_per_seq, const int32_t* context_lens,
                                        int32_t num_seqs, int32_t num_q_heads,
                                        int32_t num_kv_heads, int32_t head_dim,
                                        int32_t block_size, int32_t num_blocks, float scale,
                                        void* out, float* weight_sums, int32_t sums_cols,
                                        int64_t max_tokens, void* workspace,
                                        size_t workspace_bytes, int32_t num_warps, int32_t dtype,
                                        void* stream) {
  PKV_REQUIRE(codes == 0 || codes == PKV_FP8_E4M3 || codes == PKV_INT8, PKV_ERR_DTYPE,
              "codes %d are not 0, PKV_FP8_E4M3 or PKV_INT8", codes);
  HostArgs h = host_args(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                         num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                         scale, out, workspace, workspace_bytes, num_warps, dtype, stream);
  h.codes = codes;
  h.k_scale = k_scale;
  h.v_scale = v_scale;
  return weights_entry(h, weight_sums, sums_cols, max_tokens);
}

}  // extern "C"
