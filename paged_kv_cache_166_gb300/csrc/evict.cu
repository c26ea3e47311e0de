// Eviction from the paged cache by accumulated attention weight.
//
// Select: for every sequence s and KV head h, of the t cached tokens n = min(keep, t) stay:
// the first `first`, the last `recent`, and of those between the ones with the largest
// sums (ties: the lower position).  Their positions come out ascending, so the order of
// the tokens is kept and "recent" means the same after the next eviction.
// Gather: the kept tokens' K and V rows move to positions 0..n-1 of a new block table.
// The rows are copied into blocks that the sequence alone holds rather than moved within
// the old ones: those may be shared with other sequences (fork, common prefixes), and
// every row can then move at once.
//
// Select is exact: the m-th largest sum is found by its bits, most significant digits
// first (a histogram a digit), and the tokens above it, plus the lowest positions equal to
// it, are compacted with prefix counts.  A row of sums is read from memory once: a
// cluster of CTAs holds it in shared memory, one slice each, and adds its histograms over
// distributed shared memory.  Gather is a copy, bound by memory.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "quant8.cuh"

namespace cg = cooperative_groups;

namespace pkv {
namespace {

// ---- select ---------------------------------------------------------------------

constexpr int kDigitBins = 2048;  // 11, 11 and 10 bits of a key
constexpr int kPasses = 3;
constexpr int kMaxCluster = 8;

struct SelectArgs {
  const float* sums;
  const int32_t* context_lens;
  const int32_t* keep_lens;
  int32_t* kept;
  float* new_sums;
  int32_t* new_lens;
  int32_t* status;  // or NULL
  int32_t Hkv, cols, kept_cols, new_cols, first, recent;
  int32_t slots;  // floats of a row slice that shared memory holds
};

// Unsigned key in the order of the values: larger sum, larger key.  NaN counts as
// -infinity and -0 as +0.
__device__ __forceinline__ uint32_t key_of(float x) {
  uint32_t u = __float_as_uint(x);
  if (x != x) u = 0xff800000u;
  if (x == 0.f) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum of v over the block's threads; the block's total in *total.
template <int kThreads>
__device__ __forceinline__ int block_prefix(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // warp_sums may still be read from the call before
  if (lane == 31) warp_sums[w] = x;
  __syncthreads();
  int base = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    const int y = warp_sums[i];
    if (i < w) base += y;
    all += y;
  }
  *total = all;
  return base + x - v;
}

// One cluster per (sequence, KV head).
template <int kThreads>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const SelectArgs a) {
  extern __shared__ float slice_s[];
  __shared__ int hist[kPasses][kDigitBins];
  __shared__ int warp_sums[kThreads / 32];
  __shared__ int counts[2];        // this CTA's tokens above the threshold, and equal to it
  __shared__ int warp_gt[kThreads / 32], warp_eq[kThreads / 32];
  __shared__ uint32_t found_bin;
  __shared__ int found_above;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int64_t row = blockIdx.x / C;
  const int s = static_cast<int>(row / a.Hkv);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  int c = a.context_lens[s], n = a.keep_lens[s];
  bool bad = c < 0 || c > a.cols;
  c = min(max(c, 0), a.cols);
  n = min(max(n, 0), c);
  bad |= n > a.kept_cols || n > a.new_cols;
  n = min(n, min(a.kept_cols, a.new_cols));
  const bool lead = rank == 0 && tid == 0 && row % a.Hkv == 0;
  if (lead) {
    a.new_lens[s] = n;
    if (bad && a.status != nullptr) atomicOr(a.status, PKV_DEV_BAD_CONTEXT_LEN);
  }
  const int r = min(a.recent, n), f = min(a.first, n - r), m = n - r - f;
  const int M = c - r - f;  // candidates: positions f .. f + M - 1, m of which stay
  const float* const sums = a.sums + row * a.cols;
  int32_t* const kept = a.kept + row * a.kept_cols;
  float* const out = a.new_sums + row * a.new_cols;

  // this CTA's slice of the candidates
  const int per = (M + C - 1) / C;
  const int lo = f + min(M, rank * per), len = max(0, min(per, f + M - lo));
  const float* vals = sums + lo;
  if (len <= a.slots) {
    for (int i = tid; i < len; i += kThreads) slice_s[i] = sums[lo + i];
    vals = slice_s;
  }
  for (int i = tid; i < kPasses * kDigitBins; i += kThreads) (&hist[0][0])[i] = 0;
  if (tid < 2) counts[tid] = 0;
  // the ends that stay whatever their sums
  for (int i = rank * kThreads + tid; i < f + r; i += C * kThreads) {
    const int j = i < f ? i : n - r + (i - f), p = i < f ? i : c - r + (i - f);
    kept[j] = p;
    out[j] = sums[p];
  }
  __syncthreads();

  // The threshold: the m-th largest key, digit by digit; `above` keys are larger.
  uint32_t prefix = 0;
  int above = 0;
  if (m > 0 && m < M) {
    int shift = 32;
    for (int pass = 0; pass < kPasses; ++pass) {
      const int bits = pass < 2 ? 11 : 10;
      const uint32_t fixed = shift == 32 ? 0u : ~0u << shift;
      shift -= bits;
      for (int i = tid; i < len; i += kThreads) {
        const uint32_t k = key_of(vals[i]);
        if ((k & fixed) == prefix) atomicAdd(&hist[pass][(k >> shift) & ((1u << bits) - 1)], 1);
      }
      cluster.sync();
      // bins from the top: thread t holds those from (kThreads - 1 - t) * kPer on
      constexpr int kPer = kDigitBins / kThreads;
      const int b0 = (kThreads - 1 - tid) * kPer;
      int n_bin[kPer], sum = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        int v = 0;
        for (int q = 0; q < C; ++q) v += cluster.map_shared_rank(&hist[pass][0], q)[b0 + i];
        n_bin[i] = v;
        sum += v;
      }
      int total;
      int before = above + block_prefix<kThreads>(sum, warp_sums, &total);
#pragma unroll
      for (int i = kPer - 1; i >= 0; --i) {
        if (before < m && before + n_bin[i] >= m) {
          found_bin = static_cast<uint32_t>(b0 + i);
          found_above = before;
        }
        before += n_bin[i];
      }
      __syncthreads();
      prefix |= found_bin << shift;
      above = found_above;
      __syncthreads();
    }
  }
  // m == M: everything is above a threshold of 0 (no key is 0); m == 0: nothing stays
  const bool all = m == M;
  const int ties = all ? 0 : m - above;

  // Compaction, ascending: warps take consecutive parts of the slice.
  constexpr int kWarps = kThreads / 32;
  const int part = ((len + kWarps - 1) / kWarps + 31) & ~31;
  const int p0 = min(len, warp * part), p1 = min(len, p0 + part);
  int gt = 0, eq = 0;
  if (m > 0) {
    for (int i = p0 + lane; i < p1; i += 32) {
      const uint32_t k = key_of(vals[i]);
      gt += all || k > prefix;
      eq += !all && k == prefix;
    }
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    warp_gt[warp] = gt;
    warp_eq[warp] = eq;
    atomicAdd(&counts[0], gt);
    atomicAdd(&counts[1], eq);
  }
  cluster.sync();
  if (m > 0) {
    int gt0 = 0, eq0 = 0;
    for (int q = 0; q < rank; ++q) {
      const int* cq = cluster.map_shared_rank(&counts[0], q);
      gt0 += cq[0];
      eq0 += cq[1];
    }
    for (int w = 0; w < warp; ++w) {
      gt0 += warp_gt[w];
      eq0 += warp_eq[w];
    }
    for (int i0 = p0; i0 < p1; i0 += 32) {
      const int i = i0 + lane;
      const float x = i < p1 ? vals[i] : 0.f;
      const uint32_t k = key_of(x);
      const bool g = i < p1 && (all || k > prefix), e = i < p1 && !all && k == prefix;
      const uint32_t mg = __ballot_sync(0xffffffffu, g), me = __ballot_sync(0xffffffffu, e);
      const uint32_t below = (1u << lane) - 1;
      const int ng = gt0 + __popc(mg & below), ne = eq0 + __popc(me & below);
      if (g || (e && ne < ties)) {
        const int j = f + ng + min(ne, ties);
        kept[j] = lo + i;
        out[j] = x;
      }
      gt0 += __popc(mg);
      eq0 += __popc(me);
    }
  }
  cluster.sync();  // no CTA leaves while others read its counts
}

// ---- gather ---------------------------------------------------------------------

constexpr int kGatherThreads = 256;
constexpr int kGatherTokens = 64;  // kept tokens of one CTA

struct GatherArgs {
  uint4* kc;
  uint4* vc;
  const int32_t* tables;
  const int32_t* kept;
  const int32_t* new_lens;
  const int32_t* new_tables;
  int32_t* status;  // or NULL
  int32_t Hkv, B, NB, MAXB, NEWB, kept_cols, row_vecs, D;
};

// Slot row (in rows of the cache) of position p of a table row, or -1.
__device__ __forceinline__ int64_t cache_row(const int32_t* table, int max_blocks, int p, int B,
                                             int NB, int Hkv, int h) {
  if (p < 0 || p >= max_blocks * B) return -1;
  const int j = p / B;
  const int b = __ldg(table + j);
  if (b < 0 || b >= NB) return -1;
  return (static_cast<int64_t>(b) * Hkv + h) * B + (p - j * B);
}

// grid: (pieces of kGatherTokens kept tokens, KV heads, sequences).  kV: the V rows are
// laid out like the K rows (16- and 32-bit caches).
template <bool kV>
__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(const GatherArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int s = blockIdx.z, h = blockIdx.y;
  const int n = min(max(a.new_lens[s], 0), a.kept_cols);
  const int j0 = blockIdx.x * kGatherTokens, j1 = min(n, j0 + kGatherTokens);
  if (j0 >= n) return;
  const int rows = kGatherThreads / a.row_vecs;
  const int v = threadIdx.x % a.row_vecs, r = threadIdx.x / a.row_vecs;
  if (r >= rows) return;
  const int32_t* const kept = a.kept + (static_cast<int64_t>(s) * a.Hkv + h) * a.kept_cols;
  const int32_t* const table = a.tables + static_cast<int64_t>(s) * a.MAXB;
  const int32_t* const fresh = a.new_tables + static_cast<int64_t>(s) * a.NEWB;
  constexpr int U = 4;
  for (int j = j0 + r; j < j1; j += U * rows) {
    int64_t dst[U];
    uint4 kx[U], vx[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int ju = j + u * rows;
      dst[u] = -1;
      if (ju < j1) {
        const int64_t src = cache_row(table, a.MAXB, __ldg(kept + ju), a.B, a.NB, a.Hkv, h);
        dst[u] = cache_row(fresh, a.NEWB, ju, a.B, a.NB, a.Hkv, h);
        if (src < 0 || dst[u] < 0) {
          if (a.status != nullptr && v == 0) atomicOr(a.status, PKV_DEV_BAD_BLOCK_ID);
          dst[u] = -1;
        } else {
          kx[u] = a.kc[src * a.row_vecs + v];
          if constexpr (kV) vx[u] = a.vc[src * a.row_vecs + v];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (dst[u] >= 0) {
        a.kc[dst[u] * a.row_vecs + v] = kx[u];
        if constexpr (kV) a.vc[dst[u] * a.row_vecs + v] = vx[u];
      }
    }
  }
}

// V of 8-bit caches: tiles [D x 16 bytes], a token one byte of every row.  A CTA fills
// one new tile, a thread whole 16-byte rows of it; consecutive kept tokens often come
// from one old tile, whose row is then read once.
__global__ void __launch_bounds__(kGatherThreads) evict_gather_v8_kernel(const GatherArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ int64_t src_tile[16];
  __shared__ int src_byte[16];
  const int s = blockIdx.z, h = blockIdx.y;
  const int n = min(max(a.new_lens[s], 0), a.kept_cols);
  const int j0 = blockIdx.x * 16;
  if (j0 >= n) return;
  const int count = min(16, n - j0);
  const int64_t to = cache_row(a.new_tables + static_cast<int64_t>(s) * a.NEWB, a.NEWB, j0, 16,
                               a.NB, a.Hkv, h);
  if (threadIdx.x < 16) {
    int64_t row = -1;
    if (static_cast<int>(threadIdx.x) < count)
      row = cache_row(a.tables + static_cast<int64_t>(s) * a.MAXB, a.MAXB,
                      __ldg(a.kept + (static_cast<int64_t>(s) * a.Hkv + h) * a.kept_cols + j0 +
                            threadIdx.x),
                      16, a.NB, a.Hkv, h);
    src_tile[threadIdx.x] = row < 0 ? -1 : row >> 4;
    src_byte[threadIdx.x] = row < 0 ? 0 : fp8_v_pos(static_cast<int>(row & 15));
  }
  __syncthreads();
  if (to < 0) return;  // reported by the K rows' kernel
  for (int d = threadIdx.x; d < a.D; d += kGatherThreads) {
    uint4* const dst = a.vc + (to >> 4) * a.D + d;
    // bytes of tokens that do not move (past n, or from a bad block) stay as they are
    uint4 w = count < 16 ? *dst : make_uint4(0u, 0u, 0u, 0u);
    uint8_t* const wb = reinterpret_cast<uint8_t*>(&w);
    int64_t have = -1;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      const int64_t tile = src_tile[t];
      if (tile < 0) continue;
      if (tile != have) {
        x = a.vc[tile * a.D + d];
        have = tile;
      }
      const int b = src_byte[t];
      const uint32_t word = (b >> 2) == 0 ? x.x : (b >> 2) == 1 ? x.y : (b >> 2) == 2 ? x.z : x.w;
      const int at = t < 8 ? 4 * (t >> 1) + (t & 1) : 4 * ((t - 8) >> 1) + 2 + (t & 1);
      wb[at] = static_cast<uint8_t>(word >> (8 * (b & 3)));
    }
    *dst = w;
  }
}

template <int kThreads>
int launch_select(const SelectArgs& a0, int64_t rows, int cluster, int slice, cudaStream_t st) {
  SelectArgs a = a0;
  a.slots = slice;
  const size_t smem = static_cast<size_t>(slice) * sizeof(float);
  PKV_CUDA(cudaFuncSetAttribute(evict_select_kernel<kThreads>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(smem)));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  PKV_CUDA(cudaLaunchKernelEx(&cfg, evict_select_kernel<kThreads>, a));
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_evict_select(const float* weight_sums, int32_t sums_cols, const int32_t* context_lens,
                     const int32_t* keep_lens, int32_t num_seqs, int32_t num_kv_heads,
                     int32_t first, int32_t recent, int32_t* kept, int32_t kept_cols,
                     float* new_sums, int32_t new_cols, int32_t* new_lens, int32_t* status,
                     void* stream) {
  PKV_REQUIRE(num_seqs >= 0 && num_kv_heads > 0 && sums_cols > 0 && kept_cols > 0 && new_cols > 0,
              PKV_ERR_INVALID_ARG, "sizes must be positive (num_seqs >= 0)");
  PKV_REQUIRE(first >= 0 && recent >= 0, PKV_ERR_INVALID_ARG, "negative first or recent");
  PKV_REQUIRE(static_cast<int64_t>(num_seqs) * num_kv_heads * kMaxCluster < (int64_t(1) << 31),
              PKV_ERR_UNSUPPORTED, "num_seqs * num_kv_heads * %d >= 2^31", kMaxCluster);
  if (num_seqs == 0) return ok();
  PKV_REQUIRE(weight_sums && context_lens && keep_lens && kept && new_sums && new_lens,
              PKV_ERR_INVALID_ARG, "NULL pointer");
  PKV_REQUIRE(aligned(weight_sums, 4) && aligned(context_lens, 4) && aligned(keep_lens, 4) &&
                  aligned(kept, 4) && aligned(new_sums, 4) && aligned(new_lens, 4) &&
                  aligned(status, 4),
              PKV_ERR_INVALID_ARG, "a pointer is not 4-byte aligned");
  PKV_REQUIRE(weight_sums != new_sums && context_lens != new_lens, PKV_ERR_INVALID_ARG,
              "new_sums and new_lens must not be the inputs");
  SelectArgs a{};
  a.sums = weight_sums;
  a.context_lens = context_lens;
  a.keep_lens = keep_lens;
  a.kept = kept;
  a.new_sums = new_sums;
  a.new_lens = new_lens;
  a.status = status;
  a.Hkv = num_kv_heads;
  a.cols = sums_cols;
  a.kept_cols = kept_cols;
  a.new_cols = new_cols;
  a.first = first;
  a.recent = recent;
  const int64_t rows = static_cast<int64_t>(num_seqs) * num_kv_heads;
  // Short rows: one small CTA each.  Long ones: a slice of at most 16,384 sums (64 KB, so
  // that three CTAs share an SM) a CTA, up to eight CTAs; what does not fit then is read
  // from memory once a pass instead.
  int rc;
  if (sums_cols <= 2048) {
    rc = launch_select<128>(a, rows, 1, sums_cols, static_cast<cudaStream_t>(stream));
  } else {
    int cluster = 1;
    while (cluster < kMaxCluster && static_cast<int64_t>(cluster) * 16384 < sums_cols) cluster *= 2;
    const int slice = (sums_cols + cluster - 1) / cluster;
    rc = launch_select<512>(a, rows, cluster, slice <= 40960 ? slice : 0,
                            static_cast<cudaStream_t>(stream));
  }
  return rc == PKV_OK ? ok() : rc;
}

int pkv_evict_gather(void* k_cache, void* v_cache, const int32_t* block_tables,
                     int32_t max_blocks_per_seq, const int32_t* kept, int32_t kept_cols,
                     const int32_t* new_lens, const int32_t* new_tables, int32_t max_new_blocks,
                     int32_t num_seqs, int32_t num_blocks, int32_t num_kv_heads,
                     int32_t block_size, int32_t head_dim, int32_t* status, int32_t dtype,
                     void* stream) {
  const int elt = element_bytes(dtype);
  const bool codes = dtype == PKV_FP8_E4M3 || dtype == PKV_INT8;
  PKV_REQUIRE(elt != 0, PKV_ERR_DTYPE, "unknown dtype %d", dtype);
  PKV_REQUIRE(num_seqs >= 0 && num_blocks > 0 && num_kv_heads > 0 && block_size > 0 &&
                  head_dim > 0 && kept_cols > 0 && max_blocks_per_seq > 0 && max_new_blocks > 0,
              PKV_ERR_INVALID_ARG, "sizes must be positive (num_seqs >= 0)");
  PKV_REQUIRE(num_seqs <= 65535 && num_kv_heads <= 65535, PKV_ERR_UNSUPPORTED,
              "num_seqs %d or num_kv_heads %d above 65535", num_seqs, num_kv_heads);
  PKV_REQUIRE(!codes || block_size == 16, PKV_ERR_UNSUPPORTED,
              "8-bit caches use block_size 16, not %d", block_size);
  const int64_t row_bytes = static_cast<int64_t>(head_dim) * elt;
  PKV_REQUIRE(row_bytes % 16 == 0 && row_bytes <= 16 * kGatherThreads, PKV_ERR_INVALID_ARG,
              "head_dim * element size must be a multiple of 16 bytes, at most %d",
              16 * kGatherThreads);
  PKV_REQUIRE(static_cast<int64_t>(num_blocks) * block_size < (int64_t(1) << 31) &&
                  static_cast<int64_t>(max_blocks_per_seq) * block_size < (int64_t(1) << 31) &&
                  static_cast<int64_t>(max_new_blocks) * block_size < (int64_t(1) << 31),
              PKV_ERR_INVALID_ARG, "blocks * block_size must be < 2^31");
  if (num_seqs == 0) return ok();
  PKV_REQUIRE(k_cache && v_cache && block_tables && kept && new_lens && new_tables,
              PKV_ERR_INVALID_ARG, "NULL pointer");
  PKV_REQUIRE(aligned(k_cache, 16) && aligned(v_cache, 16), PKV_ERR_INVALID_ARG,
              "caches must be 16-byte aligned");
  PKV_REQUIRE(aligned(block_tables, 4) && aligned(kept, 4) && aligned(new_lens, 4) &&
                  aligned(new_tables, 4) && aligned(status, 4),
              PKV_ERR_INVALID_ARG, "a pointer is not 4-byte aligned");
  PKV_REQUIRE(block_tables != new_tables, PKV_ERR_INVALID_ARG,
              "new_tables must not be block_tables: rows move into other blocks");
  GatherArgs a{};
  a.kc = static_cast<uint4*>(k_cache);
  a.vc = static_cast<uint4*>(v_cache);
  a.tables = block_tables;
  a.kept = kept;
  a.new_lens = new_lens;
  a.new_tables = new_tables;
  a.status = status;
  a.Hkv = num_kv_heads;
  a.B = block_size;
  a.NB = num_blocks;
  a.MAXB = max_blocks_per_seq;
  a.NEWB = max_new_blocks;
  a.kept_cols = kept_cols;
  a.row_vecs = static_cast<int32_t>(row_bytes / 16);
  a.D = head_dim;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((kept_cols + kGatherTokens - 1) / kGatherTokens, num_kv_heads, num_seqs);
  cfg.blockDim = dim3(kGatherThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (!codes) {
    PKV_CUDA(cudaLaunchKernelEx(&cfg, evict_gather_kernel<true>, a));
    return ok();
  }
  PKV_CUDA(cudaLaunchKernelEx(&cfg, evict_gather_kernel<false>, a));
  cfg.gridDim = dim3((kept_cols + 15) / 16, num_kv_heads, num_seqs);
  PKV_CUDA(cudaLaunchKernelEx(&cfg, evict_gather_v8_kernel, a));
  return ok();
}

}  // extern "C"
