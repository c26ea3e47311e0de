// The accepted path of every sequence's drafted tokens, moved to where its next tokens belong,
// in the caches of all layers in one launch.
//
// Sequence s has t cached tokens, the last c of them drafted; with base = t - c its j-th
// accepted token's row, position base + path[s, j], goes to position base + j, j < n.  A token
// of a tree is drafted after its ancestors, so path[s, j] >= j, and rows are moved in
// ascending j: position base + j is written after every earlier row has been read, and no later
// one (path[s, i] >= i > j) lies there.  Each thread moves its own 16 bytes of a row through all
// j, so no two threads need an order between them.
//
// Bound by memory for many layers (each row read and written once), else by the chain of
// lengths, path, tables and rows: a CTA looks a sequence's rows up once and goes through its
// layers with them.  Measured: 64 paths of up to 8 tokens in 32 layers of 8 heads of 128, bf16, 14.6
// us (10.6 with the rows in L2), 4 paths in 2 layers 3.0, one launch.
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "quant8.cuh"

namespace pkv {
namespace {

constexpr int kCommitThreads = 128;
constexpr int kCommitRows = 64;  // rows looked up at once

struct CommitCaches {
  void* k[kMaxCopyLayers];
  void* v[kMaxCopyLayers];
};

struct CommitArgs {
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;
  const int32_t* path;       // [S, P]
  const int32_t* path_lens;  // [S]
  int32_t* status;           // or NULL
  int32_t S, MAXB, P, NB, Hkv, B, L;
  int32_t row_bytes;         // of a token and KV head
  int32_t codes;             // 8-bit caches: V tiles transposed
};

__device__ __forceinline__ void commit_flag(const CommitArgs& a, int bits) {
  if (a.status != nullptr && blockIdx.y == 0) atomicOr(a.status, bits);
}

// Grid: sequences, shares of the layers.
__global__ void __launch_bounds__(kCommitThreads)
    tree_commit_kernel(const __grid_constant__ CommitCaches caches, const CommitArgs a) {
  // rows to move: block and place in it, of the source and the target
  __shared__ int2 from_s[kCommitRows], to_s[kCommitRows];
  __shared__ int count_s;
  const int s = blockIdx.x, tid = threadIdx.x;
  const int t = __ldg(a.context_lens + s);
  const int c = __ldg(a.query_start + s + 1) - __ldg(a.query_start + s);
  int n = __ldg(a.path_lens + s);
  if (t < 0 || t > static_cast<int64_t>(a.MAXB) * a.B || c < 0 || c > t) {
    if (tid == 0) commit_flag(a, PKV_DEV_BAD_CONTEXT_LEN);
    return;
  }
  if (n < 0 || n > min(c, a.P)) {
    if (tid == 0) commit_flag(a, PKV_DEV_BAD_POSITION);
    n = n < 0 ? 0 : min(c, a.P);
  }
  const int base = t - c;
  const int32_t* const table = a.block_tables + static_cast<int64_t>(s) * a.MAXB;
  for (int j0 = 0; j0 < n; j0 += kCommitRows) {
    if (tid < 32) {  // ascending rows, those that stay left out
      int count = 0;
      for (int b = 0; b < kCommitRows && j0 + b < n; b += 32) {
        const int j = j0 + b + tid;
        bool moves = false;
        int2 from = make_int2(0, 0), to = make_int2(0, 0);
        if (j < n) {
          const int p = __ldg(a.path + static_cast<int64_t>(s) * a.P + j);
          if (p < j || p >= c) {
            commit_flag(a, PKV_DEV_BAD_POSITION);
          } else if (p != j) {
            const int x = base + p, y = base + j;
            const int bx = __ldg(table + x / a.B), by = __ldg(table + y / a.B);
            if (static_cast<uint32_t>(bx) >= static_cast<uint32_t>(a.NB) ||
                static_cast<uint32_t>(by) >= static_cast<uint32_t>(a.NB)) {
              commit_flag(a, PKV_DEV_BAD_BLOCK_ID);
            } else {
              moves = true;
              from = make_int2(bx, x % a.B);
              to = make_int2(by, y % a.B);
            }
          }
        }
        const uint32_t on = __ballot_sync(0xffffffffu, moves);
        if (moves) {
          const int at = count + __popc(on & ((1u << tid) - 1u));
          from_s[at] = from;
          to_s[at] = to;
        }
        count += __popc(on);
      }
      if (tid == 0) count_s = count;
    }
    __syncthreads();
    const int m = count_s;
    const int pieces = a.row_bytes / 16, items = a.Hkv * pieces;
    for (int l = blockIdx.y; l < a.L && m > 0; l += gridDim.y) {
      uint4* const kc = static_cast<uint4*>(caches.k[l]);
      uint4* const vc = static_cast<uint4*>(caches.v[l]);
      for (int i = tid; i < items; i += kCommitThreads) {
        const int g = i / pieces, d = i - g * pieces;
        auto at = [&](int2 x) {
          return ((static_cast<int64_t>(x.x) * a.Hkv + g) * a.B + x.y) * pieces + d;
        };
        for (int j = 0; j < m; j += 4) {
          uint4 kx[4], vx[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if (j + u >= m) continue;
            kx[u] = kc[at(from_s[j + u])];
            if (a.codes == 0) vx[u] = vc[at(from_s[j + u])];
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if (j + u >= m) continue;
            kc[at(to_s[j + u])] = kx[u];
            if (a.codes == 0) vc[at(to_s[j + u])] = vx[u];
          }
        }
      }
      if (a.codes != 0) {  // a token is a byte of each of a tile's 16-byte rows
        uint8_t* const vb = static_cast<uint8_t*>(caches.v[l]);
        for (int i = tid; i < a.Hkv * a.row_bytes; i += kCommitThreads) {
          const int g = i / a.row_bytes, d = i - g * a.row_bytes;
          auto at = [&](int2 x) {
            return ((static_cast<int64_t>(x.x) * a.Hkv + g) * a.row_bytes + d) * 16 +
                   fp8_v_pos(x.y);
          };
          for (int j = 0; j < m; j += 4) {
            uint8_t x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (j + u < m) x[u] = vb[at(from_s[j + u])];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (j + u < m) vb[at(to_s[j + u])] = x[u];
          }
        }
      }
    }
    __syncthreads();
  }
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_tree_commit(void* const* k_caches, void* const* v_caches, int32_t num_layers,
                               const int32_t* block_tables, int32_t max_blocks_per_seq,
                               const int32_t* context_lens, const int32_t* query_start,
                               const int32_t* path, int32_t path_cols, const int32_t* path_lens,
                               int32_t num_seqs, int32_t num_blocks, int32_t num_kv_heads,
                               int32_t block_size, int32_t head_dim, int32_t* status,
                               int32_t dtype, void* stream) {
  const int elt = element_bytes(dtype);
  PKV_REQUIRE(elt > 0, PKV_ERR_DTYPE, "unknown dtype %d", dtype);
  const bool codes = dtype == PKV_FP8_E4M3 || dtype == PKV_INT8;
  PKV_REQUIRE(num_layers >= 1 && num_layers <= kMaxCopyLayers, PKV_ERR_UNSUPPORTED,
              "num_layers %d outside [1, %d]", num_layers, kMaxCopyLayers);
  PKV_REQUIRE(num_seqs >= 0 && path_cols >= 0 && max_blocks_per_seq > 0 && num_blocks > 0 &&
                  num_kv_heads > 0 && block_size > 0 && head_dim > 0,
              PKV_ERR_INVALID_ARG, "sizes must be positive (num_seqs, path_cols >= 0)");
  PKV_REQUIRE(!codes || block_size == 16, PKV_ERR_UNSUPPORTED,
              "8-bit caches use block_size 16, not %d", block_size);
  PKV_REQUIRE(head_dim <= 4096 && (head_dim * elt) % 16 == 0, PKV_ERR_INVALID_ARG,
              "head_dim * element size must be a multiple of 16 bytes (head_dim at most 4096)");
  PKV_REQUIRE(num_kv_heads <= 65535, PKV_ERR_UNSUPPORTED, "num_kv_heads %d above 65535",
              num_kv_heads);
  PKV_REQUIRE(static_cast<int64_t>(max_blocks_per_seq) * block_size < (int64_t(1) << 31) &&
                  static_cast<int64_t>(num_blocks) * block_size < (int64_t(1) << 31),
              PKV_ERR_UNSUPPORTED, "tables or pool of 2^31 tokens or more");
  PKV_REQUIRE(k_caches && v_caches, PKV_ERR_INVALID_ARG, "NULL cache list");
  CommitCaches caches{};
  for (int l = 0; l < num_layers; ++l) {
    PKV_REQUIRE(k_caches[l] && v_caches[l], PKV_ERR_INVALID_ARG, "NULL cache of layer %d", l);
    PKV_REQUIRE(aligned(k_caches[l], 16) && aligned(v_caches[l], 16), PKV_ERR_INVALID_ARG,
                "caches of layer %d must be 16-byte aligned", l);
    for (int m = 0; m < l; ++m)  // two CTAs would move its rows at the same time
      PKV_REQUIRE(k_caches[l] != k_caches[m] && v_caches[l] != v_caches[m] &&
                      k_caches[l] != v_caches[m] && v_caches[l] != k_caches[m],
                  PKV_ERR_INVALID_ARG, "layers %d and %d share a cache", m, l);
    caches.k[l] = k_caches[l];
    caches.v[l] = v_caches[l];
  }
  if (num_seqs == 0 || path_cols == 0) return ok();
  PKV_REQUIRE(block_tables && context_lens && query_start && path && path_lens,
              PKV_ERR_INVALID_ARG, "NULL pointer");
  PKV_REQUIRE(aligned(block_tables, 4) && aligned(context_lens, 4) && aligned(query_start, 4) &&
                  aligned(path, 4) && aligned(path_lens, 4) && aligned(status, 4),
              PKV_ERR_INVALID_ARG, "a pointer is not aligned to its element");
  int sms = 0, dev = 0;
  const int rc = device_sm_count(&sms, &dev);
  if (rc != PKV_OK) return rc;
  CommitArgs a{};
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.query_start = query_start;
  a.path = path;
  a.path_lens = path_lens;
  a.status = status;
  a.S = num_seqs;
  a.MAXB = max_blocks_per_seq;
  a.P = path_cols;
  a.NB = num_blocks;
  a.Hkv = num_kv_heads;
  a.B = block_size;
  a.L = num_layers;
  a.row_bytes = head_dim * elt;
  a.codes = codes;
  // layers of a sequence spread over CTAs until the SMs have 16 each
  int shares = num_layers;
  while (shares > 1 && static_cast<int64_t>(shares) * num_seqs > 16 * sms)
    shares = (shares + 1) / 2;
  tree_commit_kernel<<<dim3(num_seqs, shares), kCommitThreads, 0,
                       static_cast<cudaStream_t>(stream)>>>(caches, a);
  PKV_CUDA(cudaGetLastError());
  return ok();
}
