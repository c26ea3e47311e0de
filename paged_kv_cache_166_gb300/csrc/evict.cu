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
// Select is exact: the m-th largest sum is found by its bits, and the tokens above it, plus
// the lowest positions equal to it, are compacted with prefix counts.  A row of sums is read
// from memory once: a short row's keys stay in a warp's registers, a long row's upper halves
// in the shared memory of a cluster of CTAs, a slice each, whose histograms of the keys'
// digits are added over distributed shared memory.  Gather is a copy, bound by memory.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "quant8.cuh"

namespace cg = cooperative_groups;

namespace pkv {
namespace {

// ---- select ---------------------------------------------------------------------

constexpr int kMaxCols = 1 << 30;  // of sums and positions: indices stay within 32 bits
constexpr int kDigitBins = 2048;  // 11, 5, 11 and 5 bits of a key
constexpr int kPasses = 4;
constexpr int kMaxCluster = 8;    // eight threads add a bin's shares

struct SelectArgs {
  const float* sums;
  const int32_t* context_lens;
  const int32_t* keep_lens;
  int32_t* kept;
  float* new_sums;
  int32_t* new_lens;
  int32_t* status;  // or NULL
  int32_t Hkv, cols, kept_cols, new_cols, first, recent;
};

// Unsigned key in the order of the values: larger sum, larger key.  NaN counts as
// -infinity and -0 as +0.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(fmaxf(x + 0.f, -INFINITY));
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

// A row's ends, and the candidates between them.
struct Row {
  int c, n, r, f, m, M;  // tokens, kept ones, last and first kept ones, picked of M between
  const float* sums;
  int32_t* kept;
  float* out;
};

// Reads the row's lengths; `lead` (one thread of a sequence) writes the new length.
__device__ __forceinline__ Row row_of(const SelectArgs& a, int64_t row, bool lead) {
  Row w;
  const int s = static_cast<int>(row / a.Hkv);
  int c = a.context_lens[s], n = a.keep_lens[s];
  bool bad = c < 0 || c > a.cols;
  c = min(max(c, 0), a.cols);
  n = min(max(n, 0), c);
  const int most = min(a.kept_cols, a.new_cols);
  bad |= n > most;
  n = min(n, most);
  if (lead && row % a.Hkv == 0) {
    a.new_lens[s] = n;
    if (bad && a.status != nullptr) atomicOr(a.status, PKV_DEV_BAD_CONTEXT_LEN);
  }
  w.c = c;
  w.n = n;
  w.r = min(a.recent, n);
  w.f = min(a.first, n - w.r);
  w.m = n - w.r - w.f;
  w.M = c - w.r - w.f;
  w.sums = a.sums + row * a.cols;
  w.kept = a.kept + row * a.kept_cols;
  w.out = a.new_sums + row * a.new_cols;
  return w;
}

// The ends, which stay whatever their sums, by threads t of T.
__device__ __forceinline__ void keep_ends(const Row& w, int t, int T) {
  for (int i = t; i < w.f + w.r; i += T) {
    const int j = i < w.f ? i : w.n - w.r + (i - w.f), p = i < w.f ? i : w.c - w.r + (i - w.f);
    w.kept[j] = p;
    w.out[j] = w.sums[p];
  }
}

// Where the kept ones of 32 consecutive candidates go: those above the threshold, and
// equal ones while `ties` last; gt and eq count the ones before, and move on.
__device__ __forceinline__ int place_of(bool g, bool e, int ties, int lane, int& gt, int& eq) {
  const uint32_t mg = __ballot_sync(0xffffffffu, g), me = __ballot_sync(0xffffffffu, e);
  const uint32_t below = (1u << lane) - 1;
  const int ng = gt + __popc(mg & below), ne = eq + __popc(me & below);
  gt += __popc(mg);
  eq += __popc(me);
  return g || (e && ne < ties) ? ng + min(ne, ties) : -1;
}

// ---- short rows: a warp each, the keys in registers -------------------------------

constexpr int kShortCols = 2048;
constexpr int kShortWarps = 4;

// kKeys keys a lane, M <= 32 kKeys.  The threshold's bits are found one at a time, from the
// highest in which the keys differ, by counting the keys it would leave: a few tens of
// register compares and one warp sum a bit, and no barrier; it is done early once the
// count is the number wanted.
// Bound by the longest rows' chains of such bits: 2,560 rows of 2,048 in 33 us, of 400 in 8.9
// (21 and 4 MB); with rows of all lengths 15% of the warps are active and the SM is at 12%.
template <int kKeys>
__device__ __forceinline__ void select_short(const Row& w, int lane) {
  uint32_t key[kKeys];
  const float* const vals = w.sums + w.f;
#pragma unroll
  for (int i = 0; i < kKeys; ++i) {
    const int p = 32 * i + lane;
    key[i] = p < w.M ? key_of(vals[p]) : 0u;  // 0: no token
  }
  uint32_t t = 1;  // everything stays
  int ties = 0;
  if (w.m < w.M) {
    uint32_t hi = 0, lo = ~0u;
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      hi = max(hi, key[i]);
      lo = min(lo, key[i] == 0 ? ~0u : key[i]);
    }
    hi = __reduce_max_sync(0xffffffffu, hi);
    lo = __reduce_min_sync(0xffffffffu, lo);
    int bit = 31 - __clz(hi ^ lo);  // -1 if all are equal
    t = bit < 0 ? hi : (hi >> bit >> 1) << bit << 1;
    int count = w.M;                // keys >= t
    for (; bit >= 0 && count != w.m; --bit) {
      const uint32_t u = t | (1u << bit);
      int n = 0;
#pragma unroll
      for (int i = 0; i < kKeys; ++i) n += key[i] >= u;
      n = __reduce_add_sync(0xffffffffu, n);
      if (n >= w.m) {
        t = u;
        count = n;
      }
    }
    if (count != w.m) {  // t is the m-th largest key itself, and more keys equal it than fit
      int above = 0;
#pragma unroll
      for (int i = 0; i < kKeys; ++i) above += key[i] > t;
      ties = w.m - __reduce_add_sync(0xffffffffu, above);
    } else {
      t -= 1;  // keys above t - 1
    }
  } else {
    t = 0;
  }
  int gt = 0, eq = 0;
#pragma unroll
  for (int i = 0; i < kKeys; ++i) {
    if (32 * i < w.M) {
      const int at = place_of(key[i] > t, ties > 0 && key[i] == t, ties, lane, gt, eq);
      if (at >= 0) {
        const int p = 32 * i + lane;
        w.kept[w.f + at] = w.f + p;
        w.out[w.f + at] = vals[p];
      }
    }
  }
}

__global__ void __launch_bounds__(kShortWarps * 32, 5)
    evict_select_short_kernel(const SelectArgs a, int64_t rows) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kShortWarps + (threadIdx.x >> 5);
  if (row >= rows) return;
  const Row w = row_of(a, row, lane == 0);
  keep_ends(w, lane, 32);
  if (w.m == 0) return;
  if (w.M <= 256) select_short<8>(w, lane);
  else if (w.M <= 512) select_short<16>(w, lane);
  else if (w.M <= 1024) select_short<32>(w, lane);
  else select_short<kShortCols / 32>(w, lane);
}

// ---- long rows: a cluster of CTAs each, the keys' upper halves in shared memory -----
//
// The threshold is found by its digits, 11, 5, 11 and 5 bits, from histograms of the keys
// that agree with it so far; once few are left, every CTA of the cluster takes them all and
// goes on alone.  Halves take 2 bytes a key, so a CTA holds 32,768 of them, two CTAs fit an
// SM and 64 rows of 131,072 are worked on at once; with whole keys in registers (16,384 a
// CTA) they took a second round of CTAs: 41.7 us against 26.1 (33.5 MB, of which reading
// them takes 5.2).  The loops over eight keys a thread are short code run many times: the
// same keys unrolled in registers took 31.9 us, much of it waiting for instructions.  What is
// left is latency: of some 38,000 cycles the loads and first histogram take 12,000 (6.5 TB/s),
// the bin's keys 5,000, the cluster's sums and barriers 8,000, the output 5,000.

constexpr int kLongThreads = 512;
constexpr int kLongKeys = 32768;                        // keys of a CTA at once, at most
constexpr int kSlice = 4096;                            // keys a CTA is left with, if possible
constexpr int kSmallSlice = 8192;                       // keys of a CTA of which four fit an SM
constexpr int kWarps = kLongThreads / 32;
constexpr int kCoarse = 64;                             // sums of 32 bins each
constexpr int kTailKeys = 4;
constexpr int kTail = kLongThreads * kTailKeys;         // keys resolved without histograms
constexpr int kTailBins = 128;

// Exclusive prefix sum of v over the block's threads; the sum of all in *total.
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
  for (int i = 0; i < kWarps; ++i) {
    const int y = warp_sums[i];
    base += i < w ? y : 0;
    all += y;
  }
  *total = all;
  return base + x - v;
}

// Bits of eight keys whose upper halves, masked, are above u (over) or u itself (same).
__device__ __forceinline__ void compare8(const uint4& q, uint32_t mask, uint32_t u, uint32_t& over,
                                         uint32_t& same) {
  const uint32_t h[4] = {q.x, q.y, q.z, q.w};
  over = same = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = h[i] & mask, b = (h[i] >> 16) & mask;
    over |= (a > u ? 1u << (2 * i) : 0u) | (b > u ? 2u << (2 * i) : 0u);
    same |= (a == u ? 1u << (2 * i) : 0u) | (b == u ? 2u << (2 * i) : 0u);
  }
}

// The few keys whose lower half matters, those with the threshold's upper half, are read
// again (from L2).  cap: keys of the CTA at once, a multiple of 32.  kCtas: CTAs of an SM.
template <int kCtas>
__global__ void __launch_bounds__(kLongThreads, kCtas)
    evict_select_long_kernel(const SelectArgs a, int cap) {
  extern __shared__ uint4 eights[];
  __shared__ __align__(16) int hist[kDigitBins];  // of 11 bits
  __shared__ int coarse[kCoarse], low[32];        // its sums; of 5 bits
  __shared__ uint32_t tail[kTail];                // this CTA's keys in the threshold's bin
  __shared__ int tail_at[kTail];                  // and where they are
  __shared__ __align__(16) int tail_hist[3][kTailBins];  // of seven bits
  __shared__ uint32_t mask_gt[kLongKeys / 32], mask_eq[kLongKeys / 32];
  __shared__ int warp_sums[kWarps];
  __shared__ int bins[kCoarse];                   // the cluster's sums of the bins looked at
  __shared__ int tail_count, counts[2];
  __shared__ int found_bin, found_above, found_count;
  uint16_t* const halves = reinterpret_cast<uint16_t*>(eights);
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Row w = row_of(a, blockIdx.x / C, rank == 0 && tid == 0);

  // this CTA's slice of the candidates, in rounds of cap
  const int per = (w.M + C - 1) / C;
  const int lo = w.f + min(w.M, rank * per), len = max(0, min(per, w.f + w.M - lo));
  const int rounds = (per + cap - 1) / cap;
  const float* const vals = w.sums + lo;
  auto load = [&](int round, bool count) {
    constexpr int U = kCtas == 2 ? 16 : 8;  // loads in flight
    const float* const at = vals + static_cast<int64_t>(round) * cap;
    const int n = min(len - round * cap, cap), n8 = (n + 7) & ~7;
    for (int p0 = tid; p0 < n8; p0 += U * kLongThreads) {
      float x[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int p = p0 + i * kLongThreads;
        x[i] = p < n ? __ldg(at + p) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int p = p0 + i * kLongThreads;
        const uint32_t k = p < n ? key_of(x[i]) : 0u;  // 0: no token
        if (p < n8) halves[p] = static_cast<uint16_t>(k >> 16);
        if (count && p < n) atomicAdd(&hist[k >> 21], 1);
      }
    }
    __syncthreads();
  };
  auto eights_of = [&](int round) { return (max(0, min(len - round * cap, cap)) + 7) / 8; };
  // use(bit, key) for each key of `same` of the eight at v: all of them read at once
  auto each = [&](int round, int v, uint32_t same, auto use) {
    const float* const at = vals + static_cast<int64_t>(round) * cap + 8 * v;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = same >> i & 1 ? __ldg(at + i) : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (same >> i & 1) use(i, key_of(x[i]));
  };
  for (int i = tid; i < kDigitBins; i += kLongThreads) hist[i] = 0;
  for (int i = tid; i < kLongKeys / 32; i += kLongThreads) mask_gt[i] = mask_eq[i] = 0;
  if (tid < 32) low[tid] = 0;
  if (tid < 3 * kTailBins) (&tail_hist[0][0])[tid] = 0;
  if (tid == 0) tail_count = 0;
  __syncthreads();
  // a row of one round is read from memory once
  const bool cuts = w.m > 0 && w.m < w.M;
  if (rounds == 1) load(0, cuts);
  keep_ends(w, rank * kLongThreads + tid, C * kLongThreads);

  // The threshold t: the m-th largest key; `above` keys are larger.  m == M: everything is
  // above 0.
  uint32_t t = 0;
  int above = 0;
  bool masked = false;  // the masks are there
  if (cuts) {
    int shift = 32;
    for (int pass = 0; pass < kPasses; ++pass) {
      const int bits = pass % 2 == 0 ? 11 : 5;
      shift -= bits;
      if (pass == 2) {  // every CTA is past its reads of the first two passes
        for (int i = tid; i < kDigitBins; i += kLongThreads) hist[i] = 0;
      }
      if (pass == 3 && tid < 32) low[tid] = 0;
      __syncthreads();
      for (int round = 0; round < rounds; ++round) {
        if (rounds > 1) load(round, pass == 0);
        if (pass == 0) continue;
        for (int v = tid; v < eights_of(round); v += kLongThreads) {
          uint32_t over, same;
          const uint4 q = eights[v];
          compare8(q, pass == 1 ? 0xffe0u : 0xffffu, t >> 16, over, same);
          if (pass == 1) {
            const uint32_t h[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (same >> i & 1) atomicAdd(&low[h[i / 2] >> (16 * (i % 2)) & 31], 1);
          } else if (same != 0) {
            each(round, v, same, [&](int, uint32_t k) {
              if (pass == 2) atomicAdd(&hist[k >> 5 & 2047], 1);
              else if (k >> 5 == t >> 5) atomicAdd(&low[k & 31], 1);
            });
          }
        }
        if (rounds > 1) __syncthreads();
      }
      __syncthreads();
      if (bits == 11) {
        const int4 h = *reinterpret_cast<const int4*>(&hist[4 * tid]);
        int n = h.x + h.y + h.z + h.w;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
        if ((tid & 7) == 0) coarse[tid >> 3] = n;
      }
      cluster.sync();
      // the cluster's sums of 64 runs of 32 bins, then of the bins of the run that counts:
      // eight threads a sum, a CTA's share each
      for (int level = bits == 11 ? 0 : 1; level < 2; ++level) {
        const int width = level == 0 ? kCoarse : 32;
        const int first = level == 0 || bits == 5 ? 0 : 32 * found_bin;
        const int q = tid & 7, at = tid >> 3;
        int n = 0;
        if (q < C && at < width)
          n = *cluster.map_shared_rank(bits == 5    ? &low[at]
                                       : level == 0 ? &coarse[at]
                                                    : &hist[first + at], q);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
        if (q == 0) bins[at] = at < width ? n : 0;
        __syncthreads();
        if (warp == 0) {  // from the top: lane l holds bins 63 - 2 l and 62 - 2 l
          const int hi = bins[kCoarse - 1 - 2 * lane], lw = bins[kCoarse - 2 - 2 * lane];
          int x = hi + lw;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
          }
          const int before = above + x - hi - lw;  // keys in the bins above this lane's
          __syncwarp();
          if (before < w.m && before + hi >= w.m) {
            found_bin = first + kCoarse - 1 - 2 * lane;
            found_above = before;
            found_count = hi;
          } else if (before + hi < w.m && before + hi + lw >= w.m) {
            found_bin = first + kCoarse - 2 - 2 * lane;
            found_above = before + hi;
            found_count = lw;
          }
        }
        __syncthreads();
        above = found_above;
      }
      t |= static_cast<uint32_t>(found_bin) << shift;
      int left = found_count;  // keys in the bin
      if (shift == 0) break;
      if (left > kTail || shift < 16) {
        __syncthreads();  // found_* may be written again
        continue;
      }
      // Few keys in the bin: every CTA takes them all and finds the rest of the threshold's
      // bits by counting, from the highest; done early once the count is the number wanted.
      for (int round = 0; round < rounds; ++round) {
        if (rounds > 1) load(round, false);
        for (int v = tid; v < eights_of(round); v += kLongThreads) {
          uint32_t over, same;
          compare8(eights[v], 0xffffu << (shift - 16) & 0xffffu, t >> 16, over, same);
          if (rounds == 1) reinterpret_cast<uint8_t*>(mask_gt)[v] = static_cast<uint8_t>(over);
          for (; same != 0; same &= same - 1)
            tail_at[atomicAdd(&tail_count, 1)] = round * cap + 8 * v + __ffs(same) - 1;
        }
        if (rounds > 1) __syncthreads();
      }
      masked = rounds == 1;
      __syncthreads();
      const int mine = tail_count;
      for (int i = tid; i < mine; i += kLongThreads) tail[i] = key_of(__ldg(vals + tail_at[i]));
      cluster.sync();
      uint32_t k[kTailKeys] = {};
      int begin = 0;
      for (int q = 0; q < C; ++q) {
        const int n = *cluster.map_shared_rank(&tail_count, q);
        const uint32_t* const from = cluster.map_shared_rank(&tail[0], q);
#pragma unroll
        for (int i = 0; i < kTailKeys; ++i) {
          const int at = i * kLongThreads + tid - begin;
          if (at >= 0 && at < n) k[i] = from[at];
        }
        begin += n;
      }
      // The rest of the threshold, seven bits at a time, until all keys of a bin stay.
      for (int i = 0; shift > 0 && above + left != w.m; ++i) {
        const int bits7 = shift < 7 ? shift : 7;
        const uint32_t fixed = ~0u << shift;
        shift -= bits7;
#pragma unroll
        for (int j = 0; j < kTailKeys; ++j)
          if ((k[j] & fixed) == t) atomicAdd(&tail_hist[i][k[j] >> shift & ((1u << bits7) - 1)], 1);
        __syncthreads();
        if (warp == 0) {  // from the top: lane l holds bins 127 - 4 l .. 124 - 4 l
          const int4 h = *reinterpret_cast<const int4*>(&tail_hist[i][kTailBins - 4 - 4 * lane]);
          const int sum = h.x + h.y + h.z + h.w;
          int x = sum;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
          }
          int before = above + x - sum;
          const int n[4] = {h.w, h.z, h.y, h.x};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (before < w.m && before + n[j] >= w.m) {
              found_bin = kTailBins - 1 - 4 * lane - j;
              found_above = before;
              found_count = n[j];
            }
            before += n[j];
          }
        }
        __syncthreads();
        t |= static_cast<uint32_t>(found_bin) << shift;
        above = found_above;
        left = found_count;
      }
      if (above + left == w.m) {
        t -= 1;  // all keys of at least t stay: those above t - 1, and none equal to it
        above = w.m;
      }
      if (masked) {  // the keys of the bin join those above it
        for (int i = tid; i < mine; i += kLongThreads) {
          const int p = tail_at[i];
          if (tail[i] > t) atomicOr(&mask_gt[p >> 5], 1u << (p & 31));
          else if (tail[i] == t) atomicOr(&mask_eq[p >> 5], 1u << (p & 31));
        }
        __syncthreads();
      }
      break;
    }
  }
  const int ties = w.m == w.M ? 0 : w.m - above;  // keys equal to t that stay

  // Bit masks of a round's keys above t, and equal to it; words behind the round's keys are
  // not used.
  auto masks = [&](int round) {
    const uint32_t th = t >> 16;
    for (int v = tid; v < eights_of(round); v += kLongThreads) {
      uint32_t over, same, equal = 0;
      compare8(eights[v], 0xffffu, th, over, same);
      if (th == 0) same = 0;  // no tokens
      if (same != 0)
        each(round, v, same, [&](int i, uint32_t k) {
          if (k > t) over |= 1u << i;
          if (k == t) equal |= 1u << i;
        });
      reinterpret_cast<uint8_t*>(mask_gt)[v] = static_cast<uint8_t>(over);
      reinterpret_cast<uint8_t*>(mask_eq)[v] = static_cast<uint8_t>(equal);
    }
    __syncthreads();
  };
  // A thread has `words` (one or two) consecutive words of a round's masks.
  const int words = (cap / 32 + kLongThreads - 1) / kLongThreads;
  auto bits_of = [&](const uint32_t* mask, int round) {
    const int i = words * tid, left = 8 * eights_of(round) - 32 * i;  // bits from there on
    uint64_t x = left > 0 ? mask[i] : 0u;
    if (words == 2 && left > 32) x |= static_cast<uint64_t>(mask[i + 1]) << 32;
    const int n = min(left, 32 * words);
    return n <= 0 || n == 64 ? x : x & ((1ull << n) - 1);
  };
  // How many of each the CTAs before have.
  int gt0 = 0, eq0 = 0;
  if (w.m > 0) {
    int total_gt = 0, total_eq = 0;
    for (int round = 0; round < rounds; ++round) {
      if (rounds > 1) load(round, false);
      if (!masked) masks(round);
      total_gt += __popcll(bits_of(mask_gt, round));
      total_eq += __popcll(bits_of(mask_eq, round));
      if (rounds > 1) __syncthreads();
    }
    int all_gt, all_eq;
    block_prefix(total_gt, warp_sums, &all_gt);
    block_prefix(total_eq, warp_sums, &all_eq);
    if (tid == 0) {
      counts[0] = all_gt;
      counts[1] = all_eq;
    }
  }
  cluster.sync();
  if (w.m > 0) {
    for (int q = 0; q < rank; ++q) {
      const int* const c = cluster.map_shared_rank(&counts[0], q);
      gt0 += c[0];
      eq0 += c[1];
    }
    for (int round = 0; round < rounds; ++round) {
      if (rounds > 1) {
        load(round, false);
        masks(round);
      }
      const uint64_t g = bits_of(mask_gt, round), e = bits_of(mask_eq, round);
      int all_gt, all_eq = 0;
      const int ng0 = gt0 + block_prefix(__popcll(g), warp_sums, &all_gt);
      const int ne0 = eq0 + (ties > 0 ? block_prefix(__popcll(e), warp_sums, &all_eq) : 0);
      // the round's tokens in order, in the keys' place, then copied side by side
      const int at0 = gt0 + min(eq0, ties);
      const int count = gt0 + all_gt + min(eq0 + all_eq, ties) - at0;
      for (uint64_t left = g | e; left != 0; left &= left - 1) {
        const uint64_t bit = left & (0ull - left);
        const int ng = ng0 + __popcll(g & (bit - 1)), ne = ne0 + __popcll(e & (bit - 1));
        if ((g & bit) || ne < ties)
          halves[ng + min(ne, ties) - at0] =
              static_cast<uint16_t>(32 * words * tid + 63 - __clzll(static_cast<long long>(bit)));
      }
      __syncthreads();
#pragma unroll 4
      for (int j = tid; j < count; j += kLongThreads) {
        const int p = round * cap + halves[j];
        w.kept[w.f + at0 + j] = lo + p;
        w.out[w.f + at0 + j] = __ldg(vals + p);
      }
      gt0 += all_gt;
      eq0 += all_eq;
      if (rounds > 1) __syncthreads();
    }
  }
  cluster.sync();  // no CTA leaves while others read its counts
}

// ---- gather ---------------------------------------------------------------------

constexpr int kGatherThreads = 256;

struct GatherArgs {
  uint4* kc;
  uint4* vc;
  const int32_t* tables;
  const int32_t* kept;
  const int32_t* new_lens;
  const int32_t* new_tables;
  int32_t* status;  // or NULL
  int32_t Hkv, B, NB, MAXB, NEWB, kept_cols, row_vecs, D;
  int32_t tokens;  // kept tokens of one CTA, at most kGatherThreads
};

// New V tiles of one CTA: a thread has one of the D rows of one.
__host__ __device__ __forceinline__ int v8_tiles(int D) {
  return D < kGatherThreads ? kGatherThreads / D : 1;
}

// Slot row (in rows of the cache) of position p of a table row, or -1.
__device__ __forceinline__ int64_t cache_row(const int32_t* table, int max_blocks, int p, int B,
                                             int NB, int Hkv, int h) {
  if (p < 0 || p >= max_blocks * B) return -1;
  const int j = p / B;
  const int b = __ldg(table + j);
  if (b < 0 || b >= NB) return -1;
  return (static_cast<int64_t>(b) * Hkv + h) * B + (p - j * B);
}

// Bound by memory: 8 sequences' 4,096 tokens of 8 heads of 128, 16-bit, 134 MB read and
// written, take 39.6 us, the copy rate.
// grid: (pieces of a.tokens kept tokens, KV heads, sequences).  Every thread looks up one
// token's two rows, then the rows are moved 16 bytes a thread, U of them in flight.
// kV: the V rows are laid out like the K rows (16- and 32-bit caches).
template <bool kV>
__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(const GatherArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ int64_t src_row[kGatherThreads], dst_row[kGatherThreads];
  const int s = blockIdx.z, h = blockIdx.y;
  const int n = min(max(a.new_lens[s], 0), a.kept_cols);
  const int j0 = blockIdx.x * a.tokens;
  if (j0 >= n) return;
  const int count = min(a.tokens, n - j0);
  if (static_cast<int>(threadIdx.x) < count) {
    const int j = j0 + threadIdx.x;
    const int p = __ldg(a.kept + (static_cast<int64_t>(s) * a.Hkv + h) * a.kept_cols + j);
    const int64_t src = cache_row(a.tables + static_cast<int64_t>(s) * a.MAXB, a.MAXB, p, a.B,
                                  a.NB, a.Hkv, h);
    const int64_t dst = cache_row(a.new_tables + static_cast<int64_t>(s) * a.NEWB, a.NEWB, j, a.B,
                                  a.NB, a.Hkv, h);
    const bool bad = src < 0 || dst < 0;
    if (bad && a.status != nullptr) atomicOr(a.status, PKV_DEV_BAD_BLOCK_ID);
    src_row[threadIdx.x] = src;
    dst_row[threadIdx.x] = bad ? -1 : dst;
  }
  __syncthreads();
  const int rows = kGatherThreads / a.row_vecs;
  const int v = threadIdx.x % a.row_vecs, r = threadIdx.x / a.row_vecs;
  if (r >= rows) return;
  constexpr int U = 4;
  for (int j = r; j < count; j += U * rows) {
    int64_t dst[U];
    uint4 kx[U], vx[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int ju = j + u * rows;
      dst[u] = ju < count ? dst_row[ju] : -1;
      if (dst[u] >= 0) {
        const int64_t at = src_row[ju] * a.row_vecs + v;
        kx[u] = __ldcs(a.kc + at);
        if constexpr (kV) vx[u] = __ldcs(a.vc + at);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (dst[u] >= 0) {
        const int64_t at = dst[u] * a.row_vecs + v;
        a.kc[at] = kx[u];
        if constexpr (kV) a.vc[at] = vx[u];
      }
    }
  }
}

// V of 8-bit caches: tiles [D x 16 bytes], a token one byte of every row.  A thread fills a
// 16-byte row of a new tile (a CTA as many tiles as it has rows for); consecutive kept tokens
// often come from one old tile, whose row is then read once, and eight tokens' rows are on
// their way together (select and gather of 82 sequences of 1,334 tokens cut to 207, 16 heads:
// 181 us with one row read behind the other and one tile a CTA, 133 now; of 8 to 131,072 cut to
// 4,096, 8 heads: 242 and 144).
__global__ void __launch_bounds__(kGatherThreads, 3) evict_gather_v8_kernel(const GatherArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ int64_t src_tile[kGatherThreads];  // of 16 tokens a tile, 16 tiles at most
  __shared__ int src_byte[kGatherThreads];
  const int s = blockIdx.z, h = blockIdx.y;
  const int n = min(max(a.new_lens[s], 0), a.kept_cols);
  const int tiles = v8_tiles(a.D), first = blockIdx.x * tiles * 16;  // of the CTA; its first token
  if (first >= n) return;
  if (static_cast<int>(threadIdx.x) < 16 * tiles) {
    const int j = first + threadIdx.x;
    int64_t row = -1;
    if (j < n)
      row = cache_row(a.tables + static_cast<int64_t>(s) * a.MAXB, a.MAXB,
                      __ldg(a.kept + (static_cast<int64_t>(s) * a.Hkv + h) * a.kept_cols + j), 16,
                      a.NB, a.Hkv, h);
    src_tile[threadIdx.x] = row < 0 ? -1 : row >> 4;
    src_byte[threadIdx.x] = row < 0 ? 0 : fp8_v_pos(static_cast<int>(row & 15));
  }
  __syncthreads();
  const int mine = tiles == 1 ? 0 : threadIdx.x / a.D, j0 = first + 16 * mine;
  if (mine >= tiles || j0 >= n) return;
  const int64_t to = cache_row(a.new_tables + static_cast<int64_t>(s) * a.NEWB, a.NEWB, j0, 16,
                               a.NB, a.Hkv, h);
  if (to < 0) return;  // reported by the K rows' kernel
  const int64_t* const tile_of = src_tile + 16 * mine;
  const int* const byte_of = src_byte + 16 * mine;
  for (int d = threadIdx.x - mine * a.D; d < a.D; d += kGatherThreads) {
    uint4* const dst = a.vc + (to >> 4) * a.D + d;
    // bytes of tokens that do not move (past n, or from a bad block) stay as they are
    bool whole = true;
#pragma unroll
    for (int t = 0; t < 16; ++t) whole &= tile_of[t] >= 0;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (!whole) w = *dst;
    uint8_t* const wb = reinterpret_cast<uint8_t*>(&w);
#pragma unroll
    for (int t0 = 0; t0 < 16; t0 += 8) {
      uint4 x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int64_t tile = tile_of[t0 + u];
        if (tile >= 0 && (u == 0 || tile != tile_of[t0 + u - 1])) x[u] = a.vc[tile * a.D + d];
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int t = t0 + u;
        const int64_t tile = tile_of[t];
        if (tile < 0) continue;
        if (u > 0 && tile == tile_of[t - 1]) x[u] = x[u > 0 ? u - 1 : 0];
        const int b = byte_of[t];
        const uint32_t word =
            (b >> 2) == 0 ? x[u].x : (b >> 2) == 1 ? x[u].y : (b >> 2) == 2 ? x[u].z : x[u].w;
        const int at = t < 8 ? 4 * (t >> 1) + (t & 1) : 4 * ((t - 8) >> 1) + 2 + (t & 1);
        wb[at] = static_cast<uint8_t>(word >> (8 * (b & 3)));
      }
    }
    *dst = w;
  }
}

template <int kCtas>
int launch_long(const SelectArgs& a, int64_t rows, int cluster, int cap, cudaStream_t st) {
  static SmemOnce once;
  const int rc = allow_dynamic_smem(
      once, reinterpret_cast<const void*>(evict_select_long_kernel<kCtas>),
      kLongKeys * sizeof(uint16_t));
  if (rc != PKV_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * cluster));
  cfg.blockDim = dim3(kLongThreads);
  cfg.dynamicSmemBytes = cap * sizeof(uint16_t);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  PKV_CUDA(cudaLaunchKernelEx(&cfg, evict_select_long_kernel<kCtas>, a, cap));
  return PKV_OK;
}

// Rows of up to 2,048 columns take a warp each: 2,560 rows of 2,048 took 33 us so, against 54
// with a CTA's histograms.  A longer row takes a cluster of as many CTAs, up to eight, as
// leave no SM idle (two on each): 8 rows of 131,072 took 20.4 us with the four CTAs that hold
// one, 15.3 with eight; 64 rows of 32,768 20.8 with one and 15.8 with four.  A row that eight
// CTAs do not hold is read once a pass.
int launch_select(const SelectArgs& a, int64_t rows, cudaStream_t st) {
  if (a.cols <= kShortCols) {
    const int64_t ctas = (rows + kShortWarps - 1) / kShortWarps;
    evict_select_short_kernel<<<static_cast<unsigned>(ctas), kShortWarps * 32, 0, st>>>(a, rows);
    PKV_CUDA(cudaGetLastError());
    return PKV_OK;
  }
  int sms = 0, dev = 0;
  const int rc = device_sm_count(&sms, &dev);
  if (rc != PKV_OK) return rc;
  int cluster = 1;
  while (cluster < kMaxCluster &&
         (static_cast<int64_t>(cluster) * kLongKeys < a.cols ||
          (a.cols / cluster > kSlice && rows * cluster <= sms)))
    cluster *= 2;
  const int per = static_cast<int>((static_cast<int64_t>(a.cols) + cluster - 1) / cluster);
  const int cap = per < kLongKeys ? (per + 31) / 32 * 32 : kLongKeys;
  // few keys a CTA and more CTAs than two an SM: four, with half the loads in flight each
  // (2,048 rows of 8,192: 111 us with two, 92 with four; 64 of 32,768: 17.4 and 19.2)
  return cap <= kSmallSlice && rows * cluster > 2 * sms
             ? launch_long<4>(a, rows, cluster, cap, st)
             : launch_long<2>(a, rows, cluster, cap, st);
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
  PKV_REQUIRE(sums_cols <= kMaxCols && kept_cols <= kMaxCols && new_cols <= kMaxCols,
              PKV_ERR_UNSUPPORTED, "more than %d columns", kMaxCols);
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
  const int rc = launch_select(a, rows, static_cast<cudaStream_t>(stream));
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
  PKV_REQUIRE(kept_cols <= kMaxCols, PKV_ERR_UNSUPPORTED, "more than %d columns", kMaxCols);
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
  // 256 tokens a CTA, or fewer while the SMs would not have a few CTAs each (select and gather
  // of one sequence, 1,024 tokens of 8 heads: 14.5 us, 16.9 with 256)
  int sms = 0, dev = 0;
  const int rc = device_sm_count(&sms, &dev);
  if (rc != PKV_OK) return rc;
  a.tokens = kGatherThreads;
  const int64_t heads = static_cast<int64_t>(num_seqs) * num_kv_heads;
  while (a.tokens > 32 && heads * ((kept_cols + a.tokens - 1) / a.tokens) < 4 * sms) a.tokens /= 2;
  cfg.gridDim = dim3((kept_cols + a.tokens - 1) / a.tokens, num_kv_heads, num_seqs);
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
  const int span = 16 * v8_tiles(head_dim);
  cfg.gridDim = dim3((kept_cols + span - 1) / span, num_kv_heads, num_seqs);
  PKV_CUDA(cudaLaunchKernelEx(&cfg, evict_gather_v8_kernel, a));
  return ok();
}

}  // extern "C"
