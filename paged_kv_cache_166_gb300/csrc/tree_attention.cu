// Attention of drafted tokens over the paged cache on the 5th-generation tensor cores.
//
// Sequence s has t cached tokens, the last c of them drafted (their K and V written before):
// a tree, or a plain chunk.  Query row q0 + i is drafted token i; with base = t - c it sees
// every key p < base and of the drafted keys base + j those of its row of the mask (no mask:
// j <= i), both only within the window:
//   x = scale * q . K[p];  cap > 0: x = cap * tanh(x / cap);  x += slope_h * (pos(p) - pos(i));
//   out = softmax_p(x) . V[p], zero where a row sees nothing,
// pos(p) = p for p < base, base + depth_j for drafted token j; window: pos(i) - pos(p) < window.
//
// How.  A unit is a tile of up to 128 rows of one (sequence, KV head): row r is drafted token
// i0 + r / G, head g * G + r % G.  Its keys come in tiles of 128 (64 at head_dim 256, where
// the output alone takes half of the tensor memory): S = Q K^T (tcgen05, operands in
// 128-byte-swizzled shared memory, S in tensor memory, two buffers), softmax by two threads a
// row with a running maximum, P rounded to the input type in tensor memory, O += P V with O in
// tensor memory.  The layout of the tiles is the paged prefill's (prefill_tcgen05.cu).
//
// Split: the key tiles of all units, one after the other, are cut into one run of equal cost
// for each CTA (one CTA an SM), so that few long contexts use every SM.  A unit that a run's
// border cuts leaves each piece's unnormalised O, maximum and sum in the workspace (fp32); a
// second kernel, its launch overlapped, joins the pieces in order.  The same bits on every run.
//
// Bound: up to 128 rows read K and V once, 512 bytes a key and KV head at head_dim 128 for
// 4 * 128 * 128 operations: memory, if the softmax of a tile (16,384 exponentials) stays below
// the 1.5 us that its 64 KB take.  Measured: trees on a 70B-shaped batch (64 / 8 heads of 128, bf16,
// 128 contexts, 976 MB) 166 us, 5.9 TB/s; on contexts of 32,768 to 131,072 270 us, 6.5 TB/s; chunks
// of 513 with slopes on 8 sequences of 40 / 40 heads, f16, 194 us, bound by the row warps' chain of
// phases, not by memory or products; the smallest calls 10 us, two launches and their chains (the
// joining kernel is launched whether a unit is cut or not).  Behind a cache write a call takes some
// 1 us more than if lengths and masks were read before that write is done (with a step's norm and
// rotary write 42.0 us against 40.8 for 16 sequences, 16.8 against 16.1 for the smallest call).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kTrMaxSeqs = 2048;
constexpr int kTrMaxGroup = 16;
constexpr int kTrMaxDepth = 1 << 29;           // positions, below 2^30 + this, fit 32 bits
constexpr uint64_t kTrWaitNs = 1000000000ull;  // 1 s per wait before giving up
constexpr int kTrRows = 128;                   // rows of a unit = tensor-memory lanes = MMA M
constexpr int kTrRowWarps = 8;                 // softmax warps 2 .. 9: a lane quarter, a half of the keys
constexpr int kTrVWarp = 10, kTrQWarp = 11;    // producer of V; query tiles, and V looked through
constexpr int kTrThreads = 12 * 32;
constexpr int kTrChunk = 128 * 128;            // one [128 rows x 128 B] swizzled chunk of Q
// Of a unit beside its key tiles, in tiles.  With 1, 2, 3, 4: trees of a 70B-shaped batch 166, 166,
// 173, 171 us, with slopes 176, 168, 172, 176; a 13B-shaped chunk with slopes 205, 195, 194, 195, without
// 190, 179, 169, 170; long contexts and heads of 256 the same.
constexpr int kTrUnitCost = 2;
constexpr float kTrRescale = 8.f;              // log2 of the growth of a maximum that moves the reference

// How q . k becomes a score: times a scale that keeps its order (and by which a slope can be
// divided); with slopes; capped, or by another scale, slopes or not; under a cap above kTrSmallCap.
// (A form for all with slopes or a cap, its unused parts jumped over: a 13B-shaped chunk with
// slopes 218 us, this one 194.  One for all caps: that chunk capped at 30, without slopes, 266 us,
// this one 259.)
constexpr float kTrLeastScale = 0x1p-40f;
constexpr float kTrSmallCap = 128.f;
enum TreeForm { kPlainScores, kSlopeScores, kAnyScores, kLargeCapScores };

// What a CTA leaves behind of the unit that its run begins and another one ends.
struct TreeCut {
  long long P, C;   // cost before the unit; of all units
  int32_t n;        // key tiles of the unit; 0: no such unit
  int32_t row0;     // row of q and out of the unit's row 0
  int32_t rows, g;  // rows of the unit, KV head
};

struct TreeArgs {
  const void* q;
  void* out;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;
  const uint32_t* mask;   // [T, W] or NULL: drafted tokens that each row sees
  const int32_t* depths;  // [T] or NULL
  const float* slopes;    // [Hq] or NULL
  const void* v_cache;
  int32_t* status;        // or NULL
  TreeCut* cuts;          // [grid]
  float* part_o;          // [2 * grid][128][D]: O of cut pieces
  float2* part_ml;        // [2 * grid][128]: reference (log2 units) and sum
  int32_t S, T, Hq, Hkv, G, MAXB, NB, bs, W, window;
  int32_t nodes, box;     // drafted tokens of a unit and of one TMA box of q
  float scale_log2;       // without cap: x in log2 units is S * scale_log2
  float cap_log2, cap_z;  // with cap: cap_log2 * tanh, 2^(S * cap_z) = e^(2 x / cap)
  float cap_inv;          // above kTrSmallCap: 1 / cap_log2
};

__device__ __forceinline__ void tr_flag(const TreeArgs& a, int bits) {
  if (a.status) atomicOr(a.status, bits);
}

// Context t, drafted tokens c and first row q0 of sequence s, clamped to 0 <= c <= t <= MAXB *
// bs (with a mask c <= 32 W) and 0 <= q0, q0 + c <= T.
__device__ __forceinline__ void tr_seq(const TreeArgs& a, int s, int& t, int& c, int& q0,
                                       bool report) {
  t = __ldg(a.context_lens + s);
  q0 = __ldg(a.query_start + s);
  const int q1 = __ldg(a.query_start + s + 1);
  const int limit = a.MAXB * a.bs;
  const int most = a.mask != nullptr && static_cast<int64_t>(a.W) * 32 < limit ? a.W * 32 : limit;
  const bool fine = t >= 0 && t <= limit && q0 >= 0 && q1 >= q0 && q1 <= a.T && q1 - q0 <= t &&
                    q1 - q0 <= most;
  c = q1 - q0;
  if (!fine) {
    if (report) tr_flag(a, PKV_DEV_BAD_CONTEXT_LEN);
    t = t < 0 ? 0 : (t > limit ? limit : t);
    q0 = q0 < 0 ? 0 : (q0 > a.T ? a.T : q0);
    const int end = q1 > a.T ? a.T : q1;
    c = end > q0 ? end - q0 : 0;
    c = c > t ? t : c;
    c = c > most ? most : c;
  }
}

__device__ __forceinline__ int tr_depth(const TreeArgs& a, int q0, int i) {
  if (a.depths == nullptr) return i;
  return min(max(__ldg(a.depths + q0 + i), 0), kTrMaxDepth);
}

__device__ __forceinline__ int tr_units(const TreeArgs& a, int c) {
  return (c + a.nodes - 1) / a.nodes;
}

// Keys [lo, hi) that some row of unit `tile` may see.
__device__ __forceinline__ void tr_keys(const TreeArgs& a, int t, int c, int tile, int& lo,
                                        int& hi) {
  const int base = t - c, i0 = tile * a.nodes;
  hi = a.mask != nullptr ? t : base + min(c, i0 + a.nodes);
  lo = 0;
  if (a.window > 0) {  // depths are not negative
    const int p = base + (a.depths != nullptr ? 0 : i0);
    lo = p >= a.window ? p - a.window + 1 : 0;
  }
}

template <int KT>
__device__ __forceinline__ int tr_tiles(const TreeArgs& a, int t, int c, int tile, int& j0) {
  int lo, hi;
  tr_keys(a, t, c, tile, lo, hi);
  j0 = lo / KT;
  return (hi - 1) / KT + 1 - j0;
}

// A unit of n key tiles costs n + kTrUnitCost: its first tile lies at cost P, tile k > 0 at
// P + k + kTrUnitCost.  First tile at or after cost x.
__device__ __forceinline__ int tr_first_tile(long long P, int n, long long x) {
  if (x <= P) return 0;
  const long long k = x - P - kTrUnitCost;
  return k < 1 ? (n < 1 ? n : 1) : (k < n ? static_cast<int>(k) : n);
}

// Where run x of `runs` begins, of C costs.
__device__ __forceinline__ long long tr_border(long long C, int x, int runs) {
  if (C < (1 << 23) && runs <= 256)  // the usual case, in 32 bits
    return static_cast<uint32_t>(C) * static_cast<uint32_t>(x) / static_cast<uint32_t>(runs);
  return C * x / runs;
}

template <int KT>
__device__ __forceinline__ long long tr_seq_cost(const TreeArgs& a, int s, bool report) {
  int t, c, q0, j0;
  tr_seq(a, s, t, c, q0, report);
  long long cost = 0;
  const int nu = tr_units(a, c);
  for (int u = 0; u < nu; ++u) cost += tr_tiles<KT>(a, t, c, u, j0) + kTrUnitCost;
  return cost * a.Hkv;
}

// A CTA's place in the list of units, and the part of the unit there that is its own.
struct TreeWalk {
  int32_t s, g, tile;
  long long P, lo, hi;  // cost before the unit; the CTA's run of costs
  int32_t t, c, q0;     // of sequence s
  int32_t j0, n;        // the unit's first key tile and how many
  int32_t ka, kb;       // of those, the CTA's
};

// Fills in the unit at (s, g, tile); false behind the CTA's last one.
template <int KT>
__device__ __forceinline__ bool tr_unit(const TreeArgs& a, TreeWalk& w) {
  for (;;) {
    if (w.s >= a.S || w.P >= w.hi) return false;
    tr_seq(a, w.s, w.t, w.c, w.q0, false);
    if (w.tile >= tr_units(a, w.c)) {
      w.tile = 0;
      if (w.c == 0 || ++w.g >= a.Hkv) {
        w.g = 0;
        ++w.s;
      }
      continue;
    }
    w.n = tr_tiles<KT>(a, w.t, w.c, w.tile, w.j0);
    w.ka = tr_first_tile(w.P, w.n, w.lo);
    w.kb = tr_first_tile(w.P, w.n, w.hi);
    if (w.kb > w.ka) return true;
    w.P += w.n + kTrUnitCost;
    ++w.tile;
  }
}
template <int KT>
__device__ __forceinline__ bool tr_next(const TreeArgs& a, TreeWalk& w) {
  w.P += w.n + kTrUnitCost;
  ++w.tile;
  return tr_unit<KT>(a, w);
}

// What the roles of a CTA need of a piece, handed out ahead of its use.
struct TreePiece {
  int32_t s, g, tile, t, c, q0, j0, n, ka, kb;  // as in TreeWalk; n = 0: no more
  int32_t pad[2];
};
constexpr int kTrAhead = 2;   // pieces handed out ahead of the one whose V is looked through
// ... and kept: when piece n is looked through, P V of the tile four (the V ring's most) before
// is done, so the pieces up to n - 6 are read out, and the slot of piece n + 2 is free.
constexpr int kTrPieces = 8;

enum {
  kTrKFull = 0,     // [6] K stage landed (TMA bytes)
  kTrKEmpty = 6,    // [6] K stage consumed (commit after S)
  kTrVFull = 12,    // [6] V stage landed
  kTrVEmpty = 18,   // [6] V stage consumed (commit after P V) and passed by the looking warp
  kTrVReady = 24,   // [6] V stage looked through (only tiles that need it)
  kTrQFull = 30,    // query tile landed
  kTrQEmpty = 31,   // query tile consumed (commit after the piece's last S)
  kTrSFull = 32,    // [2] S in tensor memory (commit)
  kTrSEmpty = 34,   // [2] S read by the row warps
  kTrPFull = 36,    // [2] P in tensor memory (row warps)
  kTrPvDone = 38,   // [2] P V done (commit)
  kTrOEmpty = 40,   // the piece's O read out by the row warps
  kTrDrain = 41,    // every MMA of the CTA done (final commit)
  kTrPiece = 42,    // [8] piece handed out
  kTrBars = 50
};
constexpr uint32_t kTrSlotOff = 8 * kTrBars;       // tensor-memory base address
constexpr uint32_t kTrDeadOff = kTrSlotOff + 8;    // [4] give-up bits of the row-warp pairs
constexpr uint32_t kTrOddOff = kTrDeadOff + 16;    // [8] a piece met values of V that are not finite
constexpr uint32_t kTrPieceOff = (kTrOddOff + 32 + 15) / 16 * 16;
constexpr uint32_t kTrBarArea = 1024;
static_assert(kTrPieceOff + kTrPieces * sizeof(TreePiece) <= kTrBarArea, "barrier area");

template <typename T, int D>
struct TreeShape {
  static constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  static constexpr int KT = D == 256 ? 64 : 128;      // keys of a tile
  static constexpr int kHalfKeys = KT / 2;            // a row thread's
  static constexpr int kChunks = D * 2 / 128;         // 128-byte column chunks of a row
  static constexpr uint32_t kQTile = kTrRows * D * 2;
  static constexpr uint32_t kTile = KT * D * 2;       // K or V tile
  static constexpr uint32_t kGroup = kChunks * 1024;  // 8 keys of a tile, every chunk
  static constexpr int kK = D == 64 ? 6 : (D == 128 ? 3 : 2);  // K ring
  static constexpr int kV = D == 64 ? 4 : 3;                   // V ring
  static constexpr uint32_t kQOff = 0;
  static constexpr uint32_t kKOff = kQTile;
  static constexpr uint32_t kVOff = kKOff + kK * kTile;
  static constexpr uint32_t kBarOff = kVOff + kV * kTile;
  static constexpr uint32_t kXchOff = kBarOff + kTrBarArea;  // [2 turns][2 halves][128] floats
  static constexpr uint32_t kBytes = kXchOff + 4 * kTrRows * 4;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kOCol = 256;                              // O: D columns
  static constexpr uint32_t kPCol = D == 256 ? 2 * KT : 384;          // P[b]: KT / 2 columns each
  static constexpr uint32_t kIdQK = ptx::idesc_f16(kTrRows, KT, kBf16, false);
  static constexpr uint32_t kIdPV = ptx::idesc_f16(kTrRows, D, kBf16, true);
  static constexpr int kHalfD = D / 2;                                // O columns of a row thread
  // P = 2^(x - m + shift): f16 loses values below 2^-24, so its P uses the range above 1 too
  static constexpr float kShift = kBf16 ? 0.f : 7.f;
  static_assert(kV <= 4 && kK <= 6, "barriers, and the pieces kept");
  static_assert(2 * KT <= kOCol && kBytes <= 232448, "tensor and shared memory");
  static_assert(D == 256 ? kPCol + KT <= kOCol : (kOCol + D <= kPCol && kPCol + KT <= kTmemCols),
                "tensor memory");
};

// 16 consecutive 32-bit columns of this thread's lane, waited for.  Whole warp.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// N consecutive 32-bit words (16-byte aligned), 32 bytes a store where the address allows it.
template <int N>
__device__ __forceinline__ void st_row(void* to, const uint32_t* y) {
  uint32_t* const p = static_cast<uint32_t*>(to);
  if ((reinterpret_cast<uintptr_t>(to) & 31u) == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 8)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + i),
                   "r"(y[i]), "r"(y[i + 1]), "r"(y[i + 2]), "r"(y[i + 3]), "r"(y[i + 4]),
                   "r"(y[i + 5]), "r"(y[i + 6]), "r"(y[i + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<uint4*>(p + i) = make_uint4(y[i], y[i + 1], y[i + 2], y[i + 3]);
  }
}
// max(a, b, c), one instruction.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// 1 / x, one instruction.
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// min(a, b), NaN if one is.
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// cap * tanh z of two scores x, 2^(x cap_z) = e^2z: tanh z = 1 - 2 / (1 + e^2z), off by some 3e-7
// of the cap, however small the score: up to kTrSmallCap that is 4e-5, below an eighth of f16's half
// step, of the probability that follows.  (One reciprocal for four scores, of their product, was 5% faster for a 70B-shaped
// batch of small trees, 206 against 216 us, and 18% slower where tiles are full, 303 against 257:
// a NaN then needs its neighbours done again, each by itself.)
__device__ __forceinline__ void tanh_cap2(uint32_t& v0, uint32_t& v1, float cap_z, float cap) {
  float x, y;
  ptx::unpair(ptx::mul2(ptx::pair(__uint_as_float(v0), __uint_as_float(v1)),
                        ptx::pair(cap_z, cap_z)), x, y);
  ptx::unpair(ptx::add2(ptx::pair(ptx::ex2(x), ptx::ex2(y)), ptx::pair(1.f, 1.f)), x, y);
  ptx::unpair(ptx::fma2(ptx::pair(rcp_approx(x), rcp_approx(y)),
                        ptx::pair(-2.f * cap, -2.f * cap), ptx::pair(cap, cap)), x, y);
  v0 = __float_as_uint(x);
  v1 = __float_as_uint(y);
}

// The same for any cap, off by some 1e-6 of the capped score itself: for |z| <= 1/2, where the form
// above cancels, x (tanh z / z) with the Taylor series of tanh z / z up to z^14 (the next term is
// below 2^-26).  Both forms are computed: a 70B-shaped batch of small trees 308 us, 215 under a small
// cap.  by: the scores' scale in log2 units; inv: 1 / cap.
__device__ __forceinline__ void tanh_any_cap2(uint32_t& v0, uint32_t& v1, float by, float inv,
                                              float cap) {
  const uint64_t x = ptx::mul2(ptx::pair(__uint_as_float(v0), __uint_as_float(v1)),
                               ptx::pair(by, by));
  const uint64_t z = ptx::mul2(x, ptx::pair(inv, inv)), u = ptx::mul2(z, z);
  constexpr float kC[7] = {21844.f / 6081075.f, -1382.f / 155925.f, 62.f / 2835.f, -17.f / 315.f,
                           2.f / 15.f,          -1.f / 3.f,         1.f};
  uint64_t p = ptx::pair(-929569.f / 638512875.f, -929569.f / 638512875.f);
#pragma unroll
  for (int i = 0; i < 7; ++i) p = ptx::fma2(p, u, ptx::pair(kC[i], kC[i]));
  float z0, z1, y0, y1, w0, w1;
  ptx::unpair(z, z0, z1);
  ptx::unpair(ptx::mul2(x, p), y0, y1);
  constexpr float kTwoLog2e = 2.8853900817779268f;
  ptx::unpair(ptx::add2(ptx::pair(ptx::ex2(z0 * kTwoLog2e), ptx::ex2(z1 * kTwoLog2e)),
                        ptx::pair(1.f, 1.f)), w0, w1);
  ptx::unpair(ptx::mul2(ptx::fma2(ptx::pair(rcp_approx(w0), rcp_approx(w1)), ptx::pair(-2.f, -2.f),
                                  ptx::pair(1.f, 1.f)), ptx::pair(cap, cap)), w0, w1);
  v0 = __float_as_uint(fabsf(z0) <= 0.5f ? y0 : w0);
  v1 = __float_as_uint(fabsf(z1) <= 0.5f ? y1 : w1);
}

__device__ __forceinline__ uint64_t low_bits(int n) {
  return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1);
}

// Bits [at, at + 64) of a row of W words (at >= 0; bits past the words are 0).
__device__ __forceinline__ uint64_t bits_of(const uint32_t* row, int W, int at) {
  const int w = at >> 5, sh = at & 31;
  const uint32_t x0 = w < W ? __ldg(row + w) : 0u;
  const uint32_t x1 = w + 1 < W ? __ldg(row + w + 1) : 0u;
  const uint32_t x2 = w + 2 < W ? __ldg(row + w + 2) : 0u;
  const uint32_t lo = __funnelshift_r(x0, x1, sh), hi = __funnelshift_r(x1, x2, sh);
  return static_cast<uint64_t>(hi) << 32 | lo;
}

// Which of the keys k0 .. k0 + n - 1 (n <= 64) drafted token i sees, bit by bit.
__device__ __forceinline__ uint64_t tr_sees(const TreeArgs& a, const TreeWalk& w, int i, int depth,
                                            int k0, int n) {
  const int base = w.t - w.c;
  uint64_t vis;
  if (a.mask == nullptr) {
    vis = low_bits(base + i + 1 - k0);
  } else {
    vis = low_bits(base - k0);
    if (k0 + n > base) {
      const uint32_t* const row = a.mask + static_cast<int64_t>(w.q0 + i) * a.W;
      const int at = k0 - base;  // drafted token of bit 0
      const uint64_t m = at >= 0 ? bits_of(row, a.W, at) : bits_of(row, a.W, 0) << -at;
      vis |= m & low_bits(w.t - k0);
    }
  }
  if (a.window > 0) {
    const int pos = base + depth;
    if (a.depths == nullptr) {
      vis &= ~low_bits(max(pos - a.window + 1, 0) - k0);
    } else {
      vis &= ~low_bits(min(max(pos - a.window + 1, 0), base) - k0);
      if (depth >= a.window) {
        for (int e = max(0, base - k0); e < n && k0 + e < w.t; ++e)
          if (depth - tr_depth(a, w.q0, k0 + e - base) >= a.window) vis &= ~(1ull << e);
      }
    }
  }
  return n >= 64 ? vis : vis & low_bits(n);
}

// Whether a drafted key's place does not tell which rows see it.
__device__ __forceinline__ bool tr_by_row(const TreeArgs& a) {
  return a.mask != nullptr || (a.depths != nullptr && a.window > 0);
}

// Keys whose values must not reach every row of a unit, as up to two ranges: those that some row
// sees and another does not, and the rest of the first and last cache blocks that are read.
// There, values of V that are not finite would (0 * infinity).  Depths let a window hide a drafted
// token from any row, in whatever order they stand.
__device__ __forceinline__ void tr_mixed(const TreeArgs& a, const TreeWalk& w, int (&from)[2],
                                         int (&to)[2]) {
  const int base = w.t - w.c, i0 = w.tile * a.nodes, last = min(w.c, i0 + a.nodes) - 1;
  int lo, hi;
  tr_keys(a, w.t, w.c, w.tile, lo, hi);
  from[1] = tr_by_row(a) ? base : base + i0 + 1;
  to[1] = (hi + a.bs - 1) & -a.bs;
  from[0] = lo & -a.bs;
  to[0] = lo;
  if (a.window > 0)
    to[0] = min(max(base + (a.depths != nullptr ? w.c - 1 : last) - a.window + 1, lo), from[1]);
}

// Whether tile k has any of them.
template <int KT>
__device__ __forceinline__ bool tr_special(const TreeArgs& a, const TreeWalk& w, int k) {
  const int k0 = (w.j0 + k) * KT;
  int from[2], to[2];
  tr_mixed(a, w, from, to);
  return max(from[0], k0) < min(to[0], k0 + KT) || max(from[1], k0) < min(to[1], k0 + KT);
}

// Two 16-bit values.
template <typename T>
using PairOf = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
template <typename T>
__device__ __forceinline__ PairOf<T> as_pair(uint32_t x) {
  return *reinterpret_cast<PairOf<T>*>(&x);
}
template <typename P>
__device__ __forceinline__ uint32_t pair_bits(P x) {
  return *reinterpret_cast<uint32_t*>(&x);
}
template <typename T>
__device__ __forceinline__ bool odd_pair(uint32_t x) {  // one of the two is not finite
  constexpr uint32_t e = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
  return (x & e) == e || (x & (e << 16)) == (e << 16);
}
template <typename T>
__device__ __forceinline__ uint32_t finite_pair(uint32_t x) {  // 0 in place of what is not finite
  constexpr uint32_t e = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
  if ((x & e) == e) x &= 0xffff0000u;
  if ((x & (e << 16)) == (e << 16)) x &= 0xffffu;
  return x;
}

template <typename T, int D, TreeForm kForm>
__global__ void __launch_bounds__(kTrThreads, 1)
    tree_attention_kernel(const __grid_constant__ CUtensorMap qmap,
                          const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap vmap, const TreeArgs a) {
  constexpr bool kSlopes = kForm != kPlainScores;
  using Sh = TreeShape<T, D>;
  constexpr int KT = Sh::KT, HK = Sh::kHalfKeys, HD = Sh::kHalfD;
  constexpr uint32_t NK = Sh::kK, NV = Sh::kV;
  // The joining kernel may be launched: it waits for the whole of this grid.  This grid itself
  // may have been launched ahead of the end of what is in front of it: nothing is read or
  // written in memory before the wait below.
  asm volatile("griddepcontrol.launch_dependents;");
  // swizzled tiles lie on 1,024-byte boundaries (there is no room to look for one)
  extern __shared__ __align__(1024) uint8_t base_p[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base_s = ptx::smem_addr(base_p);
  if ((base_s & 1023u) != 0) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x == 0) {
      tr_flag(a, PKV_DEV_WAIT_TIMEOUT);
      a.cuts[blockIdx.x] = TreeCut{0, 0, 0, 0, 0, 0};
    }
    return;
  }
  const uint32_t bars = base_s + Sh::kBarOff;
  const int BS = a.bs, bs_log = 31 - __clz(a.bs);
  auto bar = [&](int i) { return bars + 8u * static_cast<uint32_t>(i); };
  uint32_t* const slot = reinterpret_cast<uint32_t*>(base_p + Sh::kBarOff + kTrSlotOff);
  volatile int* const odd_seen = reinterpret_cast<volatile int*>(base_p + Sh::kBarOff + kTrOddOff);
  TreePiece* const pieces = reinterpret_cast<TreePiece*>(base_p + Sh::kBarOff + kTrPieceOff);

  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&qmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&vmap)) : "memory");
    for (int i = 0; i < kTrBars; ++i) {
      const bool rows = i == kTrOEmpty || (i >= kTrSEmpty && i < kTrPvDone);
      const bool two = i >= kTrVEmpty && i < kTrVReady;
      ptx::mbar_init(bar(i), rows ? kTrRowWarps : (two ? 2 : 1));
    }
    ptx::fence_barrier_init();
    for (int i = 0; i < 4; ++i) reinterpret_cast<int*>(base_p + Sh::kBarOff + kTrDeadOff)[i] = 0;
    for (int i = 0; i < 8; ++i) odd_seen[i] = 0;
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_addr(slot), Sh::kTmemCols);
    ptx::tmem_relinquish();
  }
  // Every thread waits: lengths, masks and depths may have been written by the kernel in front as well
  // as the caches, a joining kernel there may still read its cuts, and whatever comes behind this
  // call relies on all in front of it being done.
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- costs of all sequences summed up (in the K ring, free until the first load) --------
  long long* const cpre = reinterpret_cast<long long*>(base_p + Sh::kKOff);
  {
    long long* const wsum = cpre + a.S + 1;
    const int tid = threadIdx.x;
    const int per = (a.S + kTrThreads - 1) / kTrThreads;
    const int b0 = min(a.S, tid * per), b1 = min(a.S, b0 + per);
    long long local = 0;
    for (int s = b0; s < b1; ++s) local += tr_seq_cost<KT>(a, s, blockIdx.x == 0);
    long long x = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    long long run = x - local;
    for (int w = 0; w < warp; ++w) run += wsum[w];
    for (int s = b0; s < b1; ++s) {
      cpre[s] = run;
      run += per > 1 ? tr_seq_cost<KT>(a, s, false) : local;
    }
    if (tid == kTrThreads - 1) cpre[a.S] = run;
    ptx::fence_proxy_async_smem();  // the rings' copies come after these stores
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *slot;
  auto read_piece = [&](uint32_t n, TreeWalk& w) {
    const int4* const p = reinterpret_cast<const int4*>(pieces + n % kTrPieces);
    const int4 x = p[0], y = p[1], z = p[2];
    w.s = x.x, w.g = x.y, w.tile = x.z, w.t = x.w;
    w.c = y.x, w.q0 = y.y, w.j0 = y.z, w.n = y.w;
    w.ka = z.x, w.kb = z.y;
  };
  // The next piece (the n-th) of the CTA; n = 0 in it: no more.  Whole warp; false: timed out.
  auto get_piece = [&](uint32_t n, TreeWalk& w) {
    if (!__all_sync(0xffffffffu, ptx::mbar_wait(bar(kTrPiece + n % kTrPieces),
                                                (n / kTrPieces) & 1u, kTrWaitNs)))
      return false;
    read_piece(n, w);
    return true;
  };

  if (warp == kTrQWarp) {
    // ---- the CTA's run and its pieces, the query tiles (TMA), and V looked through where rows
    // of it must not reach every query ------------------------------------------------------
    TreeWalk w{};  // the next piece to hand out
    {
      // lane 0 looks for the unit in which the run begins, lane 1 for the one in which it ends
      const long long C = cpre[a.S];
      const long long lo = tr_border(C, blockIdx.x, gridDim.x);
      const long long hi = tr_border(C, blockIdx.x + 1, gridDim.x);
      const long long at = lane == 1 ? hi - 1 : lo;
      int s = a.S, g = 0, u = 0, n = 0, t = 0, c = 0, q0 = 0, j0;
      long long P = 0;
      if (lane < 2 && hi > lo) {
        int l = 0, h = a.S;  // the last sequence with cpre <= at: `at` lies in one of its units
        while (h - l > 1) {
          const int mid = (l + h) >> 1;
          if (cpre[mid] <= at) l = mid; else h = mid;
        }
        s = l;
        tr_seq(a, s, t, c, q0, false);
        const long long cost = cpre[s + 1] - cpre[s], in = at - cpre[s];
        const long long cost_g = cost < (1 << 30) ? static_cast<int>(cost) / a.Hkv : cost / a.Hkv;
        g = static_cast<int>(cost < (1 << 30) ? static_cast<int>(in) / static_cast<int>(cost_g)
                                              : in / cost_g);
        P = cpre[s] + g * cost_g;
        for (;; ++u) {
          n = tr_tiles<KT>(a, t, c, u, j0);
          if (P + n + kTrUnitCost > at) break;
          P += n + kTrUnitCost;
        }
      }
      if (lane == 1) {
        // the unit that this run begins and another ends, for the joining kernel
        TreeCut cut{0, C, 0, 0, 0, 0};
        if (hi > lo && hi < C && P >= lo && tr_first_tile(P, n, hi) < n) {
          cut.P = P;
          cut.n = n;
          cut.row0 = q0 + u * a.nodes;
          cut.rows = min(a.nodes, c - u * a.nodes) * a.G;
          cut.g = g;
        }
        a.cuts[blockIdx.x] = cut;
      }
      __syncwarp();
      w.s = __shfl_sync(0xffffffffu, s, 0);
      w.g = __shfl_sync(0xffffffffu, g, 0);
      w.tile = __shfl_sync(0xffffffffu, u, 0);
      w.P = __shfl_sync(0xffffffffu, P, 0);
      w.lo = lo;
      w.hi = hi;
    }
    uint32_t out = 0;  // pieces handed out
    bool more = tr_unit<KT>(a, w);
    auto hand_out = [&]() {
      if (lane == 0) {
        int4* const p = reinterpret_cast<int4*>(pieces + out % kTrPieces);
        p[0] = make_int4(w.s, w.g, w.tile, w.t);
        p[1] = make_int4(w.c, w.q0, w.j0, more ? w.n : 0);
        p[2] = make_int4(w.ka, w.kb, 0, 0);
        ptx::mbar_arrive(bar(kTrPiece + out % kTrPieces));
      }
      __syncwarp();
      ++out;
      if (more) more = tr_next<KT>(a, w);
    };
    uint32_t loaded = 0, it = 0;  // pieces whose queries are loaded; tiles
    bool alive = true;
    const uint64_t policy = ptx::policy_evict_first();
    auto load_q = [&](const TreeWalk& u) {
      const int here = min(a.nodes, u.c - u.tile * a.nodes);
      const int boxes = (here + a.box - 1) / a.box;
      const uint32_t box_bytes = static_cast<uint32_t>(a.box * a.G) * 128u;
      bool ok = true;
      if (lane == 0) {
        ok = ptx::mbar_wait(bar(kTrQEmpty), (loaded & 1u) ^ 1u, kTrWaitNs);
        if (ok) ptx::mbar_arrive_expect_tx(bar(kTrQFull), boxes * box_bytes * Sh::kChunks);
      }
      if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
      __syncwarp();
      for (int i = lane; i < boxes * Sh::kChunks; i += 32) {
        const int bx = i / Sh::kChunks, cc = i - bx * Sh::kChunks;
        ptx::tma_load_3d(base_s + Sh::kQOff + cc * kTrChunk + bx * box_bytes, &qmap, cc * 64,
                         u.g * a.G, u.q0 + u.tile * a.nodes + bx * a.box, bar(kTrQFull), policy);
      }
      ++loaded;
      return true;
    };
    auto look_through = [&](uint32_t vt, const TreeWalk& u, int k, uint32_t n) {
      // values that are not finite are taken out, and added to the rows that see them at the
      // end.  Products with 0, summed up, show whether there are any: one instruction for two
      // values.  (Taking nothing out costs no fence: one between this warp's stores and the
      // tensor cores' reads waits for the copies in flight, some microseconds.)
      const int k0 = (u.j0 + k) * KT;
      int from[2], to[2];
      tr_mixed(a, u, from, to);
      bool wrote = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r0 = max(0, from[e] - k0), r1 = min(KT, to[e] - k0);
        PairOf<T> sum = as_pair<T>(0u);
        for (int g = r0 >> 3; g < (r1 + 7) >> 3; ++g) {  // 8 rows: 2 * kChunks pieces a lane
          uint32_t v[2 * Sh::kChunks][4];
          const uint32_t at = vt + g * Sh::kGroup + lane * 16;
#pragma unroll
          for (int x = 0; x < 2 * Sh::kChunks; ++x)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[x][0]), "=r"(v[x][1]), "=r"(v[x][2]), "=r"(v[x][3])
                         : "r"(at + 512 * x));
#pragma unroll
          for (int x = 0; x < 2 * Sh::kChunks; ++x) {
#pragma unroll
            for (int q = 0; q < 4; ++q) sum = __hfma2(as_pair<T>(v[x][q]), as_pair<T>(0u), sum);
          }
        }
        if (r1 <= r0 || !__any_sync(0xffffffffu, odd_pair<T>(pair_bits(sum)))) continue;
        for (uint32_t i = lane; i < static_cast<uint32_t>((r1 + 7) >> 3) * (Sh::kGroup / 16);
             i += 32) {
          const int row = 8 * (i / (Sh::kGroup / 16)) + ((i >> 3) & 7);
          if (row < r0 || row >= r1) continue;
          const uint32_t at = vt + 16 * i;
          uint32_t v[4];
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                       : "r"(at));
          bool any = false;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            any |= odd_pair<T>(v[q]);
            v[q] = finite_pair<T>(v[q]);
          }
          if (any) ptx::st_shared_v4(at, v[0], v[1], v[2], v[3]);
          wrote |= any;
        }
      }
      if (__any_sync(0xffffffffu, wrote)) {
        if (lane == 0) odd_seen[n % kTrPieces] = 1;
        __threadfence_block();
        ptx::fence_proxy_async_smem();
        __syncwarp();
      }
    };
    for (int i = 0; i < kTrAhead; ++i) hand_out();
    TreeWalk u{}, next{};
    alive = get_piece(0, u);
    if (alive && u.n > 0) alive = load_q(u);
    for (uint32_t n = 0; alive && u.n > 0; ++n) {
      if (lane == 0) odd_seen[n % kTrPieces] = 0;  // (its last user has been read out)
      hand_out();
      alive = get_piece(n + 1, next);
      for (int k = u.ka; alive && k < u.kb; ++k, ++it) {
        // the next queries are loaded once the piece's last S is done, which waits for the
        // products two tiles before: for no tile of V from here on
        if (k == u.kb - 1 && next.n > 0 && !(alive = load_q(next))) break;
        // every tile is waited for, so that no phase of its barrier is missed
        const uint32_t st = it % NV;
        alive = __all_sync(0xffffffffu,
                           ptx::mbar_wait(bar(kTrVFull + st), (it / NV) & 1u, kTrWaitNs));
        if (!alive) break;
        const bool special = tr_special<KT>(a, u, k);
        if (special) look_through(base_s + Sh::kVOff + st * Sh::kTile, u, k, n);
        if (lane == 0) {
          if (special) ptx::mbar_arrive(bar(kTrVReady + st));
          ptx::mbar_arrive(bar(kTrVEmpty + st));
        }
      }
      u = next;
    }
    if (lane == 0) {
      if (!alive) tr_flag(a, PKV_DEV_WAIT_TIMEOUT);
      if (loaded > 0)  // the copy in flight lands first
        ptx::mbar_wait(bar(kTrQFull), (loaded - 1) & 1u, kTrWaitNs / 8);
    }
  } else if (warp == 0 || warp == kTrVWarp) {
    // ---- TMA producers of K (warp 0) and V (warp 10) ---------------------------------
    const bool is_k = warp == 0;
    const uint64_t policy = ptx::policy_evict_normal();
    const int32_t groups_total = a.NB * a.Hkv * (BS / 8);  // 8-row groups of the cache
    const int nblk = KT >> bs_log;                         // cache blocks of a tile
    const CUtensorMap* const map = is_k ? &kmap : &vmap;
    const int full0 = is_k ? kTrKFull : kTrVFull, empty0 = is_k ? kTrKEmpty : kTrVEmpty;
    const uint32_t ring = base_s + (is_k ? Sh::kKOff : Sh::kVOff);
    const uint32_t NS = is_k ? NK : NV;
    uint32_t it = 0;
    TreeWalk w{};
    bool alive = true;
    for (uint32_t n = 0; alive; ++n) {
      if (!get_piece(n, w)) { alive = false; break; }
      if (w.n == 0) break;
      int lo, hi;
      tr_keys(a, w.t, w.c, w.tile, lo, hi);
      for (int k = w.ka; k < w.kb; ++k, ++it) {
        const uint32_t st = it % NS;
        const int bi = nblk * (w.j0 + k) + (lane & (nblk - 1));
        int32_t y = groups_total;  // a box wholly past the end: zero-filled
        // blocks behind the last key, and those that the window has left behind, are not read
        if (lane < nblk && bi * BS < hi && (bi + 1) * BS > lo) {
          const int id = __ldg(a.block_tables + static_cast<int64_t>(w.s) * a.MAXB + bi);
          if (static_cast<uint32_t>(id) < static_cast<uint32_t>(a.NB))
            y = (id * a.Hkv + w.g) * (BS / 8);
          else if (is_k)
            tr_flag(a, PKV_DEV_BAD_BLOCK_ID);
        }
        bool ok = true;
        if (lane == 0) {
          ok = ptx::mbar_wait(bar(empty0 + st), ((it / NS) & 1u) ^ 1u, kTrWaitNs);
          if (ok) ptx::mbar_arrive_expect_tx(bar(full0 + st), Sh::kTile);
        }
        if (!__shfl_sync(0xffffffffu, ok, 0)) { alive = false; break; }
        __syncwarp();
        if (lane < nblk)
          ptx::tma_load_4d(ring + st * Sh::kTile + lane * (BS / 8) * Sh::kGroup, map, 0, 0, 0, y,
                           bar(full0 + st), policy);
      }
    }
    if (lane == 0) {
      if (!alive) tr_flag(a, PKV_DEV_WAIT_TIMEOUT);
      for (uint32_t k = it > NS ? it - NS : 0; k < it; ++k)  // copies in flight land first
        ptx::mbar_wait(bar(full0 + k % NS), (k / NS) & 1u, kTrWaitNs / 8);
    }
  } else if (warp == 1) {
    // ---- MMA issuer: S of a tile ahead of P V of the one before, across pieces too --------
    uint32_t it = 0;
    bool alive = true;
    auto wait1 = [&](uint32_t b, uint32_t parity) {
      return __all_sync(0xffffffffu, ptx::mbar_wait(b, parity, kTrWaitNs)) != 0;
    };
    uint32_t ready = 0;  // phases of the V stages' kTrVReady
    // O (+)= P V for tile k of piece n (the x-th tile of the CTA)
    auto pv = [&](uint32_t x, bool begins, bool special, uint32_t n) {
      const int b = static_cast<int>(x & 1u);
      const uint32_t st = x % NV;
      if (begins && !wait1(bar(kTrOEmpty), (n & 1u) ^ 1u)) return false;
      if (!wait1(bar(kTrVFull + st), (x / NV) & 1u)) return false;
      if (special) {
        if (!wait1(bar(kTrVReady + st), (ready >> st) & 1u)) return false;
        ready ^= 1u << st;
      }
      if (!wait1(bar(kTrPFull + b), (x >> 1) & 1u)) return false;
      ptx::tc_fence_after();
      const uint32_t vt = base_s + Sh::kVOff + st * Sh::kTile;
      const uint32_t pt = tmem + Sh::kPCol + b * (KT / 2);
#pragma unroll
      for (int ks = 0; ks < KT / 16; ++ks)  // 16 keys = 8 packed columns of P
        ptx::umma_f16_ta_elect(tmem + Sh::kOCol, pt + ks * 8,
                               ptx::smem_desc_sw128(vt + ks * 2 * Sh::kGroup, 1024, Sh::kGroup),
                               Sh::kIdPV, !begins || ks > 0);
      ptx::umma_commit_elect(bar(kTrPvDone + b));
      ptx::umma_commit_elect(bar(kTrVEmpty + st));
      __syncwarp();
      return true;
    };
    bool pending = false;  // a P V not issued yet: the px-th tile, in piece pn
    uint32_t px = 0, pn = 0;
    bool p_begins = false, p_special = false;
    TreeWalk w{};
    for (uint32_t n = 0; alive; ++n) {
      if (!get_piece(n, w)) { alive = false; break; }
      if (w.n == 0) break;
      if (!wait1(bar(kTrQFull), n & 1u)) { alive = false; break; }
      ptx::tc_fence_after();
      for (int k = w.ka; k < w.kb; ++k, ++it) {
        const uint32_t st = it % NK;
        const int b = static_cast<int>(it & 1u);
        if (!wait1(bar(kTrKFull + st), (it / NK) & 1u) ||
            !wait1(bar(kTrSEmpty + b), ((it >> 1) & 1u) ^ 1u)) {
          alive = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t qa = base_s + Sh::kQOff;
        const uint32_t kb = base_s + Sh::kKOff + st * Sh::kTile;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t kin = (ks & 3) * 32;  // 16 columns inside a 128-byte chunk
          ptx::umma_f16_elect(tmem + b * KT,
                              ptx::smem_desc_sw128(qa + (ks >> 2) * kTrChunk + kin, 16, 1024),
                              ptx::smem_desc_sw128(kb + (ks >> 2) * 1024 + kin, 16, Sh::kGroup),
                              Sh::kIdQK, ks > 0);
        }
        ptx::umma_commit_elect(bar(kTrSFull + b));
        ptx::umma_commit_elect(bar(kTrKEmpty + st));
        if (k == w.kb - 1) ptx::umma_commit_elect(bar(kTrQEmpty));
        __syncwarp();
        if (pending && !pv(px, p_begins, p_special, pn)) { alive = false; break; }
        pending = true;
        px = it;
        pn = n;
        p_begins = k == w.ka;
        p_special = tr_special<KT>(a, w, k);
      }
    }
    if (alive && pending && !pv(px, p_begins, p_special, pn)) alive = false;
    if (lane == 0) {
      if (!alive) tr_flag(a, PKV_DEV_WAIT_TIMEOUT);
      ptx::umma_commit(bar(kTrDrain));  // lands once every MMA issued above is done
      ptx::mbar_wait(bar(kTrDrain), 0, kTrWaitNs);
    }
    __syncwarp();
  } else {
    // ---- row threads: scores, softmax, output ------------------------------------------
    // The two warps of a lane quarter meet at every exchange (named barrier).  A warp whose wait
    // ran out flags itself, arrives there once without waiting, and leaves; the other one
    // finds the flag at its next exchange.  A quarter without rows only keeps the hand-offs going.
    const int q4 = warp & 3, h = (warp - 2) >> 2;
    const int r = 32 * q4 + lane;  // tile row = tensor-memory lane
    const int rn = r / a.G, rh = r - rn * a.G;
    const uint32_t lane_off = static_cast<uint32_t>(32 * q4) << 16;
    const uint32_t pcol = tmem + lane_off + Sh::kPCol + h * (HK / 2);
    const uint32_t oa = tmem + lane_off + Sh::kOCol + h * HD;  // this thread's half of O
    float* const xch = reinterpret_cast<float*>(base_p + Sh::kXchOff);
    int* const dead_bits = reinterpret_cast<int*>(base_p + Sh::kBarOff + kTrDeadOff);
    const uint32_t pair_bar = 1 + q4;
    bool gone = false;       // this warp leaves: a wait ran out, or the other one has left
    bool pair_dead = false;  // ... the latter
    // the other half's x for this row; two buffers in turn: a value has been read once its
    // reader comes to the next exchange
    uint32_t turn = 0;
    auto exchange = [&](float x) {
      float* const at = xch + (turn ^= 2 * kTrRows);
      at[h * kTrRows + r] = x;
      ptx::named_bar_sync(pair_bar, 64);
      pair_dead = *reinterpret_cast<volatile int*>(dead_bits + q4) != 0;
      gone |= pair_dead;
      return at[(1 - h) * kTrRows + r];
    };
    auto wait_all = [&](uint32_t b, uint32_t parity) {
      gone = !__all_sync(0xffffffffu, ptx::mbar_wait(b, parity, kTrWaitNs));
      return !gone;
    };
    // A piece's output is written after the first tile of the next (its last P V is done by
    // then), so that the tensor cores are not left waiting on it.
    bool pend = false, pend_live = false, pend_valid = false;
    float pend_m = 0.f, pend_l = 0.f;
    uint32_t pend_x = 0, pend_n = 0;
    auto epilogue = [&]() {
      pend = false;
      float lt = pend_l;
      if (pend_live) lt += exchange(pend_l);
      if (gone || !wait_all(bar(kTrPvDone + (pend_x & 1u)), (pend_x >> 1) & 1u)) return;
      if (pend_live) {
        ptx::tc_fence_after();
        TreeWalk pu;
        read_piece(pend_n, pu);
        const bool whole = pu.ka == 0 && pu.kb == pu.n;
        // a piece that begins its unit is the run's last one, another its first
        const int64_t cut_row =
            (2 * static_cast<int64_t>(blockIdx.x) + (pu.ka == 0 ? 1 : 0)) * kTrRows + r;
        const int node = pu.tile * a.nodes + rn;
        T* const out_row = static_cast<T*>(a.out) +
                           (static_cast<int64_t>(pu.q0 + node) * a.Hq + pu.g * a.G + rh) * D +
                           h * HD;
        float* const part_row = a.part_o + cut_row * D + h * HD;
        if (!whole && pend_valid && h == 0) a.part_ml[cut_row] = make_float2(pend_m, lt);
        const float inv = whole ? (lt == 0.f ? 0.f : 1.f / lt) : 1.f;
        const bool odd = odd_seen[pend_n % kTrPieces] != 0;
#pragma unroll 1
        for (int c0 = 0; c0 < HD; c0 += 32) {
          uint32_t o[32];
          ptx::tmem_ld32(oa + c0, o);
          if (!pend_valid) continue;
          if (odd) {  // values of V that are not finite, for the rows that see them
            int from[2], to[2];
            tr_mixed(a, pu, from, to);
            const int first_key = (pu.j0 + pu.ka) * KT, last_key = (pu.j0 + pu.kb) * KT;
            const int depth = tr_depth(a, pu.q0, node);
            for (int e = 0; e < 2; ++e) {
              for (int p = max(from[e], first_key); p < min(to[e], last_key); ++p) {
                if (tr_sees(a, pu, node, depth, p, 1) == 0) continue;
                const int id =
                    __ldg(a.block_tables + static_cast<int64_t>(pu.s) * a.MAXB + (p >> bs_log));
                if (static_cast<uint32_t>(id) >= static_cast<uint32_t>(a.NB)) continue;
                const T* const vr =
                    static_cast<const T*>(a.v_cache) +
                    ((static_cast<int64_t>(id) * a.Hkv + pu.g) * BS + (p & (BS - 1))) * D +
                    h * HD + c0;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  const float v = ptx::to_float(vr[i]);
                  if (!isfinite(v)) o[i] = __float_as_uint(__uint_as_float(o[i]) + v);
                }
              }
            }
          }
          if (whole) {
            uint32_t y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              y[i] = ptx::pack2<T>(__uint_as_float(o[2 * i]) * inv,
                                   __uint_as_float(o[2 * i + 1]) * inv);
            st_row<16>(out_row + c0, y);
          } else {
            st_row<32>(part_row + c0, o);
          }
        }
        ptx::tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(kTrOEmpty));
    };
    uint32_t it = 0;
    TreeWalk w{};
    for (uint32_t n = 0; !gone; ++n) {
      if (!get_piece(n, w)) { gone = true; break; }
      if (w.n == 0) break;
      const int here = min(a.nodes, w.c - w.tile * a.nodes);
      const bool live = 32 * q4 < here * a.G;  // a row of this quarter
      const bool valid = rn < here;
      const int node = w.tile * a.nodes + (valid ? rn : 0);
      const int base = w.t - w.c;
      const int depth = live ? tr_depth(a, w.q0, node) : 0;
      // keys at these places are seen whatever the mask: no need to look at each
      const int clear_to = tr_by_row(a) ? base : base + node + 1;
      const int clear_from = a.window > 0 ? max(base + depth - a.window + 1, 0) : 0;
      float slope = 0.f, slope_by = 0.f;  // in log2 units, in those of the scores as they come
      float by = a.scale_log2;
      if constexpr (kForm == kAnyScores) {
        if (a.cap_log2 > 0.f || by < kTrLeastScale) by = 1.f;
      }
      if constexpr (kForm == kLargeCapScores) by = 1.f;
      if constexpr (kSlopes) {
        if (live && a.slopes != nullptr) {
          slope = __ldg(a.slopes + w.g * a.G + rh) * 1.4426950408889634f;
          slope_by = min_nan(-min_nan(-slope / by, 0x1p90f), 0x1p90f);
          slope = slope_by * by;  // (beyond that, the nearest key that is seen takes all)
        }
      }
      if (live && a.depths != nullptr && h == 0 && valid && w.ka == 0 &&
          __ldg(a.depths + w.q0 + node) != depth)
        tr_flag(a, PKV_DEV_BAD_POSITION);
      float m = -INFINITY, l = 0.f;
      for (int k = w.ka; k < w.kb; ++k, ++it) {
        const int b = static_cast<int>(it & 1u);
        // (S of this tile was issued after P V of two tiles ago: its P buffer is free, too)
        if (!wait_all(bar(kTrSFull + b), (it >> 1) & 1u)) break;
        if (live) {
          uint32_t v[HK];
          const int k0 = (w.j0 + k) * KT + h * HK;
          ptx::tc_fence_after();
          const uint32_t sa = tmem + lane_off + b * KT + h * HK;
#pragma unroll
          for (int i = 0; i < HK; i += 32)
            ptx::tmem_ld32_nowait(sa + i, *reinterpret_cast<uint32_t(*)[32]>(&v[i]));
          ptx::tmem_wait_ld();
          float off = 0.f;  // a score in log2 units: v * by + off
          if constexpr (kForm == kLargeCapScores) {
#pragma unroll
            for (int i = 0; i < HK; i += 2)
              tanh_any_cap2(v[i], v[i + 1], a.scale_log2, a.cap_inv, a.cap_log2);
          }
          if constexpr (kForm == kAnyScores) {
            if (a.cap_log2 > 0.f) {
#pragma unroll
              for (int i = 0; i < HK; i += 2) tanh_cap2(v[i], v[i + 1], a.cap_z, a.cap_log2);
            }
            if (a.cap_log2 <= 0.f && a.scale_log2 < kTrLeastScale) {
#pragma unroll
              for (int i = 0; i < HK; ++i)
                v[i] = __float_as_uint(__uint_as_float(v[i]) * a.scale_log2);
            }
          }
          if constexpr (kSlopes) {
            if (kForm == kSlopeScores || a.slopes != nullptr) {
              int own = depth;
              if (a.depths != nullptr && k0 + HK > base) {
                // drafted tokens: how far each one's position is from its place in the chunk
                own = node;
                int there[HK / 32];  // of a lane's keys
#pragma unroll
                for (int e = 0; e < HK / 32; ++e) {
                  const int j = k0 + 32 * e + lane - base;
                  there[e] = j < 0 || j >= w.c ? 0 : tr_depth(a, w.q0, j) - j;
                }
#pragma unroll
                for (int i = 0; i < HK; ++i) {
                  const int x = __shfl_sync(0xffffffffu, there[i >> 5], i & 31) - (depth - node);
                  v[i] = __float_as_uint(
                      fmaf(slope_by, static_cast<float>(x), __uint_as_float(v[i])));
                }
              }
              // neighbouring keys lie a position apart: multiples of the slope beside the scores,
              // the first key's distance beside the reference
              off = slope * static_cast<float>(k0 - base - own);
#pragma unroll
              for (int i = 0; i < HK; ++i)
                v[i] = __float_as_uint(
                    fmaf(slope_by, static_cast<float>(i), __uint_as_float(v[i])));
            }
          }
          // keys that the row does not see score -inf
          if (__any_sync(0xffffffffu, valid && (k0 < clear_from || k0 + HK > clear_to))) {
            const uint64_t vis = valid ? tr_sees(a, w, node, depth, k0, HK) : 0ull;
            const uint32_t v0 = static_cast<uint32_t>(vis), v1 = static_cast<uint32_t>(vis >> 32);
#pragma unroll
            for (int i = 0; i < HK; ++i)
              if (!((i < 32 ? v0 >> (i & 31) : v1 >> (i & 31)) & 1u))
                v[i] = __float_as_uint(-INFINITY);
          }
          float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < HK; i += 2)
            mx4[(i >> 1) & 3] =
                max3(mx4[(i >> 1) & 3], __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
          // the row's maximum over this tile, log2 units
          float mt = fmaf(max3(fmaxf(mx4[0], mx4[1]), mx4[2], mx4[3]), by, off);
          mt = fmaxf(mt, exchange(mt));
          if (gone) break;
          // The reference m moves only when the maximum grows by more than 2^8 (at first from
          // -inf): O and l are scaled once the product before has landed.  The accesses are
          // warp-wide: the whole warp takes the branch, the other rows scale by 1.
          const bool move = mt > m + kTrRescale;
          if (k > w.ka && __any_sync(0xffffffffu, move)) {
            const float al = move ? ptx::ex2(m - mt) : 1.f;  // 2^-inf = 0
            if (!wait_all(bar(kTrPvDone + (b ^ 1)), ((it - 1) >> 1) & 1u)) break;
            ptx::tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < HD; c0 += 32) {
              uint32_t o[32];
              ptx::tmem_ld32(oa + c0, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
              ptx::tmem_st32(oa + c0, o);
            }
            l *= al;
          }
          if (move) m = mt;
          // a row that has seen nothing yet: every exponent is -inf whatever the reference
          const float ref = m == -INFINITY ? 0.f : m - Sh::kShift;
          const float less = off - ref;
          float s0 = 0.f, s1 = 0.f;
          uint32_t pk[HK / 2];
#pragma unroll
          for (int i = 0; i < HK / 2; ++i) {  // keys 2i, 2i + 1 of the half
            const float x0 = ptx::ex2(fmaf(__uint_as_float(v[2 * i]), by, less));
            const float x1 = ptx::ex2(fmaf(__uint_as_float(v[2 * i + 1]), by, less));
            pk[i] = ptx::pack2<T>(x0, x1);
            s0 += x0;
            s1 += x1;
          }
          if constexpr (HK == 64) ptx::tmem_st32(pcol + b * (KT / 2), pk);
          else tmem_st16(pcol + b * (KT / 2), pk);
          l += s0 + s1;
          ptx::tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(bar(kTrSEmpty + b));
          ptx::mbar_arrive(bar(kTrPFull + b));
        }
        if (k == w.ka && pend) {  // the previous piece's output
          epilogue();
          if (gone) break;
        }
      }
      if (gone) break;
      pend = true;
      pend_live = live;
      pend_valid = valid;
      pend_m = m == -INFINITY ? m : m - Sh::kShift;
      pend_l = l;
      pend_x = it - 1;
      pend_n = n;
    }
    if (pend && !gone) epilogue();
    if (gone) {
      if (lane == 0) {
        tr_flag(a, PKV_DEV_WAIT_TIMEOUT);
        atomicOr(dead_bits + q4, 1 << h);
        __threadfence_block();
      }
      __syncwarp();
      if (!pair_dead)
        asm volatile("bar.arrive %0, 64;" ::"r"(pair_bar) : "memory");
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc(tmem, Sh::kTmemCols);
}

// Joins the pieces of the units that runs' borders cut: CTA x looks after the unit that run x
// begins, a warp a row.  out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i, in order.
constexpr int kJoinWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) tree_join_kernel(const TreeArgs a, int runs) {
  constexpr int E = D / 32;  // elements of a lane
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const TreeCut cut = a.cuts[blockIdx.x];
  const int r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (cut.n == 0 || r >= cut.rows) return;
  // the runs that hold the unit's first and last tile; those between hold a tile or none
  const int x0 = blockIdx.x;
  const long long end = cut.P + cut.n - 1 + kTrUnitCost;
  const int x1 = static_cast<int>(((end + 1) * runs - 1) / cut.C);
  auto row = [&](int x) { return (2 * static_cast<int64_t>(x) + (x == x0)) * kTrRows + r; };
  float M = -INFINITY, total = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int b0 = x0; b0 <= x1; b0 += 32) {  // 32 pieces: a lane looks one up
    const int x = b0 + lane;
    float2 ml = make_float2(-INFINITY, 0.f);
    bool here = false;
    if (x <= x1) {
      here = tr_first_tile(cut.P, cut.n, tr_border(cut.C, x + 1, runs)) >
             tr_first_tile(cut.P, cut.n, tr_border(cut.C, x, runs));
      if (here) ml = a.part_ml[row(x)];
    }
    float top = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top > M) {  // what is there is brought to the new reference
      const float al = ptx::ex2(M - top);
      total *= al;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= al;
      M = top;
    }
    // a row that has seen nothing has sums of 0 (or of NaN), whatever the reference
    const float wt = ml.x == -INFINITY ? 1.f : ptx::ex2(ml.x - M);
    const float part = ml.y * wt;
    const uint32_t on = __ballot_sync(0xffffffffu, here);
    for (uint32_t left = on; left != 0;) {  // in order, four pieces' loads on their way
      int at[4];
      float src[4][E];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        at[u] = left != 0 ? __ffs(left) - 1 : -1;
        left &= left - 1;
        if (at[u] >= 0) {
          const float* const p = a.part_o + row(b0 + at[u]) * D + lane * E;
#pragma unroll
          for (int e = 0; e < E; e += 2)
            *reinterpret_cast<float2*>(&src[u][e]) = *reinterpret_cast<const float2*>(p + e);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (at[u] < 0) continue;
        const float wi = __shfl_sync(0xffffffffu, wt, at[u]);
        total += __shfl_sync(0xffffffffu, part, at[u]);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(src[u][e], wi, acc[e]);
      }
    }
  }
  const float inv = total == 0.f ? 0.f : 1.f / total;
  const int rn = r / a.G, rh = r - rn * a.G;
  T* const dst = static_cast<T*>(a.out) +
                 (static_cast<int64_t>(cut.row0 + rn) * a.Hq + cut.g * a.G + rh) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(dst + e) = ptx::pack2<T>(acc[e] * inv, acc[e + 1] * inv);
}

// The two launches of a call hand pieces over through the workspace: they are queued one behind the
// other, whatever other host threads queue on the stream with the same workspace.
std::mutex tree_queue;

template <typename T, int D, TreeForm kForm>
int launch_tree(const TreeArgs& a, const void* k_cache, int32_t dtype, int sms, cudaStream_t st) {
  using Sh = TreeShape<T, D>;
  static SmemOnce once;
  int rc = allow_dynamic_smem(
      once, reinterpret_cast<const void*>(tree_attention_kernel<T, D, kForm>), Sh::kBytes);
  if (rc != PKV_OK) return rc;
  static_assert((kTrMaxSeqs + 1 + 12) * 8 <= Sh::kK * Sh::kTile, "the prefix sums' room");
  CUtensorMap qmap, kmap, vmap;
  const CUtensorMapDataType ty =
      dtype == PKV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  // q [T, Hq, D]: boxes of 64 columns (128 B) x G heads x `box` drafted tokens, whole 8-row
  // swizzle atoms
  const int64_t qdims[3] = {D, a.Hq, a.T};
  const int64_t qstrides[2] = {static_cast<int64_t>(D) * 2, static_cast<int64_t>(a.Hq) * D * 2};
  const int32_t qbox[3] = {64, a.G, a.box};
  rc = encode_map_3d(&qmap, a.q, ty, 2, qdims, qstrides, qbox, CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc != PKV_OK) return rc;
  // K and V [rows, D] as (column in chunk, row in group, chunk, 8-row group): a box is a cache
  // block of one KV head, landing chunk-major within each group
  const int64_t kvdims[4] = {64, 8, Sh::kChunks, static_cast<int64_t>(a.NB) * a.Hkv * (a.bs / 8)};
  const int64_t kvstrides[3] = {static_cast<int64_t>(D) * 2, 128, 8 * static_cast<int64_t>(D) * 2};
  const int32_t kvbox[4] = {64, 8, Sh::kChunks, a.bs / 8};
  rc = encode_map_4d(&kmap, k_cache, ty, kvdims, kvstrides, kvbox, CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc != PKV_OK) return rc;
  rc = encode_map_4d(&vmap, a.v_cache, ty, kvdims, kvstrides, kvbox, CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc != PKV_OK) return rc;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(sms);
  cfg.blockDim = dim3(kTrThreads);
  cfg.dynamicSmemBytes = Sh::kBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const std::lock_guard<std::mutex> both(tree_queue);
  PKV_CUDA(cudaLaunchKernelEx(&cfg, tree_attention_kernel<T, D, kForm>, qmap, kmap, vmap, a));
  cfg.gridDim = dim3(sms, kTrRows / kJoinWarps);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.dynamicSmemBytes = 0;
  PKV_CUDA(cudaLaunchKernelEx(&cfg, tree_join_kernel<T, D>, a, sms));
  return PKV_OK;
}

template <typename T>
int launch_tree_d(const TreeArgs& a, const void* k_cache, int32_t dtype, int32_t head_dim,
                  TreeForm form, int sms, cudaStream_t st) {
#define PKV_TREE(D)                                                                          \
  (form == kPlainScores   ? launch_tree<T, D, kPlainScores>(a, k_cache, dtype, sms, st)      \
   : form == kSlopeScores ? launch_tree<T, D, kSlopeScores>(a, k_cache, dtype, sms, st)      \
   : form == kAnyScores   ? launch_tree<T, D, kAnyScores>(a, k_cache, dtype, sms, st)        \
                          : launch_tree<T, D, kLargeCapScores>(a, k_cache, dtype, sms, st))
  return head_dim == 64 ? PKV_TREE(64) : (head_dim == 128 ? PKV_TREE(128) : PKV_TREE(256));
#undef PKV_TREE
}

size_t tree_part_bytes(int sms, int head_dim) {
  return static_cast<size_t>(2) * sms * kTrRows * head_dim * sizeof(float);
}
size_t tree_ml_bytes(int sms) { return static_cast<size_t>(2) * sms * kTrRows * sizeof(float2); }

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_tree_workspace_size(int32_t head_dim, size_t* bytes) {
  PKV_REQUIRE(bytes != nullptr, PKV_ERR_INVALID_ARG, "bytes is NULL");
  PKV_REQUIRE(head_dim == 64 || head_dim == 128 || head_dim == 256, PKV_ERR_UNSUPPORTED,
              "head_dim %d not in {64, 128, 256}", head_dim);
  int sms = 0, dev = 0;
  const int rc = device_sm_count(&sms, &dev);
  if (rc != PKV_OK) return rc;
  *bytes = tree_part_bytes(sms, head_dim) + tree_ml_bytes(sms) + sms * sizeof(TreeCut);
  return ok();
}

int pkv_tree_attention(const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* block_tables, int32_t max_blocks_per_seq,
                       const int32_t* context_lens, const int32_t* query_start,
                       const int32_t* tree_mask, int32_t mask_words, const int32_t* depths,
                       const float* slopes, float cap, int32_t window, int32_t num_seqs,
                       int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads,
                       int32_t head_dim, int32_t block_size, int32_t num_blocks, float scale,
                       void* out, int32_t* status, void* workspace, size_t workspace_bytes,
                       int32_t dtype, void* stream) {
  PKV_REQUIRE(dtype == PKV_F16 || dtype == PKV_BF16, PKV_ERR_DTYPE,
              "tree attention takes f16 or bf16 (dtype %d)", dtype);
  PKV_REQUIRE(num_seqs >= 0 && num_seqs <= kTrMaxSeqs, PKV_ERR_UNSUPPORTED,
              "num_seqs %d outside [0, %d]", num_seqs, kTrMaxSeqs);
  PKV_REQUIRE(num_q_heads > 0 && num_kv_heads > 0 && num_q_heads % num_kv_heads == 0,
              PKV_ERR_INVALID_ARG, "num_q_heads %d must be a positive multiple of num_kv_heads %d",
              num_q_heads, num_kv_heads);
  const int G = num_q_heads / num_kv_heads;
  PKV_REQUIRE(G <= kTrMaxGroup, PKV_ERR_UNSUPPORTED, "query heads per KV head %d above %d", G,
              kTrMaxGroup);
  PKV_REQUIRE(head_dim == 64 || head_dim == 128 || head_dim == 256, PKV_ERR_UNSUPPORTED,
              "head_dim %d not in {64, 128, 256}", head_dim);
  PKV_REQUIRE(block_size == 8 || block_size == 16 || block_size == 32, PKV_ERR_UNSUPPORTED,
              "block_size %d not in {8, 16, 32}", block_size);
  PKV_REQUIRE(max_blocks_per_seq > 0 && num_blocks > 0, PKV_ERR_INVALID_ARG, "bad sizes");
  PKV_REQUIRE(static_cast<int64_t>(max_blocks_per_seq) * block_size < (int64_t(1) << 30),
              PKV_ERR_UNSUPPORTED, "max_blocks_per_seq * block_size >= 2^30");
  PKV_REQUIRE(static_cast<int64_t>(num_blocks) * num_kv_heads * block_size * 4 < (int64_t(1) << 31),
              PKV_ERR_UNSUPPORTED, "num_blocks * num_kv_heads * block_size * 4 >= 2^31");
  PKV_REQUIRE(num_tokens >= 0, PKV_ERR_INVALID_ARG, "negative num_tokens");
  PKV_REQUIRE(static_cast<int64_t>(num_tokens) * num_q_heads < (int64_t(1) << 31),
              PKV_ERR_UNSUPPORTED, "num_tokens * num_q_heads >= 2^31");
  PKV_REQUIRE(std::isfinite(scale), PKV_ERR_INVALID_ARG, "scale must be finite");
  PKV_REQUIRE(std::isfinite(cap) && cap >= 0.f, PKV_ERR_INVALID_ARG,
              "cap must be finite and not negative (0: none)");
  PKV_REQUIRE(window >= 0, PKV_ERR_INVALID_ARG, "window must not be negative (0: none)");
  PKV_REQUIRE(tree_mask == nullptr || mask_words > 0, PKV_ERR_INVALID_ARG,
              "a mask has at least one word a row");
  if (num_seqs == 0 || num_tokens == 0) return ok();
  PKV_REQUIRE(q && k_cache && v_cache && block_tables && context_lens && query_start && out,
              PKV_ERR_INVALID_ARG, "NULL pointer");
  PKV_REQUIRE(aligned(q, 16) && aligned(k_cache, 16) && aligned(v_cache, 16) && aligned(out, 16),
              PKV_ERR_INVALID_ARG, "q, caches and out must be 16-byte aligned");
  PKV_REQUIRE(aligned(block_tables, 4) && aligned(context_lens, 4) && aligned(query_start, 4) &&
                  aligned(tree_mask, 4) && aligned(depths, 4) && aligned(slopes, 4) &&
                  aligned(status, 4),
              PKV_ERR_INVALID_ARG, "a pointer is not aligned to its element");
  PKV_REQUIRE(workspace != nullptr && aligned(workspace, 256), PKV_ERR_INVALID_ARG,
              "workspace must be a 256-byte aligned device pointer");
  int sms = 0, dev = 0;
  int rc = device_sm_count(&sms, &dev);
  if (rc != PKV_OK) return rc;
  const size_t po = tree_part_bytes(sms, head_dim), ml = tree_ml_bytes(sms);
  PKV_REQUIRE(workspace_bytes >= po + ml + sms * sizeof(TreeCut), PKV_ERR_INVALID_ARG,
              "workspace of %zu bytes, %zu needed", workspace_bytes,
              po + ml + sms * sizeof(TreeCut));
  TreeArgs a{};
  a.q = q;
  a.out = out;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.query_start = query_start;
  a.mask = reinterpret_cast<const uint32_t*>(tree_mask);
  a.depths = depths;
  a.slopes = slopes;
  a.v_cache = v_cache;
  a.status = status;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(static_cast<char*>(workspace) + po);
  a.cuts = reinterpret_cast<TreeCut*>(static_cast<char*>(workspace) + po + ml);
  a.S = num_seqs;
  a.T = num_tokens;
  a.Hq = num_q_heads;
  a.Hkv = num_kv_heads;
  a.G = G;
  a.MAXB = max_blocks_per_seq;
  a.NB = num_blocks;
  a.bs = block_size;
  a.W = mask_words;
  a.window = window > (1 << 30) + kTrMaxDepth ? 0 : window;  // no two positions are as far apart
  // whole 8-row swizzle atoms: a box of q is 8 / gcd(G, 8) drafted tokens, a unit whole boxes (a G
  // that is no power of two leaves rows idle: 72 of 128 used for 9, 88 for 11, 104 for 13, else 112 or 120)
  a.box = G % 8 == 0 ? 1 : (G % 4 == 0 ? 2 : (G % 2 == 0 ? 4 : 8));
  a.nodes = kTrRows / G / a.box * a.box;
  const double log2e = 1.4426950408889634;
  a.scale_log2 = static_cast<float>(scale * log2e);
  // (caps next to the largest float: log2 units end there; scores that large are a tie or take all)
  const double most = FLT_MAX;
  a.cap_log2 = static_cast<float>(std::min(cap * log2e, most));
  // (kept finite: a score of 0 stays one under the smallest caps)
  a.cap_z = cap > 0.f ? static_cast<float>(std::clamp(2.0 * log2e * scale / cap, -most, most)) : 0.f;
  a.cap_inv = cap > kTrSmallCap ? static_cast<float>(1.0 / a.cap_log2) : 0.f;
  const TreeForm form = cap > kTrSmallCap                               ? kLargeCapScores
                        : cap > 0.f || !(a.scale_log2 >= kTrLeastScale) ? kAnyScores
                        : slopes != nullptr                             ? kSlopeScores
                                                                        : kPlainScores;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  rc = dtype == PKV_BF16
           ? launch_tree_d<__nv_bfloat16>(a, k_cache, dtype, head_dim, form, sms, st)
           : launch_tree_d<__half>(a, k_cache, dtype, head_dim, form, sms, st);
  return rc == PKV_OK ? ok() : rc;
}

int pkv_tree_masks(const int32_t* parents, const int32_t* query_start, int32_t num_seqs,
                   int32_t mask_words, int32_t* tree_mask, int32_t* depths) {
  PKV_REQUIRE(num_seqs >= 0 && mask_words > 0, PKV_ERR_INVALID_ARG, "bad sizes");
  PKV_REQUIRE(query_start && (num_seqs == 0 || (parents && tree_mask && depths)),
              PKV_ERR_INVALID_ARG, "NULL pointer");
  PKV_REQUIRE(num_seqs == 0 || query_start[0] >= 0, PKV_ERR_INVALID_ARG,
              "query_start must not be negative");
  // all checked before anything is written, every border before a parent is read: the last one is
  // the number of parents
  for (int32_t s = 0; s < num_seqs; ++s)
    PKV_REQUIRE(query_start[s + 1] >= query_start[s], PKV_ERR_INVALID_ARG,
                "query_start must not decrease");
  for (int32_t s = 0; s < num_seqs; ++s) {
    const int32_t q0 = query_start[s], q1 = query_start[s + 1];
    PKV_REQUIRE(q1 - q0 <= static_cast<int64_t>(mask_words) * 32, PKV_ERR_INVALID_ARG,
                "sequence %d has %d drafted tokens, a mask row holds %lld", s, q1 - q0,
                static_cast<long long>(mask_words) * 32);
    for (int32_t i = q0; i < q1; ++i)
      PKV_REQUIRE(parents[i] >= -1 && parents[i] < i - q0, PKV_ERR_INVALID_ARG,
                  "parent %d of drafted token %d is not one before it (or -1)", parents[i], i - q0);
  }
  for (int32_t s = 0; s < num_seqs; ++s) {
    const int32_t q0 = query_start[s], q1 = query_start[s + 1];
    for (int32_t i = q0; i < q1; ++i) {
      int32_t* const row = tree_mask + static_cast<int64_t>(i) * mask_words;
      const int32_t p = parents[i];
      for (int32_t x = 0; x < mask_words; ++x)
        row[x] = p < 0 ? 0 : tree_mask[static_cast<int64_t>(q0 + p) * mask_words + x];
      const int32_t j = i - q0;
      row[j / 32] = static_cast<int32_t>(static_cast<uint32_t>(row[j / 32]) | (1u << (j % 32)));
      depths[i] = p < 0 ? 0 : depths[q0 + p] + 1;
    }
  }
  return ok();
}

}  // extern "C"
