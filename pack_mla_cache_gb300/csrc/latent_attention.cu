// latent_attention.cu -- attention of new tokens over the paged latent cache in
// the absorbed MLA form (include/mla_cache.h: mla_latent_attention), on the 5th
// generation tensor cores.
//
// What it computes, per (token, head) row q of 576 elements and the cache rows
// k_p that the token sees: x_p = scale <q, k_p>, lse = ln sum exp(x_p), out =
// sum exp(x_p - lse) k_p[0:512].  All heads of a token share the rows.
//
// Shape of the work.  A sequence's query rows (token-major, heads inside) are
// cut into tiles of NR = 16, 32 or 64 rows, its cache rows into tiles of 64
// keys; one unit = (query tile, key tile).  The units of the whole call, in
// (sequence, query tile, key tile) order, are cut into equal contiguous runs,
// one per CTA (one CTA per SM), so ragged batches load every SM alike.  A
// query tile whose units fall into several CTAs leaves unnormalised fp32
// partial sums in the workspace, which a second small launch joins in the
// order of the CTAs (no atomics: equal calls give equal bits).
//
// Measured (replayed from a graph, without the profiler; 16 heads, 64-row blocks): one
// new token of 4 sequences over 131072 bf16 rows 101 us (5.97 TB/s), of 64 over 130 to
// 16384 e4m3 rows 60.3 us (5.2 TB/s), of one over 2047 bf16 rows 10.2 us; 1024 new
// tokens of 2 over 8192 bf16 rows 643 us (852 TFLOP/s).  About 10 us of a call are fixed
// (finding the run and the first rows 3, filling and draining the pipeline 4, the join 3).
//
// Both products are computed transposed, so that few query rows (a decode
// batch has 16 per token) are the N dimension of the tensor core's tile and no
// row of it is wasted:
//   scores    S^T [64 keys x NR]  = K  [64 x 576] * Q^T   (A = K as loaded)
//   outputs   O^T [512 x NR]     += V^T [512 x 64] * P^T  (A = the same shared
//             memory read MN-major: a latent row is key and value)
// A key tile is a few chunks of 64 keys x 128 bytes in the 128-byte swizzle.
// S^T (two buffers) and O^T (4 x 128 dims) stay in tensor memory.
//
// bf16 cache: 9 chunks of 64 columns, two tiles in flight (2 x 72 KB).
// fp8 cache: the codes themselves are the A operand (5 chunks, the last one
// columns 448 to 575, four tiles in flight), and the 16-bit operands are split
// into 8-bit parts: a query row, scaled by a power of two, is two e4m3 parts, q1 +
// q2 / 16; a weight is three e5m2 parts, p1 + p2 / 16 + p3 / 256.  The parts are 2 NR
// or 3 NR columns of one product, added when the sums are read.
//
// Why three e5m2 parts for a weight.  A long tail of small weights can hold most of a
// row's mass, so small weights need their 8 bits as much as large ones.  Weights reach
// 2^14 (a reference 2^10 below the maximum, which may grow by 2^4 more).  A part of a
// value in [2^k, 2^(k+1)) is off by at most 2^(k-3), which times 16 is at most 2^(k+1)
// again: three parts hold a weight to 2^-11 of itself, or to half the last part's
// smallest step, 2^-16 / 256 / 2 = 2^-25, which is 2^-34 of the row's largest weight or
// less.  (Two e4m3 parts held 8 bits down to 2^-7 of the largest weight and nothing
// below 2^-19: a tail of 131072 equal weights with 20% of the mass was lost.)
//
// Cost of a tile.  64 products in a row on resident operands take, per product, 24 / 25 /
// 33 cycles at M = 64 and N = 16 / 32 / 64, and 40 / 45 / 49 / 57 at M = 128 and N = 16 /
// 48 / 64 / 96 (the A operand's shared-memory reads bound them).  So the 36 + 16 products
// of a bf16 tile take 1500 cycles at NR = 16 and 2000 at NR = 64, the 18 + 8 of an fp8
// tile 820 and 1060: 0.4 to 1 us at 2070 MHz.  HBM's rate delivers a bf16 tile to each SM
// in 1.65 us, an fp8 one in 0.82.
//
// Roles (10 or 14 warps): 4 or 8 warps do the softmax (running maximum per query
// row, rescaling O^T only when a maximum has grown by more than 2^8, or 2^4 for
// fp8) and the output; two warps issue the matrix instructions; 4 warps load.
// Whole tiles come by TMA where a tile is a few boxes of the paged cache (block
// size a multiple of 8); the others, and the last tile of a sequence, whose rows
// behind the end are zeros, by 16-byte asynchronous copies.
//
// Rows that a token must not see: rows behind every row's view are zeros; in
// the tiles where tokens of one query tile see different rows, a row holding a
// NaN or an infinity is stored as zeros and marked, and its score becomes NaN
// for the tokens that do see it.
//
// Waits are bounded (wait_limit_ns): one that runs out marks the CTA as given up.
// Every role leaves at its next wait then, copies and products in flight are waited
// for (bounded again), and MLA_ERRBIT_TIMEOUT is set.
#include <cuda.h>

#include <atomic>
#include <type_traits>

#include "mla_device.cuh"
#include "serving.h"
#include "tensor_core.cuh"

namespace mla {
namespace {

constexpr int kKeys = 64;                 // keys per tile
constexpr int kChunk = kKeys * 128;       // bytes of a chunk
constexpr int kProdWarps = 4;
constexpr int kProdThreads = kProdWarps * 32;
constexpr int kRank = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A CTA takes at least this many units (fewer: more partial sums to join; more: fewer SMs).
// us with 1, 2 and 3, 16 heads, bf16: one decode over 512 rows 9.2, 9.5, 10.7, over 2047
// 10.7, 10.3, 11.6, over 8192 16.7, 13.7, 13.6; four over 2047 11.7, 11.4, 12.2; one of
// 128 heads over 2047 15.5, 14.8, 17.3.
constexpr int kMinUnits = 2;
constexpr float kQ2 = 0.0625f;            // query parts: q = q1 + q2 / 16
constexpr float kPStep = 16.0f;           // weight parts: p = p1 + p2 / 16 + p3 / 256

// Key flags of a tile (one byte per key).
constexpr uint32_t kAbsent = 1;  // its block was not found: left out
constexpr uint32_t kPoison = 2;  // holds a NaN or an infinity

template <int FMT, int NR>
struct Lay {
  static constexpr bool kF8 = FMT != kBF16;
  static constexpr int kN = (kF8 ? 2 : 1) * NR;         // columns of the scores: parts of the queries
  static constexpr int kParts = kF8 ? 3 : 1;            // parts of a weight
  static constexpr int kPN = kParts * NR;               // columns of the outputs
  static constexpr int kChunks = kF8 ? 5 : 9;
  static constexpr int kTile = kChunks * kChunk;
  static constexpr int kStages = kF8 ? 4 : 2;
  // Halves of a stage (chunks 0 to 3 and the rest) that fill and are freed by
  // themselves.  At 64 query rows the chain load, scores, weights, outputs of the two
  // stages is what takes the time, and a half's load overlaps the outputs of the other
  // (2 chunks of 1024 tokens over 8192 rows: 645 us, 689 with whole stages; 16 decodes of
  // 128 heads 46.1, 47.7).
  static constexpr int kHalves = NR == 64 ? 2 : 1;
  static constexpr int kQBufs = NR <= (kF8 ? 16 : 32) ? 2 : 1;
  static constexpr int kQ = kChunks * kN * 128;
  static constexpr int kSoftWarps = NR == 16 ? 4 : 8;   // one or two groups of 4 warps
  static constexpr int kCols = NR / (kSoftWarps / 4);   // query rows of a group
  static constexpr int kScoreWarp = kSoftWarps;         // issues the scores' products
  static constexpr int kOutWarp = kScoreWarp + 1;       // and the outputs'
  static constexpr int kProdWarp = kOutWarp + 1;
  static constexpr int kWarps = kProdWarp + kProdWarps;
  static constexpr int kThreads = kWarps * 32;
  // What beginning another query tile costs a CTA, in key tiles (its queries, the sums
  // of the one before): the runs are cut as if each query tile had this many more.
  // us with 0, 1, 2, 3, 4 and 6 of them (r. = ragged, 16 heads):
  //   fp8  16  64 r. e4m3 decodes           62.1 61.2 60.8 60.2 60.0 61.0
  //   fp8  32  32 r. verifications of 4     56.6 55.2 53.3 52.4 50.6 48.2
  //            32 r. verifications of 2     37.0 36.8 35.5 34.4 33.9 31.9
  //   bf16 16  64 r. decodes               103.7 103.5 103.7 104.1 104.4 105.3
  //   bf16 32  32 r. verifications of 2     45.5 45.4 43.1 42.2 41.8 42.6
  //   bf16 64  16 r. decodes, 128 heads     48.1 47.4 46.1 47.1 47.0 46.3
  //            32 r. verifications of 4     55.7 55.7 53.1 52.0 50.9 51.2
  static constexpr int kSwitch = kF8 ? (NR == 16 ? 3 : 6) : (NR == 16 ? 1 : 2);
  // The reference of a row's weights is the next whole number (log2) above its maximum
  // less kTop; a score may pass the reference by kGrow before the sums are rescaled.
  // Whole numbers, so that the weights round alike whichever rows a CTA's run begins with.
  static constexpr float kTop = kF8 ? 10.0f : 0.0f;
  static constexpr float kGrow = kF8 ? 14.0f : 8.0f;
  // shared memory
  static constexpr int q = kStages * kTile;
  static constexpr int kPBufs = NR == 64 ? 1 : 2;
  static constexpr int kP = kPN * 128;                   // kPN rows x 64 keys (fp8: half of each row)
  static constexpr int p = q + kQBufs * kQ;
  static constexpr int red = p + kPBufs * kP;               // float [2][kSoftWarps][kCols]
  static constexpr int qs = red + 2 * kSoftWarps * kCols * 4;  // float [kQBufs][NR]
  static constexpr int flags = qs + (kF8 ? kQBufs * NR * 4 : 0);  // uint8 [kStages][64]
  static constexpr int bars = flags + kStages * kKeys;
  // barriers, by index
  static constexpr int kFull = 0, kEmpty = kStages * kHalves, kQFull = 2 * kEmpty, kQEmpty = kQFull + 2,
                       kSFull = kQEmpty + 2, kPFull = kSFull + 2, kPvDone = kPFull + 2,
                       kOFree = kPvDone + 2, kBars = kOFree + 1;
  static constexpr int misc = (bars + kBars * 8 + 15) / 16 * 16;
  static constexpr int bytes = misc + 64;
  static_assert(bytes <= 232448, "shared memory of a CTA");
  // tensor memory columns: two score buffers, then the sums of 4 x 128 dims
  static constexpr int kO = 2 * kN;
  static constexpr int kCols32 = 2 * kN + 4 * kPN;
  static constexpr int kTmem = kCols32 <= 128 ? 128 : kCols32 <= 256 ? 256 : 512;
  static_assert(kCols32 <= 512, "tensor memory of an SM");
};

struct Misc {
  uint32_t tmem;
  uint32_t abort;
};
static_assert(sizeof(Misc) <= 64, "Misc fits");

// What the join needs of a split query tile: token and head of its first row, its
// rows, and the CTAs with partials, first .. first + parts - 1.  Written by each of
// them but the last (whose run goes on with other query tiles); rows 0: none.
struct Split {
  int32_t tok0, head0;
  uint16_t rows, parts;
  int32_t first;
};

struct Seq {
  int32_t t0, ntok;  // tokens t0 .. t0 + ntok - 1 are computed
  int32_t c1, kv;
  int32_t nqt;       // query tiles
};

// Token of a sequence's query row (row < 2^31).
__device__ __forceinline__ int token_of(const LatentAttnArgs& a, uint32_t row) {
  return (int)a.by_heads(row);
}

template <int NR>
__device__ __forceinline__ Seq load_seq(const LatentAttnArgs& a, int s) {
  Seq q;
  const int32_t c0 = __ldg(a.cu_q + s);
  q.c1 = __ldg(a.cu_q + s + 1);
  q.kv = __ldg(a.kv_lens + s);
  q.t0 = max(c0, 0);
  q.ntok = max(min(q.c1, a.num_tokens) - q.t0, 0);
  q.nqt = (int)(((uint32_t)q.ntok * (uint32_t)a.num_heads + NR - 1) / NR);
  return q;
}
// Rows that token t of the sequence sees.
__device__ __forceinline__ int seen_of(const LatentAttnArgs& a, const Seq& q, int t) {
  const int64_t n = (int64_t)q.kv + (a.causal ? (int64_t)t + 1 - q.c1 : 0);
  return (int)max((int64_t)0, min(n, (int64_t)a.room));
}
// Rows that the last (first) row of query tile qt sees: the most (least) of its rows.
template <int NR>
__device__ __forceinline__ int most_seen(const LatentAttnArgs& a, const Seq& q, int qt) {
  const uint32_t last = min((uint32_t)(qt + 1) * NR, (uint32_t)q.ntok * (uint32_t)a.num_heads) - 1;
  return seen_of(a, q, q.t0 + token_of(a, last));
}
// Whether a token sees rows beyond the block table's.
__device__ __forceinline__ bool over_room(const LatentAttnArgs& a, const Seq& q) {
  return (int64_t)q.kv + (a.causal ? (int64_t)q.t0 + q.ntok - q.c1 : 0) > a.room;
}
// Key tiles of a query tile that sees `most` rows (one even when it sees none: its
// rows are still written).
__device__ __forceinline__ int key_tiles(int most) { return max(1, (most + kKeys - 1) / kKeys); }

struct Tile {
  bool valid, first, last;  // first / last of this CTA's run of the query tile
  int s, qt, kt, nkt;
  int most, least;          // rows seen by the last / first row of the query tile
  int t0, ntok;             // the sequence's tokens
};

// A CTA's run of units: where it starts, and what finds the CTA of another unit.  A
// query tile is kSwitch units that stand for beginning it, then its key tiles: a run
// starts before the first of these when kt is negative.
struct Run {
  Seq q;               // of sequence s
  int s, qt, kt, count;
  int64_t begin, each; // the first unit; units of the CTAs c >= extra (each + 1 of the ones before)
  int extra;
  __device__ __forceinline__ int left() const { return count + min(kt, 0); }
};

// Walks the run; every role has its own copy.
template <int NR, int kSwitch>
struct Walk {
  Seq q;
  int s, qt, kt, nkt, most, least;
  int left;
  bool fresh;
  __device__ __forceinline__ void item(const LatentAttnArgs& a) {
    most = most_seen<NR>(a, q, qt);
    least = seen_of(a, q, q.t0 + token_of(a, (uint32_t)qt * NR));
    nkt = key_tiles(most);
    fresh = true;
  }
  __device__ __forceinline__ void start(const Run& r) {
    q = r.q;
    s = r.s;
    qt = r.qt;
    kt = max(r.kt, 0);
    left = r.left();
    nkt = 0;
  }
  // The next unit.  Each role calls this at one place only: 10 or 14 warps of
  // different code share the instruction caches.
  __device__ __forceinline__ Tile next(const LatentAttnArgs& a) {
    Tile t{};
    if (left <= 0) return t;
    if (__builtin_expect(kt >= nkt, 0)) {  // another query tile (the first: nkt is 0)
      if (nkt > 0) {
        kt = 0;
        ++qt;
        if (qt >= q.nqt) {
          qt = 0;
          do q = load_seq<NR>(a, ++s);
          while (q.nqt == 0 && s + 1 < a.num_seqs);
        }
        left -= kSwitch;
        if (left <= 0) return t;
      }
      item(a);
    }
    t.valid = true;
    t.first = fresh;
    fresh = false;
    t.s = s;
    t.qt = qt;
    t.kt = kt++;
    t.nkt = nkt;
    t.most = most;
    t.least = least;
    t.t0 = q.t0;
    t.ntok = q.ntok;
    --left;
    t.last = kt == nkt || left == 0;
    return t;
  }
};

// Bounded waits.  The loops of the roles have to stay small (10 or 14 warps of
// different code share the instruction caches; fetching was the largest stall), so all but
// the first look at a barrier is out of line.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, uint32_t abort, uint64_t limit) {
  uint64_t since = 0;
  for (uint32_t spin = 1; !mbar_try_wait(bar, parity); ++spin) {
    if (spin & 31u) continue;
    if (lds_u32(abort) != 0) return false;
    const uint64_t now = global_ns();
    if (since == 0) since = now;
    if (now - since > limit) {
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(abort), "r"(1u) : "memory");
      return false;
    }
  }
  return true;
}
struct Waiter {
  uint32_t abort;  // shared address of Misc::abort
  uint64_t limit;
  __device__ __forceinline__ bool given_up() const { return lds_u32(abort) != 0; }
  // Whether the barrier's phase completed: false once the CTA has given up.
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    return mbar_try_wait(bar, parity) || wait_on(bar, parity, abort, limit);
  }
};

__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void sts8(uint32_t addr, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void sts_u8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void sts_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
// A barrier of the four warps of one softmax group.
__device__ __forceinline__ void soft_sync(int group) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
}
// The same barrier, and whether x holds in any of its threads.
__device__ __forceinline__ bool soft_any(int group, bool x) {
  uint32_t any;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 q, %2, 0;\n"
      "  barrier.cta.red.or.pred p, %1, 128, q; selp.u32 %0, 1, 0, p; }"
      : "=r"(any)
      : "r"(1 + group), "r"(x ? 1u : 0u)
      : "memory");
  return any != 0;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Whether any of the 8 bf16 (16 fp8) values of v is a NaN or an infinity.
template <int FMT>
__device__ __forceinline__ bool any_special(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (FMT == kBF16) m |= (w[i] & 0x7FFF7FFFu) + 0x00800080u;  // exponent 255 carries
    else if constexpr (FMT == kE4M3) m |= (w[i] & 0x7F7F7F7Fu) + 0x01010101u;
    else m |= (w[i] & 0x7F7F7F7Fu) + 0x04040404u;
  }
  return (m & (FMT == kBF16 ? 0x80008000u : 0x80808080u)) != 0;
}

// The block of row p of sequence s: an id to be checked, or kUnseen when no row of
// the query tile sees it.  The table's answer is not looked at here, so its load
// runs on while the tile before is produced.
constexpr int32_t kUnseen = INT32_MIN;
__device__ __forceinline__ int32_t find_block(const LatentAttnArgs& a, const Tile& t, int p) {
  const int kb = a.bs_shift >= 0 ? p >> a.bs_shift : p / a.block_size;
  int32_t blk = kUnseen;
  if (t.valid && p < t.most) blk = __ldg(a.block_table + (int64_t)t.s * a.bt_stride + kb);
  return blk;
}
// The address of row p in that block, or nullptr: unseen, or not found (flag kAbsent).
__device__ __forceinline__ const uint8_t* row_in(const LatentAttnArgs& a, int p, int32_t blk,
                                                 uint32_t& flag) {
  const bool ok = blk >= 0 && blk < a.num_blocks;
  flag = ok || blk == kUnseen ? 0 : kAbsent;
  const int off = a.bs_shift >= 0 ? p & (a.block_size - 1) : p % a.block_size;
  const uint8_t* r = a.cache + (int64_t)blk * a.block_stride + (int64_t)off * a.entry_stride;
  return ok ? r : nullptr;
}

// Whether the tile comes by TMA: whole, and every row of the query tile sees it.
__device__ __forceinline__ bool by_box(const LatentAttnArgs& a, const Tile& t) {
  return a.box_rows != 0 && (t.kt + 1) * kKeys <= t.least;
}

// ------------------------------------------------------------------ producers
// One query tile into shared memory: bf16 rows by asynchronous copies.
template <int NR>
__device__ __forceinline__ void load_q(const LatentAttnArgs& a, const Tile& q, uint32_t dst,
                                       uint32_t bar, int pw, int lane) {
  const uint32_t rows = (uint32_t)q.ntok * (uint32_t)a.num_heads;
  const int col = lane & 7;
#pragma unroll 1
  for (int r = pw * 4 + (lane >> 3); r < NR; r += kProdWarps * 4) {
    const uint32_t row = (uint32_t)q.qt * NR + r;
    const bool ok = row < rows;
    const int tok = ok ? token_of(a, row) : 0;
    const int64_t t = ok ? q.t0 + tok : 0;
    const int64_t h = ok ? (int)row - tok * a.num_heads : 0;
    const uint8_t* c = a.q_c + t * a.qc_ts + h * a.qc_hs + col * 16;
    const uint8_t* pe = a.q_pe + t * a.qp_ts + h * a.qp_hs + col * 16;
    const uint32_t d = dst + r * 128 + ((col ^ (r & 7)) << 4);
#pragma unroll
    for (int ch = 0; ch < 8; ++ch) tc::cp_async16(d + ch * (NR * 128), c + ch * 128, ok);
    tc::cp_async16(d + 8 * (NR * 128), pe, ok);
  }
  tc::cp_async_arrive(bar);
}
// The same as two e4m3 parts of the row times a power of two: with the largest
// magnitude in [2^7, 2^8), q1 = e4m3(q) rounds by at most 8 and q2 = e4m3(16 (q -
// q1)).  q1 + q2 / 16 has every bit of a bf16 down to 2^-14 of the largest, and
// is off by at most 2^-21 of it below.  A row with a NaN or an infinity gets NaN
// as its inverse scale.  8 lanes take a row, 16 bytes of every chunk each, so a
// tile of 16 rows costs four warps one round of loads.  The producers do it, but for a
// CTA's first query tile: there the kWarps softmax warps have nothing else to do (the
// producers would do it behind the first rows).
template <int NR, int kWarps>
__device__ __forceinline__ void split_q(const LatentAttnArgs& a, const Tile& q, uint32_t dst,
                                        uint32_t scales, uint32_t bar, int pw, int lane) {
  const uint32_t rows = (uint32_t)q.ntok * (uint32_t)a.num_heads;
  const int col = lane & 7;
#pragma unroll 1
  for (int r = pw * 4 + (lane >> 3); r < NR; r += kWarps * 4) {
    const uint32_t row = (uint32_t)q.qt * NR + r;
    const bool ok = row < rows;
    const int tok = ok ? token_of(a, row) : 0;
    const int64_t t = ok ? q.t0 + tok : 0, h = ok ? (int)row - tok * a.num_heads : 0;
    const uint8_t* c = a.q_c + t * a.qc_ts + h * a.qc_hs + col * 16;
    const uint8_t* pe = a.q_pe + t * a.qp_ts + h * a.qp_hs + col * 16;
    // once for the largest magnitude, and again (from L1) to split
    uint32_t top = 0;
    {
      uint4 v[9];
#pragma unroll
      for (int ch = 0; ch < 9; ++ch) v[ch] = ld_shared_ro16(ch < 8 ? c + ch * 128 : pe);
#pragma unroll
      for (int ch = 0; ch < 9; ++ch)
        top = umax16x2(top, umax16x2(umax16x2(v[ch].x & 0x7FFF7FFFu, v[ch].y & 0x7FFF7FFFu),
                                     umax16x2(v[ch].z & 0x7FFF7FFFu, v[ch].w & 0x7FFF7FFFu)));
    }
    top = ok ? max(top & 0xFFFFu, top >> 16) : 0;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const uint32_t e = max(top >> 7, 8u);  // exponent field of the largest magnitude
    const float s = ok ? __uint_as_float((261u - e) << 23) : 0.0f;  // 2^(134 - e)
    // columns 64 ch + 8 col ..: 8 bytes at byte 64 (ch % 2) + 8 col of chunk ch / 2
    const uint32_t d = dst + r * 128 + 8 * (col & 1);
#pragma unroll 3
    for (int ch = 0; ch < 9; ++ch) {
      const uint4 v = ld_shared_ro16(ch < 8 ? c + ch * 128 : pe);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t p1[4], p2[4];  // two codes each
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x0 = ok ? bf16lo(w[i]) * s : 0.0f, x1 = ok ? bf16hi(w[i]) * s : 0.0f;
        p1[i] = pack_fp8x2<kE4M3>(x0, x1);
        float y0, y1;
        fp8x2_to_f32x2<kE4M3>(p1[i], y0, y1);
        p2[i] = pack_fp8x2<kE4M3>((x0 - y0) * 16.0f, (x1 - y1) * 16.0f);
      }
      const int unit = (ch & 1) * 4 + (col >> 1);
      const uint32_t at = d + (ch >> 1) * (2 * NR * 128) + ((unit ^ (r & 7)) << 4);
      sts8(at, p1[0] | p1[1] << 16, p1[2] | p1[3] << 16);
      sts8(at + NR * 128, p2[0] | p2[1] << 16, p2[2] | p2[3] << 16);
    }
    if (col == 0)
      sts_u32(scales + 4 * r, top >= 0x7F80u ? 0x7FC00000u : (e - 7u) << 23);  // 2^(e - 134)
  }
  __syncwarp();
  if (lane == 0) mbar_arrive_n(bar, kProdThreads / kWarps);
}

// Returns the key tiles whose copies were issued.
template <int FMT, int NR>
__device__ __forceinline__ uint32_t produce(const LatentAttnArgs& a, const CUtensorMap& map,
                                        const Run& run, uint32_t smem, const Waiter& wait, int pw,
                                        int lane, uint32_t& errbits) {
  using L = Lay<FMT, NR>;
  const uint32_t bars = smem + L::bars;
  Walk<NR, L::kSwitch> walk;
  walk.start(run);
  // Row copies: 8 lanes x 16 bytes per row and chunk; this thread has the rows
  // pw * 16 + 4 i + lane / 8.
  constexpr int kRows = 4;
  const int row0 = pw * 16 + (lane >> 3), col = lane & 7;
  // Boxes of box_rows keys x one chunk, `boxes` per chunk: number pw + 4 lane is this
  // thread's (at most 72; issuing them takes time, so the four warps share
  // them).  Lanes 28 to 31 write the flags of the warp's 16 keys, four each.
  const int boxes = 1 << a.box_shift;
  const int box = (pw + 4 * lane) & (boxes - 1), box_chunk = (pw + 4 * lane) >> a.box_shift;
  const uint32_t box_bytes = (uint32_t)((boxes * L::kChunks - pw + 3) >> 2) * a.box_rows * 128;
  const int box_key = lane < 28 ? box * a.box_rows : pw * 16 + 4 * (lane - 28);
  // Blocks are looked up two tiles ahead.
  Tile cur{}, nxt{};
  int32_t blk[kRows] = {}, nblk[kRows] = {};
  uint32_t item = 0, issued = 0;
  const uint64_t policy = tc::l2_policy(a.stream_rows);
#pragma unroll 1
  for (int step = -2;; ++step) {
    const Tile far = walk.next(a);
    int32_t fblk[kRows];
    if (__builtin_expect(by_box(a, far), 1)) {
      fblk[0] = find_block(a, far, far.kt * kKeys + box_key);
    } else {
#pragma unroll
      for (int i = 0; i < kRows; ++i) fblk[i] = find_block(a, far, far.kt * kKeys + row0 + 4 * i);
    }
    if (cur.valid) {
      const uint32_t g = step;
      const int st = g % L::kStages;
      const uint32_t full = bars + 8 * (L::kFull + st * L::kHalves), flags = smem + L::flags + st * kKeys;
      // (the halves of a stage one after the other; rows need both)
      auto freed = [&](int h) {
        return g < L::kStages ||
               __all_sync(0xFFFFFFFFu, wait(bars + 8 * (L::kEmpty + st * L::kHalves + h),
                                            (g / L::kStages - 1) & 1));
      };
      if (!freed(0)) break;
      ++issued;
      const uint32_t base = smem + st * L::kTile;
      if (__builtin_expect(by_box(a, cur), 1)) {
        const bool ok = blk[0] >= 0 && blk[0] < a.num_blocks;
        if (!ok) errbits |= kErrBlockOOB;
        if (lane >= 28) sts_u32(flags + box_key, ok ? 0u : 0x01010101u * kAbsent);
        bool gone = false;
#pragma unroll 1
        for (int h = 0; h < L::kHalves; ++h) {
          // this warp's boxes of chunks 0 to 3 are those of the lanes below `boxes`
          const bool both = L::kHalves == 1;
          if (h > 0 && !freed(h)) {
            gone = true;
            break;
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive_expect_tx(full + 8 * h, both ? box_bytes : h ? box_bytes - kChunk : (uint32_t)kChunk);
            mbar_arrive_n(full + 8 * h, 32);
          }
          __syncwarp();
          if (box_chunk < L::kChunks && (both || (lane >= boxes) == (h > 0))) {
            const int p = cur.kt * kKeys + box_key;
            const int off = a.bs_shift >= 0 ? p & (a.block_size - 1) : p % a.block_size;
            const int z = ok ? blk[0] : (int)a.num_blocks;  // outside the tensor: zeros
            tc::tma_load3(base + box_chunk * kChunk + box_key * 128, &map,
                          L::kF8 ? (box_chunk < 4 ? box_chunk * 128 : 448) : box_chunk * 64, off, z,
                          full + 8 * h, policy);
          }
        }
        if (gone) break;
      } else {
        if (L::kHalves > 1 && !freed(1)) break;
        // tokens of the query tile see different rows of this key tile
        const bool mixed = cur.least < cur.most && (cur.kt + 1) * kKeys > cur.least;
#pragma unroll 1
        for (int i = 0; i < kRows; ++i) {
          const int row = row0 + 4 * i;
          const int32_t bi = i == 0 ? blk[0] : i == 1 ? blk[1] : i == 2 ? blk[2] : blk[3];
          uint32_t flag;
          const uint8_t* src = row_in(a, cur.kt * kKeys + row, bi, flag);
          if (flag) errbits |= kErrBlockOOB;
          const uint32_t d = base + row * 128 + ((col ^ (row & 7)) << 4);
          // the 16-byte parts of this lane: chunk c, and for fp8 the rotary columns of
          // the last chunk (its upper half) in lanes 4 to 7
          auto part = [&](int c) { return !L::kF8 || c < 4 ? c * 128 + col * 16 : 512 + (col - 4) * 16; };
          auto has = [&](int c) { return !L::kF8 || c < 4 || col >= 4; };
          if (!mixed) {
#pragma unroll
            for (int c = 0; c < L::kChunks; ++c)
              if (has(c)) tc::cp_async16(d + c * kChunk, src ? src + part(c) : a.cache, src != nullptr);
          } else {
            // once to look for NaNs and infinities, and again to store
            bool sp = false;
#pragma unroll
            for (int c = 0; c < L::kChunks; ++c)
              sp |= any_special<FMT>(src && has(c) ? ld_shared_ro16(src + part(c)) : make_uint4(0, 0, 0, 0));
            const bool drop = __ballot_sync(0xFFFFFFFFu, sp) & (0xFFu << (lane & 24));
            if (drop) flag = kPoison;
#pragma unroll 1
            for (int c = 0; c < L::kChunks; ++c)
              if (has(c))
                sts16(d + c * kChunk,
                      src && !drop ? ld_shared_ro16(src + part(c)) : make_uint4(0, 0, 0, 0));
          }
          if (col == 0) sts_u8(flags + row, flag);
        }
        __syncwarp();
#pragma unroll
        for (int h = 0; h < L::kHalves; ++h) {
          if (mixed) {
            if (lane == 0) mbar_arrive_n(full + 8 * h, 33);
          } else {
            if (lane == 0) mbar_arrive(full + 8 * h);
            tc::cp_async_arrive(full + 8 * h);
          }
        }
      }
      if (__builtin_expect(cur.first, 0)) {  // the query, behind the first rows
        const int b = item % L::kQBufs;
        const uint32_t n = item / L::kQBufs;
        if (n > 0 && !__all_sync(0xFFFFFFFFu, wait(bars + 8 * (L::kQEmpty + b), (n - 1) & 1))) break;
        const uint32_t dst = smem + L::q + b * L::kQ, bar = bars + 8 * (L::kQFull + b);
        if constexpr (L::kF8) {
          if (item > 0)
            split_q<NR, kProdWarps>(a, cur, dst, smem + L::qs + b * NR * 4, bar, pw, lane);
        } else load_q<NR>(a, cur, dst, bar, pw, lane);
        ++item;
      }
    }
    cur = nxt;
    nxt = far;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      blk[i] = nblk[i];
      nblk[i] = fblk[i];
    }
    if (step >= -1 && !cur.valid) break;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  return issued;
}

// --------------------------------------------------------------- matrix issue
// The whole warp runs these; one elected lane issues.  Descriptors are made the
// same in all lanes (stage and buffer by a shuffle) and their loops have constant
// bounds without branches inside, so that they live in uniform registers.  One instance
// of each loop for all stages and buffers: the roles share the instruction caches, and
// with an instance each, fetching was the largest stall (64 ragged decodes 81 us, 71
// with one, both before later steps).
template <int FMT, int NR>
__device__ __forceinline__ void issue_scores(uint32_t smem, uint32_t tmem, bool one, int stage,
                                             int qbuf, int sbuf, int half, bool last) {
  using L = Lay<FMT, NR>;
  constexpr uint32_t kId =
      tc::instr_desc(kKeys, L::kN, false, FMT == kE4M3 ? 0 : 1, L::kF8 ? 0 : 1);
  const uint32_t st = __shfl_sync(0xFFFFFFFFu, stage, 0), qb = __shfl_sync(0xFFFFFFFFu, qbuf, 0);
  const uint32_t sb = __shfl_sync(0xFFFFFFFFu, sbuf, 0);
  const uint64_t ka = tc::smem_desc(smem + st * L::kTile, 0, 1024);
  const uint64_t qa = tc::smem_desc(smem + L::q + qb * L::kQ, 0, 1024);
  const uint32_t d = tmem + sb * L::kN;
  // a k step is 32 bytes of a row
  auto chunks = [&](auto from, auto to) {
#pragma unroll 1
    for (int c = from; c < to; ++c)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint64_t ak = ka + (c * kChunk >> 4) + 2 * k, bk = qa + (c * L::kN * 128 >> 4) + 2 * k;
        if constexpr (L::kF8) tc::mma_fp8(one, d, ak, bk, kId, c + k > 0);
        else tc::mma_bf16(one, d, ak, bk, kId, c + k > 0);
      }
  };
  using std::integral_constant;
  if (L::kHalves == 1) {
    chunks(integral_constant<int, 0>(), integral_constant<int, L::kF8 ? 4 : 9>());
  } else if (half == 0) {
    chunks(integral_constant<int, 0>(), integral_constant<int, 4>());
    return;
  } else {
    chunks(integral_constant<int, 4>(), integral_constant<int, 9>());
  }
  // the fp8 rotary columns are the upper half of their chunk, the lower half of the query's
  if constexpr (L::kF8)
#pragma unroll
    for (int k = 0; k < 2; ++k)
      tc::mma_fp8(one, d, ka + (4 * kChunk >> 4) + 2 * k + 4, qa + (4 * L::kN * 128 >> 4) + 2 * k, kId,
                  true);
  tc::commit(one, smem + L::bars + 8 * (L::kSFull + sb));
  if (last) tc::commit(one, smem + L::bars + 8 * (L::kQEmpty + qb));
}
template <int FMT, int NR>
__device__ __forceinline__ void issue_outputs(uint32_t smem, uint32_t tmem, bool one, int stage,
                                              int pbuf, bool first) {
  using L = Lay<FMT, NR>;
  constexpr uint32_t kId = tc::instr_desc(128, L::kPN, true, FMT == kE4M3 ? 0 : 1, 1);
  const uint32_t st = __shfl_sync(0xFFFFFFFFu, stage, 0), pb = __shfl_sync(0xFFFFFFFFu, pbuf, 0);
  // The K tile, MN-major.  128 dims are two bf16 chunks or one fp8 chunk; a k step
  // is 16 keys (2 groups of 8 rows) or 32.
  const uint64_t va = tc::smem_desc(smem + st * L::kTile, L::kF8 ? 0 : kChunk, 1024);
  const uint64_t pa = tc::smem_desc(smem + L::p + (pb & (L::kPBufs - 1)) * L::kP, 0, 1024);
  constexpr int kDims = L::kF8 ? kChunk : 2 * kChunk, kStep = L::kF8 ? 4096 : 2048;
#pragma unroll
  for (int h = 0; h < L::kHalves; ++h) {
#pragma unroll 1
    for (int b = h * 2; b < (h + 1 == L::kHalves ? 4 : 2); ++b)
#pragma unroll
      for (int k = 0; k < (L::kF8 ? 2 : 4); ++k) {
        const uint32_t d = tmem + L::kO + b * L::kPN;
        const uint64_t ak = va + (b * kDims >> 4) + k * (kStep >> 4), bk = pa + 2 * k;
        if constexpr (L::kF8) tc::mma_fp8(one, d, ak, bk, kId, k > 0 || !first);
        else tc::mma_bf16(one, d, ak, bk, kId, k > 0 || !first);
      }
    tc::commit(one, smem + L::bars + 8 * (L::kEmpty + st * L::kHalves + h));
  }
  tc::commit(one, smem + L::bars + 8 * (L::kPvDone + pb));
}

struct Workspace {
  Split* split;   // [ctas]
  float *m, *l;   // [2 ctas][NR]: running maximum (log2 units) and sum
  float* o;       // [2 ctas][NR][512]: unnormalised sums
};
template <int NR>
__host__ __device__ inline Workspace workspace_of(uint8_t* p, int ctas) {
  Workspace w;
  w.split = reinterpret_cast<Split*>(p);
  w.m = reinterpret_cast<float*>(p + (int64_t)ctas * sizeof(Split));
  w.l = w.m + (int64_t)ctas * 2 * NR;
  w.o = w.l + (int64_t)ctas * 2 * NR;
  return w;
}
// The CTA whose run has unit u.
__device__ __noinline__ int cta_of(int64_t u, int64_t each, int extra) {
  const int64_t longer = (each + 1) * extra;  // units of the runs of each + 1
  return (int)(u < longer ? u / (each + 1) : extra + (u - longer) / each);
}

// One warp issues the scores, another the outputs, each as soon as its operands
// are there: outputs free the stage that the rows behind need, and from one warp
// they would wait for the scores of the next tile or for its polls of both (2 chunks of
// 1024 tokens 726 us from one warp, 695 from two, both before later steps).
template <int FMT, int NR>
__device__ __forceinline__ void score_role(const LatentAttnArgs& a, const Run& run, uint32_t smem,
                                           uint32_t tmem, const Waiter& waiter) {
  using L = Lay<FMT, NR>;
  const uint32_t bars = smem + L::bars;
  auto wait = [&](int bar, uint32_t phase) { return waiter(bars + 8 * bar, phase & 1); };
  Walk<NR, L::kSwitch> walk;
  walk.start(run);
  const bool one = tc::elect();
  uint32_t item = 0;
#pragma unroll 1
  for (uint32_t g = 0;; ++g) {
    const Tile t = walk.next(a);
    if (!t.valid) break;
    const int qb = item % L::kQBufs, st = g % L::kStages;
    bool ok = !t.first || wait(L::kQFull + qb, item / L::kQBufs);
    if (g >= 2) ok &= wait(L::kPFull + (g & 1), (g - 2) >> 1);  // the score buffer is read
    ok &= wait(L::kFull + st * L::kHalves, g / L::kStages);
    if (!__all_sync(0xFFFFFFFFu, ok)) break;
    // Queries, and rows that do not come by TMA, are written by ordinary and
    // asynchronous stores of the producers; the fence towards the tensor core's reads
    // stands here, behind the barrier (in the producers it would also wait for their
    // loads in flight).
    if (t.first || !by_box(a, t)) tc::fence_smem_async();
    tc::fence_after_sync();
    issue_scores<FMT, NR>(smem, tmem, one, st, qb, g & 1, 0, t.last);
    if constexpr (L::kHalves > 1) {
      if (!__all_sync(0xFFFFFFFFu, wait(L::kFull + st * L::kHalves + 1, g / L::kStages))) break;
      tc::fence_after_sync();
      issue_scores<FMT, NR>(smem, tmem, one, st, qb, g & 1, 1, t.last);
    }
    item += t.last;
  }
}

template <int FMT, int NR>
__device__ __forceinline__ void output_role(const LatentAttnArgs& a, const Run& run, uint32_t smem,
                                            uint32_t tmem, const Waiter& waiter, int lane,
                                            const Workspace& ws) {
  using L = Lay<FMT, NR>;
  const uint32_t bars = smem + L::bars;
  auto wait = [&](int bar, uint32_t phase) { return waiter(bars + 8 * bar, phase & 1); };
  Walk<NR, L::kSwitch> walk;
  walk.start(run);
  const bool one = tc::elect();
  uint32_t item = 0;
#pragma unroll 1
  for (uint32_t g = 0;; ++g) {
    const Tile t = walk.next(a);
    if (!t.valid) break;
    bool ok = wait(L::kPFull + (g & 1), g >> 1);
    if (t.first && item > 0) ok &= wait(L::kOFree, item - 1);  // the sums of the query tile before are read
    if (!__all_sync(0xFFFFFFFFu, ok)) break;
    tc::fence_after_sync();
    issue_outputs<FMT, NR>(smem, tmem, one, g % L::kStages, g & 1, t.first);
    item += t.last;
    if (__builtin_expect(t.last && t.kt + 1 < t.nkt && lane == 0, 0)) {
      // The run ends inside the query tile: for the join.  (This warp has nothing else to
      // do now; from the softmax warps one decode took 10.6 us, 10.3 from here, both before
      // later steps.)  The run's last unit
      // is number t.kt of the tile's.
      const int64_t u0 = run.begin + run.count - 1 - t.kt;
      const int c0 = cta_of(u0, run.each, run.extra);
      const int c1 = cta_of(u0 + t.nkt - 1, run.each, run.extra);
      const uint32_t row = (uint32_t)t.qt * NR;
      const int rows = (int)min((uint32_t)NR, (uint32_t)t.ntok * (uint32_t)a.num_heads - row);
      const int dt = token_of(a, row);
      ws.split[blockIdx.x] = Split{t.t0 + dt, (int)row - dt * a.num_heads, (uint16_t)rows,
                                   (uint16_t)(c1 - c0 + 1), c0};
    }
  }
}

// ----------------------------------------------------------- softmax and output
template <int FMT, int NR>
__device__ __forceinline__ void soften(const LatentAttnArgs& a, const Run& run, uint32_t smem,
                                       uint32_t tmem, const Waiter& waiter, int warp, int lane,
                                       const Workspace& ws) {
  using L = Lay<FMT, NR>;
  constexpr int kC = L::kCols;  // query rows of this group of four warps
  constexpr int kG = kC / 8;    // a thread has the rows 8 j + 2 (lane % 4) + {0, 1} of them
  const int group = warp >> 2, w4 = warp & 3, col0 = group * kC;
  const uint32_t bars = smem + L::bars;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    waiter(bar, parity);
    __syncwarp();
  };
  const uint32_t sub = tmem + ((uint32_t)(w4 * 32) << 16);  // this warp's lanes
  const float ks = FMT == kBF16 ? 1.0f : __ldg(a.k_scale);
  const float c = a.softmax_scale * ks * kLog2e;
  const int c2 = 2 * (lane & 3);
  const int key0 = w4 * 16 + (lane >> 2);  // and + 8
  float* red = reinterpret_cast<float*>(__cvta_shared_to_generic(smem + L::red));
  float mu[kG][2], l[kG][2];
  float cs[kG][2];  // score of a product: softmax and cache scale, log2 e, the query row's scale
  Walk<NR, L::kSwitch> walk;
  walk.start(run);
  int kt_begin = 0;
  uint32_t g = 0, item = 0;
#pragma unroll 1
  for (;; ++g) {
    const Tile t = walk.next(a);
    if (!t.valid) break;
    if (t.first) {
      kt_begin = t.kt;
      const uint32_t scales = smem + L::qs + (item % L::kQBufs) * NR * 4;
      if constexpr (L::kF8) {
        if (item == 0)
          split_q<NR, L::kSoftWarps>(a, t, smem + L::q, scales, bars + 8 * L::kQFull, warp, lane);
        wait(bars + 8 * (L::kQFull + item % L::kQBufs), (item / L::kQBufs) & 1);
      }
#pragma unroll
      for (int j = 0; j < kG; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          cs[j][e] = c;
          if constexpr (L::kF8)
            cs[j][e] = c * __uint_as_float(lds_u32(scales + 4 * (col0 + 8 * j + c2 + e)));
          l[j][e] = 0.0f;
          mu[j][e] = -INFINITY;
        }
      if constexpr (L::kF8) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + 8 * (L::kQEmpty + item % L::kQBufs));
      }
      ++item;
    }
    const int b = g & 1;
    const int st = g % L::kStages;
    // The key flags, the scores, and an early look whether P's buffer is free (below): the
    // three answers are asked for together.
    const uint32_t full = bars + 8 * (L::kFull + (st + 1) * L::kHalves - 1), full_at = (g / L::kStages) & 1;
    const uint32_t o = g - L::kPBufs;  // the tile whose outputs free the buffer
    const bool flagged = mbar_try_wait(full, full_at);
    const bool scored = mbar_try_wait(bars + 8 * (L::kSFull + b), (g >> 1) & 1);
    const bool unused = g < L::kPBufs || mbar_test(bars + 8 * (L::kPvDone + (o & 1)), (o >> 1) & 1);
    if (!flagged) waiter(full, full_at);
    if (!scored) waiter(bars + 8 * (L::kSFull + b), (g >> 1) & 1);
    __syncwarp();
    tc::fence_after_sync();
    const bool dead = waiter.given_up();  // (cheaper than each wait's answer)
    float x[kG][4];
    tc::ld_16x256<kG>(sub + b * L::kN + col0, reinterpret_cast<uint32_t*>(&x[0][0]));
    if constexpr (L::kF8) {
      float y[kG][4];
      tc::ld_16x256<kG>(sub + b * L::kN + NR + col0, reinterpret_cast<uint32_t*>(&y[0][0]));
#pragma unroll
      for (int j = 0; j < kG; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[j][i] = fmaf(y[j][i], kQ2, x[j][i]);
    }
    const uint32_t f0 = lds_u8(smem + L::flags + st * kKeys + key0);
    const uint32_t f1 = lds_u8(smem + L::flags + st * kKeys + key0 + 8);
#pragma unroll
    for (int j = 0; j < kG; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[j][i] *= cs[j][i & 1];
    if (__builtin_expect((t.kt + 1) * kKeys > t.least || __any_sync(0xFFFFFFFFu, (f0 | f1) != 0), 0)) {
      const int p = t.kt * kKeys + key0;
#pragma unroll
      for (int j = 0; j < kG; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // a row behind the last one (its query is zeros) copies the last one's view
          const uint32_t row = min((uint32_t)t.qt * NR + col0 + 8 * j + c2 + e,
                                   (uint32_t)t.ntok * (uint32_t)a.num_heads - 1);
          const int seen = seen_of(a, walk.q, t.t0 + token_of(a, row));
          if (f0 == kPoison) x[j][e] = NAN;
          if (f1 == kPoison) x[j][e + 2] = NAN;
          if (p >= seen || f0 == kAbsent) x[j][e] = -INFINITY;
          if (p + 8 >= seen || f1 == kAbsent) x[j][e + 2] = -INFINITY;
        }
    }
    // Only whether a score passes its row's reference by more than 2^kGrow is asked of
    // every tile (one barrier that also ORs); the new maxima are found when one does.
    bool grown = false;
#pragma unroll
    for (int j = 0; j < kG; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        grown |= fmaxf(x[j][e], x[j][e + 2]) > mu[j][e] + L::kGrow;
    grown = soft_any(group, grown | dead);
    // P's buffer is free when the outputs of the tile that had it are done
    if (!unused) waiter(bars + 8 * (L::kPvDone + (o & 1)), (o >> 1) & 1);
    __syncwarp();
    if (__builtin_expect(grown, 0)) {
      // maximum over the tile's 64 keys: in the warp, then across the four warps
      float* mine = red + warp * kC;
      float* fac = red + (L::kSoftWarps + warp) * kC;
      float tm[kG][2];
#pragma unroll
      for (int j = 0; j < kG; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = fmaxf(x[j][e], x[j][e + 2]);
          v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
          tm[j][e] = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
        }
      if (lane < 4)
#pragma unroll
        for (int j = 0; j < kG; ++j)
          *reinterpret_cast<float2*>(mine + 8 * j + c2) = make_float2(tm[j][0], tm[j][1]);
      // All four warps leave when one has given up (or they would wait for each other):
      // it says so by a negative factor, which it alone could replace by one.
      const bool leave = __any_sync(0xFFFFFFFFu, dead);
      if (lane == 0) fac[0] = leave ? -1.0f : 0.0f;
      soft_sync(group);
      const float* said = red + (L::kSoftWarps + group * 4) * kC;
      if (__any_sync(0xFFFFFFFFu, *reinterpret_cast<const volatile float*>(said + (lane & 3) * kC) < 0.0f))
        break;
#pragma unroll
      for (int j = 0; j < kG; ++j) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 v = *reinterpret_cast<const float2*>(red + (group * 4 + w) * kC + 8 * j + c2);
          tm[j][0] = fmaxf(tm[j][0], v.x);
          tm[j][1] = fmaxf(tm[j][1], v.y);
        }
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mn = fmaxf(mu[j][e], ceilf(tm[j][e]) - L::kTop);
          f[e] = mu[j][e] == -INFINITY ? 0.0f : ex2(mu[j][e] - mn);
          l[j][e] *= f[e];
          mu[j][e] = mn;
        }
        if (lane < 4) *reinterpret_cast<float2*>(fac + 8 * j + c2) = make_float2(f[0], f[1]);
      }
      soft_sync(group);  // the maxima are read, the factors written
      if (!t.first) {  // and O^T when those of the tile before are
        wait(bars + 8 * (L::kPvDone + ((g - 1) & 1)), ((g - 1) >> 1) & 1);
        tc::fence_after_sync();
#pragma unroll 1
        for (int n = 0; n < 4 * L::kParts * kC; n += 16) {
          // 16 of this group's columns: dims n / (kParts kC), part, columns n % kC
          const int o = L::kO + n / kC * NR + col0 + n % kC;
          uint32_t r[16];
          tc::ld_32x16(sub + o, r);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            r[i] = __float_as_uint(__uint_as_float(r[i]) * fac[n % kC + i]);
          tc::st_32x16(sub + o, r);
        }
        tc::wait_st();
      }
    }
    // weights, their sums, and P^T to shared memory: row n = the 64 keys of query row n
#pragma unroll
    for (int j = 0; j < kG; j += 2) {
      uint32_t w[4];
#pragma unroll
      for (int jj = 0; jj < 2; ++jj) {
        const float m0 = mu[j + jj][0] == -INFINITY ? 0.0f : mu[j + jj][0];
        const float m1 = mu[j + jj][1] == -INFINITY ? 0.0f : mu[j + jj][1];
        const float p0 = ex2(x[j + jj][0] - m0), p1 = ex2(x[j + jj][1] - m1);
        const float p2 = ex2(x[j + jj][2] - m0), p3 = ex2(x[j + jj][3] - m1);
        l[j + jj][0] += p0 + p2;
        l[j + jj][1] += p1 + p3;
        if constexpr (!L::kF8) {
          w[2 * jj] = pack_bf16x2(p0, p1);
          w[2 * jj + 1] = pack_bf16x2(p2, p3);
        } else {
          // each weight as three e5m2 parts, in the rows n, NR + n and 2 NR + n
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float u = h ? p2 : p0, v = h ? p3 : p1;
            const int n = col0 + (j + jj) * 8 + c2;  // and n + 1
            const uint32_t in = (lane >> 2) + 8 * h;
            const uint32_t d0 = smem + L::p + (g & (L::kPBufs - 1)) * L::kP + n * 128 + ((w4 ^ (n & 7)) << 4) + in;
            const uint32_t d1 = smem + L::p + (g & (L::kPBufs - 1)) * L::kP + (n + 1) * 128 + ((w4 ^ ((n + 1) & 7)) << 4) + in;
#pragma unroll
            for (int i = 0; i < L::kParts; ++i) {
              const uint32_t part = pack_fp8x2<kE5M2>(u, v);
              sts_u8(d0 + i * NR * 128, part);
              sts_u8(d1 + i * NR * 128, part >> 8);
              float uh, vh;
              fp8x2_to_f32x2<kE5M2>(part, uh, vh);
              u = (u - uh) * kPStep;
              v = (v - vh) * kPStep;
            }
          }
        }
      }
      if constexpr (!L::kF8) {
        const int n = col0 + (j + (lane >> 4)) * 8 + (lane & 7);
        const int unit = 2 * w4 + ((lane >> 3) & 1);
        tc::st_8x8_t(smem + L::p + (g & (L::kPBufs - 1)) * L::kP + n * 128 + ((unit ^ (n & 7)) << 4), w[0], w[1], w[2], w[3]);
      }
    }
    tc::fence_smem_async();
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + 8 * (L::kPFull + b));
    if (__builtin_expect(!t.last, 1)) continue;

    // ---- the end of this CTA's run of the query tile
    wait(bars + 8 * (L::kPvDone + b), (g >> 1) & 1);
    tc::fence_after_sync();
    // the sums of the weights over lanes (and warps, below); row n's sum and maximum
    // then go to lane n
    float* part = red + warp * kC;
    float* mine = red + (L::kSoftWarps + warp) * kC;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kG; ++j) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[j][e] += __shfl_xor_sync(0xFFFFFFFFu, l[j][e], 4);
        l[j][e] += __shfl_xor_sync(0xFFFFFFFFu, l[j][e], 8);
        l[j][e] += __shfl_xor_sync(0xFFFFFFFFu, l[j][e], 16);
      }
      if (lane < 4) *reinterpret_cast<float2*>(part + 8 * j + c2) = make_float2(l[j][0], l[j][1]);
    }
    soft_sync(group);
    if (lane < 4)
#pragma unroll
      for (int j = 0; j < kG; ++j)
        *reinterpret_cast<float2*>(mine + 8 * j + c2) = make_float2(mu[j][0], mu[j][1]);
    __syncwarp();
    const bool whole = kt_begin == 0 && t.kt + 1 == t.nkt;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (kt_begin == 0 ? 1 : 0);
    const uint32_t first = (uint32_t)t.qt * NR;
    // this group's rows that exist (none or less: not one)
    const int nv = min((int)min((uint32_t)NR, (uint32_t)t.ntok * (uint32_t)a.num_heads - first) - col0, kC);
    // token and head of this group's first row
    const int dt0 = token_of(a, first + col0), tok0 = t.t0 + dt0;
    const int head0 = (int)(first + col0) - dt0 * a.num_heads;
    const bool lost = __any_sync(0xFFFFFFFFu, waiter.given_up());
    // where row `lane` of the group goes in out
    const int dt = token_of(a, head0 + lane), row_h = head0 + lane - dt * a.num_heads;
    const int64_t row_at = (int64_t)(tok0 + dt) * a.out_ts + (int64_t)row_h * a.out_hs;
    if (lane < kC) {
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w)
        sum += red[(group * 4 + w) * kC + lane];
      const float top = mine[lane];
      mine[lane] = sum == 0.0f ? 0.0f : __fdividef(ks, sum);
      if (w4 == 0 && lane < nv && !lost) {
        if (!whole) {
          ws.m[slot * NR + col0 + lane] = top;
          ws.l[slot * NR + col0 + lane] = sum;
        } else if (a.lse) {
          a.lse[(int64_t)(tok0 + dt) * a.lse_ts + (int64_t)row_h * a.lse_hs] =
              sum == 0.0f ? -INFINITY : (top + __log2f(sum)) * kLn2;
        }
      }
    }
    __syncwarp();
#pragma unroll 1
    for (int n0 = 0; n0 < nv; n0 += 16) {
#pragma unroll 1
      for (int blk = 0; blk < 4; ++blk) {
        uint32_t r[16];
        const uint32_t o = sub + L::kO + blk * L::kPN + col0 + n0;
        tc::ld_32x16(o, r);
        if constexpr (L::kF8) {
#pragma unroll
          for (int k = 1; k < L::kParts; ++k) {
            uint32_t rk[16];
            tc::ld_32x16(o + k * NR, rk);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              r[i] = __float_as_uint(fmaf(__uint_as_float(rk[i]), k == 1 ? 1 / kPStep : 1 / (kPStep * kPStep),
                                          __uint_as_float(r[i])));
          }
        }
        if (lost) continue;
        if (whole) {
          // lanes 2 i and 2 i + 1 exchange, so that each holds two neighbouring columns of out
          uint8_t* o = a.out + (blk * 128 + w4 * 32 + (lane & ~1)) * 2;
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float v0 = __uint_as_float(r[i]) * mine[n0 + i];
            const float v1 = __uint_as_float(r[i + 1]) * mine[n0 + i + 1];
            const float x = __shfl_xor_sync(0xFFFFFFFFu, (lane & 1) ? v0 : v1, 1);
            const uint32_t w = (lane & 1) ? pack_bf16x2(x, v1) : pack_bf16x2(v0, x);
            const int n = n0 + i + (lane & 1);
            const int64_t at = __shfl_sync(0xFFFFFFFFu, row_at, n);
            if (n < nv) *reinterpret_cast<uint32_t*>(o + at) = w;
          }
        } else {
          // (16 rows of a dim in a run, 16 bytes per store, took three times as long: a
          // warp's store then touches 32 lines instead of one)
          float* dst = ws.o + (slot * NR + col0 + n0) * kRank + blk * 128 + w4 * 32 + lane;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (n0 + i < nv) dst[i * kRank] = __uint_as_float(r[i]);
        }
      }
    }
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + 8 * L::kOFree);
    soft_sync(group);  // red is read: the next tile may write it
  }
}

// ------------------------------------------------------------------ the kernel
// The runs of `total` units: the first `extra` CTAs take one unit more than the
// others; fewer CTAs than the grid has when each would get less than kMinUnits.
__device__ __noinline__ int64_t divide(int64_t n, int64_t d) { return n / d; }
__device__ __forceinline__ void cut(int64_t total, Run& r) {
  const uint32_t ctas = total >= (int64_t)gridDim.x * kMinUnits
                            ? gridDim.x
                            : max(1u, (uint32_t)total / (uint32_t)kMinUnits);
  if ((total >> 32) == 0) r.each = (uint32_t)total / ctas;
  else r.each = divide(total, ctas);
  r.extra = (int)(total - r.each * ctas);
  r.begin = r.each * blockIdx.x + min((int)blockIdx.x, r.extra);
  r.count = blockIdx.x < ctas ? (int)r.each + ((int)blockIdx.x < r.extra ? 1 : 0) : 0;
}
__device__ __forceinline__ int64_t scan64(int64_t v, int lane) {  // inclusive, over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// This CTA's run.  Up to 128 sequences of at most 8 query tiles: every warp finds it
// by itself without a barrier, a lane looking at four neighbouring sequences.
constexpr int kLaneSeqs = 4, kSmallTiles = 8;
template <int NR, int kSwitch>
__device__ __forceinline__ bool schedule_small(const LatentAttnArgs& a, int lane, Run& r,
                                               uint32_t& errbits) {
  if (a.num_seqs > 32 * kLaneSeqs) return false;
  const int per = (a.num_seqs + 31) >> 5, s0 = lane * per;  // this lane's sequences
  Seq q[kLaneSeqs];
#pragma unroll
  for (int i = 0; i < kLaneSeqs; ++i) {
    q[i].nqt = 0;
    if (i < per && s0 + i < a.num_seqs) q[i] = load_seq<NR>(a, s0 + i);
  }
  bool large = false;
  int u[kLaneSeqs], sum = 0;
#pragma unroll
  for (int i = 0; i < kLaneSeqs; ++i) {
    u[i] = 0;
    if (q[i].nqt == 0) continue;
    // the last query tile has the most key tiles: the sums stay below 2^31
    large |= q[i].nqt > kSmallTiles || most_seen<NR>(a, q[i], q[i].nqt - 1) > 1 << 24;
    if (over_room(a, q[i])) errbits |= kErrBlockOOB;
#pragma unroll 1
    for (int qt = 0; qt < min(q[i].nqt, kSmallTiles); ++qt)
      u[i] += kSwitch + key_tiles(most_seen<NR>(a, q[i], qt));
    sum += u[i];
  }
  if (__any_sync(0xFFFFFFFFu, large)) return false;
  int inc = sum;  // inclusive sum over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += v;
  }
  cut(__shfl_sync(0xFFFFFFFFu, inc, 31), r);
  r.kt = 0;
  if (r.count == 0) return true;
  // the lane, sequence and query tile with the run's first unit
  int off = (int)r.begin - (inc - sum), s = s0;
  const int from = __ffs(__ballot_sync(0xFFFFFFFFu, off >= 0 && off < sum)) - 1;
#pragma unroll
  for (int i = 0; i + 1 < kLaneSeqs; ++i)
    if (s == s0 + i && off >= u[i]) {
      off -= u[i];
      ++s;
    }
  r.s = __shfl_sync(0xFFFFFFFFu, s, from);
  off = __shfl_sync(0xFFFFFFFFu, off, from);
  r.q = load_seq<NR>(a, r.s);
#pragma unroll 1
  for (r.qt = 0;; ++r.qt) {
    const int k = kSwitch + key_tiles(most_seen<NR>(a, r.q, r.qt));
    if (off < k) break;
    off -= k;
  }
  r.kt = off - kSwitch;
  return true;
}

// Any number of sequences and query tiles, by the whole CTA; the scratch is the
// (still unused) first key stage.
template <int NR, int kSwitch, int kWarps>
__device__ __noinline__ void schedule_large(const LatentAttnArgs& a, uint8_t* scratch, Run& r) {
  constexpr int kThreads = kWarps * 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t* pre = reinterpret_cast<int64_t*>(scratch);  // [num_seqs]
  int64_t* part = pre + a.num_seqs;                    // [kWarps]
  int64_t* at = part + kWarps;                         // sequence, unit in it, query tile, key tile
  for (int s = warp; s < a.num_seqs; s += kWarps) {
    const Seq q = load_seq<NR>(a, s);
    int64_t u = 0;
    for (int qt = lane; qt < q.nqt; qt += 32)
      u += kSwitch + key_tiles(most_seen<NR>(a, q, qt));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
    if (lane == 0) pre[s] = u;
    if (lane == 0 && q.nqt > 0 && over_room(a, q) && a.err) atomicOr(a.err, kErrBlockOOB);
  }
  __syncthreads();
  // prefix sums: each thread a run of sequences, then warps, then all
  const int run = (a.num_seqs + kThreads - 1) / kThreads;
  const int s0 = min((int)threadIdx.x * run, a.num_seqs), s1 = min(s0 + run, a.num_seqs);
  int64_t sum = 0;
  for (int s = s0; s < s1; ++s) sum += pre[s];
  const int64_t inc = scan64(sum, lane);
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  int64_t before = inc - sum, total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += part[w];
    total += part[w];
  }
  cut(total, r);
  r.kt = 0;
  if (r.count > 0)
    for (int s = s0; s < s1; ++s) {
      const int64_t u = pre[s];
      if (before <= r.begin && r.begin < before + u) {
        at[0] = s;
        at[1] = r.begin - before;
      }
      before += u;
    }
  __syncthreads();
  if (r.count > 0) {
    r.s = (int)at[0];
    r.q = load_seq<NR>(a, r.s);
  }
  if (r.count > 0 && warp == 0) {
    const int64_t off = at[1];
    int64_t base = 0;
    for (int q0 = 0; q0 < r.q.nqt; q0 += 32) {
      const int64_t u =
          q0 + lane < r.q.nqt ? kSwitch + key_tiles(most_seen<NR>(a, r.q, q0 + lane)) : 0;
      const int64_t in = scan64(u, lane);
      const uint32_t hit = __ballot_sync(0xFFFFFFFFu, off < base + in);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          at[2] = q0 + lane;
          at[3] = off - (base + in - u);
        }
        break;
      }
      base += __shfl_sync(0xFFFFFFFFu, in, 31);
    }
  }
  __syncthreads();
  if (r.count > 0) {
    r.qt = (int)at[2];
    r.kt = (int)at[3] - kSwitch;
  }
  tc::fence_smem_async();  // the scratch is read; copies may write there now
  __syncthreads();
}

// After giving up: waits, bounded again, for the copies into shared memory that this
// thread's warp issued, and a millisecond for matrix products in flight (they end by
// themselves within microseconds).
template <int FMT, int NR>
__device__ __noinline__ void settle(uint32_t smem, uint32_t issued, uint64_t limit) {
  using L = Lay<FMT, NR>;
  const uint64_t since = global_ns();
  for (uint32_t g = issued > L::kStages ? issued - L::kStages : 0; g < issued; ++g)
    for (int h = 0; h < L::kHalves; ++h)
      while (!mbar_try_wait(smem + L::bars + 8 * (L::kFull + g % L::kStages * L::kHalves + h),
                            (g / L::kStages) & 1) &&
             global_ns() - since <= limit) {
      }
  while (global_ns() - since <= 1000000) {
  }
}

template <int FMT, int NR>
__global__ void __launch_bounds__(Lay<FMT, NR>::kThreads, 1)
    latent_attention_kernel(const LatentAttnArgs a, const __grid_constant__ CUtensorMap map) {
  using L = Lay<FMT, NR>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t smem = smem_addr(smem_raw);
  // broadcast, so that the compiler knows the roles' branches are uniform in a warp
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  Misc& m = *reinterpret_cast<Misc*>(smem_raw + L::misc);
  pdl_trigger();
  if (threadIdx.x == 0) {
    m.abort = 0;
    const uint32_t bars = smem + L::bars;
    for (int i = 0; i < L::kStages * L::kHalves; ++i) {
      // each producer warp's key flags, and each thread's row copies
      const bool stall = blockIdx.x == 0 && a.stall_stage == i / L::kHalves + 1;  // one arrival too many
      mbar_init(bars + 8 * (L::kFull + i), kProdWarps + kProdThreads + (stall ? 1 : 0));
      mbar_init(bars + 8 * (L::kEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars + 8 * (L::kQFull + i), kProdThreads);
      // the last scores of its query tile, and for fp8 the softmax warps' look at the scales
      mbar_init(bars + 8 * (L::kQEmpty + i), 1 + (L::kF8 ? L::kSoftWarps : 0));
      mbar_init(bars + 8 * (L::kSFull + i), 1);
      mbar_init(bars + 8 * (L::kPFull + i), L::kSoftWarps);
      mbar_init(bars + 8 * (L::kPvDone + i), 1);
    }
    mbar_init(bars + 8 * L::kOFree, L::kSoftWarps);
    mbar_fence_init();
  }
  const Waiter wait{smem_addr(&m.abort), a.wait_limit_ns};
  // Tensor memory is taken behind the wait for the kernel before: holding it there could
  // keep a block of that kernel from its own.
  pdl_wait();
  if (warp == L::kScoreWarp) tc::alloc(smem_addr(&m.tmem), L::kTmem);
  const Workspace ws = workspace_of<NR>(a.workspace, gridDim.x);
  if (threadIdx.x == 0) ws.split[blockIdx.x] = Split{0, 0, 0, 0, 0};
  uint32_t errbits = 0;
  Run run;
  if (!schedule_small<NR, L::kSwitch>(a, lane, run, errbits)) {
    Run large;  // apart, so that only this branch has it in memory
    schedule_large<NR, L::kSwitch, L::kWarps>(a, smem_raw, large);
    run = large;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, m.tmem, 0);
  uint32_t issued = 0;
  if (run.left() > 0) {
    if (warp < L::kSoftWarps)
      soften<FMT, NR>(a, run, smem, tmem, wait, warp, lane, ws);
    else if (warp >= L::kProdWarp)
      issued = produce<FMT, NR>(a, map, run, smem, wait, warp - L::kProdWarp, lane, errbits);
    else if (warp == L::kScoreWarp)
      score_role<FMT, NR>(a, run, smem, tmem, wait);
    else
      output_role<FMT, NR>(a, run, smem, tmem, wait, lane, ws);
  }
  __syncwarp();
  if (a.err) {
    errbits = __reduce_or_sync(0xFFFFFFFFu, errbits);
    if (lane == 0) {
      if (wait.given_up()) errbits |= kErrTimeout;
      if (errbits) atomicOr(a.err, errbits);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (__builtin_expect(wait.given_up(), 0)) {
    settle<FMT, NR>(smem, issued, a.wait_limit_ns);
    __syncthreads();
  }
  if (warp == L::kScoreWarp) tc::dealloc(tmem, L::kTmem);
}

// ---------------------------------------------------- join of the split query tiles
// Block (r, c) looks at what CTA c left.  The blocks of all CTAs of a split query tile
// but the last (which noted another tile, or none) deal its rows out: one per group of
// 128 threads (four dims a thread) with up to kFewParts partials, else one per block, a
// group a quarter of the partials (there are at least kFewParts * NR / 8 of those, one
// for every row).  So a block mostly costs two dependent loads, whatever the batch, and
// the grid, NR / 8 blocks per CTA, is one to four rounds of resident blocks.  With NR / 4
// and the rows of few partials left to the first CTA's, most blocks found nothing to do:
// 32 verifications took 48.5 us (48.2 now), 16 decodes of 128 heads 47.3 (46.1), one
// decode 10.7 (10.3).
constexpr int kJoinGroups = 4;
constexpr int kJoinThreads = kJoinGroups * 128;
constexpr int kFewParts = 8;
constexpr int kMaxCtas = 1024;

template <int FMT, int NR>
__global__ void __launch_bounds__(kJoinThreads, 2) latent_join_kernel(const LatentAttnArgs a) {
  __shared__ float4 acc_s[kJoinGroups][128];
  __shared__ float2 sum_s[kJoinGroups];
  pdl_trigger();
  pdl_wait();
  const Workspace ws = workspace_of<NR>(a.workspace, gridDim.y);
  const int grp = threadIdx.x >> 7, d4 = threadIdx.x & 127;
  const Split sp = ws.split[blockIdx.y];
  const int c = sp.first;
  const bool few = sp.parts <= kFewParts;
  const int blocks = (sp.parts - 1) * (int)gridDim.x;
  int n = ((int)blockIdx.y - c) * (int)gridDim.x + (int)blockIdx.x;
  if (few) n = n * kJoinGroups + grp;
  if (n >= sp.rows) return;  // the whole group, and the whole block when it is shared
  const float ks = FMT == kBF16 ? 1.0f : __ldg(a.k_scale);
  do {
    float4 acc = make_float4(0, 0, 0, 0);
    float sum = 0.0f, top = -INFINITY;
    // joins `v` with weight sum lv and maximum mv to what is there
    auto add = [&](const float4& v, float lv, float mv) {
      const float m = fmaxf(top, mv), m0 = m == -INFINITY ? 0.0f : m;
      const float f = ex2(top - m0), w = ex2(mv - m0);
      acc.x = fmaf(acc.x, f, w * v.x);
      acc.y = fmaf(acc.y, f, w * v.y);
      acc.z = fmaf(acc.z, f, w * v.z);
      acc.w = fmaf(acc.w, f, w * v.w);
      sum = fmaf(sum, f, w * lv);
      top = m;
    };
    // the first partial lies in the odd slot of CTA c, the others in the even ones behind
    const int quarter = (sp.parts + kJoinGroups - 1) / kJoinGroups;
    const int i0 = few ? 0 : min(grp * quarter, (int)sp.parts);
    const int i1 = few ? sp.parts : min(i0 + quarter, (int)sp.parts);
#pragma unroll 1
    for (int i = i0; i < i1; i += 4) {
      float4 v[4];
      float lv[4], mv[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t row = (2 * (int64_t)(c + i + k) + (i + k == 0 ? 1 : 0)) * NR + n;
        v[k] = make_float4(0, 0, 0, 0);
        lv[k] = 0.0f;
        mv[k] = -INFINITY;
        if (i + k < i1) {
          v[k] = __ldcs(reinterpret_cast<const float4*>(ws.o + row * kRank) + d4);
          lv[k] = ws.l[row];
          mv[k] = ws.m[row];
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) add(v[k], lv[k], mv[k]);
    }
    if (!few) {
      acc_s[grp][d4] = acc;
      if (d4 == 0) sum_s[grp] = make_float2(sum, top);
      __syncthreads();
      if (grp != 0) return;
#pragma unroll 1
      for (int k = 1; k < kJoinGroups; ++k) add(acc_s[k][d4], sum_s[k].x, sum_s[k].y);
    }
    const int dt = token_of(a, sp.head0 + n);
    const int64_t t = sp.tok0 + dt, h = sp.head0 + n - dt * a.num_heads;
    const float inv = sum == 0.0f ? 0.0f : __fdividef(ks, sum);
    st8(a.out + t * a.out_ts + h * a.out_hs + d4 * 8,
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv)));
    if (d4 == 0 && a.lse)
      a.lse[t * a.lse_ts + h * a.lse_hs] = sum == 0.0f ? -INFINITY : (top + __log2f(sum)) * kLn2;
    n += blocks * kJoinGroups;
  } while (few && n < sp.rows);
}

// The cache as a tensor of (column, entry, block), read in boxes of one chunk of
// `rows` entries.  Without a box (entries per block not a multiple of 8, or sizes
// that a tensor map does not hold) rows are copied one by one: 64 ragged e4m3 decodes
// then take 94.0 us instead of 60.5, 4 x 131072 bf16 rows 107.5 instead of 99.4.
// Returns the entries of a box, or 0.  (All chunks of a tile as one box of a
// 4-dimensional map took the same time.)
int box_map(const LatentAttnArgs& a, bool fp8, CUtensorMap* map) {
  int rows = kKeys;
  while (a.block_size % rows) rows >>= 1;
  if (rows < 8 || a.num_blocks >= INT32_MAX) return 0;
  static const auto encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    (void)cudaGetLastError();
    return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(f);
  }();
  if (!encode) return 0;
  const cuuint64_t dims[3] = {576, (cuuint64_t)a.block_size, (cuuint64_t)a.num_blocks};
  const cuuint64_t strides[2] = {(cuuint64_t)a.entry_stride, (cuuint64_t)a.block_stride};
  const cuuint32_t box[3] = {fp8 ? 128u : 64u, (cuuint32_t)rows, 1}, unit[3] = {1, 1, 1};
  const CUresult r = encode(
      map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
      const_cast<uint8_t*>(a.cache), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? rows : 0;
}

template <int FMT, int NR>
cudaError_t launch_t(const LatentAttnArgs& a, const CUtensorMap& map, int ctas,
                     const LaunchCfg& cfg) {
  using L = Lay<FMT, NR>;
  auto kern = latent_attention_kernel<FMT, NR>;
  // the attribute stays with the device's context: set on a device's first call
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(set.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::bytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) set.fetch_or(uint64_t(1) << dev);
  }
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(ctas);
  lc.blockDim = dim3(L::kThreads);
  lc.dynamicSmemBytes = L::bytes;
  lc.stream = cfg.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = cfg.pdl ? 1 : 0;
  e = cudaLaunchKernelEx(&lc, kern, a, map);
  if (e != cudaSuccess) return e;
  lc.gridDim = dim3(NR / 8, ctas);
  lc.blockDim = dim3(kJoinThreads);
  lc.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&lc, latent_join_kernel<FMT, NR>, a);
}

template <int FMT>
cudaError_t launch_f(LatentAttnArgs a, int ctas, const LaunchCfg& cfg) {
  constexpr bool kF8 = FMT != kBF16;
  CUtensorMap map = {};
  a.box_rows = box_map(a, kF8, &map);
  for (int rows = a.box_rows; rows != 0 && rows < kKeys; rows *= 2) ++a.box_shift;
  const int nr = attention_tile_rows(a.num_tokens, a.num_heads, a.num_seqs, kF8);
  // Cache rows that up to four query tiles of a sequence read (at about the same time) are
  // the first to leave L2: 64 ragged decodes 60.5 us (62.9 without the hint), in bf16 103.5
  // (107.3), 32 verifications 48.2 (50.5), 16 decodes of 128 heads 46.1 (46.9).  The many
  // query tiles of a prefill want them kept: 2 chunks of 1024 tokens 645 us (699 with the
  // hint).  16 bf16 sequences over 8192 rows at 2, 4, 8 and 16 query tiles each: 73.7, 121.8,
  // 219.7 and 415 us with it, 74.0, 121.4, 213.6 and 391 without.
  a.stream_rows = (int64_t)a.num_tokens * a.num_heads <= (int64_t)4 * nr * a.num_seqs;
  switch (nr) {
    case 16: return launch_t<FMT, 16>(a, map, ctas, cfg);
    case 32: return launch_t<FMT, 32>(a, map, ctas, cfg);
    default:
      if constexpr (!kF8) return launch_t<FMT, 64>(a, map, ctas, cfg);
      else return cudaErrorInvalidValue;
  }
}

}  // namespace

// Calls of fewer sequences within these sizes have more rows per sequence, at most all of
// them in one: its (bf16) tile is the largest that any of them takes.
int64_t latent_attention_workspace(int32_t num_tokens, int32_t num_heads, int32_t, int num_sms) {
  const int64_t ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
  const int64_t nr = attention_tile_rows(num_tokens, num_heads, 1, false);
  return ctas * ((int64_t)sizeof(Split) + 2 * nr * (2 + kRank) * (int64_t)sizeof(float));
}

cudaError_t launch_latent_attention(const LatentAttnArgs& a, int cache_fmt, int num_sms,
                                    const LaunchCfg& cfg) {
  const int ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
  switch (cache_fmt) {
    case kBF16: return launch_f<kBF16>(a, ctas, cfg);
    case kE4M3: return launch_f<kE4M3>(a, ctas, cfg);
    case kE5M2: return launch_f<kE5M2>(a, ctas, cfg);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mla
