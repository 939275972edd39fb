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
// (query tile) whose units fall into several CTAs leaves unnormalised fp32
// partial sums in the workspace, which a second small launch joins in the
// order of the CTAs (no atomics: equal calls give equal bits).
//
// Both products are computed transposed, so that few query rows (a decode
// batch has 16 per token) are the N dimension of the tensor core's tile and no
// row of it is wasted:
//   scores    S^T [64 keys x NR]  = K  [64 x 576] * Q^T   (A = K as loaded)
//   outputs   O^T [512 x NR]     += V^T [512 x 64] * P^T  (A = the same shared
//             memory read MN-major: a latent row is key and value)
// A key tile is 9 chunks of 64 keys x 64 columns bf16 in the 128-byte swizzle.
// S^T (two buffers) and O^T (4 x 128 dims) stay in tensor memory.
//
// Roles (13 warps): 8 producer warps load and, for fp8, widen key tiles into a
// two-stage ring; one thread issues the matrix instructions; 4 warps do the
// softmax (running maximum per query row, rescaling O^T only when the maximum
// has grown by more than 2^8) and the output.  The scores of tile i + 1 are
// issued before the outputs of tile i, so they overlap the softmax.
//
// Rows that a token must not see: rows behind every row's view are loaded as
// zeros; in the tiles where tokens of one query tile see different rows, a row
// holding a NaN or an infinity is loaded as zeros and marked, and its score
// becomes NaN for the tokens that do see it.
//
// Waits are bounded (wait_limit_ns): one that runs out marks the CTA as given
// up, every later wait returns at once, and MLA_ERRBIT_TIMEOUT is set.
#include "mla_device.cuh"
#include "mla_internal.h"
#include "tensor_core.cuh"

namespace mla {
namespace {

constexpr int kKeys = 64;                    // keys per tile
constexpr int kChunk = kKeys * 128;          // bytes of a chunk: 64 keys x 64 columns
constexpr int kChunks = 9;                   // 576 columns
constexpr int kTile = kChunks * kChunk;      // 73728
constexpr int kStages = 2;
constexpr int kSoftWarps = 4;
constexpr int kMmaWarp = kSoftWarps;
constexpr int kProdWarp = kMmaWarp + 1;
constexpr int kProdWarps = 8;
constexpr int kWarps = kProdWarp + kProdWarps;
constexpr int kThreads = kWarps * 32;
constexpr int kProdThreads = kProdWarps * 32;
constexpr int kRank = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 8.0f;  // rescale when a maximum grows by more than this (log2)
constexpr int kMinUnits = 2;   // a CTA takes at least this many units

// Key flags of a tile (one byte per key).
constexpr uint32_t kAbsent = 1;  // its block was not found: left out
constexpr uint32_t kPoison = 2;  // holds a NaN or an infinity

template <int NR>
struct Lay {
  static constexpr int kQBufs = NR <= 32 ? 2 : 1;
  static constexpr int kQ = kChunks * NR * 128;
  static constexpr int q = kStages * kTile;
  static constexpr int p = q + kQBufs * kQ;          // NR x 64 keys bf16
  static constexpr int red = p + NR * 128;           // float [2][4][NR]
  static constexpr int flags = red + 2 * 4 * NR * 4; // uint8 [kStages][64]
  static constexpr int bars = flags + kStages * 64;
  static constexpr int kBars = 13;
  static constexpr int misc = bars + kBars * 8;      // Misc
  static constexpr int bytes = misc + 64;
  static constexpr int kCols = NR == 16 ? 128 : NR == 32 ? 256 : 512;
};
enum Bar { kFull = 0, kEmpty = 2, kQFull = 4, kQEmpty = 6, kSFull = 8, kPFull = 10, kPvDone = 11,
           kOFree = 12 };

struct Misc {
  uint32_t tmem;
  uint32_t abort;
  int32_t s, qt, kt, ctas;
  int64_t begin, count, total;
};
static_assert(sizeof(Misc) <= 64, "Misc fits");

// A split query tile that CTA c starts: the partials of CTAs c .. last belong to it.
struct Split {
  int32_t s, qt, last, pad;
};

struct Seq {
  int32_t t0, ntok;  // tokens t0 .. t0 + ntok - 1 are computed
  int32_t c1, kv;
  int32_t nqt;       // query tiles
};

template <int NR>
__device__ __forceinline__ Seq load_seq(const LatentAttnArgs& a, int s) {
  Seq q;
  const int32_t c0 = __ldg(a.cu_q + s);
  q.c1 = __ldg(a.cu_q + s + 1);
  q.kv = __ldg(a.kv_lens + s);
  q.t0 = max(c0, 0);
  q.ntok = max(min(q.c1, a.num_tokens) - q.t0, 0);
  q.nqt = (int)(((int64_t)q.ntok * a.num_heads + NR - 1) / NR);
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
  const int64_t last = min((int64_t)(qt + 1) * NR, (int64_t)q.ntok * a.num_heads) - 1;
  return seen_of(a, q, q.t0 + (int)(last / a.num_heads));
}
// Key tiles of a query tile that sees `most` rows (one even when it sees none: its
// rows are still written).
__device__ __forceinline__ int key_tiles(int most) { return max(1, (most + kKeys - 1) / kKeys); }

struct Tile {
  bool valid, first, last;  // first / last of this CTA's run of the query tile
  int s, qt, kt, nkt;
  int most, least;          // rows seen by the last / first row of the query tile
};

// Walks a CTA's run of units; every role has its own copy.
template <int NR>
struct Walk {
  Seq q;
  int s, qt, kt, nkt, most, least;
  int64_t left;
  bool fresh;
  __device__ __forceinline__ void item(const LatentAttnArgs& a) {
    most = most_seen<NR>(a, q, qt);
    least = seen_of(a, q, q.t0 + (int)((int64_t)qt * NR / a.num_heads));
    nkt = key_tiles(most);
    fresh = true;
  }
  __device__ __forceinline__ void start(const LatentAttnArgs& a, const Misc& m) {
    s = m.s;
    qt = m.qt;
    kt = m.kt;
    left = m.count;
    if (left > 0) {
      q = load_seq<NR>(a, s);
      item(a);
    }
  }
  __device__ __forceinline__ Tile next(const LatentAttnArgs& a) {
    Tile t{};
    if (left <= 0) return t;
    if (kt == nkt) {
      kt = 0;
      ++qt;
      while (qt >= q.nqt && s + 1 < a.num_seqs) {
        q = load_seq<NR>(a, ++s);
        qt = 0;
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
    --left;
    t.last = kt == nkt || left == 0;
    return t;
  }
};

// Bounded waits of one thread.
struct Waiter {
  uint32_t abort;  // shared address of Misc::abort
  uint64_t limit;
  __device__ __forceinline__ bool given_up() const { return lds_u32(abort) != 0; }
  __device__ __forceinline__ void operator()(uint32_t bar, uint32_t parity) const {
    if (mbar_try_wait(bar, parity)) return;
    const uint64_t t0 = global_ns();
    for (uint32_t spin = 1;; ++spin) {
      if (mbar_try_wait(bar, parity)) return;
      if ((spin & 31u) == 0) {
        if (given_up()) return;
        if (global_ns() - t0 > limit) {
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(abort), "r"(1u) : "memory");
          return;
        }
      }
    }
  }
};

__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void sts_u8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void soft_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kSoftWarps * 32) : "memory");
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

// The address of row p of sequence s, or nullptr: not seen by any row of the
// query tile (p >= most), or its block cannot be found (flag kAbsent).
__device__ __forceinline__ const uint8_t* find_row(const LatentAttnArgs& a, int s, int p, int most,
                                                   uint32_t& flag) {
  flag = 0;
  if (p >= most) return nullptr;
  const int kb = a.bs_shift >= 0 ? p >> a.bs_shift : p / a.block_size;
  const int32_t blk = __ldg(a.block_table + (int64_t)s * a.bt_stride + kb);
  if (blk < 0 || blk >= a.num_blocks) {
    flag = kAbsent;
    return nullptr;
  }
  return a.cache + (int64_t)blk * a.block_stride + (int64_t)(p - kb * a.block_size) * a.entry_stride;
}

// ------------------------------------------------------------------ producers
template <int NR>
__device__ __forceinline__ void load_q(const LatentAttnArgs& a, const Seq& q, int qt, uint32_t dst,
                                       int pw, int lane) {
  const int64_t rows = (int64_t)q.ntok * a.num_heads;
  const int col = lane & 7;
  for (int r = pw * 4 + (lane >> 3); r < NR; r += kProdWarps * 4) {
    const int64_t row = (int64_t)qt * NR + r;
    const bool ok = row < rows;
    const int64_t t = ok ? q.t0 + row / a.num_heads : 0;
    const int64_t h = ok ? row % a.num_heads : 0;
    const uint8_t* c = a.q_c + t * a.qc_ts + h * a.qc_hs + col * 16;
    const uint8_t* pe = a.q_pe + t * a.qp_ts + h * a.qp_hs + col * 16;
    const uint32_t d = dst + r * 128 + ((col ^ (r & 7)) << 4);
#pragma unroll
    for (int ch = 0; ch < 8; ++ch) tc::cp_async16(d + ch * (NR * 128), c + ch * 128, ok);
    tc::cp_async16(d + 8 * (NR * 128), pe, ok);
  }
}

template <int FMT, int NR>
__device__ __forceinline__ void produce(const LatentAttnArgs& a, const Misc& m, uint32_t smem,
                                        const Waiter& wait, int pw, int lane, uint32_t& errbits) {
  using L = Lay<NR>;
  const uint32_t bars = smem + L::bars;
  Walk<NR> walk;
  walk.start(a, m);
  // bf16: 8 lanes x 16 bytes per row, rows pw * 8 + lane / 8 and + 4.
  // fp8: 4 lanes x 16 bytes per row, row pw * 8 + lane / 4.
  constexpr int kRows = FMT == kBF16 ? 2 : 1;
  const int row0 = pw * 8 + (FMT == kBF16 ? lane >> 3 : lane >> 2);
  const int col = FMT == kBF16 ? lane & 7 : lane & 3;
  const bool marks = col == 0;  // the lane that writes its rows' flags
  Tile cur = walk.next(a);
  Seq cq = walk.q;
  const uint8_t* src[kRows];
  uint32_t flag[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    src[i] = cur.valid ? find_row(a, cur.s, cur.kt * kKeys + row0 + 4 * i, cur.most, flag[i]) : nullptr;
  uint4 reg[FMT == kBF16 ? 1 : kChunks];
  if constexpr (FMT != kBF16) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      reg[c] = src[0] ? ld_stream16(src[0] + col * 16 + c * 64) : make_uint4(0, 0, 0, 0);
  }
  uint32_t g = 0, item = 0;
  for (; cur.valid; ++g) {
    if (cur.first) {
      const int b = item % L::kQBufs;
      const uint32_t n = item / L::kQBufs;
      if (n > 0) wait(bars + 8 * (kQEmpty + b), (n - 1) & 1);
      load_q<NR>(a, cq, cur.qt, smem + L::q + b * L::kQ, pw, lane);
      tc::cp_async_arrive(bars + 8 * (kQFull + b));
      ++item;
    }
    const Tile nxt = walk.next(a);
    const uint8_t* nsrc[kRows];
    uint32_t nflag[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      nsrc[i] = nxt.valid ? find_row(a, nxt.s, nxt.kt * kKeys + row0 + 4 * i, nxt.most, nflag[i])
                          : nullptr;
    const int st = g & 1;
    const uint32_t full = bars + 8 * (kFull + st);
    if (g >= kStages) wait(bars + 8 * (kEmpty + st), ((g >> 1) - 1) & 1);
    const uint32_t base = smem + st * kTile;
    // tokens of the query tile see different rows of this key tile
    const bool mixed = cur.least < cur.most && (cur.kt + 1) * kKeys > cur.least;
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (flag[i]) errbits |= kErrBlockOOB;
    if constexpr (FMT == kBF16) {
      if (!mixed) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int row = row0 + 4 * i;
          const uint32_t d = base + row * 128 + ((col ^ (row & 7)) << 4);
          const uint8_t* p = src[i] ? src[i] + col * 16 : a.cache;
#pragma unroll
          for (int c = 0; c < kChunks; ++c) tc::cp_async16(d + c * kChunk, p + (src[i] ? c * 128 : 0), src[i] != nullptr);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int row = row0 + 4 * i;
          const uint32_t d = base + row * 128 + ((col ^ (row & 7)) << 4);
          uint4 v[kChunks];
          bool sp = false;
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            v[c] = src[i] ? ld_stream16(src[i] + col * 16 + c * 128) : make_uint4(0, 0, 0, 0);
            sp |= any_special<kBF16>(v[c]);
          }
          const uint32_t who = __ballot_sync(0xFFFFFFFFu, sp);
          if (who & (0xFFu << (lane & 24))) {
            flag[i] = kPoison;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) v[c] = make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int c = 0; c < kChunks; ++c) sts16(d + c * kChunk, v[c]);
        }
        tc::fence_smem_async();
      }
    } else {
      const int row = row0;
      if (mixed) {
        bool sp = false;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) sp |= any_special<FMT>(reg[c]);
        const uint32_t who = __ballot_sync(0xFFFFFFFFu, sp);
        if (who & (0xFu << (lane & 28))) {
          flag[0] = kPoison;
#pragma unroll
          for (int c = 0; c < kChunks; ++c) reg[c] = make_uint4(0, 0, 0, 0);
        }
      }
      const uint32_t d0 = base + row * 128 + (((2 * col) ^ (row & 7)) << 4);
      const uint32_t d1 = base + row * 128 + (((2 * col + 1) ^ (row & 7)) << 4);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const uint4 v = reg[c];
        sts16(d0 + c * kChunk, fp8x8_to_x16x8<FMT, kBF16>(make_uint2(v.x, v.y)));
        sts16(d1 + c * kChunk, fp8x8_to_x16x8<FMT, kBF16>(make_uint2(v.z, v.w)));
        reg[c] = nsrc[0] ? ld_stream16(nsrc[0] + col * 16 + c * 64) : make_uint4(0, 0, 0, 0);
      }
      tc::fence_smem_async();
    }
    if (marks) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) sts_u8(smem + L::flags + st * kKeys + row0 + 4 * i, flag[i]);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(full);
    if (FMT == kBF16 && !mixed) tc::cp_async_arrive(full);
    else mbar_arrive(full);
    cur = nxt;
    cq = walk.q;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      src[i] = nsrc[i];
      flag[i] = nflag[i];
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// --------------------------------------------------------------- matrix issue
template <int NR>
__device__ __forceinline__ void issue_mma(const LatentAttnArgs& a, const Misc& m, uint32_t smem,
                                          uint32_t tmem, const Waiter& wait) {
  using L = Lay<NR>;
  constexpr uint32_t kIdS = tc::instr_desc(kKeys, NR, false);
  constexpr uint32_t kIdO = tc::instr_desc(128, NR, true);
  const uint32_t bars = smem + L::bars;
  const uint64_t dk = tc::smem_desc(smem, 0, 1024);            // K tiles, K-major
  const uint64_t dv = tc::smem_desc(smem, kChunk, 1024);       // the same, MN-major
  const uint64_t dq = tc::smem_desc(smem + L::q, 0, 1024);
  const uint64_t dp = tc::smem_desc(smem + L::p, 0, 1024);
  Walk<NR> walk;
  walk.start(a, m);
  uint32_t items = 0;  // query tiles whose scores have begun
  auto scores = [&](const Tile& t, uint32_t g) {
    if (t.first) {
      wait(bars + 8 * (kQFull + items % L::kQBufs), (items / L::kQBufs) & 1);
      ++items;
    }
    wait(bars + 8 * (kFull + (g & 1)), (g >> 1) & 1);
    tc::fence_smem_async();
    tc::fence_after_sync();
    const int qb = (items - 1) % L::kQBufs;
    const uint64_t ka = dk + ((g & 1) * kTile >> 4);
    const uint64_t qa = dq + (qb * L::kQ >> 4);
#pragma unroll 1
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        tc::mma_bf16(tmem + (g & 1) * NR, ka + (c * kChunk >> 4) + 2 * k,
                     qa + (c * NR * 128 >> 4) + 2 * k, kIdS, c + k > 0);
    tc::commit(bars + 8 * (kSFull + (g & 1)));
    if (t.last) tc::commit(bars + 8 * (kQEmpty + qb));
  };
  Tile cur = walk.next(a);
  if (cur.valid) scores(cur, 0);
  uint32_t done_items = 0;
  for (uint32_t g = 0; cur.valid; ++g) {
    const Tile nxt = walk.next(a);
    const bool ahead = nxt.valid && (!nxt.first || L::kQBufs > 1);
    if (ahead) scores(nxt, g + 1);
    wait(bars + 8 * kPFull, g & 1);
    if (cur.first) {
      if (done_items > 0) wait(bars + 8 * kOFree, (done_items - 1) & 1);
      ++done_items;
    }
    tc::fence_after_sync();
    const uint64_t va = dv + ((g & 1) * kTile >> 4);
#pragma unroll 1
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        tc::mma_bf16(tmem + 2 * NR + b * NR, va + (2 * b * kChunk >> 4) + k * (2048 >> 4), dp + 2 * k,
                     kIdO, k > 0 || !cur.first);
    tc::commit(bars + 8 * (kEmpty + (g & 1)));
    tc::commit(bars + 8 * kPvDone);
    if (nxt.valid && !ahead) scores(nxt, g + 1);
    cur = nxt;
  }
}

// ----------------------------------------------------------- softmax and output
struct Workspace {
  Split* split;  // [ctas]
  float2* ml;    // [2 ctas][NR]: running maximum (log2 units) and sum
  float* o;      // [2 ctas][NR][512]: unnormalised sums
};
template <int NR>
__host__ __device__ inline Workspace workspace_of(uint8_t* p, int ctas) {
  Workspace w;
  w.split = reinterpret_cast<Split*>(p);
  p += (int64_t)ctas * sizeof(Split);
  w.ml = reinterpret_cast<float2*>(p);
  p += (int64_t)ctas * 2 * NR * sizeof(float2);
  w.o = reinterpret_cast<float*>(p);
  return w;
}

template <int FMT, int NR>
__device__ __forceinline__ void soften(const LatentAttnArgs& a, const Misc& m, uint32_t smem,
                                       uint32_t tmem, const Waiter& waiter, int warp, int lane,
                                       const Workspace& ws) {
  using L = Lay<NR>;
  constexpr int kG = NR / 8;  // column groups; a thread has columns 8 j + 2 (lane % 4) + {0, 1}
  const uint32_t bars = smem + L::bars;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    waiter(bar, parity);
    __syncwarp();
  };
  const uint32_t sub = tmem + ((uint32_t)(warp * 32) << 16);  // this warp's lanes
  const float ks = FMT == kBF16 ? 1.0f : __ldg(a.k_scale);
  const float c = a.softmax_scale * ks * kLog2e;
  const int c2 = 2 * (lane & 3);
  const int key0 = warp * 16 + (lane >> 2);  // and + 8
  float* red = reinterpret_cast<float*>(__cvta_shared_to_generic(smem + L::red));
  float mu[kG][2], l[kG][2];
  int seen[kG][2];
  Walk<NR> walk;
  walk.start(a, m);
  int kt_begin = 0;
  uint32_t g = 0;
  for (Tile t = walk.next(a); t.valid; t = walk.next(a), ++g) {
    if (t.first) {
      kt_begin = t.kt;
#pragma unroll
      for (int j = 0; j < kG; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // a row behind the last one (its query is zeros) copies the last one's view
          const int64_t row = min((int64_t)t.qt * NR + 8 * j + c2 + e,
                                  (int64_t)walk.q.ntok * a.num_heads - 1);
          seen[j][e] = seen_of(a, walk.q, walk.q.t0 + (int)(row / a.num_heads));
          l[j][e] = 0.0f;
          mu[j][e] = -INFINITY;
        }
    }
    const int b = g & 1;
    wait(bars + 8 * (kFull + b), (g >> 1) & 1);  // the key flags
    wait(bars + 8 * (kSFull + b), (g >> 1) & 1);
    tc::fence_after_sync();
    float x[kG][4];
    tc::ld_16x256<kG>(sub + b * NR, reinterpret_cast<uint32_t*>(&x[0][0]));
    const uint32_t f0 = lds_u8(smem + L::flags + b * kKeys + key0);
    const uint32_t f1 = lds_u8(smem + L::flags + b * kKeys + key0 + 8);
#pragma unroll
    for (int j = 0; j < kG; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[j][i] *= c;
    if ((t.kt + 1) * kKeys > t.least || __any_sync(0xFFFFFFFFu, (f0 | f1) != 0)) {
      const int p = t.kt * kKeys + key0;
#pragma unroll
      for (int j = 0; j < kG; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t f = i < 2 ? f0 : f1;
          if (f == kPoison) x[j][i] = NAN;
          if (p + (i < 2 ? 0 : 8) >= seen[j][i & 1] || f == kAbsent) x[j][i] = -INFINITY;
        }
    }
    // maximum over the tile's 64 keys: in the warp, then across the four warps
    float tm[kG][2];
    float* mine = red + (b * 4 + warp) * NR;
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
    soft_sync();
    bool grown = false;
#pragma unroll
    for (int j = 0; j < kG; ++j) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float2 v = *reinterpret_cast<const float2*>(red + (b * 4 + w) * NR + 8 * j + c2);
        tm[j][0] = fmaxf(tm[j][0], v.x);
        tm[j][1] = fmaxf(tm[j][1], v.y);
      }
      grown |= tm[j][0] > mu[j][0] + kGrow || tm[j][1] > mu[j][1] + kGrow;
    }
    // P's buffer, and O^T for the rescaling, are free when the outputs of the tile before are done
    if (g > 0) wait(bars + 8 * kPvDone, (g - 1) & 1);
    if (__any_sync(0xFFFFFFFFu, grown)) {  // the same in all four warps
      float* fac = red + ((b ^ 1) * 4 + warp) * NR;
      __syncwarp();
#pragma unroll
      for (int j = 0; j < kG; ++j) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mn = fmaxf(mu[j][e], tm[j][e]);
          f[e] = mu[j][e] == -INFINITY ? 0.0f : ex2(mu[j][e] - mn);
          l[j][e] *= f[e];
          mu[j][e] = mn;
        }
        if (lane < 4) *reinterpret_cast<float2*>(fac + 8 * j + c2) = make_float2(f[0], f[1]);
      }
      __syncwarp();
      if (!t.first) {
        tc::fence_after_sync();
#pragma unroll 1
        for (int n = 0; n < 4 * NR; n += 16) {
          uint32_t r[16];
          tc::ld_32x16(sub + 2 * NR + n, r);
  #pragma unroll
          for (int i = 0; i < 16; ++i)
            r[i] = __float_as_uint(__uint_as_float(r[i]) * fac[(n & (NR - 1)) + i]);
          tc::st_32x16(sub + 2 * NR + n, r);
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
        w[2 * jj] = pack_bf16x2(p0, p1);
        w[2 * jj + 1] = pack_bf16x2(p2, p3);
      }
      const int n = (j + (lane >> 4)) * 8 + (lane & 7);
      const int unit = 2 * warp + ((lane >> 3) & 1);
      tc::st_8x8_t(smem + L::p + n * 128 + ((unit ^ (n & 7)) << 4), w[0], w[1], w[2], w[3]);
    }
    tc::fence_smem_async();
    tc::fence_before_sync();
    mbar_arrive(bars + 8 * kPFull);
    if (!t.last) continue;

    // ---- the end of this CTA's run of the query tile
    wait(bars + 8 * kPvDone, g & 1);
    tc::fence_after_sync();
    float* part = red + ((b ^ 1) * 4 + warp) * NR;
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
    soft_sync();
    const bool whole = kt_begin == 0 && t.kt + 1 == t.nkt;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (kt_begin == 0 ? 1 : 0);
    const int64_t rows = (int64_t)walk.q.ntok * a.num_heads;
    const int64_t first = (int64_t)t.qt * NR;
    const int nv = (int)min((int64_t)NR, rows - first);
    const int tok0 = walk.q.t0 + (int)(first / a.num_heads);
    const int head0 = (int)(first % a.num_heads);
    const bool lost = waiter.given_up();
#pragma unroll
    for (int j = 0; j < kG; ++j) {
      float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float2 v = *reinterpret_cast<const float2*>(red + ((b ^ 1) * 4 + w) * NR + 8 * j + c2);
        sum.x += v.x;
        sum.y += v.y;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float s = e ? sum.y : sum.x;
        const int n = 8 * j + c2 + e;
        if (lane < 4) mine[n] = s == 0.0f ? 0.0f : ks / s;
        if (warp == 0 && lane < 4 && n < nv && !lost) {
          if (!whole) {
            ws.ml[slot * NR + n] = make_float2(mu[j][e], s);
          } else if (a.lse) {
            const int64_t hh = head0 + n;
            a.lse[(tok0 + hh / a.num_heads) * a.lse_ts + hh % a.num_heads * a.lse_hs] =
                s == 0.0f ? -INFINITY : fmaf(mu[j][e], kLn2, logf(s));
          }
        }
      }
    }
    __syncwarp();
    if (!whole && kt_begin == 0 && warp == 0 && lane == 0 && !lost) {
      const int64_t u1 = m.begin + m.count - 1 + (t.nkt - 1 - t.kt);  // the query tile's last unit
      ws.split[blockIdx.x] = Split{t.s, t.qt, (int)(((u1 + 1) * m.ctas - 1) / m.total), 0};
    }
#pragma unroll 1
    for (int blk = 0; blk < 4; ++blk) {
#pragma unroll 1
      for (int n0 = 0; n0 < nv; n0 += 16) {
        uint32_t r[16];
        tc::ld_32x16(sub + 2 * NR + blk * NR + n0, r);
        if (lost) continue;
        if (whole) {
          // lanes 2 i and 2 i + 1 exchange, so that each holds two neighbouring columns of out
          int h = head0 + n0 + (lane & 1), tok = tok0 + h / a.num_heads;
          h %= a.num_heads;
          const int d = blk * 128 + warp * 32 + (lane & ~1);
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float v0 = __uint_as_float(r[i]) * mine[n0 + i];
            const float v1 = __uint_as_float(r[i + 1]) * mine[n0 + i + 1];
            const float o = __shfl_xor_sync(0xFFFFFFFFu, (lane & 1) ? v0 : v1, 1);
            const uint32_t w = (lane & 1) ? pack_bf16x2(o, v1) : pack_bf16x2(v0, o);
            if (n0 + i + (lane & 1) < nv)
              *reinterpret_cast<uint32_t*>(a.out + (int64_t)tok * a.out_ts + (int64_t)h * a.out_hs + d * 2) = w;
            h += 2;
            while (h >= a.num_heads) {
              h -= a.num_heads;
              ++tok;
            }
          }
        } else {
          float* dst = ws.o + (slot * NR + n0) * kRank + blk * 128 + warp * 32 + lane;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (n0 + i < nv) dst[i * kRank] = __uint_as_float(r[i]);
        }
      }
    }
    tc::fence_before_sync();
    mbar_arrive(bars + 8 * kOFree);
    soft_sync();  // red is read: the next tile may write it
  }
}

// ------------------------------------------------------------------ the kernel
// Splits the call's units over the CTAs and finds this CTA's first unit; the
// scratch is the (still unused) first key stage.
template <int NR>
__device__ __forceinline__ void schedule(const LatentAttnArgs& a, uint8_t* scratch, Misc& m,
                                         uint32_t& errbits) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t* pre = reinterpret_cast<int64_t*>(scratch);  // [num_seqs + 1]
  int64_t* part = pre + a.num_seqs + 1;                // [kWarps]
  for (int s = warp; s < a.num_seqs; s += kWarps) {
    const Seq q = load_seq<NR>(a, s);
    int64_t u = 0;
    for (int qt = lane; qt < q.nqt; qt += 32) u += key_tiles(most_seen<NR>(a, q, qt));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
    if (lane == 0) {
      pre[s] = u;
      const int64_t most = (int64_t)q.kv + (a.causal ? (int64_t)q.t0 + q.ntok - q.c1 : 0);
      if (q.ntok > 0 && most > a.room) errbits |= kErrBlockOOB;
    }
  }
  __syncthreads();
  // exclusive prefix sums: each thread a run of sequences, then warps, then all
  const int run = (a.num_seqs + kThreads - 1) / kThreads;
  const int s0 = min((int)threadIdx.x * run, a.num_seqs), s1 = min(s0 + run, a.num_seqs);
  int64_t sum = 0;
  for (int s = s0; s < s1; ++s) sum += pre[s];
  int64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  int64_t before = inc - sum, total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += part[w];
    total += part[w];
  }
  const int ctas = (int)max((int64_t)1, min((int64_t)gridDim.x, total / kMinUnits));
  const int64_t begin = total * blockIdx.x / ctas, end = total * (blockIdx.x + 1) / ctas;
  const bool works = (int)blockIdx.x < ctas && end > begin;
  if (threadIdx.x == 0) {
    m.begin = begin;
    m.count = works ? end - begin : 0;
    m.total = total;
    m.ctas = ctas;
  }
  if (works)
    for (int s = s0; s < s1; ++s) {
      const int64_t u = pre[s];
      if (before <= begin && begin < before + u) {
        m.s = s;
        part[kWarps] = begin - before;
      }
      before += u;
    }
  __syncthreads();
  if (works && warp == 0) {
    const Seq q = load_seq<NR>(a, m.s);
    const int64_t off = part[kWarps];
    int64_t base = 0;
    for (int q0 = 0; q0 < q.nqt; q0 += 32) {
      const int64_t u = q0 + lane < q.nqt ? key_tiles(most_seen<NR>(a, q, q0 + lane)) : 0;
      int64_t in = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, in, o);
        if (lane >= o) in += v;
      }
      const uint32_t hit = __ballot_sync(0xFFFFFFFFu, off < base + in);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          m.qt = q0 + lane;
          m.kt = (int)(off - (base + in - u));
        }
        break;
      }
      base += __shfl_sync(0xFFFFFFFFu, in, 31);
    }
  }
  __syncthreads();
}

template <int FMT, int NR>
__global__ void __launch_bounds__(kThreads, 1) latent_attention_kernel(const LatentAttnArgs a) {
  using L = Lay<NR>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t smem = smem_addr(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Misc& m = *reinterpret_cast<Misc*>(smem_raw + L::misc);
  pdl_trigger();
  if (warp == kMmaWarp) tc::alloc(smem_addr(&m.tmem), L::kCols);
  if (threadIdx.x == 0) {
    m.abort = 0;
    const uint32_t bars = smem + L::bars;
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars + 8 * (kFull + i), kProdThreads + kProdWarps);
      mbar_init(bars + 8 * (kEmpty + i), 1);
      mbar_init(bars + 8 * (kQFull + i), kProdThreads);
      mbar_init(bars + 8 * (kQEmpty + i), 1);
      mbar_init(bars + 8 * (kSFull + i), 1);
    }
    mbar_init(bars + 8 * kPFull, kSoftWarps * 32);
    mbar_init(bars + 8 * kPvDone, 1);
    mbar_init(bars + 8 * kOFree, kSoftWarps * 32);
    mbar_fence_init();
  }
  pdl_wait();
  const Workspace ws = workspace_of<NR>(a.workspace, gridDim.x);
  if (threadIdx.x == 0) ws.split[blockIdx.x] = Split{-1, 0, 0, 0};
  uint32_t errbits = 0;
  schedule<NR>(a, smem_raw, m, errbits);
  tc::fence_after_sync();
  const uint32_t tmem = m.tmem;
  const Waiter wait{smem_addr(&m.abort), a.wait_limit_ns};
  if (m.count > 0) {
    if (warp < kSoftWarps) soften<FMT, NR>(a, m, smem, tmem, wait, warp, lane, ws);
    else if (warp >= kProdWarp) produce<FMT, NR>(a, m, smem, wait, warp - kProdWarp, lane, errbits);
    else if (lane == 0) issue_mma<NR>(a, m, smem, tmem, wait);
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
  if (warp == kMmaWarp) tc::dealloc(tmem, L::kCols);
}

// ---------------------------------------------------- join of the split query tiles
// Block (n, c): row n of the query tile that CTA c started and others went on
// with.  Four groups of 128 threads take the partials in turn, a float4 per
// thread, and are added in order.
constexpr int kJoinGroups = 4;
constexpr int kJoinThreads = kJoinGroups * 128;
constexpr int kMaxCtas = 1024;

template <int FMT, int NR>
__global__ void __launch_bounds__(kJoinThreads) latent_join_kernel(const LatentAttnArgs a) {
  __shared__ float wt[kMaxCtas];
  __shared__ float red[2][kJoinThreads / 32];
  __shared__ float4 acc_s[kJoinGroups][128];
  pdl_trigger();
  pdl_wait();
  const Workspace ws = workspace_of<NR>(a.workspace, gridDim.y);
  const int c = blockIdx.y, n = blockIdx.x;
  const Split sp = ws.split[c];
  if (sp.s < 0) return;
  const Seq q = load_seq<NR>(a, sp.s);
  const int64_t row = (int64_t)sp.qt * NR + n;
  if (row >= (int64_t)q.ntok * a.num_heads) return;
  const int parts = sp.last - c + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto slot = [&](int i) { return (2 * (int64_t)(c + i) + (i == 0 ? 1 : 0)) * NR + n; };
  // the largest maximum, the weights relative to it, and the whole sum
  float mx = -INFINITY;
  for (int i = tid; i < parts; i += kJoinThreads) mx = fmaxf(mx, ws.ml[slot(i)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  if (lane == 0) red[0][warp] = mx;
  __syncthreads();
  mx = red[0][0];
  for (int w = 1; w < kJoinThreads / 32; ++w) mx = fmaxf(mx, red[0][w]);
  const float m0 = mx == -INFINITY ? 0.0f : mx;
  float sum = 0.0f;
  for (int i = tid; i < parts; i += kJoinThreads) {
    const float2 v = ws.ml[slot(i)];
    const float w = ex2(v.x - m0);
    wt[i] = w;
    sum += w * v.y;
  }
  sum = warp_sum(sum);
  if (lane == 0) red[1][warp] = sum;
  __syncthreads();
  sum = 0.0f;
  for (int w = 0; w < kJoinThreads / 32; ++w) sum += red[1][w];
  const int grp = tid >> 7, d4 = tid & 127;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int i = grp; i < parts; i += kJoinGroups) {
    const float4 v = *reinterpret_cast<const float4*>(ws.o + slot(i) * kRank + d4 * 4);
    const float w = wt[i];
    acc.x = fmaf(w, v.x, acc.x);
    acc.y = fmaf(w, v.y, acc.y);
    acc.z = fmaf(w, v.z, acc.z);
    acc.w = fmaf(w, v.w, acc.w);
  }
  acc_s[grp][d4] = acc;
  __syncthreads();
  if (grp != 0) return;
#pragma unroll
  for (int k = 1; k < kJoinGroups; ++k) {
    const float4 v = acc_s[k][d4];
    acc.x += v.x;
    acc.y += v.y;
    acc.z += v.z;
    acc.w += v.w;
  }
  const float ks = FMT == kBF16 ? 1.0f : __ldg(a.k_scale);
  const float inv = sum == 0.0f ? 0.0f : ks / sum;
  const int64_t t = q.t0 + row / a.num_heads, h = row % a.num_heads;
  st8(a.out + t * a.out_ts + h * a.out_hs + d4 * 8,
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv)));
  if (tid == 0 && a.lse)
    a.lse[t * a.lse_ts + h * a.lse_hs] = sum == 0.0f ? -INFINITY : fmaf(m0, kLn2, logf(sum));
}

// Rows of a query tile: the average rows (tokens x heads) per sequence decide.
inline int tile_rows(int32_t num_tokens, int32_t num_heads, int32_t num_seqs) {
  const int64_t rows = (int64_t)((num_tokens + num_seqs - 1) / num_seqs) * num_heads;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

template <int FMT, int NR>
cudaError_t launch_t(const LatentAttnArgs& a, int ctas, const LaunchCfg& cfg) {
  auto kern = latent_attention_kernel<FMT, NR>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<NR>::bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(ctas);
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = Lay<NR>::bytes;
  lc.stream = cfg.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = cfg.pdl ? 1 : 0;
  e = cudaLaunchKernelEx(&lc, kern, a);
  if (e != cudaSuccess) return e;
  lc.gridDim = dim3(NR, ctas);
  lc.blockDim = dim3(kJoinThreads);
  lc.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&lc, latent_join_kernel<FMT, NR>, a);
}

template <int FMT>
cudaError_t launch_f(const LatentAttnArgs& a, int ctas, const LaunchCfg& cfg) {
  switch (tile_rows(a.num_tokens, a.num_heads, a.num_seqs)) {
    case 16: return launch_t<FMT, 16>(a, ctas, cfg);
    case 32: return launch_t<FMT, 32>(a, ctas, cfg);
    default: return launch_t<FMT, 64>(a, ctas, cfg);
  }
}

}  // namespace

// The largest call within these sizes may use any tile: enough for 64 rows.
int64_t latent_attention_workspace(int32_t, int32_t, int32_t, int num_sms) {
  const int64_t ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
  return ctas * ((int64_t)sizeof(Split) + 2 * 64 * (sizeof(float2) + kRank * sizeof(float)));
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
