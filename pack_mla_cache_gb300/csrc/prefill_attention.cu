// prefill_attention.cu -- attention of packed sequences over keys and values per head
// (include/mla_cache.h: mla_prefill_attention), on the 5th generation tensor cores.
//
// What it computes, per (token, head) row q of 128 + 64 elements and the rows of its
// sequence that the token sees: x_p = scale <q, k_p>, lse = ln sum exp(x_p), out = sum
// exp(x_p - lse) v_p.
//
// Shape of the work.  The query rows of a sequence and key head (token-major, the key
// head's query heads inside) are cut into items of 256 rows, two tiles of 128, its keys
// into tiles of 128; one unit = (item, key tile).  The units of the whole call, in
// (sequence, key head, item, key tile) order, are cut into equal contiguous runs, one per
// CTA (one CTA per SM), so ragged and causal batches load every SM alike.  An item whose
// units fall into several CTAs leaves unnormalised fp32 partial sums in the workspace, which
// a second launch joins in the order of the CTAs (no atomics: equal calls give equal bits).
//
// A unit: S_i = Q_i K^T (two tiles of 128 x 128, k = 192), weights P_i = exp2(S_i - reference)
// written over S_i in tensor memory as 16-bit values, O_i += P_i V (128 x 128).  Tensor memory
// is full: two S and two O of 128 columns.  The two tiles alternate on the tensor core: while
// one tile's weights are computed, the other tile's products run (1280 of 2560 cycles a unit
// at 8192 multiply-adds... per tile).
//
// Shared memory: the two query tiles (96 KB), and a ring of 8 slots of 128 keys x 64 columns
// (128 bytes a row, 128-byte swizzle) through which K (three slots a unit) and V (two) flow by
// TMA, a whole unit ahead of their use.
//
// Roles (20 warps): 8 warps per query tile load the queries, compute weights, two threads a row
// (64 columns each; running maximum, rescaling O only when a maximum has grown by more than
// 2^kGrow) and write the output; one per tile issues the products; one loads K and V; one looks after V rows that
// not every row of an item sees: those behind the sequence are zeroed (they may hold anything),
// those with a NaN or an infinity too, and noted, so that the sums of the rows that see them
// become NaN.
//
// Waits are bounded (wait_limit_ns): one that runs out marks the CTA as given up.  Every role
// leaves at its next wait then, copies and products in flight are waited for (bounded again),
// and MLA_ERRBIT_TIMEOUT is set.
#include <atomic>

#include "mla_device.cuh"
#include "serving.h"
#include "tensor_core.cuh"
#include "tensor_map.h"

namespace mla {
namespace {

constexpr int kSimpleThreads = 256;
constexpr int kM = 128;              // query rows of a tile
constexpr int kItemRows = 2 * kM;
constexpr int kKeys = 128;           // keys of a tile
constexpr int kV = 128;
constexpr int kSlot = kKeys * 128;   // bytes of a ring slot
constexpr int kSlots = 8;
constexpr int kUnitSlots = 5;        // 3 of K, 2 of V
constexpr int kQTile = 3 * kM * 128;
constexpr int kMmaWarp = 16, kLoadWarp = 18;  // and one more, that looks after V
constexpr int kWarps = 20, kThreads = kWarps * 32;
constexpr int kMaxCtas = 1024;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// What beginning another item costs a CTA, in units: the runs are cut as if each item had
// this many more.
constexpr int kSwitch = 1;
constexpr int kMinUnits = 2;  // a CTA takes at least this many

// The reference of a row's weights is the next whole number (log2) above its maximum less
// kTop; a score may pass the reference by kGrow before the sums are rescaled.  fp16 weights:
// up to 2^14, and 2^-25, half their smallest step, is 2^-34 of the row's largest or less.
template <int F>
struct Ref {
  static constexpr float kTop = F == kF16 ? 10.0f : 0.0f;
  static constexpr float kGrow = F == kF16 ? 14.0f : 8.0f;
};

// shared memory
struct Lay {
  static constexpr int q = 0;
  static constexpr int ring = 2 * kQTile;
  static constexpr int red = ring + kSlots * kSlot;  // float [8 pairs of warps][2][32]
  static constexpr int flags = red + 2048;           // uint32 [4 units][4]: keys with bad V rows
  static constexpr int bars = flags + 64;
  // Two of each: of units in turn (K and V), of the query tiles; the weights' by tile and half.
  static constexpr int kKFull = 0, kVFull = 2, kKEmpty = 4, kVEmpty = 6, kRaw = 8, kClean = 10,
                       kQFull = 12, kSFull = 14, kPFull = 16, kOFull = 18, kOFree = 20, kTurn = 22,
                       kBars = 24;
  static constexpr int misc = (bars + kBars * 8 + 15) / 16 * 16;
  static constexpr int bytes = misc + 64;
  static_assert(bytes <= 232448, "shared memory of a CTA");
  // tensor memory columns: S of both tiles (P in their first half), O of both tiles
  static constexpr int kO = 2 * kKeys, kTmem = 512;
};
struct Misc {
  uint32_t tmem;
  uint32_t abort;
  uint8_t left[16];  // a weights' warp that has given up, for its partner
};
static_assert(sizeof(Misc) <= 64, "Misc fits");

// How a tensor map reads row p, columns c.. of key head g: box (x_head * g + c, p, z_head * g).
struct Maps {
  CUtensorMap kn, kp, v;
  int32_t kn_x, kn_z, kp_x, kp_z, v_x, v_z;
};

// What the join needs of a split item; written by each CTA whose run ends inside it.  rows 0:
// none.
struct Split {
  int32_t tok0;        // the sequence's first computed token
  uint32_t row0;       // of the item, among the sequence's rows of a key head
  int32_t head;        // key head
  int16_t rows, parts;
  int32_t first, pad[3];
};
struct Workspace {
  Split* split;  // [ctas]
  float *m, *l;  // [2 ctas][slot_rows]: reference (log2) and sum of the weights
  float* o;      // [2 ctas][32][slot_rows][4]: 4 dims of a row lie together, so that a thread a
                 // row writes whole lines
};
__host__ __device__ inline int slot_rows(int64_t num_tokens, int group) {
  const int64_t rows = num_tokens * group;
  return rows < kItemRows ? (int)((rows + 3) / 4 * 4) : kItemRows;
}
__host__ __device__ inline Workspace workspace_of(uint8_t* p, int ctas, int rows) {
  Workspace w;
  w.split = reinterpret_cast<Split*>(p);
  w.m = reinterpret_cast<float*>(p + (int64_t)ctas * sizeof(Split));
  w.l = w.m + (int64_t)ctas * 2 * rows;
  w.o = w.l + (int64_t)ctas * 2 * rows;
  return w;
}

struct Seq {
  int32_t t0;      // first computed token
  uint32_t rows;   // query rows of a key head
  int32_t nb;      // items of a key head
  int32_t k0, m;   // its key rows that exist
  int64_t base;    // rows that token t0 sees (before clamping)
};
__device__ __forceinline__ Seq load_seq(const PrefillArgs& a, int s, uint32_t& errbits) {
  Seq q;
  const int32_t c0 = __ldg(a.cu_q + s), c1 = __ldg(a.cu_q + s + 1);
  const int32_t k0 = __ldg(a.cu_kv + s), k1 = __ldg(a.cu_kv + s + 1);
  q.t0 = max(c0, 0);
  const int32_t ntok = max(min(c1, a.num_tokens) - q.t0, 0);
  q.rows = (uint32_t)ntok * (uint32_t)a.group;
  q.nb = (int)((q.rows + kItemRows - 1) / kItemRows);
  q.k0 = k0;
  const int64_t n = (int64_t)k1 - k0;
  q.m = k0 < 0 ? 0 : (int)max((int64_t)0, min(n, (int64_t)a.num_kv - k0));
  q.base = n + (a.causal ? (int64_t)q.t0 + 1 - c1 : 0);
  if (ntok > 0 && n > q.m) errbits |= kErrPosOOB;
  return q;
}
// Key rows that the token of a query row sees.
__device__ __forceinline__ int seen_of(const PrefillArgs& a, const Seq& q, uint32_t row) {
  const int64_t n = q.base + (a.causal ? (int64_t)a.by_group(row) : 0);
  return (int)max((int64_t)0, min(n, (int64_t)q.m));
}
// Key tiles of rows of which the last sees `most` (one even when it sees none: they are still
// written).
__device__ __forceinline__ int key_tiles(int most) { return max(1, (most + kKeys - 1) / kKeys); }
__device__ __forceinline__ int item_tiles(const PrefillArgs& a, const Seq& q, int b) {
  return key_tiles(seen_of(a, q, min((uint32_t)(b + 1) * kItemRows, q.rows) - 1));
}

// A CTA's run of units: where it starts, and what finds the CTA of another unit.  An item is
// kSwitch units that stand for beginning it, then its key tiles: a run starts before the
// first of these when kt is negative.
struct Run {
  Seq q;
  int s, head, b, kt, count;
  int64_t begin, each;
  int extra;
};

// Walks the run item by item; every role has its own copy.
struct Walk {
  Seq q;
  int s, head, b, left;
  bool more;
  // the present item
  int kb, ke;              // this CTA's key tiles of it
  int nkt[2], tiles;       // key tiles of the query tiles (0: the tile has no rows), and of both
  int least, most;         // rows seen by its first and last row
  uint32_t row0;
  int rows;
  __device__ __forceinline__ void start(const Run& r) {
    q = r.q;
    s = r.s;
    head = r.head;
    b = r.b;
    left = r.count + min(r.kt, 0);
    kb = max(r.kt, 0);
    more = false;
  }
  __device__ __forceinline__ bool next(const PrefillArgs& a) {
    if (left <= 0) return false;
    if (more) {
      kb = 0;
      if (++b >= q.nb) {
        b = 0;
        if (++head >= a.kv_heads) {
          head = 0;
          uint32_t ignored = 0;
          do q = load_seq(a, ++s, ignored);
          while (q.nb == 0 && s + 1 < a.num_seqs);
        }
      }
      left -= kSwitch;
      if (left <= 0) return false;
    }
    more = true;
    row0 = (uint32_t)b * kItemRows;
    rows = (int)min((uint32_t)kItemRows, q.rows - row0);
    least = seen_of(a, q, row0);
    most = seen_of(a, q, row0 + rows - 1);
    tiles = key_tiles(most);
    nkt[0] = rows > kM ? key_tiles(seen_of(a, q, row0 + kM - 1)) : tiles;
    nkt[1] = rows > kM ? tiles : 0;
    ke = min(tiles, kb + left);
    left -= ke - kb;
    return true;
  }
  // Key tiles of query tile i in this run end here (at kb or before: none).
  __device__ __forceinline__ int end(int i) const { return min(ke, nkt[i]); }
  // The first key tile that not every row sees whole.
  __device__ __forceinline__ int ragged() const { return least / kKeys; }
  // Units of the item in this run with V rows to be looked after.
  __device__ __forceinline__ int cleaned() const { return max(0, ke - max(kb, ragged())); }
};

__device__ __forceinline__ uint32_t slot_of(uint32_t unit, int chunk) {
  return (unit * kUnitSlots + chunk) & (kSlots - 1);
}

__device__ __noinline__ int cta_of(int64_t u, int64_t each, int extra) {
  const int64_t longer = (each + 1) * extra;
  return (int)(u < longer ? u / (each + 1) : extra + (u - longer) / each);
}

// ------------------------------------------------------------------ the roles
// K and V by TMA, and where the run ends inside an item, what the join needs.  Returns the
// copies begun, in K and V of a unit, and the units whose V is looked after.  V of such a unit
// completes on a barrier of its own (two in turn), which that warp waits for: it does not follow
// the ring through the units between, and a barrier's parity tells one phase from the next
// only.
//
// The ring holds 8/5 units, so a unit's slots are those of K's last third and V of the unit two
// before, and of the first two thirds of K of the unit before.
__device__ __forceinline__ uint32_t load_role(const PrefillArgs& a, const Maps& maps, const Run& run,
                                              uint32_t smem, const Waiter& wait, int lane,
                                              const Workspace& ws, uint32_t& cleaned) {
  const uint32_t bars = smem + Lay::bars;
  // rows that one item reads leave L2 first
  const uint64_t policy =
      tc::l2_policy((int64_t)a.num_tokens * a.group <= (int64_t)kItemRows * a.num_seqs);
  Walk w;
  w.start(run);
  uint32_t g = 0;
  cleaned = 0;
  while (w.next(a)) {
    const int h = w.head;
#pragma unroll 1
    for (int kt = w.kb; kt < w.ke; ++kt, ++g) {
      const int row = w.q.k0 + kt * kKeys;
      const bool clean = kt >= w.ragged();
      auto dst = [&](int c) { return smem + Lay::ring + slot_of(g, c) * kSlot; };
      auto freed = [&](int bar, uint32_t unit) {  // K (V) of that unit is read
        return __all_sync(0xFFFFFFFFu, wait(bars + 8 * (bar + (unit & 1)), (unit >> 1) & 1));
      };
      const uint32_t kf = bars + 8 * (Lay::kKFull + (g & 1));
      if (lane == 0) {
        mbar_arrive_expect_tx(kf, 3 * kSlot);
        tc::tma_load3(dst(0), &maps.kn, h * maps.kn_x, row, h * maps.kn_z, kf, policy);
      }
      __syncwarp();
      if (g >= 2 && !freed(Lay::kVEmpty, g - 2)) return 2 * g;
      if (lane == 0) {
        tc::tma_load3(dst(1), &maps.kn, h * maps.kn_x + 64, row, h * maps.kn_z, kf, policy);
        tc::tma_load3(dst(2), &maps.kp, h * maps.kp_x, row, h * maps.kp_z, kf, policy);
      }
      __syncwarp();
      if (g >= 1 && !freed(Lay::kKEmpty, g - 1)) return 2 * g + 1;
      if (lane == 0) {
        uint32_t vf = bars + 8 * (Lay::kVFull + (g & 1));
        if (clean) {
          mbar_arrive(vf);
          vf = bars + 8 * (Lay::kRaw + (cleaned & 1));
        }
        mbar_arrive_expect_tx(vf, 2 * kSlot);
#pragma unroll
        for (int k = 0; k < 4; ++k)  // 64 keys x 64 columns each
          tc::tma_load3(dst(3 + (k >> 1)) + (k & 1) * (kSlot / 2), &maps.v, h * maps.v_x + 64 * (k & 1),
                        row + 64 * (k >> 1), h * maps.v_z, vf, policy);
      }
      __syncwarp();
      cleaned += clean;
    }
    if (w.ke < w.tiles && lane == 0) {  // the run's last item
      const int64_t u0 = run.begin + run.count - w.ke;  // the unit of its key tile 0
      const int c0 = cta_of(u0, run.each, run.extra);
      const int c1 = cta_of(u0 + w.tiles - 1, run.each, run.extra);
      ws.split[blockIdx.x] = Split{w.q.t0, w.row0, w.head, (int16_t)w.rows, (int16_t)(c1 - c0 + 1), c0, {}};
    }
  }
  return 2 * g;
}

// The V rows that not every row of an item sees.  (Units looked after use two barriers in
// turn: this role may be one unit ahead of the last look at its barrier, but not two, as V of
// the next but one waits for the scores of the next.)
template <int F>
__device__ __forceinline__ void clean_role(const PrefillArgs& a, const Run& run, uint32_t smem,
                                           const Waiter& wait, int lane) {
  const uint32_t bars = smem + Lay::bars;
  Walk w;
  w.start(run);
  uint32_t g = 0, cleaned = 0;
  const int col = lane & 7;
  while (w.next(a)) {
#pragma unroll 1
    for (int kt = max(w.kb, w.ragged()); kt < w.ke; ++kt) {
      const uint32_t u = g + kt - w.kb;
      if (!__all_sync(0xFFFFFFFFu, wait(bars + 8 * (Lay::kRaw + (cleaned & 1)), (cleaned >> 1) & 1)))
        return;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {  // 32 keys
        const int p0 = kt * kKeys + q * 32;
        uint32_t bad = 0;
        if (p0 + 32 > w.least) {
          // 64 keys to a slot: two runs of 64 columns
          const uint32_t v0 = smem + Lay::ring + slot_of(u, 3 + (q >> 1)) * kSlot + (q & 1) * 4096;
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const int key = 4 * n + (lane >> 3), p = p0 + key;
            const uint32_t at = v0 + key * 128 + col * 16;  // every column of the row, in any order
            const bool sp = any_special<F>(lds16(at)) | any_special<F>(lds16(at + kSlot / 2));
            const uint32_t votes = __ballot_sync(0xFFFFFFFFu, sp && p >= w.least && p < w.most);
            if (p >= w.most || votes & (0xFFu << (lane & 24))) {
              sts16(at, make_uint4(0, 0, 0, 0));
              sts16(at + kSlot / 2, make_uint4(0, 0, 0, 0));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (votes & (0xFFu << (8 * k))) bad |= 1u << (4 * n + k);
          }
        }
        if (lane == 0) sts_u32(smem + Lay::flags + (u & 3) * 16 + q * 4, bad);
      }
      tc::fence_smem_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (Lay::kClean + (cleaned & 1)));
      ++cleaned;
    }
    g += w.ke - w.kb;
  }
}

template <int F>
__device__ __forceinline__ void issue_scores(uint32_t smem, uint32_t tmem, bool one, int tile,
                                             uint32_t unit, uint32_t negate) {
  const uint32_t id = negate | tc::instr_desc(kM, kKeys, false, F == kBF16, F == kBF16);
  const uint32_t i = __shfl_sync(0xFFFFFFFFu, tile, 0), g = __shfl_sync(0xFFFFFFFFu, unit, 0);
  const uint64_t qa = tc::smem_desc(smem + Lay::q + i * kQTile, 0, 1024);
  const uint32_t d = tmem + i * kKeys;
#pragma unroll
  for (int c = 0; c < 3; ++c) {
    const uint64_t kb = tc::smem_desc(smem + Lay::ring + slot_of(g, c) * kSlot, 0, 1024);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      tc::mma_16bit(one, d, qa + (c * kM * 128 >> 4) + 2 * k, kb + 2 * k, id, c + k > 0);
  }
}
// V MN-major (two runs of 64 columns), half of the keys a slot.
template <int F>
__device__ __forceinline__ void issue_outputs(uint32_t smem, uint32_t tmem, bool one, int tile,
                                              uint32_t unit, bool first) {
  constexpr uint32_t kId = tc::instr_desc(kM, kV, false, F == kBF16, F == kBF16, true);
  const uint32_t i = __shfl_sync(0xFFFFFFFFu, tile, 0), g = __shfl_sync(0xFFFFFFFFu, unit, 0);
  const uint32_t p = tmem + i * kKeys, d = tmem + Lay::kO + i * kV;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint64_t vb = tc::smem_desc(smem + Lay::ring + slot_of(g, 3 + h) * kSlot, kSlot / 2, 1024);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      tc::mma_16bit_ta(one, d, p + h * 32 + 8 * k, vb + k * (2048 >> 4), kId, h + k > 0 || !first);
  }
}

// A warp issues the products of one query tile, whose chain is serial: scores of a unit behind
// the outputs of the one before, over whose weights they go.  The two warps take turns, so that
// a tile's weights are computed while the other's products run.  (One warp for both took 4900
// cycles a unit, most of them its own instructions between the products; two without turns 4600,
// both tiles waiting for the tensor core and for their weights at the same times.)  K and V of a
// unit are free when both warps have said so; a warp whose tile has no part in a unit says it
// when they have come, so that it does not run ahead.
template <int F>
__device__ __forceinline__ void mma_role(const PrefillArgs& a, const Run& run, uint32_t smem,
                                         uint32_t tmem, const Waiter& waiter, int tile, int lane) {
  const uint32_t bars = smem + Lay::bars;
  // Looks at barriers without letting itself be suspended: waking takes long.
  auto wait = [&](int bar, uint32_t phase) {
    for (int spin = 0; spin < 64; ++spin)
      if (__any_sync(0xFFFFFFFFu, mbar_test(bars + 8 * bar, phase & 1))) return true;
    return (bool)__all_sync(0xFFFFFFFFu, waiter(bars + 8 * bar, phase & 1));
  };
  const bool one = tc::elect();
  const uint32_t negate = a.softmax_scale < 0.0f ? 1u << 13 : 0u;  // of the scores, by the tensor core
  Walk w;
  w.start(run);
  uint32_t g = 0, done = 0, opened = 0, cleaned = 0;
#pragma unroll 1
  while (w.next(a)) {
    const int e = w.end(tile), from = max(w.kb, w.ragged());
    if (e > w.kb) {
      if (!wait(Lay::kQFull + tile, opened)) return;
      tc::fence_smem_async();  // the queries came by ordinary copies
    }
#pragma unroll 1
    for (int kt = w.kb; kt < w.ke; ++kt, ++g) {
      const bool act = kt < e;
      // the scores of the item's first unit; the others' follow the outputs before, below
      if (kt == w.kb) {
        if (!wait(Lay::kKFull + (g & 1), g >> 1)) return;
        if (act) {
          tc::fence_after_sync();
          issue_scores<F>(smem, tmem, one, tile, g, negate);
          tc::commit(one, bars + 8 * (Lay::kSFull + tile));
        }
        tc::commit(one, bars + 8 * (Lay::kKEmpty + (g & 1)));
      }
      // All that is usually there is asked for before the weights, which are not.
      const uint32_t n = cleaned + kt - from;
      if (!wait(Lay::kVFull + (g & 1), g >> 1)) return;
      if (act) {
        if (kt >= from && !wait(Lay::kClean + (n & 1), n >> 1)) return;
        // the sums of the item before are read
        if (kt == w.kb && opened++ > 0 && !wait(Lay::kOFree + tile, opened)) return;
      }
      if (tile + g > 0 && !wait(Lay::kTurn + tile, tile ? g : g - 1)) return;
      if (act) {
        if (!wait(Lay::kPFull + tile, done++)) return;
        tc::fence_after_sync();
        issue_outputs<F>(smem, tmem, one, tile, g, kt == w.kb);
        if (kt + 1 == e) tc::commit(one, bars + 8 * (Lay::kOFull + tile));
      }
      tc::commit(one, bars + 8 * (Lay::kVEmpty + (g & 1)));
      if (kt + 1 < w.ke && !wait(Lay::kKFull + ((g + 1) & 1), (g + 1) >> 1)) return;
      if (kt + 1 < e) {
        tc::fence_after_sync();
        issue_scores<F>(smem, tmem, one, tile, g + 1, negate);
        tc::commit(one, bars + 8 * (Lay::kSFull + tile));
      }
      if (kt + 1 < w.ke) tc::commit(one, bars + 8 * (Lay::kKEmpty + ((g + 1) & 1)));
      if (lane == 0) mbar_arrive(bars + 8 * (Lay::kTurn + (tile ^ 1)));
      __syncwarp();
    }
    cleaned += w.cleaned();
  }
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <int F>
__device__ __forceinline__ uint32_t pack16x2(float lo, float hi) {
  if constexpr (F == kF16) return pack_f16x2(lo, hi);
  else return pack_bf16x2(lo, hi);
}
// A barrier of the two warps that share 32 rows of a tile, and whether x holds in any of their
// threads.
__device__ __forceinline__ void pair_sync(int pair) {
  asm volatile("bar.sync %0, 64;" ::"r"(1 + pair) : "memory");
}
__device__ __forceinline__ bool pair_any(int pair, bool x) {
  uint32_t any;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 q, %2, 0;\n"
      "  barrier.cta.red.or.pred p, %1, 64, q; selp.u32 %0, 1, 0, p; }"
      : "=r"(any)
      : "r"(1 + pair), "r"(x ? 1u : 0u)
      : "memory");
  return any != 0;
}

// The queries of a tile by asynchronous copies, 16 rows by each of its eight warps.
__device__ __forceinline__ void load_queries(const PrefillArgs& a, const Walk& w, uint32_t smem,
                                             int tile, int warp8, int lane) {
  const int col = lane & 7;
#pragma unroll 1
  for (int r = warp8 * 16 + (lane >> 3); r < warp8 * 16 + 16; r += 4) {
    const uint32_t row = w.row0 + tile * kM + r;
    const bool ok = row < w.q.rows;
    const uint32_t dt = ok ? a.by_group(row) : 0;
    const int64_t t = ok ? w.q.t0 + (int)dt : 0;
    const int64_t h = ok ? (int64_t)w.head * a.group + (int)(row - dt * a.group) : 0;
    const uint8_t* nope = a.q_nope + t * a.qn_ts + h * a.qn_hs + col * 16;
    const uint8_t* pe = a.q_pe + t * a.qp_ts + h * a.qp_hs + col * 16;
    const uint32_t d = smem + Lay::q + tile * kQTile + r * 128 + ((col ^ (r & 7)) << 4);
    tc::cp_async16(d, nope, ok);
    tc::cp_async16(d + kM * 128, nope + 128, ok);
    tc::cp_async16(d + 2 * kM * 128, pe, ok);
  }
  tc::cp_async_arrive(smem + Lay::bars + 8 * (Lay::kQFull + tile));
}

// Weights and output of one query tile: a thread has a row's keys 64 half .. of a key tile (and
// dims 64 half .. of the output), its partner in another warp the others.  One warp for 32 whole
// rows took 2300 cycles a tile, mostly waiting for its own instructions.  The queries' place is
// free when the item's last scores have come: those of the next item are asked for before the
// output of this one is written.
template <int F>
__device__ __forceinline__ void softmax_role(const PrefillArgs& a, const Run& run, uint32_t smem,
                                             uint32_t tmem, const Waiter& waiter, int warp, int lane,
                                             const Workspace& ws, int srows, Misc& misc) {
  using R = Ref<F>;
  constexpr int kC = kKeys / 2;
  const int tile = warp >> 3, half = (warp >> 2) & 1, w4 = warp & 3, pair = tile * 4 + w4;
  const uint32_t bars = smem + Lay::bars;
  auto wait = [&](int bar, uint32_t phase) {
    return __all_sync(0xFFFFFFFFu, waiter(bars + 8 * bar, phase & 1));
  };
  const uint32_t s_at = tmem + tile * kKeys + ((uint32_t)(w4 * 32) << 16);
  const uint32_t o_at = tmem + Lay::kO + tile * kV + half * 64 + ((uint32_t)(w4 * 32) << 16);
  const float c = fabsf(a.softmax_scale) * kLog2e;  // (the scores have its sign)
  const int r = w4 * 32 + lane;
  const uint32_t red = smem + Lay::red + (pair * 2 + half) * 128 + lane * 4;  // partner: ^ 128
  volatile uint8_t* left = misc.left + pair * 2;
  Walk w;
  w.start(run);
  uint32_t n = 0, g = 0, cleaned = 0, items = 0;
  bool more = w.next(a);
  if (more && w.end(tile) > w.kb) load_queries(a, w, smem, tile, warp & 7, lane);
#pragma unroll 1
  while (more) {
    const int e = w.end(tile), mine = w.rows - tile * kM;  // rows of this tile (or less than 0)
    const bool live = w4 * 32 < mine;  // this warp has rows
    const uint32_t row = w.row0 + tile * kM + r;
    const bool ok = r < mine;
    const int seen = ok ? seen_of(a, w.q, row) - half * kC : 0;
    const int from = max(w.kb, w.ragged());
    float mu = -INFINITY, l = 0.0f;
#pragma unroll 1
    for (int kt = w.kb; kt < e; ++kt, ++n) {
      bool fine = wait(Lay::kSFull + tile, n);
      tc::fence_after_sync();
      if (live) {
        float x[kC];
        tc::ld_32x64(s_at + half * kC, reinterpret_cast<uint32_t*>(x));
        float cs = c;
        if (__builtin_expect(kt >= from, 0)) {
          const uint32_t nc = cleaned + kt - from;
          fine &= wait(Lay::kClean + (nc & 1), nc >> 1);
          const int lim = seen - kt * kKeys;
          const uint32_t at = smem + Lay::flags + ((g + kt - w.kb) & 3) * 16 + half * 8;
          bool bad = false;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int below = min(max(lim - 32 * k, 0), 32);
            bad |= (lds_u32(at + 4 * k) & (below == 32 ? 0xFFFFFFFFu : (1u << below) - 1)) != 0;
          }
          if (bad) l = NAN;
#pragma unroll
          for (int j = 0; j < kC; ++j) x[j] = j < lim ? x[j] * c : -INFINITY;
          cs = 1.0f;
        }
        float t[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int j = 4; j < kC; j += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            t[k] = j + 4 + k < kC ? fmaxf(t[k], fmaxf(x[j + k], x[j + 4 + k])) : fmaxf(t[k], x[j + k]);
        float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * cs;
        // (behind this barrier both warps have their scores: P goes over them)
        if (__builtin_expect(pair_any(pair, !fine || top > mu + R::kGrow), 0)) {
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(red), "f"(top) : "memory");
          if (lane == 0) left[half] = !fine;
          pair_sync(pair);
          if (left[0] | left[1]) return;  // both
          top = fmaxf(top, __uint_as_float(lds_u32(red ^ 128)));
          const float mn = fmaxf(mu, ceilf(top) - R::kTop);
          const float f = mu == -INFINITY ? 0.0f : ex2(mu - mn);
          l = l == 0.0f ? 0.0f : l * f;  // (a NaN stays)
          mu = mn;
          if (kt > w.kb) {  // the outputs before are done (these scores came behind them)
#pragma unroll 1
            for (int k = 0; k < 64; k += 16) {
              uint32_t y[16];
              tc::ld_32x16(o_at + k, y);
#pragma unroll
              for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * f);
              tc::st_32x16(o_at + k, y);
            }
            tc::wait_st();
          }
          pair_sync(pair);  // the maxima are read
        }
        const float m0 = mu == -INFINITY ? 0.0f : -mu;
        const uint64_t c2 = f2(cs, cs), m2 = f2(m0, m0);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int q = 0; q < 2; ++q) {  // (16 words at a time: more do not fit the registers)
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 y = unf2(fma2(f2(x[32 * q + 2 * j], x[32 * q + 2 * j + 1]), c2, m2));
            const float p0 = ex2(y.x), p1 = ex2(y.y);
            sum[j & 1] = add2(sum[j & 1], f2(p0, p1));
            pk[j] = pack16x2<F>(p0, p1);
          }
          tc::st_32x16(s_at + half * 32 + q * 16, pk);
        }
        const float2 s2 = unf2(add2(sum[0], sum[1]));
        l += s2.x + s2.y;
        tc::wait_st();
      } else if (!fine) {
        return;
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (Lay::kPFull + tile));
    }
    // ---- the end of this CTA's part of the item
    const Walk past = w;
    g += w.ke - w.kb;
    cleaned += w.cleaned();
    more = w.next(a);
    if (more && w.end(tile) > w.kb) load_queries(a, w, smem, tile, warp & 7, lane);
    const bool any = e > past.kb;
    bool fine = true;
    if (any) {
      fine = wait(Lay::kOFull + tile, items++);
      tc::fence_after_sync();
    }
    if (live) {
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(red), "f"(l) : "memory");
      if (lane == 0) left[half] = !fine;
      pair_sync(pair);
      if (left[0] | left[1]) return;  // both
      l += __uint_as_float(lds_u32(red ^ 128));
      const bool whole = past.kb == 0 && past.ke == past.tiles;
      const int64_t slot = 2 * (int64_t)blockIdx.x + (past.kb == 0 ? 1 : 0);
      const int64_t at = slot * srows + tile * kM + r;
      float* part = ws.o + slot * srows * kV + (int64_t)half * 64 * srows + (tile * kM + r) * 4;
      const uint32_t dt = a.by_group(row);
      const int64_t t = past.q.t0 + (int)dt;
      const int64_t h = (int64_t)past.head * a.group + (int)(row - dt * a.group);
      if (ok && half == 0) {
        if (!whole) {
          ws.m[at] = mu;
          ws.l[at] = l;
        } else if (a.lse) {
          a.lse[t * a.lse_ts + h * a.lse_hs] = l == 0.0f ? -INFINITY : (mu + __log2f(l)) * kLn2;
        }
      }
      const float inv = l == 0.0f ? 0.0f : __fdividef(1.0f, l);
      uint8_t* out = a.out + t * a.out_ts + h * a.out_hs + half * 128;
      if (any) {
#pragma unroll 1
        for (int k = 0; k < 64; k += 32) {
          uint32_t y[32];
          tc::ld_32x32(o_at + k, y);
          if (!ok) continue;
          if (whole) {
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              uint32_t z[4];
#pragma unroll
              for (int m = 0; m < 4; ++m)
                z[m] = pack16x2<F>(__uint_as_float(y[j + 2 * m]) * inv,
                                   __uint_as_float(y[j + 2 * m + 1]) * inv);
              st16(out + (k + j) * 2, make_uint4(z[0], z[1], z[2], z[3]));
            }
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              st16(part + (int64_t)(k + j) * srows, make_uint4(y[j], y[j + 1], y[j + 2], y[j + 3]));
          }
        }
      }
    } else if (!fine) {
      return;
    }
    if (any) {
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (Lay::kOFree + tile));
    }
  }
}

// ------------------------------------------------------------------ scheduling
__device__ __forceinline__ int64_t scan64(int64_t v, int lane) {  // inclusive, over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
// This CTA's run, by the whole CTA; the scratch is the (still unused) ring.
__device__ __noinline__ void schedule(const PrefillArgs& a, uint8_t* scratch, Run& r,
                                      uint32_t& errbits) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t* pre = reinterpret_cast<int64_t*>(scratch);  // [num_seqs]
  int64_t* part = pre + a.num_seqs;                    // [kWarps]
  int64_t* at = part + kWarps;                         // sequence, unit in it, item, key tile
  for (int s = warp; s < a.num_seqs; s += kWarps) {
    const Seq q = load_seq(a, s, errbits);
    int64_t u = 0;
    for (int b = lane; b < q.nb; b += 32) u += kSwitch + item_tiles(a, q, b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
    if (lane == 0) pre[s] = u * a.kv_heads;
  }
  __syncthreads();
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
  const int64_t ctas = max((int64_t)1, min((int64_t)gridDim.x, total / kMinUnits));
  r.each = total / ctas;
  r.extra = (int)(total - r.each * ctas);
  r.begin = r.each * blockIdx.x + min((int)blockIdx.x, r.extra);
  r.count = blockIdx.x < ctas ? (int)r.each + ((int)blockIdx.x < r.extra ? 1 : 0) : 0;
  r.kt = 0;
  if (r.count > 0)
    for (int s = s0; s < s1; ++s) {
      const int64_t u = pre[s];
      if (before <= r.begin && r.begin < before + u) {
        at[0] = s;
        at[1] = r.begin - before;
        at[2] = u;
      }
      before += u;
    }
  __syncthreads();
  if (r.count > 0) {
    uint32_t ignored = 0;
    r.s = (int)at[0];
    r.q = load_seq(a, r.s, ignored);
    const int64_t per = at[2] / a.kv_heads;
    r.head = (int)(at[1] / per);
    if (warp == 0) {
      const int64_t off = at[1] - r.head * per;
      int64_t base = 0;
      for (int b0 = 0; b0 < r.q.nb; b0 += 32) {
        const int64_t u = b0 + lane < r.q.nb ? kSwitch + item_tiles(a, r.q, b0 + lane) : 0;
        const int64_t in = scan64(u, lane);
        const uint32_t hit = __ballot_sync(0xFFFFFFFFu, off < base + in);
        if (hit) {
          if (lane == __ffs(hit) - 1) {
            at[3] = b0 + lane;
            at[4] = off - (base + in - u);
          }
          break;
        }
        base += __shfl_sync(0xFFFFFFFFu, in, 31);
      }
    }
  }
  __syncthreads();
  if (r.count > 0) {
    r.b = (int)at[3];
    r.kt = (int)at[4] - kSwitch;
  }
  tc::fence_smem_async();  // the scratch is read; copies may write there now
  __syncthreads();
}

// After giving up: waits, bounded again, for the copies into shared memory, and a
// millisecond for matrix products in flight (they end by themselves within microseconds).
__device__ __noinline__ void settle(uint32_t smem, uint32_t issued, uint32_t cleaned, uint64_t limit) {
  const uint64_t since = global_ns();
  for (uint32_t i = cleaned > 2 ? cleaned - 2 : 0; i < cleaned; ++i)
    while (!mbar_try_wait(smem + Lay::bars + 8 * (Lay::kRaw + (i & 1)), (i >> 1) & 1) &&
           global_ns() - since <= limit) {
    }
  for (uint32_t i = issued > 4 ? issued - 4 : 0; i < issued; ++i)
    while (!mbar_try_wait(smem + Lay::bars + 8 * ((i & 1 ? Lay::kVFull : Lay::kKFull) + ((i >> 1) & 1)),
                          (i >> 2) & 1) &&
           global_ns() - since <= limit) {
    }
  while (global_ns() - since <= 1000000) {
  }
}

template <int F>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_attention_kernel(const PrefillArgs a, const __grid_constant__ Maps maps) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t smem = smem_addr(smem_raw);
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  Misc& m = *reinterpret_cast<Misc*>(smem_raw + Lay::misc);
  pdl_trigger();
  if (threadIdx.x == 0) {
    m.abort = 0;
    const uint32_t bars = smem + Lay::bars;
    for (int i = 0; i < 2; ++i) {
      auto stall = [&](int n) { return blockIdx.x == 0 && a.stall_stage == n ? 1 : 0; };
      mbar_init(bars + 8 * (Lay::kKFull + i), 1 + stall(i + 1));  // (one arrival too many)
      mbar_init(bars + 8 * (Lay::kVFull + i), 1 + stall(i + 3));
      mbar_init(bars + 8 * (Lay::kKEmpty + i), 2);
      mbar_init(bars + 8 * (Lay::kVEmpty + i), 2);
      mbar_init(bars + 8 * (Lay::kTurn + i), 1);
      mbar_init(bars + 8 * (Lay::kRaw + i), 1);
      mbar_init(bars + 8 * (Lay::kClean + i), 1);
      mbar_init(bars + 8 * (Lay::kQFull + i), 8 * 32);
      mbar_init(bars + 8 * (Lay::kSFull + i), 1);
      mbar_init(bars + 8 * (Lay::kPFull + i), 8);
      mbar_init(bars + 8 * (Lay::kOFull + i), 1);
      mbar_init(bars + 8 * (Lay::kOFree + i), 8);
    }
    mbar_fence_init();
  }
  const Waiter wait{smem_addr(&m.abort), a.wait_limit_ns};
  pdl_wait();
  if (warp == kMmaWarp) tc::alloc(smem_addr(&m.tmem), Lay::kTmem);
  const int srows = slot_rows(a.num_tokens, a.group);
  const Workspace ws = workspace_of(a.workspace, gridDim.x, srows);
  if (threadIdx.x == 0) ws.split[blockIdx.x] = Split{};
  uint32_t errbits = 0;
  Run run;
  schedule(a, smem_raw + Lay::ring, run, errbits);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, m.tmem, 0);
  uint32_t issued = 0, cleaned = 0;
  if (run.count > 0) {
    if (warp < kMmaWarp) {
      softmax_role<F>(a, run, smem, tmem, wait, warp, lane, ws, srows, m);
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp < kLoadWarp) {
      mma_role<F>(a, run, smem, tmem, wait, warp - kMmaWarp, lane);
    } else if (warp == kLoadWarp) {
      issued = load_role(a, maps, run, smem, wait, lane, ws, cleaned);
    } else {
      clean_role<F>(a, run, smem, wait, lane);
    }
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
    if (warp == kLoadWarp) settle(smem, issued, cleaned, a.wait_limit_ns);
    __syncthreads();
  }
  if (warp == kMmaWarp) tc::dealloc(tmem, Lay::kTmem);
}

// -------------------------------------------------------- join of the split items
// Block (x, c) looks at what CTA c left.  An item of `parts` CTAs is dealt to the warps of the
// blocks of all of them but the last: 8 rows x 16 dims a warp, a lane four dims of a row.
constexpr int kJoinWarps = 8, kJoinBlocks = 8;

template <int F>
__global__ void __launch_bounds__(kJoinWarps * 32) prefill_join_kernel(const PrefillArgs a) {
  pdl_trigger();
  pdl_wait();
  const int srows = slot_rows(a.num_tokens, a.group);
  const Workspace ws = workspace_of(a.workspace, gridDim.y, srows);
  const Split sp = ws.split[blockIdx.y];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stride = (sp.parts - 1) * kJoinBlocks * kJoinWarps;
  for (int n = (((int)blockIdx.y - sp.first) * kJoinBlocks + (int)blockIdx.x) * kJoinWarps + warp;
       n < (sp.rows + 7) / 8 * 8; n += stride) {
    const int r = (n >> 3) * 8 + (lane & 7), quad = (n & 7) * 4 + (lane >> 3);
    if (r >= sp.rows) continue;
    float4 acc = make_float4(0, 0, 0, 0);
    float sum = 0.0f, top = -INFINITY;
    // the first partial lies in the odd slot of the first CTA, the others in the even ones behind
#pragma unroll 1
    for (int i = 0; i < sp.parts; i += 4) {
      float4 v[4];
      float lv[4], mv[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t slot = 2 * (int64_t)(sp.first + i + k) + (i + k == 0 ? 1 : 0);
        lv[k] = 0.0f;
        mv[k] = -INFINITY;
        v[k] = make_float4(0, 0, 0, 0);
        if (i + k < sp.parts) {
          lv[k] = ws.l[slot * srows + r];
          mv[k] = ws.m[slot * srows + r];
          v[k] = __ldcs(reinterpret_cast<const float4*>(ws.o + slot * srows * kV) + quad * srows + r);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (lv[k] == 0.0f) continue;  // nothing seen there (and perhaps nothing written)
        const float m = fmaxf(top, mv[k]), m0 = m == -INFINITY ? 0.0f : m;
        const float f = ex2(top - m0), w = ex2(mv[k] - m0);
        acc.x = fmaf(acc.x, f, w * v[k].x);
        acc.y = fmaf(acc.y, f, w * v[k].y);
        acc.z = fmaf(acc.z, f, w * v[k].z);
        acc.w = fmaf(acc.w, f, w * v[k].w);
        sum = fmaf(sum, f, w * lv[k]);
        top = m;
      }
    }
    const uint32_t row = sp.row0 + r, dt = a.by_group(row);
    const int64_t t = sp.tok0 + (int)dt, h = (int64_t)sp.head * a.group + (int)(row - dt * a.group);
    const float inv = sum == 0.0f ? 0.0f : __fdividef(1.0f, sum);
    st8(a.out + t * a.out_ts + h * a.out_hs + quad * 8,
        make_uint2(pack16x2<F>(acc.x * inv, acc.y * inv), pack16x2<F>(acc.z * inv, acc.w * inv)));
    if (quad == 0 && a.lse)
      a.lse[t * a.lse_ts + h * a.lse_hs] = sum == 0.0f ? -INFINITY : (top + __log2f(sum)) * kLn2;
  }
}

// ------------------------------------------------------------------ launches
// Rows of keys (or values) of all heads as a tensor map with boxes of 64 columns and
// `box_rows` rows.  Heads inside a row are columns of it, so that any head stride does; otherwise (heads
// apart) the third dimension.  `base` stands in for arrays without rows.
bool make_map(CUtensorMap* map, const void* base, int fmt, int width, int64_t hs, int heads, int64_t ts,
              int64_t rows, int box_rows, int32_t* x_head, int32_t* z_head) {
  const TensorMapEncode encode = tensor_map_encode();
  if (!encode) return false;
  const int es = is16(fmt) ? 2 : 1;
  *x_head = *z_head = 0;
  const int64_t flat = (heads - 1) * hs + (int64_t)width * es;
  cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)rows, 1};
  cuuint64_t strides[2] = {(cuuint64_t)ts, (cuuint64_t)ts};
  if (rows <= 1) strides[0] = strides[1] = (cuuint64_t)((flat + 15) / 16 * 16);
  if (heads > 1 && hs > 0) {
    if (rows <= 1 || flat <= ts) {
      dims[0] = (cuuint64_t)(flat / es);
      *x_head = (int32_t)(hs / es);
    } else {
      dims[2] = (cuuint64_t)heads;
      strides[1] = (cuuint64_t)hs;
      *z_head = 1;
    }
  }
  if (dims[0] > INT32_MAX) return false;
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1}, unit[3] = {1, 1, 1};
  const CUtensorMapDataType type =
      fmt == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return encode(map, type, 3, const_cast<void*>(base), dims, strides, box, unit,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int F>
cudaError_t launch_tc(const PrefillArgs& a, int ctas, const LaunchCfg& cfg) {
  Maps maps = {};
  const bool none = a.num_kv == 0;
  const int64_t rows = none ? 1 : a.num_kv;
  const int heads = none ? 1 : a.kv_heads;
  if (!make_map(&maps.kn, none ? a.q_nope : a.k_nope, F, 128, a.kn_hs, heads, a.kn_ts, rows, kKeys,
                &maps.kn_x, &maps.kn_z) ||
      !make_map(&maps.kp, none ? a.q_nope : a.k_pe, F, 64, a.kp_hs, heads, a.kp_ts, rows, kKeys,
                &maps.kp_x, &maps.kp_z) ||
      !make_map(&maps.v, none ? a.q_nope : a.v, F, 128, a.v_hs, heads, a.v_ts, rows, kKeys / 2,
                &maps.v_x, &maps.v_z))
    return cudaErrorInvalidValue;
  auto kern = prefill_attention_kernel<F>;
  // the attribute stays with the device's context: set on a device's first call
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(set.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::bytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) set.fetch_or(uint64_t(1) << dev);
  }
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(ctas);
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = Lay::bytes;
  lc.stream = cfg.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = cfg.pdl ? 1 : 0;
  e = cudaLaunchKernelEx(&lc, kern, a, maps);
  if (e != cudaSuccess) return e;
  lc.gridDim = dim3(kJoinBlocks, ctas);
  lc.blockDim = dim3(kJoinWarps * 32);
  lc.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&lc, prefill_join_kernel<F>, a);
}

template <int F>
__device__ __forceinline__ float value_at(const uint8_t* row, int i) {
  if constexpr (F == kBF16) return bf16lo(*reinterpret_cast<const uint16_t*>(row + 2 * i));
  else if constexpr (F == kF16) return f16lo(*reinterpret_cast<const uint16_t*>(row + 2 * i));
  else {
    float x, y;
    fp8x2_to_f32x2<F>(row[i], x, y);
    return x;
  }
}

template <int F, int KF>
__global__ void __launch_bounds__(kSimpleThreads) prefill_simple_kernel(const PrefillArgs a) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)a.num_tokens * a.num_heads;
  const int64_t warps = ((int64_t)gridDim.x * kSimpleThreads) >> 5;
  const float ks = KF == kE4M3 || KF == kE5M2 ? *a.kv_scale : 1.0f;
  uint32_t errbits = 0;
  for (int64_t row = ((int64_t)blockIdx.x * kSimpleThreads + threadIdx.x) >> 5; row < rows; row += warps) {
    const int t = (int)(row / a.num_heads), h = (int)(row - (int64_t)t * a.num_heads);
    int s = -1;
    for (int i = 0; i < a.num_seqs; ++i)
      if (a.cu_q[i] <= t && t < a.cu_q[i + 1]) s = i;
    if (s < 0) continue;
    const int c1 = a.cu_q[s + 1], k0 = a.cu_kv[s];
    int64_t m = (int64_t)a.cu_kv[s + 1] - k0;
    if (a.causal) m += t + 1 - c1;
    if (k0 < 0 || k0 + m > a.num_kv) {
      if (m > 0) errbits |= kErrPosOOB;
      m = k0 < 0 ? 0 : a.num_kv - k0;
    }
    const int g = h / a.group;
    const uint8_t* qn = a.q_nope + t * a.qn_ts + h * a.qn_hs;
    const uint8_t* qp = a.q_pe + t * a.qp_ts + h * a.qp_hs;
    float q[6], o[4] = {0, 0, 0, 0}, top = -INFINITY, sum = 0.0f;
    for (int i = 0; i < 4; ++i) q[i] = value_at<F>(qn, 32 * i + lane);
    for (int i = 0; i < 2; ++i) q[4 + i] = value_at<F>(qp, 32 * i + lane);
    for (int64_t p = k0; p < k0 + m; ++p) {
      const uint8_t* kn = a.k_nope + p * a.kn_ts + g * a.kn_hs;
      const uint8_t* kp = a.k_pe + p * a.kp_ts + g * a.kp_hs;
      float x = 0.0f;
      for (int i = 0; i < 4; ++i) x = fmaf(q[i], value_at<KF>(kn, 32 * i + lane), x);
      for (int i = 0; i < 2; ++i) x = fmaf(q[4 + i], value_at<KF>(kp, 32 * i + lane), x);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
      x *= a.softmax_scale * ks * kLog2e;
      const float mx = fmaxf(top, x), f = exp2f(top - mx), w = exp2f(x - mx);
      const uint8_t* v = a.v + p * a.v_ts + g * a.v_hs;
      for (int i = 0; i < 4; ++i) o[i] = fmaf(o[i], f, w * value_at<KF>(v, 32 * i + lane));
      sum = fmaf(sum, f, w);
      top = mx;
    }
    for (int i = 0; i < 4; ++i) {
      const float y = sum == 0.0f ? 0.0f : o[i] * ks / sum;
      uint16_t b = (uint16_t)pack_bf16x2(y, 0.0f);
      if (F == kF16) asm("cvt.rn.f16.f32 %0, %1;" : "=h"(b) : "f"(y));
      *reinterpret_cast<uint16_t*>(a.out + t * a.out_ts + h * a.out_hs + 2 * (32 * i + lane)) = b;
    }
    if (a.lse && lane == 0)
      a.lse[t * a.lse_ts + h * a.lse_hs] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
  }
  if (errbits && lane == 0 && a.err) atomicOr(a.err, errbits);
}

template <int F, int KF>
cudaError_t launch_simple(const PrefillArgs& a, const LaunchCfg& cfg) {
  const auto kern = prefill_simple_kernel<F, KF>;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(capped_grid(reinterpret_cast<const void*>(kern), kSimpleThreads,
                                ((int64_t)a.num_tokens * a.num_heads + kSimpleThreads / 32 - 1) / (kSimpleThreads / 32)));
  lc.blockDim = dim3(kSimpleThreads);
  lc.stream = cfg.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = cfg.pdl ? 1 : 0;
  return cudaLaunchKernelEx(&lc, kern, a);
}


}  // namespace

int64_t prefill_attention_workspace(int32_t num_tokens, int32_t num_heads, int32_t kv_heads, int32_t,
                                    int num_sms) {
  const int64_t ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
  return ctas * ((int64_t)sizeof(Split) +
                 2 * slot_rows(num_tokens, num_heads / kv_heads) * (2 + kV) * (int64_t)sizeof(float));
}

cudaError_t launch_prefill_attention(const PrefillArgs& a, int fmt, int kv_fmt, int num_sms,
                                     const LaunchCfg& cfg) {
  const int ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
  if (fmt == kBF16) {
    if (kv_fmt == kBF16) return launch_tc<kBF16>(a, ctas, cfg);
    return kv_fmt == kE4M3 ? launch_simple<kBF16, kE4M3>(a, cfg) : launch_simple<kBF16, kE5M2>(a, cfg);
  }
  if (kv_fmt == kF16) return launch_tc<kF16>(a, ctas, cfg);
  return kv_fmt == kE4M3 ? launch_simple<kF16, kE4M3>(a, cfg) : launch_simple<kF16, kE5M2>(a, cfg);
}

}  // namespace mla
