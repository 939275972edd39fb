// prefill_attention.cu -- attention of packed sequences over keys and values per head
// (include/mla_cache.h: mla_prefill_attention), on the 5th generation tensor cores.
//
// What it computes, per (token, head) row q of 128 + 64 elements and the rows of its
// sequence that the token sees: x_p = scale <q, k_p>, lse = ln sum exp(x_p), out = sum
// exp(x_p - lse) v_p.
//
// Shape of the work.  The query rows of a sequence and key head (token-major, the key
// head's query heads inside) are cut into items of 256 rows, two tiles of 128, its keys
// into tiles of 64; one unit = (item, key tile).  The units of the whole call, in
// (sequence, key head, item, key tile) order, are cut into equal contiguous runs, one per
// CTA (one CTA per SM), so ragged and causal batches load every SM alike.  An item whose
// units fall into several CTAs leaves unnormalised fp32 partial sums in the workspace, which
// a second launch joins in the order of the CTAs (no atomics: equal calls give equal bits).
//
// A unit: S_i = Q_i K^T (two tiles of 128 x 64, k = 192), weights P_i = exp2(S_i - reference)
// written to tensor memory as 16-bit values, O_i += P_i V (128 x 128, k = 64).  Tensor memory is
// full: per query tile S of 64 columns, P of 32, O of 128 and the queries' rotary columns, 32.  The
// weights' warps read the whole of S before they compute, so that the next scores come meanwhile.
//
// Measured (replayed from a graph, 16 heads): one prompt of 16384 tokens 950 us (1450 TFLOP/s; 950
// to 990 from one GPU to another), of 300 tokens 11.9 us; 16 prompts of 37 to 2048 tokens 142 us;
// 1024 new tokens of 2 sequences over 8192 e4m3 rows each 151 us (1140 TFLOP/s); single tokens of
// 32 sequences over 500 to 4096 rows 133 us (5.8 TB/s), over as many e4m3 rows 149 us (2.6 TB/s:
// a unit of one query row still pays the widening and products of 128 rows).
//
// Why 64 keys.  Beside the queries (96 KB) there is room for 1.6 units of 128 keys, and K of a
// unit came later than the products before it were done (2000 cycles for 32 KB; 16384 tokens
// 1100 us, in every order of the products tried).  Three stages of 64 keys hold two units ahead.
// The price: shared memory's reads bound the scores.  A product 128 x 64 x 16 with both operands
// there takes 49 cycles (6 KB at 128 bytes a cycle) where one of 128 columns takes 64, so a unit
// of both tiles would be 1690 cycles where 1280 of the tensor core would do.  The queries' rotary
// third in tensor memory takes 32 KB of a unit's 216 away (grouped heads 182.6 us without, 173.6
// with it; 2048 tokens 35.5, 34.4; 300 tokens 11.4, 11.7).  Long prompts come to 1600 to 2000 a
// unit, at the clock that the power limit leaves (1.84 GHz).
//
// Shared memory: the two query tiles (96 KB), three stages of K (24 KB: three runs of 64 columns)
// and of V (16 KB: two), in rows of 128 bytes with the 128-byte swizzle, by TMA.
//
// fp8 keys and values are widened to fp16 (exactly) on their way into the stages: two of these
// then, and two of raw codes (20 KB) in the place of the third.  That is another 80 KB of shared
// memory's traffic a unit, 2000 cycles in all; a unit takes 2200.  bf16 queries become fp16 times a
// power of two per row, in place.
//
// Roles (13 warps): 4 warps per query tile compute weights, a thread a row (running maximum;
// O is rescaled only when one has grown by more than 2^kGrow, and only that row's) and write the
// output; two per tile issue the products, scores and outputs; one plans the CTA's items, describes
// them to the others in shared memory and loads Q, K and V.  V rows that not every row of an item
// sees are looked after by the scores' warps, half a tile each, ahead of their products (16 ragged
// prompts 154 us; 156 by the outputs' warps; 180 by the weights' warps, before the weights): those
// behind the sequence are zeroed (they may hold anything), those with a NaN or an infinity too, and
// noted, so that the sums of the rows that see them become NaN.  With fp8, three more warps widen
// the codes and look after V on the way.
//
// Weights are 16-bit operands, as the tensor core takes them beside 16-bit values: bf16 ones (2^-8
// of themselves, as the bf16 result) beside bf16, fp16 ones (2^-11) beside fp16 and widened fp8.
// Against 64 bits a bf16 call is off by 0.0021 to 0.0024, relative, where weights in 32 bits would
// give 0.0016; a second bf16 part of each weight would be another product per unit.  Scores, sums
// and references are fp32.
//
// Code that runs once an item is as short as it can be: the roles' loops push it out of the
// instruction caches, and each of its instructions takes about 40 cycles.
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

constexpr int kM = 128;              // query rows of a tile
constexpr int kItemRows = 2 * kM;
constexpr int kKeys = 64;            // keys of a tile
constexpr int kV = 128;
constexpr int kRun = kKeys * 128;    // bytes of 64 columns of a key tile
constexpr int kQTile = 3 * kM * 128;
constexpr int kScoreWarp = 8, kOutWarp = 10, kLoadWarp = 12;
constexpr int kWideWarp = 13, kWideWarps = 3;  // (fp8 only)
__host__ __device__ constexpr int warps_of(int kf) { return is16(kf) ? 13 : kWideWarp + kWideWarps; }
constexpr int kItems = 4;            // item descriptions in shared memory
constexpr int kLooks = 8;            // notes of units whose V was looked after
constexpr int kMaxCtas = 1024;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// What beginning another item costs a CTA, in units: the runs are cut as if each item had
// this many more.  An item's change takes about 7000 cycles (the last output's way out, then the
// next scores' weights) where a unit takes 1600 to 2000.  With 2 and 4, medians of 5: 4 ragged
// prompts of grouped heads 182 us (180 to 183) and 175 (174 to 178), 16 ragged prompts 144.8 and
// 142.2, 6 chunks of 300 to 900 tokens over up to 4109 rows 92.0 and 90.3, 32 single tokens over
// e4m3 rows 150.7 and 149.4; where items are long or few the other way round, and less: 24 fp16
// prompts of up to 1300 tokens, 8 heads, 72.6 and 73.7, 21 of up to 503, 2 heads, 17.2 and 17.7.
constexpr int kSwitch = 4;
// A CTA takes at least this many units, so that a short call is not cut into runs that are all
// beginning and join: 21 prompts of 6 to 503 tokens, 2 heads, 17.7 us with 4 and 19.7 with 8.
constexpr int kMinUnits = 4;
// A sequence of at most this many items (of a key head) is counted by one lane, beside 31 others; a
// longer one by the whole warp.  With 4 and 12: 16 prompts of up to 8 items 144.0 and 142.2 us, 24
// of up to 6 75.0 and 73.7; 4 of 22 to 47 items, which neither deals to a lane, the same within
// their spread (172 to 178).
constexpr int kFewItems = 12;
// Calls of at most this many key rows, and of no more items than CTAs, give every CTA a whole
// item: nothing is cut, and nothing has to be joined.  Whole against cut, one prompt (us):
//   tokens       100         300         500         600         700         768
//   1 head    7.9  11.4  11.5  13.8  14.6  15.5  14.9  15.0  16.0  15.0  18.0  15.7
//   4 heads   8.0  11.7  11.5  15.3  15.1  15.9  15.3  16.1  16.5  15.8  18.1  16.0
//   16 heads  8.2  12.0  11.9  15.9  15.4  16.5  15.8  18.0  17.1  18.4  19.2  18.3
// and 8 prompts of 40 to 96, 1 head 8.3 and 12.1.  (With few heads a limit of 600 would do better
// by up to 2 us, with 16 worse by 1.4: whole items are one CTA's units in turn, cut ones a second
// launch and, with many heads, more of them than CTAs.)
constexpr int kWholeKeys = 768;

// The reference of a row's weights is the next whole number (log2) above its maximum less
// kTop; a score may pass the reference by kGrow before the sums are rescaled.  fp16 weights:
// up to 2^14, and 2^-25, half their smallest step, is 2^-34 of the row's largest or less.
template <int F>
struct Ref {
  static constexpr float kTop = F == kF16 ? 10.0f : 0.0f;
  static constexpr float kGrow = F == kF16 ? 14.0f : 8.0f;
};

// shared memory; KF: format of keys and values
template <int KF>
struct Lay {
  static constexpr bool kF8 = !is16(KF);
  static constexpr int kStages = kF8 ? 2 : 3;
  static constexpr int kRawStages = 2;
  static constexpr int kRawK = kKeys * 192, kRawV = kKeys * 128;  // bytes of a unit's codes
  static constexpr int q = 0;
  static constexpr int k = 2 * kQTile;                    // [kStages][3 runs]
  static constexpr int v = k + kStages * 3 * kRun;        // [kStages][2 runs]
  static constexpr int raw = v + kStages * 2 * kRun;      // [kRawStages][128 + 64 columns of K, V]
  static constexpr int items = raw + (kF8 ? kRawStages * (kRawK + kRawV) : 0);  // Item [kItems]
  static constexpr int flags = items + kItems * 64;       // [kLooks][16 bytes]: keys with bad V rows, a bit
                                                          // each; fp8: four to a byte
  static constexpr int bars = flags + kLooks * 16;
  // Barriers: of the stages; of units looked after, in turn; of the query tiles (scores, weights
  // and outputs two each, in turn: a warp may wait for a unit's before all have seen the one
  // before, and a phase's parity has to be told from the last); of the items.
  static constexpr int kKFull = 0, kVFull = kKFull + kStages, kKEmpty = kVFull + kStages,
                       kVEmpty = kKEmpty + kStages, kRawFull = kVEmpty + kStages,
                       kRawEmpty = kRawFull + kRawStages, kClean = kRawEmpty + kRawStages,
                       kQFull = kClean + kLooks, kQReady = kQFull + 2,
                       kQEmpty = kQReady + 2, kSFull = kQEmpty + 2, kSFree = kSFull + 4, kPFull = kSFree + 2,
                       kPvDone = kPFull + 4, kItemFull = kPvDone + 4,
                       kItemFree = kItemFull + kItems, kBars = kItemFree + kItems;
  static constexpr int misc = (bars + kBars * 8 + 15) / 16 * 16;
  static constexpr int bytes = misc + 64;
  static_assert(bytes <= 232448, "shared memory of a CTA");
};
// tensor memory columns: S of both tiles, P, the queries' rotary columns, O
constexpr int kP = 2 * kKeys, kQr = 3 * kKeys, kO = 4 * kKeys, kTmem = 512;
struct Misc {
  uint32_t tmem;
  uint32_t abort;
};

// How a tensor map reads row p, columns c.. of key head g: box (x_head * g + c, p, z_head * g).
struct Maps {
  CUtensorMap kn, kp, v;
  CUtensorMap qn, qp;  // (column, head, token); only where q_tokens is not 0
  int32_t kn_x, kn_z, kp_x, kp_z, v_x, v_z;
  int32_t q_tokens;  // tokens of a query tile that comes in boxes; 0: rows are copied one by one
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
  float *m, *l, *d;  // [2 ctas][slot_rows]: reference (log2), sum of the weights, and what it is
                     // divided by less that
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
  w.d = w.l + (int64_t)ctas * 2 * rows;
  w.o = w.d + (int64_t)ctas * 2 * rows;
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
__device__ __forceinline__ int seen_of(const PrefillArgs& a, int64_t base, int m, uint32_t row) {
  const int64_t n = base + (a.causal ? (int64_t)a.by_group(row) : 0);
  return (int)max((int64_t)0, min(n, (int64_t)m));
}
// Key tiles of rows of which the last sees `most` (one even when it sees none: they are still
// written).
__device__ __forceinline__ int key_tiles(int most) { return max(1, (most + kKeys - 1) / kKeys); }
__device__ __forceinline__ int item_tiles(const PrefillArgs& a, const Seq& q, int b) {
  return key_tiles(seen_of(a, q.base, q.m, min((uint32_t)(b + 1) * kItemRows, q.rows) - 1));
}

// Units of an item; one where a CTA takes whole items.
__device__ __forceinline__ int item_units(const PrefillArgs& a, const Seq& q, int b) {
  return a.whole ? 1 : kSwitch + item_tiles(a, q, b);
}

// A CTA's part of an item.
struct Item {
  int kb, ke;          // its key tiles of it; ke < 0: no more items
  int end[2];          // where those of the query tiles end (at kb or before: none)
  int tiles;           // of the whole item
  int least, most;     // keys seen by its first and last row
  uint32_t row0;       // first row, among the sequence's of the key head
  int rows, t0, head;
  int k0, m;           // the sequence's first key row, and how many exist
  int64_t base;        // keys that its token t0 sees (before clamping)
  // (an index that is not known would put the whole description into local memory)
  __device__ __forceinline__ int end_of(int tile) const { return tile ? end[1] : end[0]; }
  // The first key tile that not every row sees whole.
  __device__ __forceinline__ int ragged() const { return max(kb, least / kKeys); }
  // Units with V rows to be looked after.
  __device__ __forceinline__ int cleaned() const { return max(0, ke - ragged()); }
};
static_assert(sizeof(Item) <= 64, "an item's description");

// Reads the descriptions in their order, a whole warp at a time.
template <int KF>
struct Items {
  using L = Lay<KF>;
  uint32_t smem, next;
  // The next one, left there (peek) or given back.
  __device__ __forceinline__ bool get(const Waiter& wait, Item& it, bool peek = false) {
    const uint32_t i = next & (kItems - 1), bars = smem + L::bars;
    if (!__all_sync(0xFFFFFFFFu, wait(bars + 8 * (L::kItemFull + i), (next / kItems) & 1))) return false;
    const uint32_t at = smem + L::items + i * 64;
    const uint4 w0 = lds16(at), w1 = lds16(at + 16), w2 = lds16(at + 32), w3 = lds16(at + 48);
    it.kb = w0.x, it.ke = w0.y, it.end[0] = w0.z, it.end[1] = w0.w;
    it.tiles = w1.x, it.least = w1.y, it.most = w1.z, it.row0 = w1.w;
    it.rows = w2.x, it.t0 = w2.y, it.head = w2.z, it.k0 = w2.w;
    it.m = w3.x, it.base = (int64_t)((uint64_t)w3.w << 32 | w3.z);
    if (!peek) {
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(bars + 8 * (L::kItemFree + i));
      ++next;
    }
    return it.ke >= 0;
  }
};

// A place in a ring of N stages: which stage, and the parity of its phase.
template <int N>
struct Stage {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step() {
    if (++at == N) {
      at = 0;
      phase ^= 1;
    }
  }
};

// -------------------------------------------------------------- plan and load
__device__ __noinline__ int64_t divide(int64_t n, int64_t d) {
  return (n | d) >> 32 ? n / d : (int64_t)((uint32_t)n / (uint32_t)d);
}
template <typename I>
__device__ __forceinline__ I scan(I v, int lane) {  // inclusive, over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// The run of one CTA, walked item by item, by one warp.  An item is kSwitch units that stand
// for beginning it, then its key tiles: a run starts before the first of these when kt is
// negative.  I: of numbers of units (32 bits do for all but the largest calls).
template <typename I>
struct Plan {
  Seq q;
  int s, head, b, kt, left;
  I begin, each;   // the first unit; units of the CTAs c >= extra (each + 1 of the ones before)
  int extra, count;
  static __device__ __forceinline__ I over(I n, I d) {
    if constexpr (sizeof(I) == 4) return (uint32_t)n / (uint32_t)d;
    else return divide(n, d);
  }
  __device__ __forceinline__ int cta_of(I u) const {
    const I longer = (each + 1) * extra;
    return (int)(u < longer ? over(u, each + 1) : extra + over(u - longer, each));
  }
  // Where the run starts; pre: scratch for num_seqs numbers.
  __device__ __forceinline__ void find(const PrefillArgs& a, I* pre, int lane, uint32_t& errbits) {
    I total = 0;
    uint32_t ignored = 0;
#pragma unroll 1
    for (int s0 = 0; s0 < a.num_seqs; s0 += 32) {
      I u = 0;
      int nb = 0;
      if (s0 + lane < a.num_seqs) {
        const Seq one = load_seq(a, s0 + lane, errbits);
        nb = one.nb;
        if (nb <= kFewItems)
#pragma unroll 1
          for (int i = 0; i < nb; ++i) u += item_units(a, one, i);
      }
      // sequences of many items: by the whole warp
      for (uint32_t many = __ballot_sync(0xFFFFFFFFu, nb > kFewItems); many; many &= many - 1) {
        const int from = __ffs(many) - 1;
        const Seq one = load_seq(a, s0 + from, ignored);
        I sum = 0;
#pragma unroll 1
        for (int i = lane; i < one.nb; i += 32) sum += item_units(a, one, i);
        sum = __shfl_sync(0xFFFFFFFFu, scan<I>(sum, lane), 31);
        if (lane == from) u = sum;
      }
      u *= a.kv_heads;
      const I in = scan<I>(u, lane);
      if (s0 + lane < a.num_seqs) pre[s0 + lane] = total + in - u;
      total += __shfl_sync(0xFFFFFFFFu, in, 31);
    }
    __syncwarp();
    const I ctas = a.whole ? max((I)1, total) : max((I)1, min((I)gridDim.x, total / (I)kMinUnits));
    each = over(total, ctas);
    extra = (int)(total - each * ctas);
    begin = each * blockIdx.x + min((int)blockIdx.x, extra);
    count = blockIdx.x < ctas ? (int)each + ((int)blockIdx.x < extra ? 1 : 0) : 0;
    left = 0;
    if (count == 0) return;
    // the last sequence that begins at or before the run (those without units begin where the
    // one behind them does)
    int lo = 0;
#pragma unroll 1
    for (int step = a.num_seqs > 32 ? 2048 : 16; step > 0; step >>= 1)
      if (lo + step < a.num_seqs && pre[lo + step] <= begin) lo += step;
    s = lo;
    q = load_seq(a, s, ignored);
    I off = begin - pre[s];
    const I per = over((s + 1 < a.num_seqs ? pre[s + 1] : total) - pre[s], a.kv_heads);
    head = (int)over(off, per);
    off -= head * per;
    I base = 0;
#pragma unroll 1
    for (int b0 = 0;; b0 += 32) {
      const I u = b0 + lane < q.nb ? item_units(a, q, b0 + lane) : 0;
      const I in = scan<I>(u, lane);
      const uint32_t hit = __ballot_sync(0xFFFFFFFFu, off < base + in);
      if (hit) {
        const int at = __ffs(hit) - 1;
        b = b0 + at;
        kt = (int)(off - base - __shfl_sync(0xFFFFFFFFu, in - u, at)) - kSwitch;
        break;
      }
      base += __shfl_sync(0xFFFFFFFFu, in, 31);
    }
    left = a.whole ? item_tiles(a, q, b) : count + min(kt, 0);
    kt = max(kt, 0);
  }
  // The next item (the first call: the run's first).
  __device__ __forceinline__ Item next(const PrefillArgs& a) {
    Item it;
    it.ke = -1;
    if (left <= 0) return it;
    it.kb = kt;
    it.row0 = (uint32_t)b * kItemRows;
    it.rows = (int)min((uint32_t)kItemRows, q.rows - it.row0);
    it.least = seen_of(a, q.base, q.m, it.row0);
    it.most = seen_of(a, q.base, q.m, it.row0 + it.rows - 1);
    it.tiles = key_tiles(it.most);
    it.ke = min(it.tiles, kt + left);
    const int first = it.rows > kM ? key_tiles(seen_of(a, q.base, q.m, it.row0 + kM - 1)) : it.tiles;
    it.end[0] = min(it.ke, first);
    it.end[1] = it.rows > kM ? it.ke : 0;
    it.t0 = q.t0;
    it.head = head;
    it.k0 = q.k0;
    it.m = q.m;
    it.base = q.base;
    left -= it.ke - kt + kSwitch;
    kt = 0;
    if (left > 0 && ++b >= q.nb) {
      b = 0;
      if (++head >= a.kv_heads) {
        head = 0;
        uint32_t ignored = 0;
        q.nb = 0;
#pragma unroll 1
        while (q.nb == 0 && ++s < a.num_seqs) q = load_seq(a, s, ignored);
        if (q.nb == 0) left = 0;
      }
    }
    return it;
  }
};

// Plans the items and describes them, one ahead; Q, K and V by TMA; where the run ends inside
// an item, what the join needs.  Returns the copies begun, in K and V of a unit (fp8: in units);
// filled: how often the queries' boxes of each tile.
template <int KF, typename I>
__device__ __forceinline__ uint32_t load_role(const PrefillArgs& a, const Maps& maps, uint8_t* smem_raw,
                                              uint32_t smem, const Waiter& wait, int lane,
                                              const Workspace& ws, uint32_t& errbits,
                                              uint32_t (&filled)[2]) {
  using L = Lay<KF>;
  const uint32_t bars = smem + L::bars;
  auto waited = [&](int bar, uint32_t phase) {
    return __all_sync(0xFFFFFFFFu, wait(bars + 8 * bar, phase & 1));
  };
  // rows that one item reads leave L2 first
  const uint64_t policy =
      tc::l2_policy((int64_t)a.num_tokens * a.group <= (int64_t)kItemRows * a.num_seqs);
  Plan<I> plan;
  plan.find(a, reinterpret_cast<I*>(smem_raw + L::k), lane, errbits);
  tc::fence_smem_async();  // the scratch is read; copies may write there now
  __syncwarp();
  uint32_t g = 0, told = 0;
  Stage<L::kF8 ? L::kRawStages : L::kStages> st;
  Item it;
  it.ke = 0;
  // The first round only plans.
#pragma unroll 1
  for (bool first = true;; first = false) {
    const Item nxt = plan.next(a);
    if (first || it.ke >= 0) {
      const uint32_t i = told & (kItems - 1);
      if (told >= kItems && !waited(L::kItemFree + i, told / kItems - 1)) return L::kF8 ? g : 2 * g;
      if (lane == 0) {
        *reinterpret_cast<Item*>(smem_raw + L::items + i * 64) = nxt;
        mbar_arrive(bars + 8 * (L::kItemFull + i));
      }
      __syncwarp();
      ++told;
    }
    if (!first) {
      if (it.ke < 0) break;
      const int h = it.head;
      // the queries of a tile; they come behind the item's first keys, so that the first scores
      // wait for no more than they need
      auto queries = [&](int i) {
        if (maps.q_tokens == 0 || it.end[i] <= it.kb) return true;
        if (filled[i] > 0 && !waited(L::kQEmpty + i, filled[i] - 1)) return false;
        ++filled[i];
        if (lane == 0) {
          const uint32_t qf = bars + 8 * (L::kQFull + i), dst = smem + L::q + i * kQTile;
          const int t = it.t0 + ((int)(it.row0 / (uint32_t)kM) + i) * maps.q_tokens;
          mbar_arrive_expect_tx(qf, kQTile);
          tc::tma_load3(dst, &maps.qn, 0, h * a.group, t, qf, policy);
          tc::tma_load3(dst + kM * 128, &maps.qn, 64, h * a.group, t, qf, policy);
          tc::tma_load3(dst + 2 * kM * 128, &maps.qp, 0, h * a.group, t, qf, policy);
        }
        __syncwarp();
        return true;
      };
#pragma unroll 1
      for (int kt = it.kb; kt < it.ke; ++kt, ++g, st.step()) {
        const int row = it.k0 + kt * kKeys;
        if constexpr (L::kF8) {
          const uint32_t rf = bars + 8 * (L::kRawFull + st.at);
          const uint32_t k = smem + L::raw + st.at * (L::kRawK + L::kRawV);
          if (g >= L::kRawStages && !waited(L::kRawEmpty + st.at, st.phase ^ 1)) return g;
          if (lane == 0) {
            mbar_arrive_expect_tx(rf, L::kRawK + L::kRawV);
            tc::tma_load3(k, &maps.kn, h * maps.kn_x, row, h * maps.kn_z, rf, policy);
            tc::tma_load3(k + kKeys * 128, &maps.kp, h * maps.kp_x, row, h * maps.kp_z, rf, policy);
            tc::tma_load3(k + L::kRawK, &maps.v, h * maps.v_x, row, h * maps.v_z, rf, policy);
          }
          __syncwarp();
          if (kt == it.kb && !(queries(0) && queries(1))) return g + 1;
          continue;
        }
        const uint32_t kf = bars + 8 * (L::kKFull + st.at), vf = bars + 8 * (L::kVFull + st.at);
        const uint32_t k = smem + L::k + st.at * 3 * kRun, v = smem + L::v + st.at * 2 * kRun;
        if (g >= L::kStages && !waited(L::kKEmpty + st.at, st.phase ^ 1)) return 2 * g;
        if (lane == 0) {
          mbar_arrive_expect_tx(kf, 3 * kRun);
          tc::tma_load3(k, &maps.kn, h * maps.kn_x, row, h * maps.kn_z, kf, policy);
          tc::tma_load3(k + kRun, &maps.kn, h * maps.kn_x + 64, row, h * maps.kn_z, kf, policy);
          tc::tma_load3(k + 2 * kRun, &maps.kp, h * maps.kp_x, row, h * maps.kp_z, kf, policy);
        }
        __syncwarp();
        if (kt == it.kb && !queries(0)) return 2 * g + 1;
        if (g >= L::kStages && !waited(L::kVEmpty + st.at, st.phase ^ 1)) return 2 * g + 1;
        if (lane == 0) {
          mbar_arrive_expect_tx(vf, 2 * kRun);
          tc::tma_load3(v, &maps.v, h * maps.v_x, row, h * maps.v_z, vf, policy);
          tc::tma_load3(v + kRun, &maps.v, h * maps.v_x + 64, row, h * maps.v_z, vf, policy);
        }
        __syncwarp();
        if (kt == it.kb && !queries(1)) return 2 * g + 2;
      }
      if (it.ke < it.tiles && lane == 0) {  // the run's last item
        const I u0 = plan.begin + plan.count - it.ke;  // the unit of its key tile 0
        const int c0 = plan.cta_of(u0), c1 = plan.cta_of(u0 + it.tiles - 1);
        ws.split[blockIdx.x] = Split{it.t0, it.row0, it.head, (int16_t)it.rows, (int16_t)(c1 - c0 + 1), c0, {}};
      }
    }
    it = nxt;
  }
  return L::kF8 ? g : 2 * g;
}

// ------------------------------------------------------------------- widening
// Two fp8 codes (the low 16 bits) as two fp16 values, exactly.
template <int KF>
__device__ __forceinline__ uint32_t widen2(uint32_t w) {
  uint32_t r;
  if constexpr (KF == kE4M3) asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
  else asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
  return r;
}
// Columns 16 j .. of a row of a tile of runs of 64 columns.
template <int KF>
__device__ __forceinline__ void widen16(uint32_t tile, int row, int j, uint4 w) {
  const uint32_t at = tile + (j >> 2) * kRun + row * 128, u = 2 * (j & 3), x = row & 7;
  sts16(at + ((u ^ x) << 4), make_uint4(widen2<KF>(w.x), widen2<KF>(w.x >> 16), widen2<KF>(w.y),
                                        widen2<KF>(w.y >> 16)));
  sts16(at + (((u + 1) ^ x) << 4), make_uint4(widen2<KF>(w.z), widen2<KF>(w.z >> 16), widen2<KF>(w.w),
                                              widen2<KF>(w.w >> 16)));
}
// fp8 codes of K and V from the raw stages to the fp16 ones; V rows that not every row of an item
// sees are looked after on the way (as by look_after).
template <int KF>
__device__ __forceinline__ void widen_role(uint32_t smem, const Waiter& waiter, int cw, int lane) {
  using L = Lay<KF>;
  const uint32_t bars = smem + L::bars;
  auto wait = [&](int bar, uint32_t phase) {
    return __all_sync(0xFFFFFFFFu, waiter(bars + 8 * bar, phase & 1));
  };
  Stage<L::kRawStages> sr;
  Stage<L::kStages> st;
  uint32_t g = 0, cleaned = 0;
  int turn = cw;  // the 8 groups of 8 rows are dealt to three warps: who has two of them changes
  Items<KF> items{smem, 0};
  Item it;
#pragma unroll 1
  while (items.get(waiter, it)) {
    const int ragged = it.ragged();
#pragma unroll 1
    for (int kt = it.kb; kt < it.ke; ++kt, ++g, sr.step(), st.step(), turn = turn == 2 ? 0 : turn + 1) {
      const uint32_t raw = smem + L::raw + sr.at * (L::kRawK + L::kRawV);
      const uint32_t k = smem + L::k + st.at * 3 * kRun, v = smem + L::v + st.at * 2 * kRun;
      if (!wait(L::kRawFull + sr.at, sr.phase)) return;
      if (g >= L::kStages && !wait(L::kKEmpty + st.at, st.phase ^ 1)) return;
      // 8 rows x 8 pieces of 16 columns each (two rounds at once), then the rotary ones 8 x 4
#pragma unroll 1
      for (int r = turn * 8 + (lane >> 3); r < kKeys; r += kWideWarps * 8) {
        const int j = lane & 7;
        const uint4 w0 = lds16(raw + r * 128 + j * 16), w1 = lds16(raw + (r + 4) * 128 + j * 16);
        widen16<KF>(k, r, j, w0);
        widen16<KF>(k, r + 4, j, w1);
        const int rr = (r & ~7) + (lane >> 2);
        widen16<KF>(k + 2 * kRun, rr, lane & 3, lds16(raw + kKeys * 128 + rr * 64 + (lane & 3) * 16));
      }
      tc::fence_smem_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (L::kKFull + st.at));
      if (g >= L::kStages && !wait(L::kVEmpty + st.at, st.phase ^ 1)) return;
      const uint32_t flags = smem + L::flags + (g & (kLooks - 1)) * 16;
#pragma unroll 1
      for (int r = (turn == 2 ? 0 : turn + 1) * 8 + (lane >> 3); r < kKeys; r += kWideWarps * 8) {
        const int j = lane & 7;
        uint4 w[2] = {lds16(raw + L::kRawK + r * 128 + j * 16), lds16(raw + L::kRawK + (r + 4) * 128 + j * 16)};
        if (__builtin_expect(kt >= ragged, 0)) {
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int p = kt * kKeys + r + 4 * n;
            const uint32_t votes =
                __ballot_sync(0xFFFFFFFFu, any_special<KF>(w[n]) && p >= it.least && p < it.most);
            if (p >= it.most || votes & (0xFFu << (lane & 24))) w[n] = make_uint4(0, 0, 0, 0);
            uint32_t bad = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (votes & (0xFFu << (8 * i))) bad |= 1u << i;
            if (lane == 0) sts_u8(flags + (r >> 2) + n, bad);
          }
        }
        widen16<KF>(v, r, j, w[0]);
        widen16<KF>(v, r + 4, j, w[1]);
      }
      tc::fence_smem_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bars + 8 * (L::kVFull + st.at));
        mbar_arrive(bars + 8 * (L::kRawEmpty + sr.at));
        if (kt >= ragged) mbar_arrive(bars + 8 * (L::kClean + ((cleaned + kt - ragged) & (kLooks - 1))));
      }
    }
    cleaned += it.cleaned();
  }
}

// ------------------------------------------------------------ matrix products
// A query tile's rotary columns to tensor memory, where every unit's scores read them.
template <int KF>
__device__ __forceinline__ void move_rotary(uint32_t smem, uint32_t tmem, bool one, int tile) {
  const uint32_t i = __shfl_sync(0xFFFFFFFFu, tile, 0);
  const uint64_t qr = tc::smem_desc(smem + Lay<KF>::q + i * kQTile + 2 * kM * 128, 0, 1024);
#pragma unroll
  for (int k = 0; k < 4; ++k) tc::copy_k16(one, tmem + kQr + i * (kKeys / 2) + 8 * k, qr + 2 * k);
}
template <int F, int KF>
__device__ __forceinline__ void issue_scores(uint32_t smem, uint32_t tmem, bool one, int tile, int stage,
                                             uint32_t negate) {
  using L = Lay<KF>;
  const uint32_t id = negate | tc::instr_desc(kM, kKeys, false, F == kBF16, F == kBF16);
  const uint32_t i = __shfl_sync(0xFFFFFFFFu, tile, 0), st = __shfl_sync(0xFFFFFFFFu, stage, 0);
  const uint64_t qa = tc::smem_desc(smem + L::q + i * kQTile, 0, 1024);
  const uint64_t kb = tc::smem_desc(smem + L::k + st * 3 * kRun, 0, 1024);
  const uint32_t d = tmem + i * kKeys;
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      tc::mma_16bit(one, d, qa + (c * kM * 128 >> 4) + 2 * k, kb + (c * kRun >> 4) + 2 * k, id, c + k > 0);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    tc::mma_16bit_ta(one, d, tmem + kQr + i * (kKeys / 2) + 8 * k, kb + (2 * kRun >> 4) + 2 * k, id, true);
}
// V MN-major (two runs of 64 columns).
template <int F, int KF>
__device__ __forceinline__ void issue_outputs(uint32_t smem, uint32_t tmem, bool one, int tile, int stage,
                                              bool first) {
  using L = Lay<KF>;
  constexpr uint32_t kId = tc::instr_desc(kM, kV, false, F == kBF16, F == kBF16, true);
  const uint32_t i = __shfl_sync(0xFFFFFFFFu, tile, 0), st = __shfl_sync(0xFFFFFFFFu, stage, 0);
  const uint32_t p = tmem + kP + i * (kKeys / 2), d = tmem + kO + i * kV;
  const uint64_t vb = tc::smem_desc(smem + L::v + st * 2 * kRun, kRun, 1024);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    tc::mma_16bit_ta(one, d, p + 8 * k, vb + k * (2048 >> 4), kId, k > 0 || !first);
}

// Four warps issue the products: scores and outputs of a query tile each.  An issue waits for
// the products before it, and what a warp does between two of its products (looks at barriers,
// signals) leaves the tensor core idle unless another warp's products are there: 16384 tokens
// took 1380 us with one warp for all, 1060 with these.  K and V of a unit are free when
// both tiles' warps have said so; a warp whose tile has no part in a unit says it when they have
// come, so that it does not run ahead.
//
// Looks at a barrier without letting the warp be suspended: waking takes long.  Every lane has
// to see the phase complete: the lane that issues, and those that read what has come.
__device__ __forceinline__ bool spin(const Waiter& waiter, uint32_t bar, uint32_t phase) {
#pragma unroll 1
  for (int n = 0; n < 64; ++n)
    if (__all_sync(0xFFFFFFFFu, mbar_test(bar, phase & 1))) return true;
  return __all_sync(0xFFFFFFFFu, waiter(bar, phase & 1));
}
// 32 rows of V of a unit, a lane each: those from `most` on are zeroed, those from `least` on with a
// NaN or an infinity too, and noted in flags, a bit each.
template <int F>
__device__ __noinline__ void look_after(uint32_t v, uint32_t flags, int least, int most) {
  const int lane = threadIdx.x & 31;
  const uint32_t at = v + lane * 128;
  uint32_t bad = 0;
  if (least < 32) {
    uint32_t top[4] = {0, 0, 0, 0};
#pragma unroll 1
    for (int c = 0; c < 8; c += 4) {  // every column of the row, in any order
      uint4 w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = lds16(at + (i & 1) * kRun + (((c + (i >> 1)) ^ (lane & 7)) << 4));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        top[i & 3] = umax16x2(top[i & 3], umax16x2(umax16x2(w[i].x & 0x7FFF7FFFu, w[i].y & 0x7FFF7FFFu),
                                                   umax16x2(w[i].z & 0x7FFF7FFFu, w[i].w & 0x7FFF7FFFu)));
    }
    const uint32_t all = umax16x2(umax16x2(top[0], top[1]), umax16x2(top[2], top[3]));
    const bool sp = max(all & 0xFFFFu, all >> 16) >= (F == kBF16 ? 0x7F80u : 0x7C00u);
    bad = __ballot_sync(0xFFFFFFFFu, sp && lane >= least && lane < most);
    if (bad != 0 || most < 32) {
      if (lane >= most || bad >> lane & 1)
#pragma unroll 1
        for (int c = 0; c < 128; c += 16) {
          sts16(at + c, make_uint4(0, 0, 0, 0));
          sts16(at + kRun + c, make_uint4(0, 0, 0, 0));
        }
      tc::fence_smem_async();
    }
  }
  if (lane == 0) sts_u32(flags, bad);
  __syncwarp();
}
template <int F, int QF, int KF>
__device__ __forceinline__ void score_role(float scale, uint32_t smem, uint32_t tmem, const Waiter& waiter,
                                           int tile) {
  using L = Lay<KF>;
  const uint32_t bars = smem + L::bars;
  auto wait = [&](int bar, uint32_t phase) { return spin(waiter, bars + 8 * bar, phase); };
  const bool one = tc::elect();
  const uint32_t negate = scale < 0.0f ? 1u << 13 : 0u;  // of the scores, by the tensor core
  uint32_t n = 0, g = 0, opened = 0, cleaned = 0;  // units of this tile, and of all; items; units looked after
  Stage<L::kStages> st;
  Items<KF> items{smem, 0};
  Item it;
#pragma unroll 1
  while (items.get(waiter, it)) {
    const int e = it.end_of(tile), kb = it.kb, ke = it.ke, ragged = it.ragged();
    if (kb < e) {
      if (!wait((F == QF ? L::kQFull : L::kQReady) + tile, opened++)) return;
      tc::fence_smem_async();  // (the queries may have come by ordinary stores)
      // (the item before's last scores are done, or these queries would not have come)
      tc::fence_after_sync();
      move_rotary<KF>(smem, tmem, one, tile);
    }
#pragma unroll 1
    for (int kt = kb; kt < ke; ++kt, ++g) {
      // the scores before these are read
      if (kt < e && n >= 1 && !wait(L::kSFree + tile, n - 1)) return;
      if (!wait(L::kKFull + st.at, st.phase)) return;
      if (kt < e) {
        tc::fence_after_sync();
        issue_scores<F, KF>(smem, tmem, one, tile, st.at, negate);
        tc::commit(one, bars + 8 * (L::kSFull + 2 * tile + (n & 1)));
        if (kt + 1 == e) tc::commit(one, bars + 8 * (L::kQEmpty + tile));
        ++n;
      }
      // V of every unit is seen to come, though only some are looked after: a wait for one must know
      // that the stage's last has come (or it would take that phase for its own: a tile without rows
      // in an item is held back by nothing else), and the stage's next must not have come (it does
      // not before this K is free).
      if (!L::kF8 && !wait(L::kVFull + st.at, st.phase)) return;
      tc::commit(one, bars + 8 * (L::kKEmpty + st.at));
      if (!L::kF8 && kt >= ragged) {  // half of V each
        const int row = kt * kKeys + tile * 32;
        look_after<F>(smem + L::v + st.at * 2 * kRun + tile * 32 * 128,
                      smem + L::flags + (g & (kLooks - 1)) * 16 + tile * 4, it.least - row, it.most - row);
        if ((threadIdx.x & 31) == 0) mbar_arrive(bars + 8 * (L::kClean + (cleaned & (kLooks - 1))));
        ++cleaned;
      }
      st.step();
    }
  }
}
template <int F, int KF>
__device__ __forceinline__ void output_role(uint32_t smem, uint32_t tmem, const Waiter& waiter, int tile) {
  using L = Lay<KF>;
  const uint32_t bars = smem + L::bars;
  auto wait = [&](int bar, uint32_t phase) { return spin(waiter, bars + 8 * bar, phase); };
  const bool one = tc::elect();
  uint32_t n = 0, cleaned = 0;  // units of this tile; units looked after
  Stage<L::kStages> st;
  Items<KF> items{smem, 0};
  Item it;
#pragma unroll 1
  while (items.get(waiter, it)) {
    const int e = it.end_of(tile), kb = it.kb, ke = it.ke, ragged = it.ragged();
    const uint32_t c0 = cleaned - ragged;
    cleaned += it.cleaned();
#pragma unroll 1
    for (int kt = kb; kt < ke; ++kt) {
      if (!wait(L::kVFull + st.at, st.phase)) return;
      if (kt < e) {
        const uint32_t nc = c0 + kt;
        if (!L::kF8 && kt >= ragged && !wait(L::kClean + (nc & (kLooks - 1)), nc / kLooks)) return;
        // (an item's first weights: each warp has read its sums of the item before, too)
        if (!wait(L::kPFull + 2 * tile + (n & 1), n >> 1)) return;
        tc::fence_after_sync();
        issue_outputs<F, KF>(smem, tmem, one, tile, st.at, kt == kb);
        tc::commit(one, bars + 8 * (L::kPvDone + 2 * tile + (n & 1)));
        ++n;
      }
      tc::commit(one, bars + 8 * (L::kVEmpty + st.at));
      st.step();
    }
  }
}

// -------------------------------------------------------- weights and output
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

// The queries of a tile by asynchronous copies, by the tile's four warps (where they do not come
// in boxes: a group of query heads that does not divide a tile, or heads with a stride of 0).
template <int KF>
__device__ __forceinline__ void load_queries(const PrefillArgs& a, const Item& it, uint32_t smem,
                                             int tile, int w4, int lane) {
  const int col = lane & 7;
#pragma unroll 1
  for (int r = w4 * 32 + (lane >> 3); r < w4 * 32 + 32; r += 4) {
    const bool ok = tile * kM + r < it.rows;
    const uint32_t row = it.row0 + tile * kM + r;
    const uint32_t dt = ok ? a.by_group(row) : 0;
    const int64_t t = ok ? it.t0 + (int)dt : 0;
    const int64_t h = ok ? (int64_t)it.head * a.group + (int)(row - dt * a.group) : 0;
    const uint8_t* nope = a.q_nope + t * a.qn_ts + h * a.qn_hs + col * 16;
    const uint8_t* pe = a.q_pe + t * a.qp_ts + h * a.qp_hs + col * 16;
    const uint32_t d = smem + tile * kQTile + r * 128 + ((col ^ (r & 7)) << 4);
    tc::cp_async16(d, nope, ok);
    tc::cp_async16(d + kM * 128, nope + 128, ok);
    tc::cp_async16(d + 2 * kM * 128, pe, ok);
  }
  tc::cp_async_arrive(smem + Lay<KF>::bars + 8 * (Lay<KF>::kQFull + tile));
}

// A bf16 query row in shared memory as fp16 times a power of two that puts its largest magnitude
// into [2^14, 2^15): exact down to 2^-31 of that, off by at most 2^-39 of it below.  Returns the
// inverse power; NaN for a row with a NaN or an infinity.
__device__ __noinline__ float narrow_row(uint32_t at, int row) {
  uint32_t top = 0;
#pragma unroll 1
  for (int k = 0; k < 24; k += 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 w = lds16(at + ((k + i) >> 3) * (kM * 128) + ((((k + i) ^ row) & 7) << 4));
      top = umax16x2(top, umax16x2(umax16x2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                   umax16x2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu)));
    }
  }
  top = max(top & 0xFFFFu, top >> 16);
  const uint32_t e = min(max(top >> 7, 15u), 254u);         // exponent of the largest magnitude
  const float s = __uint_as_float((268u - e) << 23);        // 2^(141 - e)
#pragma unroll 1
  for (int k = 0; k < 24; k += 2) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t p = at + ((k + i) >> 3) * (kM * 128) + ((((k + i) ^ row) & 7) << 4);
      const uint4 w = lds16(p);
      sts16(p, make_uint4(pack_f16x2(bf16lo(w.x) * s, bf16hi(w.x) * s), pack_f16x2(bf16lo(w.y) * s, bf16hi(w.y) * s),
                          pack_f16x2(bf16lo(w.z) * s, bf16hi(w.z) * s), pack_f16x2(bf16lo(w.w) * s, bf16hi(w.w) * s)));
    }
  }
  return top >= 0x7F80u ? NAN : __uint_as_float((e - 14u) << 23);  // 2^(e - 141)
}

// What the weights of an item's units need to know; key tiles count from the part's first.
struct Part {
  uint32_t smem, s_at, p_at, o_at;  // tensor memory: this warp's scores, weights and sums
  uint32_t n, g, cleaned;     // units of this tile, of all, and looked after, before the part
  int tile, count, from;      // key tiles, and the first that not every row sees whole
  int seen;                   // keys that this thread's row sees, from the first tile on
  bool live;                  // the warp has rows
  bool head;                  // the part begins with the item's first key tile
  float c;                    // weights: exp2(c score - reference)
};
// The weights of an item's units: the row's reference, the sum of its weights, and how much more
// they are as they are rounded.  (The last is counted in an item's first key tile, by warps with a
// row that ends there: a row of few keys is divided by the weights that its products had, so that
// their rounding does not scale it.  In longer rows the roundings cancel, and the count would cost
// each unit.)
// False: given up.
template <int F, int KF>
__device__ __forceinline__ bool unit_weights(Part s, const Waiter waiter, float& mu_out, float& l_out, float& d_out) {
  using R = Ref<F>;
  using L = Lay<KF>;
  const int lane = threadIdx.x & 31;
  auto wait = [&](int bar, uint32_t phase) {
    return __all_sync(0xFFFFFFFFu, waiter(s.smem + L::bars + 8 * bar, phase & 1));
  };
  float mu = -INFINITY, l = 0.0f, d = 0.0f;
#pragma unroll 1
  for (int kt = 0; kt < s.count; ++kt, ++s.n) {
    if (!wait(L::kSFull + 2 * s.tile + (s.n & 1), s.n >> 1)) return false;
    tc::fence_after_sync();
    const uint32_t bars = s.smem + L::bars;
    if (!s.live) {
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (L::kSFree + s.tile));
      // (every warp waits for every unit's outputs, so that none mistakes a phase later on)
      if (kt > 0 && !wait(L::kPvDone + 2 * s.tile + ((s.n - 1) & 1), (s.n - 1) >> 1)) return false;
      if (lane == 0) mbar_arrive(bars + 8 * (L::kPFull + 2 * s.tile + (s.n & 1)));
      continue;
    }
    float x[kKeys];
    tc::ld_32x64(s.s_at, reinterpret_cast<uint32_t*>(x));
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + 8 * (L::kSFree + s.tile));
    const int lim = s.seen - kt * kKeys;
    const bool cut = kt >= s.from && __any_sync(0xFFFFFFFFu, lim < kKeys);
    if (__builtin_expect(cut, 0)) {
#pragma unroll
      for (int j = 0; j < kKeys; ++j) x[j] = j < lim ? x[j] : -INFINITY;
    }
    float t[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
    for (int j = 4; j < kKeys; j += 8)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        t[k] = j + 4 + k < kKeys ? fmaxf(t[k], fmaxf(x[j + k], x[j + 4 + k])) : fmaxf(t[k], x[j + k]);
    const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * s.c;
    if (__builtin_expect(__any_sync(0xFFFFFFFFu, top > mu + R::kGrow), 0)) {
      // Only the rows that have grown: with the others' references a row's roundings would depend
      // on keys that it does not see, and on the queries behind the sequence's last.
      const bool up = top > mu + R::kGrow;
      const float mn = up ? ceilf(top) - R::kTop : mu;
      const float f = up ? ex2(mu - mn) : 1.0f;
      l = l == 0.0f ? 0.0f : l * f;  // (a NaN stays)
      d *= f;
      mu = mn;
      if (kt > 0) {
        if (!wait(L::kPvDone + 2 * s.tile + ((s.n - 1) & 1), (s.n - 1) >> 1)) return false;
        tc::fence_after_sync();
#pragma unroll 1
        for (int k = 0; k < kV; k += 16) {
          uint32_t y[16];
          tc::ld_32x16(s.o_at + k, y);
#pragma unroll
          for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * f);
          tc::st_32x16(s.o_at + k, y);
        }
        tc::wait_st();
      }
    }
    const float m0 = mu == -INFINITY ? 0.0f : -mu;
    const uint64_t c2 = f2(s.c, s.c), m2 = f2(m0, m0);
    uint64_t sum[2] = {0, 0};
    uint32_t* pk = reinterpret_cast<uint32_t*>(x);
#pragma unroll
    for (int j = 0; j < kKeys / 2; ++j) {
      const float2 y = unf2(fma2(f2(x[2 * j], x[2 * j + 1]), c2, m2));
      const float p0 = ex2(y.x), p1 = ex2(y.y);
      sum[j & 1] = add2(sum[j & 1], f2(p0, p1));
      pk[j] = pack16x2<F>(p0, p1);
    }
    // the weights before these are read
    if (kt > 0 && !wait(L::kPvDone + 2 * s.tile + ((s.n - 1) & 1), (s.n - 1) >> 1)) return false;
    tc::fence_after_sync();
    tc::st_32x32(s.p_at, pk);
    const float2 s2 = unf2(add2(sum[0], sum[1]));
    l += s2.x + s2.y;
    if (__builtin_expect(cut && s.head && kt == 0, 0)) {
      float r0 = 0.0f, r1 = 0.0f;
#pragma unroll
      for (int j = 0; j < kKeys / 2; ++j) {
        r0 += x16lo<F>(pk[j]);
        r1 += x16hi<F>(pk[j]);
      }
      d += (r0 - s2.x) + (r1 - s2.y);
    }
    // (before the weights are handed on, without which no note is written over)
    if (__builtin_expect(kt >= s.from, 0)) {
      const uint32_t nc = s.cleaned + kt - s.from, flags = s.smem + L::flags + ((s.g + kt) & (kLooks - 1)) * 16;
      if (!wait(L::kClean + (nc & (kLooks - 1)), nc / kLooks)) return false;
      const uint4 f = lds16(flags);
      if constexpr (L::kF8) {
        if (__builtin_expect((f.x | f.y | f.z | f.w) != 0, 0))
#pragma unroll 1
          for (int k = 0; k < kKeys; ++k)
            if (k < lim && lds_u8(flags + (k >> 2)) >> (k & 3) & 1) l = NAN;
      } else if (__builtin_expect((f.x | f.y) != 0, 0)) {
        const uint64_t bits = (uint64_t)f.y << 32 | f.x;
        if (lim > 0 && bits << (kKeys - min(lim, kKeys))) l = NAN;
      }
    }
    tc::wait_st();
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + 8 * (L::kPFull + 2 * s.tile + (s.n & 1)));
  }
  mu_out = mu;
  l_out = l;
  d_out = d;
  return true;
}

__device__ __forceinline__ void st32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Weights and output of one query tile; a thread has a row.
template <int F, int QF, int KF>
__device__ __forceinline__ void softmax_role(const PrefillArgs& a, bool boxes, uint32_t smem, uint32_t tmem,
                                             const Waiter& waiter, int tile, int w4, int lane,
                                             const Workspace& ws, int srows) {
  using L = Lay<KF>;
  const uint32_t bars = smem + L::bars;
  const uint32_t s_at = tmem + tile * kKeys + ((uint32_t)(w4 * 32) << 16);
  const uint32_t p_at = tmem + kP + tile * (kKeys / 2) + ((uint32_t)(w4 * 32) << 16);
  const uint32_t o_at = tmem + kO + tile * kV + ((uint32_t)(w4 * 32) << 16);
  const int r = w4 * 32 + lane;
  uint32_t n = 0, g = 0, cleaned = 0, opened = 0;
  const float ks = L::kF8 ? __ldg(a.kv_scale) : 1.0f, scale = fabsf(a.softmax_scale * ks) * kLog2e;
  Items<KF> items{smem, 0};
  Item it;
  // The queries' place is free when the item's last scores have come: those of the next item are
  // asked for before the output of this one is written.
  auto queries = [&] {
    Item nxt;
    if (!boxes && items.get(waiter, nxt, true) && nxt.end_of(tile) > nxt.kb)
      load_queries<KF>(a, nxt, smem, tile, w4, lane);
  };
  queries();
#pragma unroll 1
  while (items.get(waiter, it)) {
    const int count = max(it.end_of(tile) - it.kb, 0), mine = it.rows - tile * kM;
    const bool live = w4 * 32 < mine, ok = r < mine;
    const uint32_t row = it.row0 + tile * kM + r;
    const int seen = ok ? seen_of(a, it.base, it.m, row) : 0, shift = it.kb * kKeys;
    float c = scale, mu, l, d;
    if constexpr (F != QF) {
      if (count > 0) {
        if (!__all_sync(0xFFFFFFFFu, waiter(bars + 8 * (L::kQFull + tile), opened++ & 1))) return;
        c *= narrow_row(smem + L::q + tile * kQTile + r * 128, r & 7);
        tc::fence_smem_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + 8 * (L::kQReady + tile));
      }
    }
    // (a masked score times it is -infinity, also where a row that sees nothing asks with a NaN)
    c = c < 1e-37f || seen <= shift ? 1e-37f : c;
    if (!unit_weights<F, KF>(Part{smem, s_at, p_at, o_at, n, g, cleaned, tile, count,
                                  it.ragged() - it.kb, seen - shift, live, it.kb == 0, c},
                             waiter, mu, l, d))
      return;
    n += count;
    g += it.ke - it.kb;
    cleaned += it.cleaned();
    queries();
    // ---- the end of this CTA's part of the item
    // (what needs no sums, while the last of them are added up)
    const bool whole = it.kb == 0 && it.ke == it.tiles;
    const float inv = l == 0.0f ? 0.0f : __fdividef(ks, l + d);
    uint8_t* to;  // where the row goes
    if (whole) {
      const uint32_t dt = a.by_group(row), t = it.t0 + dt, h = it.head * a.group + (row - dt * a.group);
      to = a.out + t * a.out_ts + h * a.out_hs;
      if (ok && a.lse) a.lse[t * a.lse_ts + h * a.lse_hs] = l == 0.0f ? -INFINITY : (mu + __log2f(l)) * kLn2;
    } else {
      const uint32_t slot = (2 * blockIdx.x + (it.kb == 0 ? 1 : 0)) * srows, at = slot + tile * kM + r;
      to = reinterpret_cast<uint8_t*>(ws.o + (int64_t)slot * kV + (tile * kM + r) * 4);  // [dims / 4][rows][4]
      if (ok) {
        ws.m[at] = mu;
        ws.l[at] = l;
        ws.d[at] = d;
      }
    }
    if (count > 0) {
      if (!__all_sync(0xFFFFFFFFu, waiter(bars + 8 * (L::kPvDone + 2 * tile + ((n - 1) & 1)), ((n - 1) >> 1) & 1))) return;
      tc::fence_after_sync();
    }
    if (count > 0 && live) {
#pragma unroll 1
      for (int k = 0; k < kV; k += 32) {
        uint32_t y[32];
        tc::ld_32x32(o_at + k, y);
        if (ok && whole) {
          uint32_t z[16];
#pragma unroll
          for (int j = 0; j < 16; ++j)
            z[j] = pack16x2<QF>(__uint_as_float(y[2 * j]) * inv, __uint_as_float(y[2 * j + 1]) * inv);
          if (a.out_32) {
            st32(to, z);
            st32(to + 32, z + 8);
          } else {
#pragma unroll
            for (int j = 0; j < 16; j += 4) st16(to + 4 * j, make_uint4(z[j], z[j + 1], z[j + 2], z[j + 3]));
          }
          to += 64;
        } else if (ok) {
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            st16(to, make_uint4(y[j], y[j + 1], y[j + 2], y[j + 3]));
            to += (int64_t)srows * 16;
          }
        }
      }
    }
  }
}

// ------------------------------------------------------------------ the kernel
// After giving up: waits, bounded again, for the copies into shared memory (keys, values and the
// queries' boxes; another CTA may own it next), and a millisecond for matrix products in flight
// (they end by themselves within microseconds).
template <int KF>
__device__ __noinline__ void settle(uint32_t smem, uint32_t issued, uint32_t filled0, uint32_t filled1,
                                    uint64_t limit) {
  using L = Lay<KF>;
  const uint64_t since = global_ns();
  auto past = [&](int bar, uint32_t phase) {
    while (!mbar_try_wait(smem + L::bars + 8 * bar, phase & 1) && global_ns() - since <= limit) {
    }
  };
  if constexpr (L::kF8) {
    for (uint32_t u = issued > L::kRawStages ? issued - L::kRawStages : 0; u < issued; ++u)
      past(L::kRawFull + u % L::kRawStages, u / L::kRawStages);
  } else {
    for (uint32_t i = issued > 2 * L::kStages ? issued - 2 * L::kStages : 0; i < issued; ++i)
      past((i & 1 ? L::kVFull : L::kKFull) + (i >> 1) % L::kStages, (i >> 1) / L::kStages);
  }
  if (filled0 > 0) past(L::kQFull, filled0 - 1);
  if (filled1 > 0) past(L::kQFull + 1, filled1 - 1);
  while (global_ns() - since <= 1000000) {
  }
}

template <int F, int QF, int KF>
__global__ void __launch_bounds__(warps_of(KF) * 32, 1)
    prefill_attention_kernel(const PrefillArgs a, const __grid_constant__ Maps maps) {
  using L = Lay<KF>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t smem = smem_addr(smem_raw);
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  Misc& m = *reinterpret_cast<Misc*>(smem_raw + L::misc);
  pdl_trigger();
  if (threadIdx.x == 0) m.abort = 0;
  if (warp == 0) {
    // arrivals of a phase, by barrier
    for (int i = lane; i < L::kBars; i += 32) {
      auto of = [&](int bar, int many) { return i >= bar && i < bar + many; };
      int n = of(L::kKEmpty, 2 * L::kStages) ? 2 : 1;
      if (L::kF8 && (of(L::kKFull, 2 * L::kStages) || of(L::kRawEmpty, L::kRawStages) || of(L::kClean, kLooks)))
        n = kWideWarps;
      if (!L::kF8 && of(L::kClean, kLooks)) n = 2;
      if (of(L::kQFull, 2) && maps.q_tokens == 0) n = kM;
      if (of(L::kSFree, 2) || of(L::kPFull, 4) || of(L::kQReady, 2)) n = 4;
      if (of(L::kItemFree, kItems)) n = warps_of(KF) - 1;
      // (testing: one arrival too many)
      if (blockIdx.x == 0 && i < 2 * L::kStages && a.stall_stage == i + 1) ++n;
      mbar_init(smem + L::bars + 8 * i, n);
    }
    mbar_fence_init();
  }
  if (warp == kLoadWarp && lane < (maps.q_tokens != 0 ? 5 : 3))
    tc::prefetch_map(reinterpret_cast<const CUtensorMap*>(&maps) + lane);
  const Waiter wait{smem_addr(&m.abort), a.wait_limit_ns};
  pdl_wait();
  if (warp == kScoreWarp) tc::alloc(smem_addr(&m.tmem), kTmem);
  const int srows = slot_rows(a.num_tokens, a.group);
  const Workspace ws = workspace_of(a.workspace, gridDim.x, srows);
  if (threadIdx.x == kLoadWarp * 32) ws.split[blockIdx.x] = Split{};
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, m.tmem, 0);
  uint32_t errbits = 0, issued = 0, filled[2] = {0, 0};
  if (warp < kScoreWarp) {
    softmax_role<F, QF, KF>(a, maps.q_tokens != 0, smem, tmem, wait, warp >> 2, warp & 3, lane, ws, srows);
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp < kOutWarp) {
    score_role<F, QF, KF>(L::kF8 ? a.softmax_scale * __ldg(a.kv_scale) : a.softmax_scale, smem, tmem, wait, warp - kScoreWarp);
  } else if (warp < kLoadWarp) {
    output_role<F, KF>(smem, tmem, wait, warp - kOutWarp);
  } else if (warp == kLoadWarp) {
    issued = a.few_units ? load_role<KF, int32_t>(a, maps, smem_raw, smem, wait, lane, ws, errbits, filled)
                         : load_role<KF, int64_t>(a, maps, smem_raw, smem, wait, lane, ws, errbits, filled);
  } else {
    if constexpr (L::kF8) widen_role<KF>(smem, wait, warp - kWideWarp, lane);
  }
  __syncwarp();
  if (a.err && warp == kLoadWarp) {
    errbits = __reduce_or_sync(0xFFFFFFFFu, errbits);
    if (lane == 0 && errbits) atomicOr(a.err, errbits);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (__builtin_expect(wait.given_up(), 0)) {
    if (warp == kLoadWarp) settle<KF>(smem, issued, filled[0], filled[1], a.wait_limit_ns);
    if (threadIdx.x == 0 && a.err) atomicOr(a.err, kErrTimeout);
    __syncthreads();
  }
  if (warp == kScoreWarp) tc::dealloc(tmem, kTmem);
}

// -------------------------------------------------------- join of the split items
// Block (x, c) looks at what CTA c left.  An item of `parts` CTAs is dealt to the warps of the
// blocks of all of them but the last: 8 rows x 32 dims a warp, a lane two times four dims of a
// row.
constexpr int kJoinWarps = 8, kJoinBlocks = 16;

template <int QF>
__global__ void __launch_bounds__(kJoinWarps * 32) prefill_join_kernel(const PrefillArgs a) {
  pdl_trigger();
  pdl_wait();
  const int srows = slot_rows(a.num_tokens, a.group);
  const Workspace ws = workspace_of(a.workspace, gridDim.y, srows);
  const Split sp = ws.split[blockIdx.y];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stride = (sp.parts - 1) * kJoinBlocks * kJoinWarps;
  for (int n = (((int)blockIdx.y - sp.first) * kJoinBlocks + (int)blockIdx.x) * kJoinWarps + warp;
       n < (sp.rows + 7) / 8 * 4; n += stride) {
    const int r = (n >> 2) * 8 + (lane & 7), quad = (n & 3) * 8 + (lane >> 3);  // and quad + 4
    if (r >= sp.rows) continue;
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    float sum = 0.0f, more = 0.0f, top = -INFINITY;
    // the first partial lies in the odd slot of the first CTA, the others in the even ones behind
    constexpr int kAtOnce = 4;
#pragma unroll 1
    for (int i = 0; i < sp.parts; i += kAtOnce) {
      float4 v[kAtOnce][2];
      float lv[kAtOnce], dv[kAtOnce], mv[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int64_t slot = 2 * (int64_t)(sp.first + i + k) + (i + k == 0 ? 1 : 0);
        lv[k] = 0.0f;
        if (i + k < sp.parts) {
          lv[k] = ws.l[slot * srows + r];
          dv[k] = ws.d[slot * srows + r];
          mv[k] = ws.m[slot * srows + r];
          const float4* o = reinterpret_cast<const float4*>(ws.o + slot * srows * kV) + r;
          v[k][0] = __ldcs(o + quad * srows);
          v[k][1] = __ldcs(o + (quad + 4) * srows);
        }
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        if (lv[k] == 0.0f) continue;  // nothing seen there (and perhaps nothing written)
        const float m = fmaxf(top, mv[k]), m0 = m == -INFINITY ? 0.0f : m;
        const float f = ex2(top - m0), w = ex2(mv[k] - m0);
        const float x[8] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w,
                            v[k][1].x, v[k][1].y, v[k][1].z, v[k][1].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = fmaf(acc[j], f, w * x[j]);
        sum = fmaf(sum, f, w * lv[k]);
        more = fmaf(more, f, w * dv[k]);
        top = m;
      }
    }
    const uint32_t row = sp.row0 + r, dt = a.by_group(row);
    const int64_t t = sp.tok0 + (int)dt, h = (int64_t)sp.head * a.group + (int)(row - dt * a.group);
    const float ks = a.kv_scale ? __ldg(a.kv_scale) : 1.0f;
    const float inv = sum == 0.0f ? 0.0f : __fdividef(ks, sum + more);
    uint8_t* out = a.out + t * a.out_ts + h * a.out_hs + quad * 8;
#pragma unroll
    for (int j = 0; j < 8; j += 4)
      st8(out + j * 8, make_uint2(pack16x2<QF>(acc[j] * inv, acc[j + 1] * inv),
                                  pack16x2<QF>(acc[j + 2] * inv, acc[j + 3] * inv)));
    if (quad == 0 && a.lse)
      a.lse[t * a.lse_ts + h * a.lse_hs] = sum == 0.0f ? -INFINITY : (top + __log2f(sum)) * kLn2;
  }
}

// ------------------------------------------------------------------ launches
// Rows of keys (or values) of all heads as a tensor map with boxes of 64 columns (fp8: all)
// and 64 rows.  Heads inside a row are columns of it, so that any head stride does; otherwise (heads
// apart, or more columns than 31 bits count) the third dimension.  `base` stands in for arrays
// without rows.
bool make_map(CUtensorMap* map, const void* base, int fmt, int width, int64_t hs, int heads, int64_t ts,
              int64_t rows, int32_t* x_head, int32_t* z_head) {
  const TensorMapEncode encode = tensor_map_encode();
  if (!encode) return false;
  const int es = is16(fmt) ? 2 : 1;
  *x_head = *z_head = 0;
  const int64_t flat = (heads - 1) * hs + (int64_t)width * es;
  cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)rows, 1};
  // (strides of dimensions of one are not used, and may be anything)
  cuuint64_t strides[2] = {(cuuint64_t)(rows > 1 ? ts : width * es), 0};
  strides[1] = strides[0];
  if (heads > 1 && hs > 0) {
    if ((rows <= 1 || flat <= ts) && flat / es <= INT32_MAX) {
      dims[0] = (cuuint64_t)(flat / es);
      *x_head = (int32_t)(hs / es);
      if (rows <= 1) strides[0] = strides[1] = (cuuint64_t)((flat + 15) / 16 * 16);
    } else {
      dims[2] = (cuuint64_t)heads;
      strides[1] = (cuuint64_t)hs;
      *z_head = 1;
    }
  }
  const cuuint32_t box[3] = {is16(fmt) ? 64u : (cuuint32_t)width, kKeys, 1}, unit[3] = {1, 1, 1};
  const CUtensorMapDataType type = fmt == kBF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                   : fmt == kF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  return encode(map, type, 3, const_cast<void*>(base), dims, strides, box, unit,
                CU_TENSOR_MAP_INTERLEAVE_NONE, is16(fmt) ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries of a tile as boxes of 64 columns x the key head's query heads x tokens; 0 tokens
// where there is no such box.
int query_maps(const PrefillArgs& a, int fmt, Maps* maps) {
  const TensorMapEncode encode = tensor_map_encode();
  if (!encode || kM % a.group != 0) return 0;
  const cuuint32_t box[3] = {64, (cuuint32_t)a.group, (cuuint32_t)(kM / a.group)}, unit[3] = {1, 1, 1};
  const CUtensorMapDataType type =
      fmt == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  auto make = [&](CUtensorMap* map, const uint8_t* base, int width, int64_t hs, int64_t ts) {
    // (strides of dimensions of one are not used, and may be anything)
    if (a.num_heads == 1) hs = 16 * width;
    if (a.num_tokens == 1) ts = 16 * width;
    if (hs <= 0 || ts <= 0 || hs >= (int64_t(1) << 40) || ts >= (int64_t(1) << 40)) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)a.num_heads, (cuuint64_t)a.num_tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)hs, (cuuint64_t)ts};
    return encode(map, type, 3, const_cast<uint8_t*>(base), dims, strides, box, unit,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  return make(&maps->qn, a.q_nope, 128, a.qn_hs, a.qn_ts) && make(&maps->qp, a.q_pe, 64, a.qp_hs, a.qp_ts)
             ? kM / a.group
             : 0;
}

template <int F, int QF, int KF>
cudaError_t launch_tc(PrefillArgs a, int ctas, const LaunchCfg& cfg) {
  Maps maps = {};
  const bool none = a.num_kv == 0;
  const int64_t rows = none ? 1 : a.num_kv;
  const int heads = none ? 1 : a.kv_heads;
  if (!make_map(&maps.kn, none ? a.q_nope : a.k_nope, KF, 128, a.kn_hs, heads, a.kn_ts, rows,
                &maps.kn_x, &maps.kn_z) ||
      !make_map(&maps.kp, none ? a.q_nope : a.k_pe, KF, 64, a.kp_hs, heads, a.kp_ts, rows,
                &maps.kp_x, &maps.kp_z) ||
      !make_map(&maps.v, none ? a.q_nope : a.v, KF, 128, a.v_hs, heads, a.v_ts, rows,
                &maps.v_x, &maps.v_z))
    return cudaErrorInvalidValue;
  maps.q_tokens = query_maps(a, QF, &maps);
  a.out_32 = ((reinterpret_cast<uintptr_t>(a.out) | (uintptr_t)a.out_ts | (uintptr_t)a.out_hs) & 31) == 0;
  const int64_t full = ((int64_t)a.num_tokens * a.group + kItemRows - 1) / kItemRows;
  const int64_t items = (full + a.num_seqs) * a.kv_heads;
  // (every sequence taken as long as all: whatever the offsets hold, the count does not overflow)
  a.few_units = full * a.num_seqs * a.kv_heads < INT32_MAX / (a.num_kv / kKeys + 2 + kSwitch);
  a.whole = items <= ctas && a.num_kv <= kWholeKeys;
  auto kern = prefill_attention_kernel<F, QF, KF>;
  // the attribute stays with the device's context: set on a device's first call
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(set.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<KF>::bytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) set.fetch_or(uint64_t(1) << dev);
  }
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(ctas);
  lc.blockDim = dim3(warps_of(KF) * 32);
  lc.dynamicSmemBytes = Lay<KF>::bytes;
  lc.stream = cfg.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = cfg.pdl ? 1 : 0;
  e = cudaLaunchKernelEx(&lc, kern, a, maps);
  if (e != cudaSuccess || a.whole) return e;
  lc.gridDim = dim3(kJoinBlocks, ctas);
  lc.blockDim = dim3(kJoinWarps * 32);
  lc.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&lc, prefill_join_kernel<QF>, a);
}

}  // namespace

int64_t prefill_attention_workspace(int32_t num_tokens, int32_t num_heads, int32_t kv_heads, int32_t,
                                    int num_sms) {
  const int64_t ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
  return ctas * ((int64_t)sizeof(Split) +
                 2 * slot_rows(num_tokens, num_heads / kv_heads) * (3 + kV) * (int64_t)sizeof(float));
}

cudaError_t launch_prefill_attention(const PrefillArgs& a, int fmt, int kv_fmt, int num_sms,
                                     const LaunchCfg& cfg) {
  const int ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
  if (fmt == kBF16) {
    if (kv_fmt == kBF16) return launch_tc<kBF16, kBF16, kBF16>(a, ctas, cfg);
    return kv_fmt == kE4M3 ? launch_tc<kF16, kBF16, kE4M3>(a, ctas, cfg) : launch_tc<kF16, kBF16, kE5M2>(a, ctas, cfg);
  }
  if (kv_fmt == kF16) return launch_tc<kF16, kF16, kF16>(a, ctas, cfg);
  return kv_fmt == kE4M3 ? launch_tc<kF16, kF16, kE4M3>(a, ctas, cfg) : launch_tc<kF16, kF16, kE5M2>(a, ctas, cfg);
}

}  // namespace mla
