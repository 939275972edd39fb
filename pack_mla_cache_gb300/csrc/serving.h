// Internal (not installed): launch interfaces of the operators that a serving loop
// runs next to the data movement (attention over the cache, merge, block copies).
#pragma once

#include "mla_internal.h"

namespace mla {

constexpr int kF32 = 4;  // beside the formats of Fmt: fp32 (merge only)

// Block copies over the layers' caches (bytes; a row = the copied part of an entry).
struct CopyBlocksArgs {
  const int64_t* cache_ptrs;
  int32_t num_layers;
  int64_t num_blocks, block_stride, entry_stride;
  int32_t block_size;
  int32_t row_chunks;  // 16-byte chunks of a row
  bool dense;          // entry_stride == row bytes: a block's rows are one run
  const int32_t* src;
  const int32_t* dst;
  const int32_t* rows;  // may be null (block_size)
  int32_t num_copies;
  uint32_t* err;
};

// Division by an invariant d >= 1 using multiplication (Granlund and Montgomery,
// PLDI 1994): shift = ceil(log2 d), mul = floor(2^32 (2^shift - d) / d) + 1; exact
// for n < 2^31 (the sum below stays in 32 bits).
struct Divider {
  uint32_t mul, shift;
  static Divider by(uint32_t d) {
    Divider r{0, 0};
    while ((uint64_t(1) << r.shift) < d) ++r.shift;
    r.mul = (uint32_t)((((uint64_t(1) << r.shift) - d) << 32) / d + 1);
    return r;
  }
#ifdef __CUDACC__
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
    return (__umulhi(n, mul) + n) >> shift;
  }
#endif
};

// Join of partial attention results (bytes; lse strides in elements).
struct MergeArgs {
  const uint8_t* parts;
  int64_t ps, ts, hs;
  const float* lse;
  int64_t lps, lts, lhs;
  int32_t num_parts, num_tokens, num_heads;
  int32_t row_chunks;  // 16-byte chunks of a row
  Divider by_units, by_heads;  // by_units (of a row) set by the launch
  float shift;                 // log2 of the weights' scale, set by the launch
  uint8_t* out;
  int64_t ots, ohs;
  float* lse_out;  // may be null
  int64_t lots, lohs;
};

// Attention over the paged latent cache (bytes; lse strides in elements).
struct LatentAttnArgs {
  const uint8_t* q_c;
  int64_t qc_ts, qc_hs;
  const uint8_t* q_pe;
  int64_t qp_ts, qp_hs;
  int32_t num_tokens, num_heads;
  Divider by_heads;
  const uint8_t* cache;
  int64_t block_stride, entry_stride, num_blocks;
  int32_t block_size, bs_shift;  // bs_shift = log2(block_size) or -1
  int32_t box_rows;              // entries of a TMA box (set by the launch), 0 = row copies
  int32_t box_shift;             // log2 of the boxes that a key tile's column of entries takes
  bool stream_rows;              // cache rows leave L2 first (set by the launch)
  const int32_t* block_table;
  int64_t bt_stride;  // elements
  int32_t room;       // rows that a table row can hold (below 2^31 - 127)
  const int32_t* cu_q;
  const int32_t* kv_lens;
  int32_t num_seqs;
  float softmax_scale;
  const float* k_scale;  // fp8 caches only
  bool causal;
  uint8_t* out;
  int64_t out_ts, out_hs;
  float* lse;  // may be null
  int64_t lse_ts, lse_hs;
  uint8_t* workspace;
  uint32_t* err;
  uint64_t wait_limit_ns;
  int32_t stall_stage;  // testing: this pipeline stage (from 1) of CTA 0 never fills
  const uint32_t* tree;  // trees only: ancestor bits, tree_words words a token
  int64_t tree_ts;       // words
  uint32_t tree_words;   // at most kMaxTree / 32
};

// Drafted tokens that a tree's masks can name.
constexpr int kMaxTree = 32768;

// Accepted rows moved to the front of the drafted ones (bytes; a row = the moved part of an
// entry).
struct CompactArgs {
  const int64_t* cache_ptrs;
  int32_t num_layers;
  int64_t num_blocks, block_stride, entry_stride;
  int32_t block_size;
  Divider by_block;
  int32_t row_chunks;  // 16-byte chunks of a row
  const int32_t* block_table;
  int64_t bt_stride;  // elements
  int32_t room;       // rows that a table row can hold (below 2^31)
  const int32_t* starts;
  const int32_t* rows;
  int64_t rows_stride;  // elements
  int32_t width;        // of a list in rows
  const int32_t* counts;
  int32_t num_seqs;
  uint32_t* err;
};
// The longest list of accepted rows.
constexpr int kMaxAccepted = 1024;

// Attention of packed sequences over keys and values per head (bytes; lse strides in
// elements).
struct PrefillArgs {
  const uint8_t* q_nope;
  int64_t qn_ts, qn_hs;
  const uint8_t* q_pe;
  int64_t qp_ts, qp_hs;
  int32_t num_tokens, num_heads;
  const uint8_t* k_nope;
  int64_t kn_ts, kn_hs;
  const uint8_t* k_pe;
  int64_t kp_ts, kp_hs;  // kp_hs 0: one rotary row for all heads
  const uint8_t* v;
  int64_t v_ts, v_hs;
  int32_t num_kv, kv_heads;
  int32_t group;  // query heads of a key head
  Divider by_group;
  const int32_t* cu_q;
  const int32_t* cu_kv;
  int32_t num_seqs;
  float softmax_scale;
  const float* kv_scale;  // fp8 keys and values only
  bool causal;
  // (set by the launch) units are counted in 32 bits; out rows on 32-byte boundaries; an item a CTA
  bool few_units, out_32, whole;
  uint8_t* out;
  int64_t out_ts, out_hs;
  float* lse;  // may be null
  int64_t lse_ts, lse_hs;
  uint8_t* workspace;
  uint32_t* err;
  uint64_t wait_limit_ns;
  int32_t stall_stage;  // testing: this pipeline stage (from 1) of CTA 0 never fills
};

// Rows of a query tile of the attention: the average rows (tokens x heads) per sequence
// decide.  fp8 tiles stop at 32: their split sums take three columns of tensor memory each.
// Measured: 16 rows per sequence 59.7 us in tiles of 16 (67.1 in tiles of 32; 64 ragged
// e4m3 decodes; in bf16 104.7 and 107.3), 32 bf16 rows 40.3 in tiles of 32 (55.6 in 16), 64
// e5m2 rows 45.3 in tiles of 32 (64.7 in 16), 128 bf16 rows 43.5 and 16384 rows 632 in tiles
// of 64 (56.5 and 1111 in 32).  One size for the whole call: a chunk of 1024 tokens beside 63
// ragged decodes of 16 heads takes 442 us in bf16 and 470 in e4m3 (327 + 101 and 412 + 58
// apart), one of 2048 beside 255 decodes of one head, in tiles of 16, 492 and 291 (56 + 370
// and 62 + 202 apart).
inline int attention_tile_rows(int32_t num_tokens, int32_t num_heads, int32_t num_seqs, bool fp8) {
  const int64_t rows = ((int64_t)num_tokens + num_seqs - 1) / num_seqs * num_heads;
  return rows <= 16 ? 16 : rows <= 32 || fp8 ? 32 : 64;
}

cudaError_t launch_copy_blocks(const CopyBlocksArgs& a, const LaunchCfg& cfg);
// fmt: kBF16, kF16 or kF32.
cudaError_t launch_merge(const MergeArgs& a, int fmt, const LaunchCfg& cfg);
cudaError_t launch_latent_attention(const LatentAttnArgs& a, int cache_fmt, int num_sms,
                                    const LaunchCfg& cfg);
cudaError_t launch_latent_tree_attention(const LatentAttnArgs& a, int cache_fmt, int num_sms,
                                         const LaunchCfg& cfg);
cudaError_t launch_compact_rows(const CompactArgs& a, const LaunchCfg& cfg);
// fmt: of the queries and the output (kBF16 or kF16); kv_fmt: of keys and values.
cudaError_t launch_prefill_attention(const PrefillArgs& a, int fmt, int kv_fmt, int num_sms,
                                     const LaunchCfg& cfg);
int64_t prefill_attention_workspace(int32_t num_tokens, int32_t num_heads, int32_t kv_heads,
                                    int32_t num_seqs, int num_sms);
// Bytes of workspace of such a call on a device of num_sms SMs.
int64_t latent_attention_workspace(int32_t num_tokens, int32_t num_heads, int32_t num_seqs,
                                   int num_sms);

}  // namespace mla
