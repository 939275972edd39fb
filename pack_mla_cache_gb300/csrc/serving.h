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
};

// Rows of a query tile of the attention: the average rows (tokens x heads) per sequence
// decide.  fp8 tiles stop at 32: their split sums take three columns of tensor memory each.
// Measured: 16 rows per sequence 60.5 us in tiles of 16 (67.7 in tiles of 32; 64 ragged
// e4m3 decodes; in bf16 103.5 and 105.7), 32 bf16 rows 43.7 in tiles of 32 (57.5 in 16), 64
// e5m2 rows 48.2 in tiles of 32 (65.5 in 16), 128 bf16 rows 46.1 and 16384 rows 645 in tiles
// of 64 (61.9 and 1120 in 32).  One size for the whole call: a chunk of 1024 tokens beside 63
// ragged decodes of 16 heads takes 444 us in bf16 and 478 in e4m3 (334 + 101 and 420 + 59
// apart), one of 2048 beside 255 decodes of one head, in tiles of 16, 494 and 291 (62 + 371
// and 64 + 203 apart).
inline int attention_tile_rows(int32_t num_tokens, int32_t num_heads, int32_t num_seqs, bool fp8) {
  const int64_t rows = ((int64_t)num_tokens + num_seqs - 1) / num_seqs * num_heads;
  return rows <= 16 ? 16 : rows <= 32 || fp8 ? 32 : 64;
}

cudaError_t launch_copy_blocks(const CopyBlocksArgs& a, const LaunchCfg& cfg);
// fmt: kBF16, kF16 or kF32.
cudaError_t launch_merge(const MergeArgs& a, int fmt, const LaunchCfg& cfg);
cudaError_t launch_latent_attention(const LatentAttnArgs& a, int cache_fmt, int num_sms,
                                    const LaunchCfg& cfg);
// Bytes of workspace of such a call on a device of num_sms SMs.
int64_t latent_attention_workspace(int32_t num_tokens, int32_t num_heads, int32_t num_seqs,
                                   int num_sms);

}  // namespace mla
