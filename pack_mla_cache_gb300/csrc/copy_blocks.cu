// copy_blocks.cu -- copy, fork or clear blocks of every layer's paged cache in
// one launch (the block layout and the per-layer pointer array of the grouped
// insert, "PR #55356 [Kimi Perf] Group fp8 mla cache insertion").
//
// What it computes: rows [0, n) of block dst become those of block src, or
// zeros.  Bound by HBM: every byte is read once and written once.
//
// Design: a warp takes one item = a run of 4 x 32 16-byte chunks of one (copy,
// layer), all four loads of a lane issued before its stores.  Items of a copy
// are consecutive, so neighbouring warps stream neighbouring addresses, and a
// call of a few blocks still spreads over many SMs (one 36 KB fp8 block = 18
// items).  When entries are contiguous a block's rows are one run; otherwise a
// chunk's row and column come from one 32-bit division.
//
// Measured (64 x 576 blocks in 5 layers): 1024 bf16 blocks 122 us (6.2 TB/s), 512 e5m2
// forks of random row counts 17.4 us, 4 e4m3 forks 2.3 us.
#include "mla_device.cuh"
#include "serving.h"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kChunks = 4;              // 16-byte chunks per lane
constexpr int kItem = 32 * kChunks;     // chunks per item

__global__ void __launch_bounds__(kThreads) copy_blocks_kernel(const CopyBlocksArgs a) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const uint32_t block_chunks = (uint32_t)a.block_size * (uint32_t)a.row_chunks;
  const uint32_t pieces = (block_chunks + kItem - 1) / kItem;  // items per (copy, layer)
  const int64_t items = (int64_t)a.num_copies * a.num_layers * pieces;
  const int64_t nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
  uint32_t errbits = 0;
  for (int64_t it = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; it < items;
       it += nwarps) {
    const int64_t cl = it / pieces;
    const uint32_t piece = (uint32_t)(it - cl * pieces);
    const int32_t c = (int32_t)(cl / a.num_layers);
    const int32_t l = (int32_t)(cl - (int64_t)c * a.num_layers);
    const int32_t src = a.src[c], dst = a.dst[c];
    const int32_t n = a.rows ? a.rows[c] : a.block_size;
    const int64_t base = a.cache_ptrs[l];
    if (dst == -1 || n == 0) continue;  // padding
    if (src < -1 || dst < -1 || src >= a.num_blocks || dst >= a.num_blocks || n < 0 ||
        n > a.block_size) {
      errbits |= kErrBlockOOB;
      continue;
    }
    if (base == 0 || (base & 15)) {
      errbits |= kErrMisaligned;
      continue;
    }
    if (src == dst) continue;
    const uint32_t total = (uint32_t)n * (uint32_t)a.row_chunks;  // chunks to move
    const uint32_t c0 = piece * kItem + lane;
    const uint8_t* from = reinterpret_cast<const uint8_t*>(base) + (int64_t)src * a.block_stride;
    uint8_t* to = reinterpret_cast<uint8_t*>(base) + (int64_t)dst * a.block_stride;
    uint4 v[kChunks];
    int64_t off[kChunks];
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      const uint32_t ch = c0 + 32 * k;
      v[k] = make_uint4(0, 0, 0, 0);
      if (a.dense) {
        off[k] = (int64_t)ch * 16;
      } else {
        const uint32_t row = ch / (uint32_t)a.row_chunks;
        off[k] = (int64_t)row * a.entry_stride + (int64_t)(ch - row * a.row_chunks) * 16;
      }
      if (src >= 0 && ch < total) v[k] = ld_stream16(from + off[k]);
    }
#pragma unroll
    for (int k = 0; k < kChunks; ++k)
      if (c0 + 32 * k < total) st16(to + off[k], v[k]);
  }
  errbits = __reduce_or_sync(0xFFFFFFFFu, errbits);
  if (errbits && lane == 0 && a.err) atomicOr(a.err, errbits);
}

}  // namespace

cudaError_t launch_copy_blocks(const CopyBlocksArgs& a, const LaunchCfg& cfg) {
  const int64_t pieces = ((int64_t)a.block_size * a.row_chunks + kItem - 1) / kItem;
  const int64_t items = (int64_t)a.num_copies * a.num_layers * pieces;
  const int64_t ctas = (items + kThreads / 32 - 1) / (kThreads / 32);
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(capped_grid(reinterpret_cast<const void*>(copy_blocks_kernel), kThreads, ctas));
  lc.blockDim = dim3(kThreads);
  lc.stream = cfg.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = cfg.pdl ? 1 : 0;
  return cudaLaunchKernelEx(&lc, copy_blocks_kernel, a);
}

}  // namespace mla
