// compact_rows.cu -- the rows of accepted drafted tokens moved to the front of the drafted
// ones in every layer's paged cache (include/mla_cache.h: mla_cache_compact_rows).
//
// What it computes: row start + i of a sequence becomes its row start + rows[i], for a
// strictly increasing list, so rows[i] >= i.  Bound by HBM and by the latency of the lists,
// the table and the rows behind them: every moved byte is read once and written once.
//
// Order.  A 16-byte column of the rows depends on that column alone, so a thread takes one
// (layer, column) of a sequence and walks the list in steps of kStep rows: all loads of a
// step, then its stores.  Stores of a step write rows below start + i + kStep, loads of the
// later ones read rows at or above that: nothing is read after it was overwritten.
//
// A block has the list, as byte offsets of its source and destination rows, in shared
// memory; blocks of one sequence check its whole list each, so that all of them skip a bad
// one.
//
// Measured (replayed from a graph): 5 rows of one sequence, 5 e4m3 layers, 2.4 us (a launch, and
// three loads that wait for one another); 1 to 9 rows of 512 sequences, 5 bf16 layers, 6.1 us
// (4.8 TB/s); 16 of 2048, 5 bf16 layers, 67.8 us (5.6 TB/s).
#include "mla_device.cuh"
#include "serving.h"

namespace mla {
namespace {

constexpr int kThreads = 128;
constexpr int kStep = 8;

__global__ void __launch_bounds__(kThreads) compact_rows_kernel(const CompactArgs a) {
  __shared__ int64_t from_s[kMaxAccepted], to_s[kMaxAccepted];
  __shared__ uint32_t bad_s;
  pdl_trigger();
  if (threadIdx.x == 0) bad_s = 0;
  pdl_wait();
  const uint32_t columns = (uint32_t)a.num_layers * (uint32_t)a.row_chunks;
  const uint32_t pieces = (columns + kThreads - 1) / kThreads;
  const uint32_t items = pieces * (uint32_t)a.num_seqs;
  for (uint32_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int s = (int)(it / pieces);
    const uint32_t col = (it - s * pieces) * kThreads + threadIdx.x;
    const int n = a.counts[s], start = a.starts[s];
    __syncthreads();  // the lists of the item before are read, bad_s is set
    uint32_t bad = n < 0 || n > a.width || (n > 0 && start < 0) ? kErrPosOOB : 0;
    if (!bad)
      for (int i = threadIdx.x; i < n; i += kThreads) {
        const int32_t* list = a.rows + (int64_t)s * a.rows_stride + i;
        const int r = list[0];
        if (r < 0 || (i > 0 && list[-1] >= r)) {
          bad |= kErrPosOOB;
          continue;
        }
        auto offset = [&](int64_t p) -> int64_t {
          if (p >= a.room) {
            bad |= kErrBlockOOB;
            return 0;
          }
          const uint32_t kb = a.by_block((uint32_t)p);
          const int32_t blk = a.block_table[(int64_t)s * a.bt_stride + kb];
          if (blk < 0 || blk >= a.num_blocks) bad |= kErrBlockOOB;
          return (int64_t)blk * a.block_stride + ((int64_t)p - (int64_t)kb * a.block_size) * a.entry_stride;
        };
        from_s[i] = offset((int64_t)start + r);
        to_s[i] = offset((int64_t)start + i);
      }
    if (bad) atomicOr(&bad_s, bad);
    __syncthreads();
    bad = bad_s;
    __syncthreads();
    if (threadIdx.x == 0) {
      if (bad && a.err) atomicOr(a.err, bad);
      bad_s = 0;
    }
    if (bad || n == 0 || col >= columns) continue;
    const int l = (int)(col / (uint32_t)a.row_chunks);
    const int64_t base = a.cache_ptrs[l];
    if (base == 0 || (base & 15)) {
      if (a.err) atomicOr(a.err, kErrMisaligned);
      continue;
    }
    uint8_t* at = reinterpret_cast<uint8_t*>(base) + (int64_t)(col - l * a.row_chunks) * 16;
    for (int i0 = 0; i0 < n; i0 += kStep) {
      uint4 v[kStep];
#pragma unroll
      for (int k = 0; k < kStep; ++k)
        if (i0 + k < n) v[k] = *reinterpret_cast<const uint4*>(at + from_s[i0 + k]);
#pragma unroll
      for (int k = 0; k < kStep; ++k)
        if (i0 + k < n && from_s[i0 + k] != to_s[i0 + k]) st16(at + to_s[i0 + k], v[k]);
    }
  }
}

}  // namespace

cudaError_t launch_compact_rows(const CompactArgs& a, const LaunchCfg& cfg) {
  const int64_t pieces = ((int64_t)a.num_layers * a.row_chunks + kThreads - 1) / kThreads;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(capped_grid(reinterpret_cast<const void*>(compact_rows_kernel), kThreads,
                                pieces * a.num_seqs));
  lc.blockDim = dim3(kThreads);
  lc.stream = cfg.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = cfg.pdl ? 1 : 0;
  return cudaLaunchKernelEx(&lc, compact_rows_kernel, a);
}

}  // namespace mla
