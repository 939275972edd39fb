// latent_attention.cu -- attention of new tokens over the paged latent cache in
// the absorbed MLA form (include/mla_cache.h: mla_latent_attention).
//
// What it computes, per (token, head) row q of 576 elements and the cache rows
// r_p that the token sees: x_p = scale <q, r_p>, lse = ln sum exp(x_p), out =
// sum exp(x_p - lse) r_p[0:512].
//
// Design: one warp per (token, head).  Lane l holds query elements
// [16 l, 16 l + 16) and 512 + 2 l, 2 l + 1, so a row costs two (bf16) or one
// (fp8) 16-byte load, one 4- or 2-byte load and a warp sum; the running
// maximum and sum rescale the accumulator when the maximum grows.
#include "mla_device.cuh"
#include "mla_internal.h"
#include "paged.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;

template <int FMT>
__device__ __forceinline__ void load_row(const uint8_t* p, int lane, float* kv, float* pe) {
  uint4 a, b;
  uint32_t r;
  if constexpr (FMT == kBF16) {
    a = ld_shared_ro16(p + lane * 32);
    b = ld_shared_ro16(p + lane * 32 + 16);
    r = __ldg(reinterpret_cast<const uint32_t*>(p + 1024) + lane);
  } else {
    const uint4 v = ld_shared_ro16(p + lane * 16);
    a = fp8x8_to_x16x8<FMT, kBF16>(make_uint2(v.x, v.y));
    b = fp8x8_to_x16x8<FMT, kBF16>(make_uint2(v.z, v.w));
    r = fp8x2_to_bf16x2<FMT>(__ldg(reinterpret_cast<const uint16_t*>(p + 512) + lane));
  }
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    kv[2 * i] = bf16lo(w[i]);
    kv[2 * i + 1] = bf16hi(w[i]);
  }
  pe[0] = bf16lo(r);
  pe[1] = bf16hi(r);
}

template <int FMT>
__global__ void __launch_bounds__(kThreads) latent_attention_kernel(const LatentAttnArgs a) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)a.num_tokens * a.num_heads;
  const int64_t nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
  const float ks = FMT == kBF16 ? 1.0f : *a.k_scale;
  uint32_t errbits = 0;
  for (int64_t w = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; w < rows; w += nwarps) {
    const int64_t t = w / a.num_heads;
    const int32_t h = (int32_t)(w - t * a.num_heads);
    const int s = find_seq(a.cu_q, a.num_seqs, t);
    if (s < 0 || s >= a.num_seqs) continue;  // owned by no sequence
    int64_t seen = a.kv_lens[s];
    if (a.causal) seen += t + 1 - a.cu_q[s + 1];
    if (seen > a.room) {
      errbits |= kErrBlockOOB;
      seen = a.room;
    }
    float q[16], qr[2], kv[16], pe[2], acc[16];
    load_row<kBF16>(a.q_c + t * a.qc_ts + h * a.qc_hs, lane, q, pe);
    {
      const uint32_t r = __ldg(reinterpret_cast<const uint32_t*>(a.q_pe + t * a.qp_ts + h * a.qp_hs) + lane);
      qr[0] = bf16lo(r);
      qr[1] = bf16hi(r);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
    float m = -INFINITY, sum = 0.0f;
    for (int64_t p = 0; p < seen; ++p) {
      const int64_t kb = a.bs_shift >= 0 ? p >> a.bs_shift : p / a.block_size;
      const int32_t blk = a.block_table[s * a.bt_stride + kb];
      if (blk < 0 || blk >= a.num_blocks) {
        errbits |= kErrBlockOOB;
        continue;
      }
      load_row<FMT>(a.cache + blk * a.block_stride + (p - kb * a.block_size) * a.entry_stride,
                    lane, kv, pe);
      float d = qr[0] * pe[0] + qr[1] * pe[1];
#pragma unroll
      for (int i = 0; i < 16; ++i) d = fmaf(q[i], kv[i], d);
      const float x = warp_sum(d) * (a.softmax_scale * ks);
      const float mn = fmaxf(m, x);
      const float f = m == -INFINITY ? 0.0f : expf(m - mn), e = expf(x - mn);
      m = mn;
      sum = fmaf(sum, f, e);
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] = fmaf(acc[i], f, e * kv[i]);
    }
    const float inv = sum > 0.0f ? ks / sum : (sum == 0.0f ? 0.0f : NAN);
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = pack_bf16x2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    uint8_t* out = a.out + t * a.out_ts + h * a.out_hs + lane * 32;
    st16(out, make_uint4(o[0], o[1], o[2], o[3]));
    st16(out + 16, make_uint4(o[4], o[5], o[6], o[7]));
    if (a.lse && lane == 0)
      a.lse[t * a.lse_ts + h * a.lse_hs] = sum == 0.0f ? -INFINITY : m + logf(sum);
  }
  errbits = __reduce_or_sync(0xFFFFFFFFu, errbits);
  if (errbits && lane == 0 && a.err) atomicOr(a.err, errbits);
}

template <int FMT>
cudaError_t launch_t(const LatentAttnArgs& a, const LaunchCfg& cfg) {
  const int64_t rows = (int64_t)a.num_tokens * a.num_heads;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(capped_grid(reinterpret_cast<const void*>(latent_attention_kernel<FMT>),
                                kThreads, (rows + kThreads / 32 - 1) / (kThreads / 32)));
  lc.blockDim = dim3(kThreads);
  lc.stream = cfg.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = cfg.pdl ? 1 : 0;
  return cudaLaunchKernelEx(&lc, latent_attention_kernel<FMT>, a);
}

}  // namespace

int64_t latent_attention_workspace(int32_t, int32_t, int32_t, int) { return 16; }

cudaError_t launch_latent_attention(const LatentAttnArgs& a, int cache_fmt, const LaunchCfg& cfg) {
  switch (cache_fmt) {
    case kBF16: return launch_t<kBF16>(a, cfg);
    case kE4M3: return launch_t<kE4M3>(a, cfg);
    case kE5M2: return launch_t<kE5M2>(a, cfg);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mla
