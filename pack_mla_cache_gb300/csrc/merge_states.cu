// merge_states.cu -- join attention results over disjoint parts of the context
// by their log-sum-exp (the end of the chunked-context loop, "PR #51772
// [Attention][MLA] Fuse Kimi-K3 chunked-context K/V packing", Implementation
// items 1-2, and of a shared prefix with each sequence's suffix).
//
// What it computes: with m = max_i lse_i and w_i = exp(lse_i - m),
//   out = sum_i w_i part_i / sum_i w_i,   lse = m + ln(sum_i w_i),
// in fp32, rounded once; a part with lse -inf has weight 0, whatever its row holds.
// Bound by HBM: every part is read once, the result written once.
//
// Design: a thread owns one 16-byte chunk of an output row.  The lse of its
// row are read twice (for m, then for the weights); the threads of a row read
// the same words, so the second pass and all but one thread's first hit L1.
// Parts are taken four at a time, their loads issued before their sums; the first
// four parts' before the lse are looked at.  Row, token and head of a chunk come
// from multiplications by reciprocals: 4 parts of 8192 x 16 rows of 128 bf16 take 30.3
// us (5.6 TB/s; 39 us with 64-bit divisions), 2 parts of 64 x 16 rows of 512 2.4 us.
#include "mla_device.cuh"
#include "serving.h"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // parts in flight per thread

template <int F>
__device__ __forceinline__ void add_weighted(uint4 v, float w, float* acc) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  if constexpr (F == kF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(w, __uint_as_float(u[i]), acc[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[2 * i] = fmaf(w, x16lo<F>(u[i]), acc[2 * i]);
      acc[2 * i + 1] = fmaf(w, x16hi<F>(u[i]), acc[2 * i + 1]);
    }
  }
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int F>
__global__ void __launch_bounds__(kThreads) merge_states_kernel(const MergeArgs a) {
  constexpr int kElts = F == kF32 ? 4 : 8;  // elements of a 16-byte chunk
  pdl_trigger();
  pdl_wait();
  const uint32_t chunks = (uint32_t)a.num_tokens * a.num_heads * a.row_chunks;  // < 2^31
  for (uint32_t u = blockIdx.x * kThreads + threadIdx.x; u < chunks; u += gridDim.x * kThreads) {
    const uint32_t row = a.by_chunks(u), ch = u - row * a.row_chunks;
    const uint32_t t = a.by_heads(row), h = row - t * a.num_heads;
    const float* lse = a.lse + (int64_t)t * a.lts + (int64_t)h * a.lhs;
    const uint8_t* src = a.parts + (int64_t)t * a.ts + (int64_t)h * a.hs + (int64_t)ch * 16;
    uint4 v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (k < a.num_parts) v[k] = ld_stream16(src + k * a.ps);
    float m = -INFINITY, bad = 0.0f;
    for (int i = 0; i < a.num_parts; ++i) {
      const float x = __ldg(lse + i * a.lps);
      if (!(x < INFINITY)) bad = NAN;  // +inf or NaN
      m = fmaxf(m, x);
    }
    const float m0 = m == -INFINITY ? 0.0f : m;
    float acc[kElts];
#pragma unroll
    for (int e = 0; e < kElts; ++e) acc[e] = 0.0f;
    float sum = 0.0f;
    for (int i0 = 0;; i0 += kBatch) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (i0 + k < a.num_parts) {
          const float x = __ldg(lse + (i0 + k) * a.lps);
          if (x != -INFINITY) {  // a part without weight has no influence, whatever it holds
            const float w = expf(x - m0);
            sum += w;
            add_weighted<F>(v[k], w, acc);
          }
        }
      }
      if (i0 + kBatch >= a.num_parts) break;
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (i0 + kBatch + k < a.num_parts) v[k] = ld_stream16(src + (i0 + kBatch + k) * a.ps);
    }
    const float inv = (sum > 0.0f ? __frcp_rn(sum) : 0.0f) + bad;
    uint4 o;
    if constexpr (F == kF32) {
      o = make_uint4(__float_as_uint(acc[0] * inv), __float_as_uint(acc[1] * inv),
                     __float_as_uint(acc[2] * inv), __float_as_uint(acc[3] * inv));
    } else if constexpr (F == kBF16) {
      o = make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                     pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
    } else {
      o = make_uint4(pack_f16x2(acc[0] * inv, acc[1] * inv), pack_f16x2(acc[2] * inv, acc[3] * inv),
                     pack_f16x2(acc[4] * inv, acc[5] * inv), pack_f16x2(acc[6] * inv, acc[7] * inv));
    }
    st16(a.out + (int64_t)t * a.ots + (int64_t)h * a.ohs + (int64_t)ch * 16, o);
    if (ch == 0 && a.lse_out)
      a.lse_out[(int64_t)t * a.lots + (int64_t)h * a.lohs] = m0 + logf(sum) + bad;
  }
}

template <int F>
cudaError_t launch_t(MergeArgs a, const LaunchCfg& cfg) {
  cudaLaunchConfig_t lc = {};
  lc.blockDim = dim3(kThreads);
  lc.stream = cfg.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = cfg.pdl ? 1 : 0;
  // chunk numbers stay below 2^31 - 2^24 (the last stride of the grid included): larger
  // calls, of many GiB, go in several launches
  const int64_t per_token = (int64_t)a.num_heads * a.row_chunks;
  const int64_t most = (INT32_MAX - (1 << 24)) / per_token, tokens = a.num_tokens;
  for (int64_t t0 = 0; t0 < tokens; t0 += most) {
    a.num_tokens = (int32_t)(tokens - t0 < most ? tokens - t0 : most);
    const int64_t chunks = a.num_tokens * per_token;
    lc.gridDim = dim3(capped_grid(reinterpret_cast<const void*>(merge_states_kernel<F>), kThreads,
                                  (chunks + kThreads - 1) / kThreads));
    const cudaError_t e = cudaLaunchKernelEx(&lc, merge_states_kernel<F>, a);
    if (e != cudaSuccess) return e;
    a.parts += most * a.ts;
    a.lse += most * a.lts;
    a.out += most * a.ots;
    if (a.lse_out) a.lse_out += most * a.lots;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_merge(const MergeArgs& a, int fmt, const LaunchCfg& cfg) {
  switch (fmt) {
    case kBF16: return launch_t<kBF16>(a, cfg);
    case kF16: return launch_t<kF16>(a, cfg);
    case kF32: return launch_t<kF32>(a, cfg);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mla
