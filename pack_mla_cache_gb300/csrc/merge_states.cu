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
// Design: a thread owns two 16-byte chunks of an output row (half a row apart), or one
// where a row has an odd number; the weights are computed once for both.  The lse of
// its row are read twice (for m, then for the weights); the threads of a row read the
// same words, so the second pass and all but one thread's first hit L1.  Parts are
// taken four at a time, their loads issued before their sums; the first four parts'
// before the lse are looked at.  Row, token and head of a chunk come from
// multiplications by reciprocals.  Weights are 2^((lse_i - m) log2 e - s) with 2^s >=
// the number of parts, so that sums of rows near the type's largest value stay finite.
//
// Measured: 4 parts of 8192 x 16 rows of 128 bf16 28.6 us (6.0 TB/s; 29.8 with one chunk
// per thread, 30.4 with expf besides, 39 with 64-bit divisions; 5 blocks per SM of 48
// registers 32.7), 2 parts of 64 x 16 rows of 512 2.3 us.
#include "mla_device.cuh"
#include "serving.h"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // parts in flight per thread
constexpr float kLog2e = 1.4426950408889634f;

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

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// C chunks per thread: chunk ch, and for C = 2 also ch + row_chunks / 2.
template <int F, int C>
__global__ void __launch_bounds__(kThreads) merge_states_kernel(const MergeArgs a) {
  constexpr int kElts = F == kF32 ? 4 : 8;  // elements of a 16-byte chunk
  pdl_trigger();
  pdl_wait();
  const uint32_t units = (uint32_t)a.num_tokens * a.num_heads * (a.row_chunks / C);  // < 2^31
  const int64_t step = (int64_t)(a.row_chunks / C) * 16;  // bytes between a thread's chunks
  for (uint32_t u = blockIdx.x * kThreads + threadIdx.x; u < units; u += gridDim.x * kThreads) {
    const uint32_t row = a.by_units(u), ch = u - row * (a.row_chunks / C);
    const uint32_t t = a.by_heads(row), h = row - t * a.num_heads;
    const float* lse = a.lse + (int64_t)t * a.lts + (int64_t)h * a.lhs;
    const uint8_t* src = a.parts + (int64_t)t * a.ts + (int64_t)h * a.hs + (int64_t)ch * 16;
    uint4 v[kBatch][C];
    auto load = [&](int i0) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (i0 + k < a.num_parts) v[k][c] = ld_stream16(src + (i0 + k) * a.ps + c * step);
    };
    load(0);
    float m = -INFINITY, bad = 0.0f;
    for (int i = 0; i < a.num_parts; ++i) {
      const float x = __ldg(lse + i * a.lps);
      if (!(x < INFINITY)) bad = NAN;  // +inf or NaN
      m = fmaxf(m, x);
    }
    const float m0 = m == -INFINITY ? 0.0f : m;
    float acc[C][kElts];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < kElts; ++e) acc[c][e] = 0.0f;
    float sum = 0.0f;
    for (int i0 = 0;; i0 += kBatch) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (i0 + k < a.num_parts) {
          const float x = __ldg(lse + (i0 + k) * a.lps);
          if (x != -INFINITY) {  // a part without weight has no influence, whatever it holds
            const float w = exp2_approx(fmaf(x - m0, kLog2e, -a.shift));
            sum += w;
#pragma unroll
            for (int c = 0; c < C; ++c) add_weighted<F>(v[k][c], w, acc[c]);
          }
        }
      }
      if (i0 + kBatch >= a.num_parts) break;
      load(i0 + kBatch);
    }
    const float inv = (sum > 0.0f ? __frcp_rn(sum) : 0.0f) + bad;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float* x = acc[c];
      uint4 o;
      if constexpr (F == kF32) {
        o = make_uint4(__float_as_uint(x[0] * inv), __float_as_uint(x[1] * inv),
                       __float_as_uint(x[2] * inv), __float_as_uint(x[3] * inv));
      } else if constexpr (F == kBF16) {
        o = make_uint4(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv),
                       pack_bf16x2(x[4] * inv, x[5] * inv), pack_bf16x2(x[6] * inv, x[7] * inv));
      } else {
        o = make_uint4(pack_f16x2(x[0] * inv, x[1] * inv), pack_f16x2(x[2] * inv, x[3] * inv),
                       pack_f16x2(x[4] * inv, x[5] * inv), pack_f16x2(x[6] * inv, x[7] * inv));
      }
      st16(a.out + (int64_t)t * a.ots + (int64_t)h * a.ohs + (int64_t)ch * 16 + c * step, o);
    }
    if (ch == 0 && a.lse_out)
      a.lse_out[(int64_t)t * a.lots + (int64_t)h * a.lohs] = m0 + logf(sum * exp2_approx(a.shift)) + bad;
  }
}

template <int F, int C>
cudaError_t launch_t(MergeArgs a, const LaunchCfg& cfg) {
  a.by_units = Divider::by((uint32_t)a.row_chunks / C);
  // the weights are scaled down by at least the number of parts: sums of rows near the
  // type's largest value stay finite
  while ((1 << (int)a.shift) < a.num_parts) a.shift += 1.0f;
  cudaLaunchConfig_t lc = {};
  lc.blockDim = dim3(kThreads);
  lc.stream = cfg.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = cfg.pdl ? 1 : 0;
  // unit numbers stay below 2^31 - 2^24 (the last stride of the grid included): larger
  // calls, of many GiB, go in several launches
  const int64_t per_token = (int64_t)a.num_heads * (a.row_chunks / C);
  const int64_t most = (INT32_MAX - (1 << 24)) / per_token, tokens = a.num_tokens;
  for (int64_t t0 = 0; t0 < tokens; t0 += most) {
    a.num_tokens = (int32_t)(tokens - t0 < most ? tokens - t0 : most);
    const int64_t units = a.num_tokens * per_token;
    lc.gridDim = dim3(capped_grid(reinterpret_cast<const void*>(merge_states_kernel<F, C>),
                                  kThreads, (units + kThreads - 1) / kThreads));
    const cudaError_t e = cudaLaunchKernelEx(&lc, merge_states_kernel<F, C>, a);
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
  const bool pairs = a.row_chunks % 2 == 0;
  switch (fmt) {
    case kBF16: return pairs ? launch_t<kBF16, 2>(a, cfg) : launch_t<kBF16, 1>(a, cfg);
    case kF16: return pairs ? launch_t<kF16, 2>(a, cfg) : launch_t<kF16, 1>(a, cfg);
    case kF32: return pairs ? launch_t<kF32, 2>(a, cfg) : launch_t<kF32, 1>(a, cfg);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mla
