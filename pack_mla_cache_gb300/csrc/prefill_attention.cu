// prefill_attention.cu -- attention of packed sequences over keys and values per head
// (include/mla_cache.h: mla_prefill_attention).
//
// What it computes, per (token, head) row q of 128 + 64 elements and the rows of its
// sequence that the token sees: x_p = scale <q, k_p>, lse = ln sum exp(x_p), out = sum
// exp(x_p - lse) v_p.
//
// A warp takes one (token, head): lanes hold 4 + 2 elements of q and 4 of the output, one
// key after the other with a running maximum and sum.
#include "mla_device.cuh"
#include "serving.h"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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
__global__ void __launch_bounds__(kThreads) prefill_attention_kernel(const PrefillArgs a) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)a.num_tokens * a.num_heads;
  const int64_t warps = ((int64_t)gridDim.x * kThreads) >> 5;
  const float ks = KF == kE4M3 || KF == kE5M2 ? *a.kv_scale : 1.0f;
  uint32_t errbits = 0;
  for (int64_t row = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; row < rows; row += warps) {
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
cudaError_t launch_t(const PrefillArgs& a, const LaunchCfg& cfg) {
  const auto kern = prefill_attention_kernel<F, KF>;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(capped_grid(reinterpret_cast<const void*>(kern), kThreads,
                                ((int64_t)a.num_tokens * a.num_heads + kThreads / 32 - 1) / (kThreads / 32)));
  lc.blockDim = dim3(kThreads);
  lc.stream = cfg.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = cfg.pdl ? 1 : 0;
  return cudaLaunchKernelEx(&lc, kern, a);
}

}  // namespace

int64_t prefill_attention_workspace(int32_t, int32_t, int32_t, int32_t, int) { return 16; }

cudaError_t launch_prefill_attention(const PrefillArgs& a, int fmt, int kv_fmt, int,
                                     const LaunchCfg& cfg) {
  if (fmt == kBF16) {
    if (kv_fmt == kBF16) return launch_t<kBF16, kBF16>(a, cfg);
    return kv_fmt == kE4M3 ? launch_t<kBF16, kE4M3>(a, cfg) : launch_t<kBF16, kE5M2>(a, cfg);
  }
  if (kv_fmt == kF16) return launch_t<kF16, kF16>(a, cfg);
  return kv_fmt == kE4M3 ? launch_t<kF16, kE4M3>(a, cfg) : launch_t<kF16, kE5M2>(a, cfg);
}

}  // namespace mla
