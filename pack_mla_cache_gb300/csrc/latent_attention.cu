// latent_attention.cu -- the attention over the paged latent cache whose tokens see a number
// of rows each (mla_latent_attention); the kernel is in latent_attention.cuh.
#include "latent_attention.cuh"

namespace mla {

// Calls of fewer sequences within these sizes have more rows per sequence, at most all of
// them in one: its (bf16) tile is the largest that any of them takes.
int64_t latent_attention_workspace(int32_t num_tokens, int32_t num_heads, int32_t, int num_sms) {
  const int64_t ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
  const int64_t nr = attention_tile_rows(num_tokens, num_heads, 1, false);
  return ctas * ((int64_t)sizeof(Split) + 2 * nr * (2 + kRank) * (int64_t)sizeof(float));
}

cudaError_t launch_latent_attention(const LatentAttnArgs& a, int cache_fmt, int num_sms,
                                    const LaunchCfg& cfg) {
  return launch_attention<false>(a, cache_fmt, num_sms, cfg);
}

}  // namespace mla
