// latent_tree_attention.cu -- the attention over the paged latent cache for trees of drafted
// tokens (mla_latent_tree_attention); the kernel is in latent_attention.cuh.
#include "latent_attention.cuh"

namespace mla {

cudaError_t launch_latent_tree_attention(const LatentAttnArgs& a, int cache_fmt, int num_sms,
                                         const LaunchCfg& cfg) {
  return launch_attention<true>(a, cache_fmt, num_sms, cfg);
}

}  // namespace mla
