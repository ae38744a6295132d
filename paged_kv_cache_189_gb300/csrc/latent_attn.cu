// latent_attn.cu -- attention over paged latent rows and over expanded keys.
#include "latent.h"

namespace pkv {

LatentPlan plan_latent(int, int, int, int, int) { return LatentPlan{}; }

cudaError_t launch_latent_attn(const LatentParams& p, const LatentPlan&, void*, const void*, cudaStream_t s) {
    return launch_latent_simt(p, s);
}

cudaError_t launch_ragged_attn(const RaggedParams& p, const void*, const void*, const void*, cudaStream_t s) {
    return launch_ragged_simt(p, s);
}

}  // namespace pkv
