// Absorbed latent attention of groups of requests that share a prefix (kda_latent_decode_shared).
//
// Each request over all of its tokens: right, and no use made of the sharing yet.
#include "kda_internal.h"

namespace kda {

size_t latent_shared_workspace(int64_t batch, int64_t, int32_t L, int32_t h, int32_t dl) { return latent_decode_workspace(batch, L, h, dl); }

cudaError_t launch_latent_decode_shared(const LatentDecodeArgs &a, const SharedGroups &, cudaStream_t st)
{
    return launch_latent_decode(a, st);
}

}  // namespace kda
