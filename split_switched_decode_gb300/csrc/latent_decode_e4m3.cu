// latent_decode_e4m3.cu -- the latent attention kernel for e4m3 caches.
#include "latent_decode.cuh"

namespace ssd {

cudaError_t launch_latent_e4m3(const AttnParams &p, int width, int rows, const LatentLaunch &a,
                               cudaStream_t s) {
  return launch_latent<true>(p, width, rows, a, s);
}

}  // namespace ssd
